// y = x W^T for a few rows of x (fp8_linear), gfx950.
#include "fp8moe_launch.h"
#include "fp8rows_device.h"

namespace fp8blk {

namespace {

template <int W, int RT, int TT, int D, class S>
__global__ __launch_bounds__(64 * W) void linear_rows_kernel(int64_t M, int64_t N, int64_t K, const uint16_t* __restrict__ x, int64_t ld_x,
                                   const uint8_t* __restrict__ qw, const float* __restrict__ sw, RowsOut out) {
  extern __shared__ v4f red[];  // [waves][RT * TT][64]
  const uint32_t lane = threadIdx.x & 63, r = lane & 15, c = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t n0 = (int64_t)blockIdx.x * (16 * RT), m0 = (int64_t)blockIdx.y * (16 * TT);
  const int nkb = (int)(K / 128);

  const uint8_t* wp[RT];
  const float* sp[RT];
  const uint16_t* xp[TT];
#pragma unroll
  for (int rt = 0; rt < RT; ++rt) {
    wp[rt] = qw + (n0 + rt * 16 + r) * K + c * 16;
    sp[rt] = sw + (n0 + rt * 16) / 128 * nkb;
  }
#pragma unroll
  for (int tt = 0; tt < TT; ++tt) {
    const int64_t m = m0 + tt * 16 + r;
    xp[tt] = x + (m < M ? m : M - 1) * ld_x + c * 16;
  }
  v4f acc[RT][TT];
#pragma unroll
  for (int rt = 0; rt < RT; ++rt)
#pragma unroll
    for (int tt = 0; tt < TT; ++tt) acc[rt][tt] = v4f{};
  rows_product<RT, TT, D, S>(wp, sp, xp, wave * nkb / W, (wave + 1) * nkb / W, acc);

#pragma unroll
  for (int rt = 0; rt < RT; ++rt)
#pragma unroll
    for (int tt = 0; tt < TT; ++tt) red[(wave * RT * TT + rt * TT + tt) * 64 + lane] = acc[rt][tt];
  __syncthreads();
  for (int u = threadIdx.x; u < RT * TT * 64; u += 64 * W) {
    v4f v = red[u];
    for (int w = 1; w < W; ++w) v += red[w * RT * TT * 64 + u];
    const int tile = u >> 6, l = u & 63;
    const int64_t m = m0 + (tile % TT) * 16 + (l & 15), n = n0 + (tile / TT) * 16 + 4 * (l >> 4);
    if (m >= M) continue;
    if (out.f32) {
      v4f* y = reinterpret_cast<v4f*>(static_cast<float*>(out.y) + m * N + n);
      *y = out.accumulate ? *y + v : v;
    } else {
      *reinterpret_cast<uint2*>(static_cast<uint16_t*>(out.y) + m * N + n) =
          make_uint2(bf16x2_rne(v[0], v[1]), bf16x2_rne(v[2], v[3]));
    }
  }
}

template <int W, int RT, int TT, int D, class S>
hipError_t launch(int64_t M, int64_t N, int64_t K, const uint16_t* x, int64_t ld_x, const uint8_t* qw,
                  const float* sw, RowsOut out, hipStream_t stream) {
  const dim3 grid((uint32_t)(N / (16 * RT)), (uint32_t)((M + 16 * TT - 1) / (16 * TT)));
  hipLaunchKernelGGL((linear_rows_kernel<W, RT, TT, D, S>), grid, dim3(64 * W), W * RT * TT * 64 * sizeof(v4f),
                     stream, M, N, K, x, ld_x, qw, sw, out);
  return hipGetLastError();
}

template <int RT, int TT, class S>
hipError_t launch_tile(int64_t M, int64_t N, int64_t K, const uint16_t* x, int64_t ld_x, const uint8_t* qw,
                       const float* sw, RowsOut out, hipStream_t stream) {
  constexpr int W = RT * TT > 6 ? 4 : 8;
  return launch<W, RT, TT, 1, S>(M, N, K, x, ld_x, qw, sw, out, stream);
}

template <int TT, class S>
hipError_t launch_tokens(int64_t M, int64_t N, int64_t K, const uint16_t* x, int64_t ld_x, const uint8_t* qw,
                         const float* sw, RowsOut out, hipStream_t stream) {
  const int64_t tiles = N / 16;
  if (tiles >= 1024) return launch_tile<4, TT, S>(M, N, K, x, ld_x, qw, sw, out, stream);
  if (tiles >= 768 && tiles % 3 == 0) return launch_tile<3, TT, S>(M, N, K, x, ld_x, qw, sw, out, stream);
  if (tiles >= 512) return launch_tile<2, TT, S>(M, N, K, x, ld_x, qw, sw, out, stream);
  return launch_tile<1, TT, S>(M, N, K, x, ld_x, qw, sw, out, stream);
}

template <class S>
hipError_t launch_scale(int64_t M, int64_t N, int64_t K, const uint16_t* x, int64_t ld_x, const uint8_t* qw,
                        const float* sw, RowsOut out, hipStream_t stream) {
  if (M <= 16) return launch_tokens<1, S>(M, N, K, x, ld_x, qw, sw, out, stream);
  if (M <= 32) return launch_tokens<2, S>(M, N, K, x, ld_x, qw, sw, out, stream);
  return launch_tokens<3, S>(M, N, K, x, ld_x, qw, sw, out, stream);
}

}  // namespace

hipError_t launch_linear_rows(int64_t M, int64_t N, int64_t K, const uint16_t* x, int64_t ld_x, const uint8_t* qw,
                              const float* sw, RowsOut out, bool fp32_scale, hipStream_t stream) {
  return fp32_scale ? launch_scale<Fp32Scale>(M, N, K, x, ld_x, qw, sw, out, stream)
                    : launch_scale<Pow2Scale>(M, N, K, x, ld_x, qw, sw, out, stream);
}

}  // namespace fp8blk
