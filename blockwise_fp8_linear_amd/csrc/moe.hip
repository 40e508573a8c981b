// A mixture-of-experts layer for a few tokens (include/fp8moe.h), gfx950.
#include "fp8moe_launch.h"
#include "fp8route_device.h"
#include "fp8rows_device.h"

namespace fp8blk {

namespace {

constexpr int kWaves = 8;  // of every kernel that multiplies

// ---------------------------------------------------------------------------
// Router logits x wr^T, fp32: 16 experts x 16 tokens per workgroup, the waves
// split H.
// ---------------------------------------------------------------------------
__global__ __launch_bounds__(64 * kWaves) void logits_kernel(int T, int E, int H, const uint16_t* __restrict__ x,
                                                             int64_t ld_x, const uint16_t* __restrict__ wr,
                                                             float* __restrict__ logits) {
  __shared__ v4f red[kWaves][64];
  const int lane = threadIdx.x & 63, r = lane & 15, c = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int e0 = blockIdx.x * 16, t0 = blockIdx.y * 16, nkb = H / 128;
  const uint16_t* wp = wr + (int64_t)min(e0 + r, E - 1) * H + c * 16;
  const uint16_t* xp = x + (int64_t)min(t0 + r, T - 1) * ld_x + c * 16;
  v4f acc{};
  for (int b = wave; b < nkb; b += kWaves) {
    const RawFrag w = load_raw(wp + b * 128), v = load_raw(xp + b * 128);
#pragma unroll
    for (int j = 0; j < 4; ++j)
      acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8bf_t, w.w[j]),
                                                    __builtin_bit_cast(v8bf_t, v.w[j]), acc, 0, 0, 0);
  }
  red[wave][lane] = acc;
  __syncthreads();
  if (wave == 0) {
#pragma unroll
    for (int w = 1; w < kWaves; ++w) acc += red[w][lane];
    const int t = t0 + r;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (t < T && e0 + 4 * c + i < E) logits[(int64_t)t * E + e0 + 4 * c + i] = acc[i];
  }
}

// The choice of one token by one wave, from its logits.
template <int NI>
__device__ __forceinline__ RouteChoice choose(const float* __restrict__ row, int E, int k, bool renorm, int lane) {
  float v[NI];
#pragma unroll
  for (int i = 0; i < NI; ++i) v[i] = lane + i * 64 < E ? row[lane + i * 64] : -INFINITY;
  return route_choose<64, NI>(v, k, renorm, lane);
}
__device__ __forceinline__ RouteChoice choose(const float* __restrict__ row, int E, int k, bool renorm, int lane) {
  if (E <= 64) return choose<1>(row, E, k, renorm, lane);
  if (E <= 128) return choose<2>(row, E, k, renorm, lane);
  if (E <= 256) return choose<4>(row, E, k, renorm, lane);
  return choose<16>(row, E, k, renorm, lane);
}

// ---------------------------------------------------------------------------
// One workgroup per token: its choice (where there are logits) and its row of
// x quantized, 16 lanes per group of 128.
// ---------------------------------------------------------------------------
template <class S>
__global__ __launch_bounds__(256) void prepare_kernel(MoeArgs a, const float* __restrict__ logits,
                                                      uint8_t* __restrict__ qx, float* __restrict__ sx) {
  const int t = blockIdx.x, l16 = threadIdx.x & 15;
  for (int g = threadIdx.x >> 4; g < a.H / 128; g += 16) {
    const u32x4 v = *reinterpret_cast<const u32x4*>(a.x + t * a.ld_x + g * 128 + l16 * 8);
    uint32_t m = pk_max_u16(pk_max_u16(abs2(v[0]), abs2(v[1])), pk_max_u16(abs2(v[2]), abs2(v[3])));
    m = row16_max(max(m & 0xFFFFu, m >> 16));
    const S sc(m);
    *reinterpret_cast<uint2*>(qx + (int64_t)t * a.H + g * 128 + l16 * 8) =
        make_uint2(quant4(v[0], v[1], sc), quant4(v[2], v[3], sc));
    if (l16 == 0) sx[(int64_t)t * (a.H / 128) + g] = sc.s;
  }
  if (logits && threadIdx.x < 64) {
    const RouteChoice c = choose(logits + (int64_t)t * a.E, a.E, a.k, a.renorm, threadIdx.x);
    if ((int)threadIdx.x < a.k) {
      a.ids[t * a.k + threadIdx.x] = c.id;
      a.weights[t * a.k + threadIdx.x] = c.weight;
    }
  }
}

// The rows t k + j (j-th choice of token t) that chose expert e, in order, into
// `list`; their number.  Every thread of the workgroup calls it.
__device__ __forceinline__ int rows_of_expert(const int32_t* __restrict__ ids, int n, int e, uint16_t* list,
                                              int* scratch) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, waves = blockDim.x >> 6;
  int found = 0;
  for (int s0 = 0; s0 < n; s0 += blockDim.x) {
    const int s = s0 + threadIdx.x;
    const bool hit = s < n && ids[s] == e;
    const uint64_t mask = __ballot(hit);
    if (lane == 0) scratch[wave] = __popcll(mask);
    __syncthreads();
    int before = found;
    for (int w = 0; w < waves; ++w) {
      if (w < wave) before += scratch[w];
      found += scratch[w];
    }
    if (hit) list[before + __popcll(mask & ((1ull << lane) - 1))] = (uint16_t)s;
    __syncthreads();
  }
  return found;
}

__device__ __forceinline__ float silu(float g) { return g / (1.0f + expf(-g)); }

// ---------------------------------------------------------------------------
// h[row] = bf16(silu(G x) * (U x)) for the rows that chose expert blockIdx.y:
// 16 columns of I per workgroup.
// ---------------------------------------------------------------------------
template <int W, int TT, class S>
__global__ __launch_bounds__(64 * W) void gate_up_kernel(MoeArgs a, uint16_t* __restrict__ h) {
  __shared__ uint16_t list[8192];
  __shared__ int scratch[W];
  extern __shared__ v4f red[];  // [W][2 * TT][64]
  const int lane = threadIdx.x & 63, r = lane & 15, c = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int e = blockIdx.y, n0 = blockIdx.x * 16, nkb = a.H / 128;
  const int rows = rows_of_expert(a.ids, a.T * a.k, e, list, scratch);

  const uint8_t* base = a.qw1 + (int64_t)e * 2 * a.I * a.H;
  const float* sbase = a.sw1 + (int64_t)e * (2 * a.I / 128) * nkb;
  const uint8_t* const wp[2] = {base + (int64_t)(n0 + r) * a.H + c * 16, base + (int64_t)(a.I + n0 + r) * a.H + c * 16};
  const float* const sp[2] = {sbase + n0 / 128 * nkb, sbase + (a.I + n0) / 128 * nkb};
  for (int r0 = 0; r0 < rows; r0 += 16 * TT) {
    const uint16_t* xp[TT];
#pragma unroll
    for (int tt = 0; tt < TT; ++tt)
      xp[tt] = a.x + (list[min(r0 + tt * 16 + r, rows - 1)] / a.k) * a.ld_x + c * 16;
    v4f acc[2][TT];
#pragma unroll
    for (int tt = 0; tt < TT; ++tt) acc[0][tt] = acc[1][tt] = v4f{};
    rows_product<2, TT, 1, S>(wp, sp, xp, wave * nkb / W, (wave + 1) * nkb / W, acc);
    if (r0) __syncthreads();  // the previous tile's sums have been read
#pragma unroll
    for (int rt = 0; rt < 2; ++rt)
#pragma unroll
      for (int tt = 0; tt < TT; ++tt) red[(wave * 2 * TT + rt * TT + tt) * 64 + lane] = acc[rt][tt];
    __syncthreads();
    for (int u = threadIdx.x; u < TT * 64; u += 64 * W) {
      v4f g = red[u], up = red[TT * 64 + u];
      for (int w = 1; w < W; ++w) {
        g += red[w * 2 * TT * 64 + u];
        up += red[w * 2 * TT * 64 + TT * 64 + u];
      }
      const int row = r0 + (u >> 6) * 16 + (u & 15);
      if (row < rows)
        *reinterpret_cast<uint2*>(h + (int64_t)list[row] * a.I + n0 + 4 * ((u & 63) >> 4)) =
            make_uint2(bf16x2_rne(silu(g[0]) * up[0], silu(g[1]) * up[1]),
                       bf16x2_rne(silu(g[2]) * up[2], silu(g[3]) * up[3]));
    }
  }
}

// ---------------------------------------------------------------------------
// partial[row] = weight * Wd h[row], fp32, for the rows that chose expert
// blockIdx.y: 16 RT columns of H per workgroup.
// ---------------------------------------------------------------------------
template <int W, int RT, int TT, class S>
__global__ __launch_bounds__(64 * W) void down_kernel(MoeArgs a, const uint16_t* __restrict__ h,
                                                      float* __restrict__ partial) {
  __shared__ uint16_t list[8192];
  __shared__ int scratch[W];
  extern __shared__ v4f red[];  // [W][RT * TT][64]
  const int lane = threadIdx.x & 63, r = lane & 15, c = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int e = blockIdx.y, n0 = blockIdx.x * 16 * RT, nkb = a.I / 128;
  const int rows = rows_of_expert(a.ids, a.T * a.k, e, list, scratch);

  const uint8_t* wp[RT];
  const float* sp[RT];
#pragma unroll
  for (int rt = 0; rt < RT; ++rt) {
    wp[rt] = a.qw2 + ((int64_t)e * a.H + n0 + rt * 16 + r) * a.I + c * 16;
    sp[rt] = a.sw2 + ((int64_t)e * (a.H / 128) + (n0 + rt * 16) / 128) * nkb;
  }
  for (int r0 = 0; r0 < rows; r0 += 16 * TT) {
    const uint16_t* xp[TT];
#pragma unroll
    for (int tt = 0; tt < TT; ++tt) xp[tt] = h + (int64_t)list[min(r0 + tt * 16 + r, rows - 1)] * a.I + c * 16;
    v4f acc[RT][TT];
#pragma unroll
    for (int rt = 0; rt < RT; ++rt)
#pragma unroll
      for (int tt = 0; tt < TT; ++tt) acc[rt][tt] = v4f{};
    rows_product<RT, TT, 1, S>(wp, sp, xp, wave * nkb / W, (wave + 1) * nkb / W, acc);
    if (r0) __syncthreads();  // the previous tile's sums have been read
#pragma unroll
    for (int rt = 0; rt < RT; ++rt)
#pragma unroll
      for (int tt = 0; tt < TT; ++tt) red[(wave * RT * TT + rt * TT + tt) * 64 + lane] = acc[rt][tt];
    __syncthreads();
    for (int u = threadIdx.x; u < RT * TT * 64; u += 64 * W) {
      v4f v = red[u];
      for (int w = 1; w < W; ++w) v += red[w * RT * TT * 64 + u];
      const int tile = u >> 6, l = u & 63, row = r0 + (tile % TT) * 16 + (l & 15);
      if (row < rows) {
        const int s = list[row];
        *reinterpret_cast<v4f*>(partial + (int64_t)s * a.H + n0 + (tile / TT) * 16 + 4 * (l >> 4)) = v * a.weights[s];
      }
    }
  }
}

// ---------------------------------------------------------------------------
// The same two products for many rows per launch: each wave owns 16 columns of
// I (their G and their U rows), or 16 RT columns of H, over the whole
// reduction, and the eight waves of a workgroup share the tokens' codes
// through the caches.  128 columns of I in one workgroup are one group of h,
// so h leaves quantized.
// ---------------------------------------------------------------------------
template <int TT, class S>
__global__ __launch_bounds__(512) void gate_up_wide_kernel(MoeArgs a, const uint8_t* __restrict__ qx,
                                                           const float* __restrict__ sx, uint8_t* __restrict__ qh,
                                                           float* __restrict__ sh) {
  extern __shared__ uint16_t list[];
  __shared__ int scratch[8];
  __shared__ uint32_t amax[8][16 * TT];
  const int lane = threadIdx.x & 63, r = lane & 15, c = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int e = blockIdx.y, n0 = blockIdx.x * 128 + wave * 16, nkb = a.H / 128;
  const int rows = rows_of_expert(a.ids, a.T * a.k, e, list, scratch);

  const uint8_t* base = a.qw1 + (int64_t)e * 2 * a.I * a.H;
  const float* sbase = a.sw1 + (int64_t)e * (2 * a.I / 128) * nkb;
  const uint8_t* const wp[2] = {base + (int64_t)(n0 + r) * a.H + c * 16, base + (int64_t)(a.I + n0 + r) * a.H + c * 16};
  const float* const sp[2] = {sbase + n0 / 128 * nkb, sbase + (a.I + n0) / 128 * nkb};
  for (int r0 = 0; r0 < rows; r0 += 16 * TT) {
    const uint8_t* xp[TT];
    const float* xs[TT];
    const int tiles = min(TT, (rows - r0 + 15) / 16);
#pragma unroll
    for (int tt = 0; tt < TT; ++tt) {
      const int t = list[min(r0 + tt * 16 + r, rows - 1)] / a.k;
      xp[tt] = qx + (int64_t)t * a.H + c * 16;
      xs[tt] = sx + (int64_t)t * nkb;
    }
    v4f acc[2][TT];
#pragma unroll
    for (int tt = 0; tt < TT; ++tt) acc[0][tt] = acc[1][tt] = v4f{};
    rows_stream<2, TT>(wp, sp, xp, xs, tiles, nkb, acc);
    uint32_t h[TT][2];
#pragma unroll
    for (int tt = 0; tt < TT; ++tt) {
      const v4f g = acc[0][tt], u = acc[1][tt];
      h[tt][0] = bf16x2_rne(silu(g[0]) * u[0], silu(g[1]) * u[1]);
      h[tt][1] = bf16x2_rne(silu(g[2]) * u[2], silu(g[3]) * u[3]);
      const uint32_t m = pk_max_u16(abs2(h[tt][0]), abs2(h[tt][1]));
      amax[wave][tt * 16 + r] = quarter_max(max(m & 0xFFFFu, m >> 16));
    }
    __syncthreads();
#pragma unroll
    for (int tt = 0; tt < TT; ++tt) {
      uint32_t m = 0;
#pragma unroll
      for (int w = 0; w < 8; ++w) m = max(m, amax[w][tt * 16 + r]);
      const S sc(m);
      const int row = r0 + tt * 16 + r;
      if (row < rows) {
        const int64_t s = list[row];
        *reinterpret_cast<uint32_t*>(qh + s * a.I + n0 + 4 * c) = quant4(h[tt][0], h[tt][1], sc);
        if (wave == 0 && c == 0) sh[s * (a.I / 128) + blockIdx.x] = sc.s;
      }
    }
    __syncthreads();  // before the next rows' maxima
  }
}

template <int RT, int TT>
__global__ __launch_bounds__(512) void down_wide_kernel(MoeArgs a, const uint8_t* __restrict__ qh,
                                                        const float* __restrict__ sh, float* __restrict__ partial) {
  extern __shared__ uint16_t list[];
  __shared__ int scratch[8];
  const int lane = threadIdx.x & 63, r = lane & 15, c = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int e = blockIdx.y, n0 = (blockIdx.x * 8 + wave) * 16 * RT, nkb = a.I / 128;
  const int rows = rows_of_expert(a.ids, a.T * a.k, e, list, scratch);
  if (n0 >= a.H) return;

  const uint8_t* wp[RT];
  const float* sp[RT];
#pragma unroll
  for (int rt = 0; rt < RT; ++rt) {
    wp[rt] = a.qw2 + ((int64_t)e * a.H + n0 + rt * 16 + r) * a.I + c * 16;
    sp[rt] = a.sw2 + ((int64_t)e * (a.H / 128) + (n0 + rt * 16) / 128) * nkb;
  }
  for (int r0 = 0; r0 < rows; r0 += 16 * TT) {
    const uint8_t* xp[TT];
    const float* xs[TT];
    const int tiles = min(TT, (rows - r0 + 15) / 16);
#pragma unroll
    for (int tt = 0; tt < TT; ++tt) {
      const int64_t s = list[min(r0 + tt * 16 + r, rows - 1)];
      xp[tt] = qh + s * a.I + c * 16;
      xs[tt] = sh + s * nkb;
    }
    v4f acc[RT][TT];
#pragma unroll
    for (int rt = 0; rt < RT; ++rt)
#pragma unroll
      for (int tt = 0; tt < TT; ++tt) acc[rt][tt] = v4f{};
    rows_stream<RT, TT>(wp, sp, xp, xs, tiles, nkb, acc);
#pragma unroll
    for (int tt = 0; tt < TT; ++tt) {
      const int row = r0 + tt * 16 + r;
      if (row < rows) {
        const int64_t s = list[row];
        const float w = a.weights[s];
#pragma unroll
        for (int rt = 0; rt < RT; ++rt)
          *reinterpret_cast<v4f*>(partial + s * a.H + n0 + rt * 16 + 4 * c) = acc[rt][tt] * w;
      }
    }
  }
}

// y[t] = the sum of the token's terms in the order of its choice; ids that are
// none have no term.
__global__ __launch_bounds__(256) void combine_kernel(MoeArgs a, const float* __restrict__ partial) {
  const int u = blockIdx.x * 256 + threadIdx.x, per = a.H / 4;
  const int t = u / per, n = (u - t * per) * 4;
  if (t >= a.T) return;
  v4f v{};
  for (int j = 0; j < a.k; ++j) {
    const int s = t * a.k + j, id = a.ids[s];
    if (id >= 0 && id < a.E) v += *reinterpret_cast<const v4f*>(partial + (int64_t)s * a.H + n);
  }
  if (a.out.f32)
    *reinterpret_cast<v4f*>(static_cast<float*>(a.out.y) + (int64_t)t * a.H + n) = v;
  else
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out.y) + (int64_t)t * a.H + n) =
        make_uint2(bf16x2_rne(v[0], v[1]), bf16x2_rne(v[2], v[3]));
}

template <int W, int TT, class S>
hipError_t experts(const MoeArgs& a, uint16_t* h, float* partial, hipStream_t stream) {
  hipLaunchKernelGGL((gate_up_kernel<W, TT, S>), dim3(a.I / 16, a.E), dim3(64 * W), W * 2 * TT * 64 * sizeof(v4f),
                     stream, a, h);
  if (hipError_t e = hipGetLastError()) return e;
  hipLaunchKernelGGL((down_kernel<W, 2, TT, S>), dim3(a.H / 32, a.E), dim3(64 * W), W * 2 * TT * 64 * sizeof(v4f),
                     stream, a, h, partial);
  if (hipError_t e = hipGetLastError()) return e;
  hipLaunchKernelGGL(combine_kernel, dim3((a.T * (a.H / 4) + 255) / 256), dim3(256), 0, stream, a, partial);
  return hipGetLastError();
}

template <class S>
hipError_t experts_by_tokens(const MoeArgs& a, uint16_t* h, float* partial, hipStream_t stream) {
  if (a.T <= 16) return experts<8, 1, S>(a, h, partial, stream);
  if (a.T <= 32) return experts<8, 2, S>(a, h, partial, stream);
  return experts<4, 4, S>(a, h, partial, stream);
}

template <int TT, class S>
hipError_t experts_wide(const MoeArgs& a, const uint8_t* qx, const float* sx, uint8_t* qh, float* sh, float* partial,
                        hipStream_t stream) {
  const size_t lds = (size_t)a.T * a.k * sizeof(uint16_t);
  hipLaunchKernelGGL((gate_up_wide_kernel<TT, S>), dim3(a.I / 128, a.E), dim3(512), lds, stream, a, qx, sx, qh, sh);
  if (hipError_t e = hipGetLastError()) return e;
  hipLaunchKernelGGL((down_wide_kernel<2, TT>), dim3((a.H + 255) / 256, a.E), dim3(512), lds, stream, a, qh, sh,
                     partial);
  if (hipError_t e = hipGetLastError()) return e;
  hipLaunchKernelGGL(combine_kernel, dim3((a.T * (a.H / 4) + 255) / 256), dim3(256), 0, stream, a, partial);
  return hipGetLastError();
}

template <class S>
hipError_t moe_wide(const MoeArgs& a, const MoeWorkspace& w, const float* logits, hipStream_t stream) {
  char* ws = static_cast<char*>(a.ws);
  uint8_t* qx = reinterpret_cast<uint8_t*>(ws + w.qx);
  float* sx = reinterpret_cast<float*>(ws + w.sx);
  uint8_t* qh = reinterpret_cast<uint8_t*>(ws + w.h);
  float* sh = reinterpret_cast<float*>(ws + w.sh);
  float* partial = reinterpret_cast<float*>(ws + w.partial);
  hipLaunchKernelGGL(prepare_kernel<S>, dim3(a.T), dim3(256), 0, stream, a, logits, qx, sx);
  if (hipError_t e = hipGetLastError()) return e;
  const int rows = a.T * a.k / a.E;
  if (rows <= 8) return experts_wide<1, S>(a, qx, sx, qh, sh, partial, stream);
  if (rows <= 20) return experts_wide<2, S>(a, qx, sx, qh, sh, partial, stream);
  return experts_wide<4, S>(a, qx, sx, qh, sh, partial, stream);
}

}  // namespace

hipError_t launch_moe(const MoeArgs& a, hipStream_t stream) {
  const MoeWorkspace w = moe_workspace(a.T, a.H, a.I, a.E, a.k);
  char* ws = static_cast<char*>(a.ws);
  uint16_t* h = reinterpret_cast<uint16_t*>(ws + w.h);
  float* partial = reinterpret_cast<float*>(ws + w.partial);
  float* const logits = a.wr ? reinterpret_cast<float*>(ws + w.logits) : nullptr;
  if (a.wr) {
    hipLaunchKernelGGL(logits_kernel, dim3((a.E + 15) / 16, (a.T + 15) / 16), dim3(64 * kWaves), 0, stream, a.T, a.E,
                       a.H, a.x, a.ld_x, a.wr, logits);
    if (hipError_t e = hipGetLastError()) return e;
  }
  if (a.T > 16)
    return a.fp32_scale ? moe_wide<Fp32Scale>(a, w, logits, stream) : moe_wide<Pow2Scale>(a, w, logits, stream);
  if (a.wr)
    if (hipError_t e = launch_moe_route(a.T, a.E, a.k, logits, true, a.E, a.renorm, a.ids, a.weights, stream)) return e;
  return a.fp32_scale ? experts_by_tokens<Fp32Scale>(a, h, partial, stream)
                      : experts_by_tokens<Pow2Scale>(a, h, partial, stream);
}

}  // namespace fp8blk
