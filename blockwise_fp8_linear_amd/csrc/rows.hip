// y = x W^T for a few rows of x (fp8_linear), gfx950.  Bound by reading W: N K
// bytes, against which 16 rows of x cost 1/4 to 1 of a byte of L2 traffic per
// byte of W, by the number of columns that share them.  One row through
// 12288 x 2048 takes 4.8 us above an empty launch: 5.2 TB/s.
#include "fp8blk_launch.h"
#include "fp8moe_launch.h"
#include "fp8rows_device.h"

namespace fp8blk {

namespace {

// The tile that a workgroup of a launch of columns x rows tiles takes.
// Consecutive workgroups go to the eight XCDs in turn, each with an L2 of its
// own: here every XCD gets a contiguous range of tiles in the order in which
// neighbours share the larger operand, W (rows first) or x.  (Where the columns
// are a multiple of eight the launch's own order keeps a column on one XCD.)
// 470 x 3712 (K 4352) 30.0 us without and 25.4 with, 200 x 3712 22.5 and 19.3;
// 12288 columns, a multiple, 130 rows 17.0 and 18.5.
struct TilePlace {
  uint32_t column, row;
};
__device__ __forceinline__ TilePlace tile_place(bool share_w) {
  constexpr uint32_t kXcds = 8;
  const uint32_t columns = gridDim.x, rows = gridDim.y;
  if (rows == 1 || (share_w && columns % kXcds == 0)) return {blockIdx.x, blockIdx.y};
  const uint32_t id = blockIdx.y * columns + blockIdx.x, n = columns * rows, xcd = id % kXcds;
  const uint32_t at = xcd * (n / kXcds) + min(xcd, n % kXcds) + id / kXcds;
  return share_w ? TilePlace{at / rows, at % rows} : TilePlace{at % columns, at / columns};
}

// One workgroup: 16 RT columns of y, 16 TT rows, the W waves splitting the
// reduction (K / 128 blocks are few: two per wave at 2048, all in flight at
// once).  RAW: xv is x in bf16 (ld_x elements apart) and quantized here;
// otherwise its codes [M][K], with the scales transposed, xs[K / 128][M].
template <int W, int RT, int TT, int XL, int D, bool RAW, class S>
__global__ __launch_bounds__(64 * W) void linear_rows_kernel(int64_t M, int64_t N, int64_t K, const uint8_t* xv,
                                                             int64_t row_bytes, const float* __restrict__ xs,
                                                             const uint8_t* __restrict__ qw,
                                                             const float* __restrict__ sw, RowsOut out) {
  extern __shared__ uint8_t lds[];  // the waves' areas; then their sums, [W][RT * TT][64] v4f
  const uint32_t lane = threadIdx.x & 63, r = lane & 15;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const TilePlace place = tile_place(M < N);
  const int64_t n0 = (int64_t)place.column * (16 * RT), m0 = (int64_t)place.row * (16 * TT);
  const int nkb = (int)(K / 128), rows = (int)(M - m0 < 16 * TT ? M - m0 : 16 * TT);

  const uint8_t* wp[RT];
  const float* sp[RT];
  const float* xsp[TT];
  uint32_t xoff[TT][XL];
#pragma unroll
  for (int rt = 0; rt < RT; ++rt) {
    wp[rt] = qw + (n0 + rt * 16) * K;
    sp[rt] = sw + (n0 + rt * 16) / 128 * nkb;
  }
#pragma unroll
  for (int tt = 0; tt < TT; ++tt) {
#pragma unroll
    for (int u = 0; u < XL; ++u) {
      const int row = tt * 16 + (int)(RAW ? raw_row(lane, u) : code_row(lane, u));
      xoff[tt][u] = (uint32_t)(min(row, rows - 1) * row_bytes) + (RAW ? (lane & 15) * 16 : code_chunk(lane, u));
    }
    xsp[tt] = RAW ? nullptr : xs + m0 + min(tt * 16 + (int)r, rows - 1);
  }
  v4f acc[RT][TT];
#pragma unroll
  for (int rt = 0; rt < RT; ++rt)
#pragma unroll
    for (int tt = 0; tt < TT; ++tt) acc[rt][tt] = v4f{};
  rows_product<RT, TT, XL, D, RAW, S>(lds + wave * D * rows_stage_bytes<RT, TT, RAW, XL>(), wp, sp, K,
                                      xv + m0 * row_bytes, xoff, xsp, M, wave * nkb / W, (wave + 1) * nkb / W, acc);

  v4f* red = reinterpret_cast<v4f*>(lds);
  __syncthreads();
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
    store_rows<true>(out, m * N + n, v);
  }
}

template <int W, int RT, int TT, int XL, int D, bool RAW, class S>
hipError_t launch(int64_t M, int64_t N, int64_t K, const void* x, int64_t row_bytes, const float* xs,
                  const uint8_t* qw, const float* sw, RowsOut out, hipStream_t stream) {
  const dim3 grid((uint32_t)(N / (16 * RT)), (uint32_t)((M + 16 * TT - 1) / (16 * TT)));
  constexpr int area = D * rows_stage_bytes<RT, TT, RAW, XL>(), sums = RT * TT * 64 * (int)sizeof(v4f);
  constexpr int lds = W * (area > sums ? area : sums);
  static std::atomic<uint64_t> raised{0};
  if (hipError_t e = ensure_lds_limit(reinterpret_cast<const void*>(&linear_rows_kernel<W, RT, TT, XL, D, RAW, S>), lds,
                                      &raised))
    return e;
  hipLaunchKernelGGL((linear_rows_kernel<W, RT, TT, XL, D, RAW, S>), grid, dim3(64 * W), lds, stream, M, N, K,
                     static_cast<const uint8_t*>(x), row_bytes, xs, qw, sw, out);
  return hipGetLastError();
}

// Many rows, but too few for the GEMMs' 256x256 tiles: 128 columns of y and 64
// rows per workgroup, whole reduction, x's codes shared in LDS, the fp8 matrix
// instruction.  Bound by what the tiles load from L2 (192 bytes per 8192
// multiply-adds) and by one block's latency.  (Columns x rows) 128 x 32, 128 x
// 128, 256 x 64 and 256 x 128 measured slower: 1024 x 4096 x 2048 16.9 us, and
// 23.1, 18.6, 20.2, 28.7.  On the bf16 instruction, whose sums are fp32's (1e-7
// of the norm instead of 4e-5), 512 x 4096 x 2048 takes 23.0 instead of 16.8 us,
// 3000 x 9216 x 4224 324 instead of 183: the fp8 one, which is what the same rows
// get from the GEMMs when there are more of them.
template <int SLOTS>
__global__ __launch_bounds__(512) void linear_wide_kernel(int64_t M, int64_t N, int64_t K,
                                                          const uint8_t* __restrict__ q, const float* __restrict__ xs,
                                                          const uint8_t* __restrict__ qw,
                                                          const float* __restrict__ sw, RowsOut out) {
  extern __shared__ uint8_t lds[];
  constexpr int TT = kWideTiles;
  const int lane = threadIdx.x & 63, r = lane & 15, c = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const TilePlace place = tile_place(M < N);
  const int64_t n0 = ((int64_t)place.column * 8 + wave) * 16, m0 = (int64_t)place.row * 16 * TT;
  const int nkb = (int)(K / 128), rows = (int)(M - m0 < 16 * TT ? M - m0 : 16 * TT);
  const uint8_t* const wp[1] = {qw + n0 * K};
  const float* const sp[1] = {sw + n0 / 128 * nkb};
  const int load = wave % (2 * TT), row = (load >> 1) * 16 + (int)code_row(lane, load & 1);
  const uint32_t xoff = (uint32_t)(min(row, rows - 1) * K) + code_chunk(lane, load & 1);
  v4f acc[1][TT] = {};
  rows_ring<1, TT, SLOTS, true>(
      lds, wp, sp, K, q + m0 * K, xoff, xs + m0, M, [&](int i) { return min(i, rows - 1); }, nkb, acc);
#pragma unroll
  for (int tt = 0; tt < TT; ++tt)
    if (tt * 16 + r < rows) store_rows<true>(out, (m0 + tt * 16 + r) * N + n0 + 4 * c, acc[0][tt]);
}

// ---------------------------------------------------------------------------
// Codes of all rows of x, with the scales transposed ([K / 128][M]): what the
// tiles of several rows load.  16 lanes per group of 128, which take the next
// ones where there are more than kQuantGrid workgroups' (a launch has fewer
// than 2^32 threads).
// ---------------------------------------------------------------------------
constexpr int64_t kQuantGrid = 65536;
template <class S>
__global__ __launch_bounds__(256) void quantize_rows_kernel(int64_t M, int nkb, const uint16_t* __restrict__ x,
                                                            int64_t ld_x, uint8_t* __restrict__ q,
                                                            float* __restrict__ s) {
  const int l16 = threadIdx.x & 15;
  for (int64_t u = (int64_t)blockIdx.x * 16 + (threadIdx.x >> 4); u < M * nkb; u += (int64_t)gridDim.x * 16) {
    const int64_t m = u / nkb;
    const int g = (int)(u - m * nkb);
    const u32x4 v = *reinterpret_cast<const u32x4*>(x + m * ld_x + g * 128 + l16 * 8);
    float scale;
    *reinterpret_cast<uint2*>(q + u * 128 + l16 * 8) = quantize8<S>(v, &scale);
    if (l16 == 0) s[g * M + m] = scale;
  }
}

// Tiles are chosen so that a launch has about one workgroup of eight waves per
// CU.  Times below are us as a graph node at K = 2048 (an empty node takes 2.1),
// power-of-two scales.

// rows_raw(): one launch that quantizes as it multiplies.  16 tokens per
// workgroup (more rows per tile only pay at large N: 32 x 12288 9.7 with two
// tiles of tokens, 10.3 with one).  1, 2, 3, 4 tiles of columns:
//   16 x 4096   4.9  5.2   -    -       24 x 4096   6.1  5.2   -    -
//   64 x 4096   -    6.7   -   6.3      16 x 12288  9.7  9.7  8.0  8.2
//   24 x 12288  -   10.2 10.2   -  (four tiles: 1.5 rounds of one workgroup per CU, 13.4)
// 16 waves for one tile: 16 x 4096 4.7 instead of 4.9, 16 x 2048 (K 6144) 9.2
// instead of 10.1; a single row is no faster with them at K = 2048.
template <int XL, class S>
hipError_t launch_raw(int64_t M, int64_t N, int64_t K, const uint16_t* x, int64_t ld_x, const uint8_t* qw,
                      const float* sw, RowsOut out, hipStream_t stream) {
  const int64_t tiles = N / 16, all = tiles * ((M + 15) / 16);
#define FP8_RAW(W, RT) launch<W, RT, 1, XL, 1, true, S>(M, N, K, x, ld_x * 2, nullptr, qw, sw, out, stream)
  if (all <= 256) return XL > 1 || K >= 4096 ? FP8_RAW(16, 1) : FP8_RAW(8, 1);
  if (all <= 512) return FP8_RAW(8, 2);
  if (tiles % 3 == 0 && all <= 1536) return FP8_RAW(8, 3);
  if (all <= 1024) return FP8_RAW(8, 4);
  return tiles % 3 == 0 ? FP8_RAW(4, 3) : FP8_RAW(4, 2);
#undef FP8_RAW
}

template <int SLOTS>
hipError_t launch_wide(int64_t M, int64_t N, int64_t K, const uint8_t* q, const float* s, const uint8_t* qw,
                       const float* sw, RowsOut out, hipStream_t stream) {
  constexpr int lds = rows_ring_bytes<1, kWideTiles, SLOTS>();
  static std::atomic<uint64_t> raised{0};
  const auto k = &linear_wide_kernel<SLOTS>;
  if (hipError_t e = ensure_lds_limit(reinterpret_cast<const void*>(k), lds, &raised)) return e;
  const dim3 grid((uint32_t)(N / 128), (uint32_t)((M + 16 * kWideTiles - 1) / (16 * kWideTiles)));
  hipLaunchKernelGGL(k, grid, dim3(512), lds, stream, M, N, K, q, s, qw, sw, out);
  return hipGetLastError();
}

// More rows: x quantized once (2.2 us), then the kernel of codes_tile().
hipError_t launch_codes(int64_t M, int64_t N, int64_t K, const uint8_t* q, const float* s, const uint8_t* qw,
                        const float* sw, RowsOut out, hipStream_t stream) {
  const RowsTile t = codes_tile(M, N);
  if (t.slots)
    return t.slots == 4 ? launch_wide<4>(M, N, K, q, s, qw, sw, out, stream)
                        : launch_wide<2>(M, N, K, q, s, qw, sw, out, stream);
#define FP8_CODES(W, RT, TT)                             \
  if (t.waves == W && t.columns == RT && t.tokens == TT) \
  return launch<W, RT, TT, 2, 1, false, Pow2Scale>(M, N, K, q, K, s, qw, sw, out, stream)
  FP8_CODES(16, 1, 1);
  FP8_CODES(8, 2, 1);
  FP8_CODES(8, 2, 2);
  FP8_CODES(8, 4, 2);
  FP8_CODES(8, 4, 4);
  FP8_CODES(4, 3, 2);
  FP8_CODES(4, 4, 2);
#undef FP8_CODES
  return hipErrorInvalidValue;
}

template <class S>
hipError_t launch_scale(int64_t M, int64_t N, int64_t K, const uint16_t* x, int64_t ld_x, const uint8_t* qw,
                        const float* sw, RowsOut out, bool raw, void* ws, hipStream_t stream) {
  if (raw) {
    if (M <= 4) return launch_raw<1, S>(M, N, K, x, ld_x, qw, sw, out, stream);
    if (M <= 8) return launch_raw<2, S>(M, N, K, x, ld_x, qw, sw, out, stream);
    return launch_raw<4, S>(M, N, K, x, ld_x, qw, sw, out, stream);
  }
  const int nkb = (int)(K / 128);
  uint8_t* q = static_cast<uint8_t*>(ws);
  float* s = reinterpret_cast<float*>(q + rows_scales_at(M, K));
  const int64_t grid = (M * nkb + 15) / 16;
  hipLaunchKernelGGL(quantize_rows_kernel<S>, dim3((uint32_t)(grid < kQuantGrid ? grid : kQuantGrid)), dim3(256), 0,
                     stream, M, nkb, x, ld_x, q, s);
  if (hipError_t e = hipGetLastError()) return e;
  return launch_codes(M, N, K, q, s, qw, sw, out, stream);
}

}  // namespace

hipError_t launch_linear_rows(int64_t M, int64_t N, int64_t K, const uint16_t* x, int64_t ld_x, const uint8_t* qw,
                              const float* sw, RowsOut out, bool fp32_scale, void* ws, hipStream_t stream) {
  const bool raw = rows_raw(M, N, K, fp32_scale);
  return fp32_scale ? launch_scale<Fp32Scale>(M, N, K, x, ld_x, qw, sw, out, raw, ws, stream)
                    : launch_scale<Pow2Scale>(M, N, K, x, ld_x, qw, sw, out, raw, ws, stream);
}

}  // namespace fp8blk
