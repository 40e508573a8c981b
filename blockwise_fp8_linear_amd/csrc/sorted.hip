// Rows in sorted order and back (include/fp8train.h): the gather that quantizes
// a token's row for each of its experts, the weighted sum of a token's rows, and
// the gradient of the weights.
//
//   gather    row r = x[source[r] / k] (times weights[source[r]], rounded to bf16)
//   combine   y[t] = sum_i w[t][i] z[rows[t][i]]
//   dweights  dw[t][i] = sum_h dy[t][h] z[rows[t][i]][h]
//
// All are bound by memory: a row is read or written k times a token, for a few
// operations a value.
#include "fp8blk_device.h"
#include "fp8tile_device.h"
#include "fp8train_launch.h"
#include "fp8used_device.h"

namespace fp8blk {

namespace {

constexpr int kThreads = 256;

// Two bf16 times w, rounded to bf16.
__device__ __forceinline__ uint32_t scaled2(uint32_t v, float w) {
  return bf16x2_rne(bf16_lo(v) * w, bf16_hi(v) * w);
}

// ---------------------------------------------------------------------------
// Row groups only.  A wave takes kRowCols columns of a run of rows: everything
// about a row (its source, its addresses, its weight) is the same for the whole
// wave and costs no vector instructions, of which the quantizing alone takes 35 a
// KiB -- with a row per 16 lanes instead the kernel was bound by them (16384 tokens
// to 8 experts each, 2048 wide: 126 us).  A row's source has to be there before
// its values can be loaded, so the run's sources come first, in one load, and the
// next row's values are on the way while one is quantized.
// ---------------------------------------------------------------------------
constexpr int kRowSteps = 4, kRowCols = kRowSteps * 512;
constexpr int kMaxRun = 16;

// The order in which pairs of runs are taken (GatherArgs::order): by the token of a
// pair's first row.  A token's rows are far apart, one in each of its experts'
// segments; taken in the order of the rows they are fetched from memory k times
// (16384 tokens to 8 of 128 experts: 511 MB, with 295 MB of codes 121 us; in this
// order 126 MB and 74 us).  By
// tokens, and each XCD with a range of its own, a token's rows are taken at about
// the same time by CUs that share an L2.  Each of kOrderBlocks workgroups looks at
// all pairs, counts those before its share of the token ranges, and in LDS those of
// each range of it, and places them -- those of a range in no particular order,
// which changes no result.  (One workgroup for all: 19 us, most of it scattered
// stores; each counting every range: 12.)
constexpr int kOrderThreads = 1024, kOrderKeys = (int)(kOrderPairs / kOrderThreads), kOrderRanges = 1024;
constexpr uint32_t kOrderBlocks = 16, kOrderShare = kOrderRanges / kOrderBlocks;
static_assert(kOrderShare == 64, "a lane per range");

__global__ __launch_bounds__(kOrderThreads) void gather_order_kernel(GatherArgs a, uint32_t pair, int shift) {
  __shared__ uint32_t count[kOrderShare], wave_before[kOrderThreads / 64];
  const uint32_t t = threadIdx.x, lane = t & 63, wave = t >> 6;
  const uint32_t pairs = (used_tiles(a.used, a.R) * 128 + pair - 1) / pair;
  const uint32_t n = (uint32_t)(a.T * a.k), first = blockIdx.x * kOrderShare;
  if (t < kOrderShare) count[t] = 0;
  __syncthreads();
  uint32_t key[kOrderKeys], before = 0;
#pragma unroll
  for (int i = 0; i < kOrderKeys; ++i) {
    const uint32_t r = i * kOrderThreads + t;
    key[i] = r < pairs ? (uint32_t)a.source[(int64_t)r * pair] : 0;
  }
#pragma unroll
  for (int i = 0; i < kOrderKeys; ++i) {
    const uint32_t r = i * kOrderThreads + t;
    // choices are in the order of their tokens; padding goes anywhere, but not all
    // of it to one counter; what is behind the last pair nowhere
    const uint32_t range = r >= pairs ? kOrderRanges : key[i] < n ? key[i] >> shift : r % kOrderRanges;
    before += range < first ? 1 : 0;
    key[i] = range - first;
    if (key[i] < kOrderShare) atomicAdd(&count[key[i]], 1u);
  }
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) before += (uint32_t)__shfl_xor((int)before, d, 64);
  if (lane == 0) wave_before[wave] = before;
  __syncthreads();
  if (wave == 0) {
    const uint32_t mine = count[lane];
    uint32_t upto = mine;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const uint32_t o = (uint32_t)__shfl_up((int)upto, d, 64);
      if ((int)lane >= d) upto += o;
    }
    uint32_t at = upto - mine;
#pragma unroll
    for (int w = 0; w < kOrderThreads / 64; ++w) at += wave_before[w];
    count[lane] = at;
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kOrderKeys; ++i)
    if (key[i] < kOrderShare) a.order[atomicAdd(&count[key[i]], 1u)] = i * kOrderThreads + t;
}

template <class S, bool W, bool NT>
__global__ __launch_bounds__(kThreads) void gather_rows_kernel(GatherArgs a, uint32_t run, uint32_t parts) {
  const uint32_t lane = threadIdx.x & 63, l16 = lane & 15;
  const int64_t rows = (int64_t)used_tiles(a.used, a.R) * 128;
  uint32_t item = blockIdx.x * (kThreads / 64) + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  if (a.order) {
    // an eighth of the ordered pairs for each XCD
    const uint32_t pairs = (uint32_t)((rows + 2 * run - 1) / (2 * run)), per = (pairs + 7) / 8, xcd = blockIdx.x % 8;
    const uint32_t at = (blockIdx.x / 8) * (kThreads / 64) + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const uint32_t in = at / (2 * parts), nth = xcd * per + in;
    if (in >= per || nth >= pairs) return;
    item = a.order[nth] * 2 * parts + at % (2 * parts);
  }
  const uint32_t part = item % parts;
  const int64_t r0 = (int64_t)(item / parts) * run;
  if (r0 >= rows) return;
  const int n_rows = (int)(rows - r0 < run ? rows - r0 : run);
  const int64_t n = a.T * a.k, G = a.H / 128;
  const int32_t c0 = (int32_t)(part * kRowCols + lane * 8);  // the lane's first column
  const int32_t left = (int32_t)(a.H - part * kRowCols);     // the wave's columns: steps behind them are left out
  // lane i: the i-th row's source and weight
  int32_t src = (int)lane < n_rows ? a.source[r0 + lane] : -1;
  if (src >= n) src = -1;
  float weight = 1.0f;
  if constexpr (W) weight = src >= 0 ? a.weights[src] : 0.0f;
  const auto load = [&](int i, u32x4 (&v)[kRowSteps]) {
    const int32_t s = __builtin_amdgcn_readlane(src, i);
    if (s < 0) {
#pragma unroll
      for (int u = 0; u < kRowSteps; ++u) v[u] = u32x4{0, 0, 0, 0};
      return;
    }
    const uint16_t* row = a.x + (int64_t)((uint32_t)s / (uint32_t)a.k) * a.ld_x;
#pragma unroll
    for (int u = 0; u < kRowSteps; ++u)
      if (u * 512 < left)
        v[u] = c0 + u * 512 < a.H ? *reinterpret_cast<const u32x4*>(row + c0 + u * 512) : u32x4{0, 0, 0, 0};
  };
  u32x4 v[kRowSteps], w[kRowSteps];
  load(0, v);
  for (int i = 0; i < n_rows; ++i) {
    if (i + 1 < n_rows) load(i + 1, w);
    const float wt = W ? __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(weight), i)) : 1.0f;
    uint8_t* const q = a.q.q + (r0 + i) * a.q.ld;
    float* const s = a.q.s + (r0 + i) * G;
#pragma unroll
    for (int u = 0; u < kRowSteps; ++u) {
      if (u * 512 >= left) break;
      u32x4 x = v[u];
      if constexpr (W) x = u32x4{scaled2(x.x, wt), scaled2(x.y, wt), scaled2(x.z, wt), scaled2(x.w, wt)};
      tile_u32x2 o;
      const float scale = quant_group<S>(x, o);
      if (c0 + u * 512 < a.H) {
        store_codes<NT>(q + c0 + u * 512, o);
        if (l16 == 0) s[(c0 + u * 512) >> 7] = scale;
      }
      v[u] = w[u];
    }
  }
}

// ---------------------------------------------------------------------------
// Both orientations: a 128 x 128 tile a workgroup, as the one-pass quantizer.
// ---------------------------------------------------------------------------
// The eight values of the thread's 8 sorted rows, from column c on: zeros where a row's
// source is no choice.  Such a row loads token 0's: behind a branch for each row the
// loads waited for each other (20608 rows of 2048, of 4095 tokens, 24 us and now 22,
// amax / 448 33 and 29).  A choice's token is its number over k, by the multiplier 2^32
// / k rounded up, exact for choices below 2^28 and k up to 16.
template <bool W>
__device__ __forceinline__ void gathered(u32x4 (&v)[8], const GatherArgs& a, const int32_t* __restrict__ source,
                                         int64_t c) {
  const uint32_t n = (uint32_t)(a.T * a.k), per_k = (uint32_t)(((uint64_t(1) << 32) + a.k - 1) / (uint32_t)a.k);
  uint32_t src[8];
  float w[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) src[i] = (uint32_t)source[i];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t from = src[i] < n ? src[i] : 0, t = a.k > 1 ? __umulhi(from, per_k) : from;
    v[i] = *reinterpret_cast<const u32x4*>(a.x + (int64_t)t * a.ld_x + c);
    if constexpr (W) w[i] = a.weights[from];
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if constexpr (W) v[i] = u32x4{scaled2(v[i].x, w[i]), scaled2(v[i].y, w[i]), scaled2(v[i].z, w[i]), scaled2(v[i].w, w[i])};
    const uint32_t keep = src[i] < n ? ~0u : 0u;
    v[i] = u32x4{v[i].x & keep, v[i].y & keep, v[i].z & keep, v[i].w & keep};
  }
}

// mine: the column tiles that are one XCD's for all rows, or 0.  Where an eighth of
// x's columns fits an XCD's L2 with room to spare (kSliceL2), a token's rows beyond
// the first are read from there: 4095 tokens to 4 of 60 experts, 2048 wide,
// 27.6 us and 26.6, amax / 448 35.2 and 32.4; 16384 tokens, whose slices do not fit, 152
// to 164 us either way.
constexpr int64_t kSliceL2 = int64_t(5) << 19;

template <class S, bool W, bool NT>
__global__ __launch_bounds__(kTileThreads, 6) void gather_both_kernel(GatherArgs a, TileGrid grid, uint32_t mine) {
  __shared__ TileLds lds;
  const uint32_t row_tiles = grid.row_tiles, col_tiles = grid.col_tiles;
  uint32_t rt, ct;
  if (mine) {
    const uint32_t xcd = blockIdx.x % 8, j = blockIdx.x / 8;
    rt = j / mine;
    ct = xcd * mine + (j - rt * mine);
  } else {
    tile_of(blockIdx.x, col_tiles, grid.blocked, rt, ct);
  }
  if (ct >= col_tiles || rt >= used_tiles(a.used, a.R)) return;
  const uint32_t rb = threadIdx.x >> 4, cb = threadIdx.x & 15;
  const int64_t m0 = (int64_t)rt * 128, c0 = (int64_t)ct * 128;
  u32x4 v[8];
  gathered<W>(v, a, a.source + m0 + rb * 8, c0 + cb * 8);
  tile_row_groups<S, NT>(v, a.q.q + m0 * a.q.ld + c0 + cb * 8, a.q.ld, a.q.s + m0 * col_tiles + ct, col_tiles, rb, cb);
  tile_col_groups<S, NT>(v, lds, a.qT.q + c0 * a.qT.ld + m0, a.qT.ld, a.qT.s + c0 * row_tiles + rt, row_tiles, rb, cb);
}

// ---------------------------------------------------------------------------
// Back to the tokens.  A wave takes 512 columns of a token, 16 bytes of each of
// its rows a lane; the rows are loaded kBatch at a time.  131072 rows of 2048 to 16384
// tokens: 110 us, 5.5 TB/s.
// ---------------------------------------------------------------------------
constexpr int kBatch = 8;

__global__ __launch_bounds__(kThreads) void combine_kernel(int64_t T, int64_t H, int64_t R, int k,
                                                           const uint16_t* __restrict__ z, int64_t ld_z,
                                                           const int32_t* __restrict__ rows,
                                                           const float* __restrict__ weights, RowsOut out,
                                                           uint32_t parts) {
  const uint32_t lane = threadIdx.x & 63;
  const int64_t item = (int64_t)blockIdx.x * (kThreads / 64) + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t t = item / parts;
  const int64_t c = (item - t * parts) * 512 + lane * 8;
  if (t >= T || c >= H) return;
  float acc[8] = {};
  for (int i0 = 0; i0 < k; i0 += kBatch) {
    u32x4 v[kBatch];
    float w[kBatch];
    bool in[kBatch];
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int32_t r = i0 + i < k ? rows[t * k + i0 + i] : -1;
      in[i] = r >= 0 && r < R;
      w[i] = in[i] ? (weights ? weights[t * k + i0 + i] : 1.0f) : 0.0f;
      v[i] = in[i] ? *reinterpret_cast<const u32x4*>(z + (int64_t)r * ld_z + c) : u32x4{0, 0, 0, 0};
    }
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      if (!in[i]) continue;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        acc[2 * j] = __builtin_fmaf(w[i], bf16_lo(v[i][j]), acc[2 * j]);
        acc[2 * j + 1] = __builtin_fmaf(w[i], bf16_hi(v[i][j]), acc[2 * j + 1]);
      }
    }
  }
  if (out.f32) {
    v4f* const y = reinterpret_cast<v4f*>(static_cast<float*>(out.y) + t * H + c);
    v4f a = {acc[0], acc[1], acc[2], acc[3]}, b = {acc[4], acc[5], acc[6], acc[7]};
    if (out.accumulate) {
      const v4f a0 = y[0], b0 = y[1];
      a = v4f{a0[0] + a[0], a0[1] + a[1], a0[2] + a[2], a0[3] + a[3]};
      b = v4f{b0[0] + b[0], b0[1] + b[1], b0[2] + b[2], b0[3] + b[3]};
    }
    y[0] = a;
    y[1] = b;
  } else {
    *reinterpret_cast<u32x4*>(static_cast<uint16_t*>(out.y) + t * H + c) =
        u32x4{bf16x2_rne(acc[0], acc[1]), bf16x2_rne(acc[2], acc[3]), bf16x2_rne(acc[4], acc[5]),
              bf16x2_rne(acc[6], acc[7])};
  }
}

// The wave's sums of eight values: lane i gets the i-th (as does every lane whose
// number ends like i's).  A lane passes on the half of its sums that belongs to the
// other side of each exchange: 10 exchanges instead of 48.
static_assert(kBatch == 8, "three halvings");
__device__ __forceinline__ float sums8(const float (&v)[kBatch], uint32_t lane) {
  float a[4], b[2];
  const bool b4 = lane & 4, b2 = lane & 2, b1 = lane & 1;
#pragma unroll
  for (int i = 0; i < 4; ++i) a[i] = (b4 ? v[i + 4] : v[i]) + __shfl_xor(b4 ? v[i] : v[i + 4], 4, 64);
#pragma unroll
  for (int i = 0; i < 2; ++i) b[i] = (b2 ? a[i + 2] : a[i]) + __shfl_xor(b2 ? a[i] : a[i + 2], 2, 64);
  float s = (b1 ? b[1] : b[0]) + __shfl_xor(b1 ? b[0] : b[1], 1, 64);
  s += __shfl_xor(s, 8, 64);
  s += __shfl_xor(s, 16, 64);
  return s + __shfl_xor(s, 32, 64);
}

// A token's columns, 512 at a time, are shared by the workgroup's waves, whose sums
// meet in LDS, in wave order (a wave a token instead is 0 to 4% slower at 512 to 16384
// tokens).  Each of the k sums is a lane's, then the wave's, then the token's, in an
// order that H decides.  131072 rows of 2048: 108 us, 5.6 TB/s.
constexpr int kMaxK = 16, kWaves = kThreads / 64;

__global__ __launch_bounds__(kThreads) void dweights_kernel(int64_t T, int64_t H, int64_t R, int k,
                                                            const uint16_t* __restrict__ dy, int64_t ld_dy,
                                                            const uint16_t* __restrict__ z, int64_t ld_z,
                                                            const int32_t* __restrict__ rows,
                                                            float* __restrict__ dweights) {
  __shared__ float part[kWaves][kMaxK];
  const uint32_t lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t t = blockIdx.x;
  for (int i0 = 0; i0 < k; i0 += kBatch) {
    float acc[kBatch] = {};
    int32_t r[kBatch];
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      r[i] = i0 + i < k ? rows[t * k + i0 + i] : -1;
      if (r[i] >= R) r[i] = -1;
    }
    for (int64_t c = wave * 512 + lane * 8; c < H; c += kWaves * 512) {
      const u32x4 d = *reinterpret_cast<const u32x4*>(dy + t * ld_dy + c);
      u32x4 v[kBatch];
#pragma unroll
      for (int i = 0; i < kBatch; ++i)
        v[i] = r[i] >= 0 ? *reinterpret_cast<const u32x4*>(z + (int64_t)r[i] * ld_z + c) : u32x4{0, 0, 0, 0};
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        if (r[i] < 0) continue;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          acc[i] = __builtin_fmaf(bf16_lo(d[j]), bf16_lo(v[i][j]), acc[i]);
          acc[i] = __builtin_fmaf(bf16_hi(d[j]), bf16_hi(v[i][j]), acc[i]);
        }
      }
    }
    const float mine = sums8(acc, lane);
    if ((int)lane < kBatch && i0 + (int)lane < k) part[wave][i0 + lane] = mine;
  }
  __syncthreads();
  if (threadIdx.x < (uint32_t)k) {
    float sum = 0.0f;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) sum += part[w][threadIdx.x];
    dweights[t * k + threadIdx.x] = sum;
  }
}

template <class S, bool W, bool NT>
hipError_t gather_as(const GatherArgs& a, hipStream_t stream) {
  if (a.qT.q) {
    TileGrid g = tile_grid(a.R, a.H);
    const uint32_t mine = g.col_tiles % 8 == 0 && a.k > 1 && a.T * a.H * 2 / 8 <= kSliceL2 ? g.col_tiles / 8 : 0;
    if (mine) g.workgroups = g.row_tiles * g.col_tiles;
    hipLaunchKernelGGL((gather_both_kernel<S, W, NT>), dim3(g.workgroups), dim3(kTileThreads), 0, stream, a, g, mine);
  } else {
    const int64_t parts = (a.H + kRowCols - 1) / kRowCols, per = kThreads / 64;
    int64_t run, waves;
    if (a.order) {
      run = order_run(a.R);
      waves = ((a.R + 2 * run - 1) / (2 * run) + 7) / 8 * 2 * parts;  // of an XCD
      waves = (waves + per - 1) / per * per * 8;
      int shift = 0;
      while (((a.T * a.k - 1) >> shift) >= kOrderRanges) ++shift;
      hipLaunchKernelGGL(gather_order_kernel, dim3(kOrderBlocks), dim3(kOrderThreads), 0, stream, a, (uint32_t)(2 * run), shift);
      if (hipError_t e = hipGetLastError()) return e;
    } else {
      // as many rows a wave as leave 8192 waves, which fill the GPU
      const int64_t most = a.R * parts / 8192;
      run = most < 1 ? 1 : most < kMaxRun ? most : kMaxRun;
      waves = (a.R + run - 1) / run * parts;
    }
    hipLaunchKernelGGL((gather_rows_kernel<S, W, NT>), dim3((uint32_t)((waves + per - 1) / per)), dim3(kThreads), 0,
                       stream, a, (uint32_t)run, (uint32_t)parts);
  }
  return hipGetLastError();
}

template <class S, bool W>
hipError_t gather(const GatherArgs& a, hipStream_t stream) {
  return a.R * a.H * (a.qT.q ? 2 : 1) > kStoreNt ? gather_as<S, W, true>(a, stream) : gather_as<S, W, false>(a, stream);
}

}  // namespace

hipError_t launch_moe_gather(const GatherArgs& a, hipStream_t stream) {
  if (a.weights) return a.fp32_scale ? gather<Fp32Scale, true>(a, stream) : gather<Pow2Scale, true>(a, stream);
  return a.fp32_scale ? gather<Fp32Scale, false>(a, stream) : gather<Pow2Scale, false>(a, stream);
}

hipError_t launch_moe_combine(int64_t T, int64_t H, int64_t R, int k, const uint16_t* z, int64_t ld_z,
                              const int32_t* rows, const float* weights, RowsOut out, hipStream_t stream) {
  const uint32_t parts = (uint32_t)((H + 511) / 512);
  const int64_t waves = T * parts, per = kThreads / 64;
  hipLaunchKernelGGL(combine_kernel, dim3((uint32_t)((waves + per - 1) / per)), dim3(kThreads), 0, stream, T, H, R, k,
                     z, ld_z, rows, weights, out, parts);
  return hipGetLastError();
}

hipError_t launch_moe_combine_dweights(int64_t T, int64_t H, int64_t R, int k, const uint16_t* dy, int64_t ld_dy,
                                       const uint16_t* z, int64_t ld_z, const int32_t* rows, float* dweights,
                                       hipStream_t stream) {
  hipLaunchKernelGGL(dweights_kernel, dim3((uint32_t)T), dim3(kThreads), 0, stream, T, H, R, k, dy, ld_dy, z, ld_z,
                     rows, dweights);
  return hipGetLastError();
}

}  // namespace fp8blk
