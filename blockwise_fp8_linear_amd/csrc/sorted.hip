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

// Eight values of sorted row r, from column c on: zeros where the row has no
// choice of its own.
template <bool W>
__device__ __forceinline__ u32x4 gathered(const GatherArgs& a, int32_t src, int64_t n, int64_t c) {
  if (src < 0 || src >= n) return u32x4{0, 0, 0, 0};
  u32x4 v = *reinterpret_cast<const u32x4*>(a.x + (int64_t)((uint32_t)src / (uint32_t)a.k) * a.ld_x + c);
  if constexpr (W) {
    const float w = a.weights[src];
    v = u32x4{scaled2(v.x, w), scaled2(v.y, w), scaled2(v.z, w), scaled2(v.w, w)};
  }
  return v;
}

// ---------------------------------------------------------------------------
// Row groups only: 16 lanes to a group, four rows' groups a wave and step.
// ---------------------------------------------------------------------------
constexpr int kRowUnroll = 4;
constexpr int kGroupsPerWave = 4 * kRowUnroll;

template <class S, bool W>
__global__ __launch_bounds__(kThreads) void gather_rows_kernel(GatherArgs a) {
  const uint32_t lane = threadIdx.x & 63, sub = lane >> 4, l16 = lane & 15;
  const uint32_t G = (uint32_t)(a.H / 128);
  const uint32_t rows = (uint32_t)used_tiles(a.used, a.R) * 128, total = rows * G;
  const uint32_t g0 = (blockIdx.x * (kThreads / 64) + (threadIdx.x >> 6)) * kGroupsPerWave;
  if (g0 >= total) return;
  const int64_t n = a.T * a.k;
  u32x4 v[kRowUnroll];
  uint32_t row[kRowUnroll], grp[kRowUnroll];
  int32_t src[kRowUnroll];
#pragma unroll
  for (int u = 0; u < kRowUnroll; ++u) {
    const uint32_t g = g0 + u * 4 + sub, gg = g < total ? g : 0;
    row[u] = gg / G;
    grp[u] = gg - row[u] * G;
    src[u] = a.source[row[u]];
  }
#pragma unroll
  for (int u = 0; u < kRowUnroll; ++u) v[u] = gathered<W>(a, src[u], n, grp[u] * 128 + l16 * 8);
#pragma unroll
  for (int u = 0; u < kRowUnroll; ++u) {
    uint32_t m = pk_max_u16(pk_max_u16(abs2(v[u].x), abs2(v[u].y)), pk_max_u16(abs2(v[u].z), abs2(v[u].w)));
    m = row16_max(max(m & 0xFFFFu, m >> 16));
    const S sc(m);
    uint2 o;
    o.x = quant4(v[u].x, v[u].y, sc);
    o.y = quant4(v[u].z, v[u].w, sc);
    if (g0 + u * 4 + sub < total) {
      *reinterpret_cast<uint2*>(a.q.q + (int64_t)row[u] * a.q.ld + grp[u] * 128 + l16 * 8) = o;
      if (l16 == 0) a.q.s[(int64_t)row[u] * G + grp[u]] = sc.s;
    }
  }
}

// ---------------------------------------------------------------------------
// Both orientations: a 128 x 128 tile a workgroup, as the one-pass quantizer.
// ---------------------------------------------------------------------------
template <class S, bool W>
__global__ __launch_bounds__(kTileThreads) void gather_both_kernel(GatherArgs a, uint32_t row_tiles,
                                                                   uint32_t col_tiles) {
  __shared__ TileLds lds;
  uint32_t rt, ct;
  tile_of(blockIdx.x, col_tiles, false, rt, ct);
  if (rt >= used_tiles(a.used, a.R)) return;
  const uint32_t rb = threadIdx.x >> 4, cb = threadIdx.x & 15;
  const int64_t m0 = (int64_t)rt * 128, c0 = (int64_t)ct * 128, n = a.T * a.k;
  int32_t src[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) src[i] = a.source[m0 + rb * 8 + i];
  u32x4 v[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = gathered<W>(a, src[i], n, c0 + cb * 8);
  tile_row_groups<S>(v, a.q.q + m0 * a.q.ld + c0 + cb * 8, a.q.ld, a.q.s + m0 * col_tiles + ct, col_tiles, rb, cb);
  tile_col_groups<S>(v, lds, a.qT.q + c0 * a.qT.ld + m0, a.qT.ld, a.qT.s + c0 * row_tiles + rt, row_tiles, rb, cb);
}

// ---------------------------------------------------------------------------
// Back to the tokens.  A wave takes 512 columns of a token, 16 bytes of each of
// its rows a lane; the rows are loaded kBatch at a time.
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

// A workgroup takes a token: its waves share the columns, 512 at a time, and
// their sums meet in LDS, in wave order.  Each of the k sums is a lane's, then
// the wave's, then the workgroup's, in an order that H alone decides.
constexpr int kMaxK = 16;

__global__ __launch_bounds__(kThreads) void dweights_kernel(int64_t H, int64_t R, int k,
                                                            const uint16_t* __restrict__ dy, int64_t ld_dy,
                                                            const uint16_t* __restrict__ z, int64_t ld_z,
                                                            const int32_t* __restrict__ rows,
                                                            float* __restrict__ dweights) {
  __shared__ float part[kThreads / 64][kMaxK];
  const uint32_t lane = threadIdx.x & 63;
  const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t t = blockIdx.x;
  for (int i0 = 0; i0 < k; i0 += kBatch) {
    float acc[kBatch] = {};
    int32_t r[kBatch];
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      r[i] = i0 + i < k ? rows[t * k + i0 + i] : -1;
      if (r[i] >= R) r[i] = -1;
    }
    for (int64_t c = wave * 512 + lane * 8; c < H; c += (kThreads / 64) * 512) {
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
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
#pragma unroll
      for (int d = 1; d < 64; d <<= 1) acc[i] += __shfl_xor(acc[i], d, 64);
      if (lane == 0 && i0 + i < k) part[wave][i0 + i] = acc[i];
    }
  }
  __syncthreads();
  if (threadIdx.x < (uint32_t)k) {
    float sum = 0.0f;
#pragma unroll
    for (int w = 0; w < kThreads / 64; ++w) sum += part[w][threadIdx.x];
    dweights[t * k + threadIdx.x] = sum;
  }
}

template <class S, bool W>
hipError_t gather(const GatherArgs& a, hipStream_t stream) {
  const uint32_t row_tiles = (uint32_t)(a.R / 128), col_tiles = (uint32_t)(a.H / 128);
  if (a.qT.q) {
    hipLaunchKernelGGL((gather_both_kernel<S, W>), dim3(row_tiles * col_tiles), dim3(kTileThreads), 0, stream, a,
                       row_tiles, col_tiles);
  } else {
    const uint32_t groups = (uint32_t)a.R * col_tiles, per = kGroupsPerWave * (kThreads / 64);
    hipLaunchKernelGGL((gather_rows_kernel<S, W>), dim3((groups + per - 1) / per), dim3(kThreads), 0, stream, a);
  }
  return hipGetLastError();
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
  hipLaunchKernelGGL(dweights_kernel, dim3((uint32_t)T), dim3(kThreads), 0, stream, H, R, k, dy, ld_dy, z, ld_z, rows,
                     dweights);
  return hipGetLastError();
}

}  // namespace fp8blk
