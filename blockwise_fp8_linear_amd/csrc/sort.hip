// Tokens sorted by expert (include/fp8train.h, fp8_moe_sort): a stable counting
// sort of the choices ids[c], c < n = T k, into segments of whole 128 rows.
//
//   count_e = |{c : ids[c] = e}|,  offsets_e = sum over e' < e of up128(count_e'),
//   rows[c] = offsets_e + |{c' < c : ids[c'] = e}|,  e = ids[c].
//
// Moves 12 bytes a choice, so it is bound by latency: few launches, each a few
// dependent steps long.  A wave finds which of its 64 lanes hold the same expert
// by one ballot per bit of the id, which gives every lane its rank among them and
// one lane the count -- no atomics, so the order is fixed.  The waves of a
// workgroup leave their counts in LDS, where a thread per expert turns them into
// the waves' first rows.  Up to kSortAloneRounds rounds of 1024 choices one
// workgroup does it all in one launch; beyond, the workgroups count in a first
// launch, and in the second each adds up the others' counts for itself.  14 choices of
// 8 experts 4.0 us, 131072 of 128 5.1 and 7.8.
#include "fp8blk_device.h"
#include "fp8train_launch.h"

namespace fp8blk {

namespace {

constexpr int kThreads = (int)kSortRound, kWaves = kThreads / 64;
constexpr int kMaxE = 1024;
static_assert(kThreads >= kMaxE, "a thread per expert");

// The lanes of the wave that hold the same id as this one (ids below 2^bits).
__device__ __forceinline__ uint64_t same_lanes(uint32_t id, int bits) {
  uint64_t m = ~uint64_t(0);
  for (int b = 0; b < bits; ++b) {
    const bool bit = (id >> b) & 1;
    const uint64_t set = __ballot(bit);
    m &= bit ? set : ~set;
  }
  return m;
}

// Choice c's expert; E for none.
__device__ __forceinline__ uint32_t expert_of(const int32_t* __restrict__ ids, int64_t c, int64_t n, int E) {
  const int32_t id = c < n ? ids[c] : -1;
  return id >= 0 && id < E ? (uint32_t)id : (uint32_t)E;
}

// Sum of the lanes before this one, over the wave.
__device__ __forceinline__ int32_t wave_before(int32_t v, uint32_t lane) {
  int32_t s = v;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int32_t o = __shfl_up(s, d, 64);
    if ((int)lane >= d) s += o;
  }
  return s - v;
}

// counts[block][e]: how many choices of the block's rounds are expert e's.
__global__ __launch_bounds__(kThreads) void sort_count_kernel(int64_t n, int E, int bits, int rounds,
                                                              const int32_t* __restrict__ ids,
                                                              int32_t* __restrict__ counts) {
  __shared__ int32_t wave_count[kWaves][kMaxE];
  const uint32_t t = threadIdx.x, lane = t & 63, wave = t >> 6;
  for (int e = lane; e < E; e += 64) wave_count[wave][e] = 0;
  __builtin_amdgcn_wave_barrier();
  const int64_t c0 = (int64_t)blockIdx.x * rounds * kThreads;
  for (int r = 0; r < rounds; ++r) {
    const uint32_t e = expert_of(ids, c0 + (int64_t)r * kThreads + t, n, E);
    const uint64_t same = same_lanes(e, bits);
    // the lowest of the lanes adds for all of them; a wave's counts are its own
    if (e < (uint32_t)E && (uint32_t)__builtin_ctzll(same) == lane) wave_count[wave][e] += (int32_t)__popcll(same);
    __builtin_amdgcn_wave_barrier();
  }
  __syncthreads();
  if (t < (uint32_t)E) {
    int32_t sum = 0;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) sum += wave_count[w][t];
    counts[(int64_t)blockIdx.x * E + t] = sum;
  }
}

// ALONE: the only workgroup, which counts for itself.
template <bool ALONE>
__global__ __launch_bounds__(kThreads) void sort_place_kernel(int64_t n, int E, int bits, int rounds, int64_t R,
                                                              const int32_t* __restrict__ ids,
                                                              const int32_t* __restrict__ counts,
                                                              int32_t* __restrict__ rows, int32_t* __restrict__ source,
                                                              int32_t* __restrict__ offsets) {
  __shared__ int32_t wave_count[kWaves][kMaxE];  // of a round; then the wave's first row of each expert
  const uint32_t t = threadIdx.x, lane = t & 63, wave = t >> 6;
  const int64_t c0 = (int64_t)blockIdx.x * rounds * kThreads;
  int32_t total = 0, before = 0;  // of expert t: all choices, those of earlier workgroups
  if constexpr (ALONE) {
    for (int e = lane; e < E; e += 64) wave_count[wave][e] = 0;
    __builtin_amdgcn_wave_barrier();
    for (int r = 0; r < rounds; ++r) {
      const uint32_t e = expert_of(ids, (int64_t)r * kThreads + t, n, E);
      const uint64_t same = same_lanes(e, bits);
      if (e < (uint32_t)E && (uint32_t)__builtin_ctzll(same) == lane) wave_count[wave][e] += (int32_t)__popcll(same);
      __builtin_amdgcn_wave_barrier();
    }
    __syncthreads();
    if (t < (uint32_t)E) {
#pragma unroll
      for (int w = 0; w < kWaves; ++w) total += wave_count[w][t];
    }
  } else {
    // each expert's counts, added up by as many threads as there are for it
    const uint32_t parts = (uint32_t)kThreads / (uint32_t)E;
    int32_t* const part_total = &wave_count[0][0];             // [parts][E], parts * E <= kThreads
    int32_t* const part_before = &wave_count[kWaves / 2][0];
    const uint32_t part = t / (uint32_t)E, e = t - part * (uint32_t)E;
    if (part < parts) {
      int32_t all = 0, mine = 0;
      // eight on the way at a time
      for (uint32_t b0 = part; b0 < gridDim.x; b0 += 8 * parts) {
        int32_t v[8];
#pragma unroll
        for (uint32_t u = 0; u < 8; ++u) {
          const uint32_t b = b0 + u * parts;
          v[u] = b < gridDim.x ? counts[(int64_t)b * E + e] : 0;
        }
#pragma unroll
        for (uint32_t u = 0; u < 8; ++u) {
          all += v[u];
          mine += b0 + u * parts < blockIdx.x ? v[u] : 0;
        }
      }
      part_total[part * E + e] = all;
      part_before[part * E + e] = mine;
    }
    __syncthreads();
    if (t < (uint32_t)E) {
      for (uint32_t p = 0; p < parts; ++p) {
        total += part_total[p * E + t];
        before += part_before[p * E + t];
      }
    }
  }
  // offsets: the segments' lengths, summed over the experts before
  const int32_t length = t < (uint32_t)E ? (total + 127) & ~127 : 0;
  int32_t at = wave_before(length, lane);
  __syncthreads();  // the counts have been read
  int32_t* const wave_sum = &wave_count[0][0];
  if (lane == 63) wave_sum[wave] = at + length;
  __syncthreads();
  for (uint32_t w = 0; w < wave; ++w) at += wave_sum[w];
  int32_t end = 0;  // of all segments
#pragma unroll
  for (int w = 0; w < kWaves; ++w) end += wave_sum[w];
  if (t < (uint32_t)E) {
    if (blockIdx.x == 0) {
      offsets[t] = at;
      if (t == (uint32_t)E - 1) offsets[E] = end;
    }
  }
  // padding: an expert's by one wave of one workgroup
  __syncthreads();  // wave_sum has been read
  int32_t* const pad_from = &wave_count[0][0];
  int32_t* const pad_to = &wave_count[kWaves / 2][0];
  if (t < (uint32_t)E) {
    pad_from[t] = at + total;
    pad_to[t] = at + length;
  }
  __syncthreads();
  for (uint32_t e = blockIdx.x + wave * gridDim.x; e < (uint32_t)E; e += kWaves * gridDim.x)
    for (int32_t r = pad_from[e] + (int32_t)lane; r < pad_to[e]; r += 64) source[r] = -1;
  for (int64_t r = end + (int64_t)blockIdx.x * kThreads + t; r < R; r += (int64_t)gridDim.x * kThreads) source[r] = -1;

  int32_t next = at + before;  // the row of expert t's next choice
  for (int r = 0; r < rounds; ++r) {
    const int64_t c = c0 + (int64_t)r * kThreads + t;
    const uint32_t e = expert_of(ids, c, n, E);
    const uint64_t same = same_lanes(e, bits);
    __syncthreads();  // the round before is done with the counts
    for (int i = lane; i < E; i += 64) wave_count[wave][i] = 0;
    __builtin_amdgcn_wave_barrier();
    if (e < (uint32_t)E && (uint32_t)__builtin_ctzll(same) == lane) wave_count[wave][e] = (int32_t)__popcll(same);
    __syncthreads();
    if (t < (uint32_t)E) {
#pragma unroll
      for (int w = 0; w < kWaves; ++w) {
        const int32_t v = wave_count[w][t];
        wave_count[w][t] = next;
        next += v;
      }
    }
    __syncthreads();
    if (c < n) {
      int32_t row = -1;
      if (e < (uint32_t)E) {
        row = wave_count[wave][e] + (int32_t)__popcll(same & ((uint64_t(1) << lane) - 1));
        source[row] = (int32_t)c;
      }
      rows[c] = row;
    }
  }
}

}  // namespace

hipError_t launch_moe_sort(int64_t n, int E, int64_t R, const int32_t* ids, int32_t* rows, int32_t* source,
                           int32_t* offsets, int32_t* counts, hipStream_t stream) {
  const SortPlan p = sort_plan(n);
  int bits = 1;
  while ((1 << bits) <= E) ++bits;  // ids 0 .. E, E for none
  const dim3 grid((uint32_t)p.blocks), block(kThreads);
  if (p.blocks == 1) {
    hipLaunchKernelGGL(sort_place_kernel<true>, grid, block, 0, stream, n, E, bits, (int)p.rounds, R, ids, counts, rows,
                       source, offsets);
    return hipGetLastError();
  }
  hipLaunchKernelGGL(sort_count_kernel, grid, block, 0, stream, n, E, bits, (int)p.rounds, ids, counts);
  if (hipError_t e = hipGetLastError()) return e;
  hipLaunchKernelGGL(sort_place_kernel<false>, grid, block, 0, stream, n, E, bits, (int)p.rounds, R, ids, counts, rows,
                     source, offsets);
  return hipGetLastError();
}

}  // namespace fp8blk
