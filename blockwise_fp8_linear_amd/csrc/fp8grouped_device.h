// Which tile of which expert: the map that the grouped GEMM kernels (gemm.hip,
// gemm_mx.hip) make for themselves from the segments' offsets, so that nothing
// about the experts' loads has to be known on the host.
#pragma once

#include "fp8blk_device.h"
#include "fp8train_launch.h"

namespace fp8blk {

constexpr int kGroupedMaxE = 1024;

// starts[e]: the first tile of expert e's, starts[E] how many there are.
struct GroupedLds {
  int64_t starts[kGroupedMaxE + 1];
  int64_t wave[16];
};

// Segment e's first row and length: whole 128s inside [0, rows], whatever the
// offsets hold.
struct Segment {
  int64_t first, length;
};
__device__ __forceinline__ int64_t segment_edge(const int32_t* __restrict__ offsets, int64_t e, int64_t rows) {
  const int64_t o = offsets[e];
  return (o < 0 ? 0 : o < rows ? o : rows) & ~int64_t(127);
}
__device__ __forceinline__ Segment segment_of(const int32_t* __restrict__ offsets, int64_t e, int64_t rows) {
  const int64_t lo = segment_edge(offsets, e, rows), hi = segment_edge(offsets, e + 1, rows);
  return {lo, hi > lo ? hi - lo : 0};
}

// Fills lds.starts for tiles of tile_rows rows x tiles_n columns.  Every thread
// of a workgroup of THREADS calls it; ends with a barrier.
template <int THREADS>
__device__ __forceinline__ void grouped_starts(GroupedLds& lds, const int32_t* __restrict__ offsets, int64_t E,
                                               int64_t rows, int64_t tile_rows, int64_t tiles_n) {
  constexpr int PER = kGroupedMaxE / THREADS;
  const uint32_t t = threadIdx.x, lane = t & 63, wave = t >> 6;
  int64_t n[PER], sum = 0;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int64_t e = (int64_t)t * PER + i;
    n[i] = sum;
    if (e < E) sum += (segment_of(offsets, e, rows).length + tile_rows - 1) / tile_rows * tiles_n;
  }
  int64_t upto = sum;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int64_t o = __shfl_up(upto, d, 64);
    if ((int)lane >= d) upto += o;
  }
  if (lane == 63) lds.wave[wave] = upto;
  __syncthreads();
  int64_t before = upto - sum;
  for (uint32_t w = 0; w < wave; ++w) before += lds.wave[w];
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int64_t e = (int64_t)t * PER + i;
    if (e <= E) lds.starts[e] = before + n[i];
  }
  if (t == THREADS - 1 && E == kGroupedMaxE) lds.starts[E] = before + sum;
  __syncthreads();
}

// The expert of a tile below starts[E]: the last one that starts at or before it
// and has any.
__device__ __forceinline__ int64_t expert_of_tile(const GroupedLds& lds, int64_t E, int64_t tile) {
  int64_t lo = 0, hi = E;
  while (hi - lo > 1) {
    const int64_t mid = (lo + hi) / 2;
    if (lds.starts[mid] <= tile) lo = mid;
    else hi = mid;
  }
  return lo;
}

// The expert whose segment is the at-th longest, equal ones by index: every thread
// of a workgroup calls it (which ends with a barrier).  Each counts the experts
// before its own, four a step, so it is for a few hundred at most.
constexpr int kGroupedOrderE = 256;
struct GroupedOrder {
  __attribute__((aligned(16))) int32_t blocks[kGroupedOrderE];  // of each expert; behind the last one -1
  int found;
};
__device__ __forceinline__ int expert_by_load(GroupedOrder& lds, const int32_t* __restrict__ offsets, int E,
                                              int64_t rows, int at) {
  typedef int v4i __attribute__((ext_vector_type(4)));
  const int e = threadIdx.x;
  const int mine = e < E ? (int)(segment_of(offsets, e, rows).length / 128) : -1;
  if (e < kGroupedOrderE) lds.blocks[e] = mine;
  __syncthreads();
  if (e < E) {
    int before = 0;
#pragma unroll 8
    for (int o = 0; o < E; o += 4) {
      const v4i b = *reinterpret_cast<const v4i*>(lds.blocks + o);
#pragma unroll
      for (int i = 0; i < 4; ++i) before += b[i] > mine || (b[i] == mine && o + i < e) ? 1 : 0;
    }
    if (before == at) lds.found = e;
  }
  __syncthreads();
  return lds.found;
}

// Output element i of a matrix of fp32 or bf16.
__device__ __forceinline__ void* element(void* out, int64_t i, bool f32) {
  return f32 ? (void*)(static_cast<float*>(out) + i) : (void*)(static_cast<uint16_t*>(out) + i);
}

// The contraction of one expert's segment: rows (Fprop, Dgrad).
__device__ __forceinline__ GemmArgs expert_rows(const GroupedArgs& a, int64_t e, Segment s) {
  GemmArgs g = a.g;
  g.a += s.first * g.R;
  g.sa += s.first * (g.R / 128);
  g.b += e * a.b_stride;
  g.sb += e * a.sb_stride;
  g.out = element(g.out, s.first * g.J, g.out_f32);
  g.I = s.length;
  return g;
}

}  // namespace fp8blk
