// Which tile of which expert: the map that the grouped GEMM kernels (gemm.hip,
// gemm_mx.hip) make for themselves from the segments' offsets, so that nothing
// about the experts' loads has to be known on the host.  It stands in front of
// every workgroup's first load, so it is one round of loads, one scan in 32 bits
// and a search in LDS.
#pragma once

#include "fp8blk_device.h"
#include "fp8train_launch.h"

namespace fp8blk {

constexpr int kGroupedMaxE = 1024;

// An offset as a whole multiple of 128 inside [0, rows], whatever it holds.
__device__ __forceinline__ int32_t segment_edge(int32_t offset, int32_t rows) {
  return (offset < 0 ? 0 : offset < rows ? offset : rows) & ~127;
}

struct Segment {
  int32_t first, length;
};
__device__ __forceinline__ Segment segment_between(int32_t lo, int32_t hi) { return {lo, hi > lo ? hi - lo : 0}; }
__device__ __forceinline__ Segment segment_of(const int32_t* __restrict__ offsets, int e, int32_t rows) {
  return segment_between(segment_edge(offsets[e], rows), segment_edge(offsets[e + 1], rows));
}

// starts[e]: the first row tile of expert e's, starts[E] how many there are.
struct GroupedMap {
  uint32_t starts[kGroupedMaxE + 1];
  int32_t edges[kGroupedMaxE + 1];
  uint32_t wave[16];
};

// Fills the map for tiles of TILE rows.  Every thread of a workgroup of THREADS
// calls it; ends with a barrier.
template <int THREADS, int TILE>
__device__ __forceinline__ void grouped_map(GroupedMap& lds, const int32_t* __restrict__ offsets, int E, int32_t rows) {
  constexpr int PER = kGroupedMaxE / THREADS;
  const uint32_t t = threadIdx.x, lane = t & 63, wave = t >> 6;
  int32_t edge[PER + 1];
#pragma unroll
  for (int i = 0; i <= PER; ++i) {
    const int e = (int)t * PER + i;
    edge[i] = e <= E ? segment_edge(offsets[e], rows) : 0;
  }
  uint32_t n[PER], sum = 0;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int e = (int)t * PER + i;
    n[i] = sum;
    if (e < E) sum += (uint32_t)(segment_between(edge[i], edge[i + 1]).length + TILE - 1) / TILE;
    if (e <= E) lds.edges[e] = edge[i];
  }
  if (t == THREADS - 1 && E == kGroupedMaxE) lds.edges[E] = edge[PER];
  uint32_t upto = sum;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const uint32_t o = (uint32_t)__shfl_up((int)upto, d, 64);
    if ((int)lane >= d) upto += o;
  }
  if (lane == 63) lds.wave[wave] = upto;
  __syncthreads();
  uint32_t before = upto - sum;
#pragma unroll
  for (uint32_t w = 0; w + 1 < THREADS / 64; ++w) before += w < wave ? lds.wave[w] : 0;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int e = (int)t * PER + i;
    if (e <= E) lds.starts[e] = before + n[i];
  }
  if (t == THREADS - 1 && E == kGroupedMaxE) lds.starts[E] = before + sum;
  __syncthreads();
}

// The expert of a row tile below starts[E]: the last one that starts at or before
// it (so one that has any).
__device__ __forceinline__ int expert_of_tile(const GroupedMap& lds, int E, uint32_t tile) {
  int lo = 0, hi = E;
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (lds.starts[mid] <= tile) lo = mid;
    else hi = mid;
  }
  return __builtin_amdgcn_readfirstlane(lo);
}

// The tiles of one workgroup: at, at + step, ... below end.  How many there are is known on the device alone, so the
// XCDs (which get the workgroups in turn) have a run of tiles each by that count:
// by the grid, the last XCDs would have none.  The grid is a multiple of 8.
struct TileRun {
  uint32_t at, end, step;
};
__device__ __forceinline__ TileRun tile_run(uint32_t total) {
  const uint32_t xcd = blockIdx.x % 8, per = (total + 7) / 8, first = xcd * per;
  const uint32_t end = total < first ? first : total - first < per ? total : first + per;
  return {first + blockIdx.x / 8, end, gridDim.x / 8};
}
inline uint32_t grouped_grid(int64_t tiles, int64_t most) {  // up to `most`, a multiple of 8
  return (uint32_t)(tiles < most ? (tiles + 7) / 8 * 8 : most);
}

// Tile `in` of a segment's (or an expert's) tiles_m x tiles_n -> its row and
// column of tiles: down a group of GM tile rows before moving right, as the dense
// kernels go, so that tiles in flight together share operand panels in L2.
struct TileAt {
  uint32_t m, n;
};
template <int GM>
__device__ __forceinline__ TileAt tile_at(uint32_t in, uint32_t tiles_m, uint32_t tiles_n) {
  const uint32_t group = in / (GM * tiles_n), first = group * GM;
  const uint32_t size = tiles_m - first < GM ? tiles_m - first : GM, rest = in - first * tiles_n, n = rest / size;
  return {first + (rest - n * size), n};
}

// Output element i of a matrix of fp32 or bf16.
__device__ __forceinline__ void* element(void* out, int64_t i, bool f32) {
  return f32 ? (void*)(static_cast<float*>(out) + i) : (void*)(static_cast<uint16_t*>(out) + i);
}

// The contraction of one expert's segment: rows (Fprop, Dgrad).
__device__ __forceinline__ GemmArgs expert_rows(const GroupedArgs& a, int e, Segment s) {
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
