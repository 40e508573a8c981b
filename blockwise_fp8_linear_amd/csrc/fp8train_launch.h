// Internal launch entry points of the operators declared in include/fp8train.h.
// Arguments are validated by the C ABI layer (api_train.cpp) before any of these
// is called.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "fp8blk_launch.h"
#include "fp8moe_launch.h"

namespace fp8blk {

// The workgroups that a sort's choices are dealt to, each a run of whole rounds
// of kSortRound; one counts for itself, more leave their counts in the workspace.
constexpr int64_t kSortRound = 1024, kSortMaxBlocks = 256, kSortAloneRounds = 4;
struct SortPlan {
  int64_t blocks, rounds;
};
inline SortPlan sort_plan(int64_t n) {
  const int64_t all = (n + kSortRound - 1) / kSortRound;
  if (all <= kSortAloneRounds) return {1, all};
  const int64_t rounds = (all + kSortMaxBlocks - 1) / kSortMaxBlocks;
  return {(all + rounds - 1) / rounds, rounds};
}

hipError_t launch_moe_sort(int64_t n, int E, int64_t R, const int32_t* ids, int32_t* rows, int32_t* source,
                           int32_t* offsets, int32_t* counts, hipStream_t stream);

// Codes in one orientation: where they go (null: not wanted) and their scales.
struct CodesOut {
  uint8_t* q;
  int64_t ld;
  float* s;
};

// weights may be null, used may be null (all rows); qT.q null: row groups only.
struct GatherArgs {
  int64_t T, H, R;
  int k;
  const uint16_t* x;
  int64_t ld_x;
  const int32_t* source;
  const float* weights;
  const int32_t* used;
  CodesOut q, qT;
  bool fp32_scale;
  uint32_t* order;  // the workspace of gather_order_bytes(), or null where that is 0
};
// Row groups of many rows are gathered in the order of their tokens, in runs of a
// few rows, which a first launch finds in 6 to 9 us: where x outgrows two XCDs' L2 and
// the rows' second and further reads of it come to kOrderReread (8192 tokens, 2048
// wide, to 4 experts each, 117 MB: 38 us, unordered 33; to 8, 252 MB: 39 and 59).
constexpr int64_t kOrderReread = int64_t(160) << 20;
// Runs are ordered in pairs (one by one: 18432 instead of 9216 to look at, 12.5 us and 9).
constexpr int64_t kOrderPairs = 16384;
inline int64_t order_run(int64_t R) {
  const int64_t least = (R + 2 * kOrderPairs - 1) / (2 * kOrderPairs);
  return least <= 4 ? 4 : (least + 7) / 8 * 8;
}
inline bool gather_ordered(int64_t T, int64_t H, int64_t R, int k, bool both) {
  return !both && k > 1 && T * H * 2 > (int64_t(8) << 20) && R >= 2 * T && (R - T) * H * 2 > kOrderReread &&
         order_run(R) <= 64;
}
inline size_t gather_order_bytes(int64_t T, int64_t H, int64_t R, int k, bool both) {
  const int64_t pair = 2 * order_run(R);
  return gather_ordered(T, H, R, k, both) ? (size_t)((R + pair - 1) / pair) * sizeof(uint32_t) : 0;
}
hipError_t launch_moe_gather(const GatherArgs& a, hipStream_t stream);

hipError_t launch_moe_combine(int64_t T, int64_t H, int64_t R, int k, const uint16_t* z, int64_t ld_z,
                              const int32_t* rows, const float* weights, RowsOut out, hipStream_t stream);
hipError_t launch_moe_combine_dweights(int64_t T, int64_t H, int64_t R, int k, const uint16_t* dy, int64_t ld_dy,
                                       const uint16_t* z, int64_t ld_z, const int32_t* rows, float* dweights,
                                       hipStream_t stream);

// qc.q may be null.
hipError_t launch_gated_forward(int64_t M, int64_t I, const uint16_t* gu, int64_t ld_gu, const int32_t* used,
                                CodesOut q, CodesOut qc, bool fp32_scale, hipStream_t stream);
hipError_t launch_gated_backward(int64_t M, int64_t I, const uint16_t* dh, int64_t ld_dh, const uint8_t* qc,
                                 int64_t ld_qc, const float* sc, const int32_t* used, CodesOut q, CodesOut qT,
                                 CodesOut qhT, bool fp32_scale, hipStream_t stream);
hipError_t launch_requantize_colgroup(const uint8_t* q, int64_t rows, int64_t cols, int64_t ld_q, const float* s,
                                      const int32_t* used, CodesOut qT, bool fp32_scale, hipStream_t stream);

// Rows of a grouped product: below it an expert has fewer than 2^22 tiles of 128 rows,
// and 1024 of them, whatever the offsets hold, fewer than 2^32.
constexpr int64_t kGroupedMaxRows = int64_t(1) << 29;

// Every expert's contraction: a GemmArgs whose rows (Wgrad: reduction) are cut
// into the experts' segments; b and sb (Wgrad: out) are expert 0's.
struct GroupedArgs {
  GemmArgs g;
  const int32_t* offsets;  // [E + 1]
  int64_t E;
  int64_t b_stride, sb_stride, out_stride;  // from one expert to the next
};
hipError_t launch_grouped_rows(const GroupedArgs& a, GemmAlgo algo, hipStream_t stream);   // Fprop, Dgrad
hipError_t launch_grouped_wgrad(const GroupedArgs& a, GemmAlgo algo, hipStream_t stream);
// On the block-scaled MFMA, tiles of 256x256: Fprop and Dgrad (gemm_mx.hip) where
// gemm_mx_eligible and up to 2^22 columns; Wgrad (grouped_wgrad.hip) up to 2^22 rows,
// whole groups of four 128-blocks, their scales 16-byte aligned.
hipError_t launch_grouped_rows_mx(const GroupedArgs& a, hipStream_t stream);
hipError_t launch_grouped_wgrad_mx(const GroupedArgs& a, hipStream_t stream);

// Wgrad's times on the two kernels, in quarters of a us, if every segment is as long
// as the mean one, of b blocks.  On tiles of 256 x 256, one workgroup a CU: a tile takes
// 2 b + 4.5 us, a workgroup 5 until its first loads are there; each: the tiles a
// workgroup takes, those that end first, up to kWgradEach, so that what the longest
// segments leave is taken by others (16 measured the same).  On tiles of 128 x 128 (in
// gemm.hip), two a CU: 3 + 1.25 b us for both.  (294 rows of 11 experts, 1280 x 1152:
// 18 us on the large tiles, 12 on the small ones; 2400 of 64, 2048 x 2048: 120 and
// 141; 65536 of 64: 386 and 593.)
constexpr int64_t kWgradEach = 8;
struct WgradPlan {
  int64_t each, large, small;
};
inline WgradPlan wgrad_plan(const GroupedArgs& a) {
  const int64_t cus = 256, tile = 8 * (a.g.R / 128) / a.E + 18;
  const int64_t tiles = a.E * ((a.g.I + 255) / 256) * ((a.g.J + 255) / 256), tiles128 = a.E * (a.g.I / 128) * (a.g.J / 128);
  WgradPlan p{1, INT64_MAX, (tiles128 + 2 * cus - 1) / (2 * cus) * (12 + 5 * (a.g.R / 128) / a.E)};
  for (int64_t n = 1; n <= kWgradEach; ++n) {
    const int64_t rounds = ((tiles + n - 1) / n + cus - 1) / cus, time = rounds * (n * tile + 20);
    if (time <= p.large) p.large = time, p.each = n;
  }
  return p;
}

// Which kernel: tiles of 256 x 256 (Large), of 128 x 128, or of 64 x 128 (Few).
enum class GroupedTiles { Large, Small, Few };
inline GroupedTiles grouped_rows_tiles(const GroupedArgs& a, GemmAlgo algo) {
  // no more than a tile of 128 x 128 a CU, whatever the segments
  if ((a.g.I / 128 + a.E) * (a.g.J / 128) <= 256) return GroupedTiles::Few;
  // the large tiles take whole groups of four 128-blocks (others on them, their scales
  // one by one, were 53 us where the small tiles take 48, 73 and 39, 59 and 47); per-lane
  // 32-bit offsets of 128 rows
  return algo == GemmAlgo::ScaledMfma && gemm_mx_eligible(a.g) && a.g.J <= (int64_t(1) << 22) ? GroupedTiles::Large
                                                                                            : GroupedTiles::Small;
}
inline GroupedTiles grouped_wgrad_tiles(const GroupedArgs& a, GemmAlgo algo) {
  // the large tiles take scales in 16-byte groups of four, per-lane 32-bit offsets of 256
  // rows of R bytes
  const auto quads = [](const float* s) { return reinterpret_cast<uintptr_t>(s) % 16 == 0; };
  if (algo != GemmAlgo::ScaledMfma || a.g.R > (int64_t(1) << 22) || a.g.R % 512 != 0 || !quads(a.g.sa) || !quads(a.g.sb))
    return GroupedTiles::Small;
  const WgradPlan p = wgrad_plan(a);
  return p.large <= p.small ? GroupedTiles::Large : GroupedTiles::Small;
}

}  // namespace fp8blk
