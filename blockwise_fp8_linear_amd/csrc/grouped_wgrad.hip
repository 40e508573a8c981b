// Every expert's Wgrad on the block-scaled MFMA (include/fp8train.h, power-of-two
// scales): dW_e[i][j] = sum over the 128-blocks b of e's segment of sa(i,b) sb(j,b)
// sum_r A[i][r] B[j][r].
//
// The tile is the dense kernel's (gemm_mx.hip): 256 x 256 of output by 4 waves of
// 128 x 128, one workgroup a CU, v_mfma_scale_f32_32x32x64_f8f6f4 on fragments from
// an LDS ring of two 128-deep pairs that direct loads fill.  But a segment is short
// -- some 8 blocks, where a dense reduction has 64 and more -- and what a tile takes
// besides its blocks (finding its expert, the first loads, the store) was half of
// the time with a tile a workgroup: 64 experts of 1024 rows each, 2048 x 2048, 552
// us.  So a workgroup takes several tiles, and its loads run through them without a
// pause: the last stages of a tile load the next one's first pairs, and its store,
// staged through 4 KiB a wave beside the ring, passes while they are on the way: 386
// us, 1.4 PFLOP/s, and 1.9 with 8 experts of 8192 rows.  What is left beyond the
// blocks is the store, 537 MB at memory's rate (fp32 instead of bf16: 455 us; added to
// what was there, whose loads wait for each other piece by piece: 614, of a floor of
// 416).
//
// The segments differ in length.  So that no XCD gets the long ones, and the last
// tiles to start are short, the experts come in the order of their loads and their
// tiles in runs (an XCD's 32 CUs share the panels of one run in L2), dealt to the
// XCDs back and forth; a workgroup's tiles are far apart in that order, so that
// workgroups have about the same work.
#include <atomic>

#include "fp8blk_device.h"
#include "fp8blk_launch.h"
#include "fp8blk_plan.h"
#include "fp8grouped_device.h"

namespace fp8blk {

namespace {

typedef int v8i __attribute__((ext_vector_type(8)));
typedef float v16f __attribute__((ext_vector_type(16)));

constexpr uint32_t TILE = (uint32_t)kMxTile, THREADS = 256;
constexpr int TM = 4, TN = 4;                    // 32 x 32 MFMA tiles of a wave
constexpr uint32_t PK = 128;                     // bytes of a row in a pair
constexpr uint32_t OPERAND = TILE * PK, SLOT = 2 * OPERAND;
// Scales come for four blocks at a time, 16 bytes a row -- one block's, 4 bytes from
// each of 512 rows, ask the L2 for as many lines as its codes do -- rows of A, then
// of B.
constexpr uint32_t SCALES = 2 * TILE * 16;
constexpr uint32_t AT_SCALES = 2 * SLOT, AT_STAGING = AT_SCALES + 2 * SCALES, STAGING = 4096;
constexpr uint32_t LDS_BYTES = AT_STAGING + (THREADS / 64) * STAGING;  // all 160 KiB
static_assert(LDS_BYTES <= 160 * 1024, "one workgroup's LDS");
constexpr int LOADS = (int)(OPERAND / 1024 / (THREADS / 64));  // of one operand's pair, 1 KiB a wave each

constexpr uint32_t RUN = 32;

// The experts in the order in which their tiles are taken: up to kOrderE longest
// first, equal ones by index; more of them as they come (finding the order takes each
// thread E steps).  The table is in registers, LDS being full: of the entries j 64 + l
// lane l holds the segment, in blocks, first and length in a half each, and the
// expert, in byte j.
constexpr int kOrderE = 256;
static_assert(THREADS >= kOrderE && kOrderE * 8 <= AT_STAGING, "a thread an expert; lengths and table in LDS at first");
struct Order {
  uint32_t segment[kOrderE / 64], expert;
};

__device__ __forceinline__ uint32_t packed(Segment s) {
  return (uint32_t)s.first / 128 | (uint32_t)s.length / 128 << 16;
}

__device__ __forceinline__ void make_order(Order& o, uint8_t* lds, const int32_t* __restrict__ offsets, int E,
                                           int32_t rows) {
  if (E > kOrderE) return;
  typedef int v4i __attribute__((ext_vector_type(4)));
  int32_t* const lengths = reinterpret_cast<int32_t*>(lds);  // behind the last expert -1
  uint32_t* const segment = reinterpret_cast<uint32_t*>(lds) + kOrderE;
  uint8_t* const expert = lds + 8 * kOrderE;
  const int e = (int)threadIdx.x;
  const Segment mine = e < E ? segment_of(offsets, e, rows) : Segment{0, -1};
  lengths[e] = mine.length;
  lds_barrier();
  if (e < E) {
    int before = 0;  // longer ones, and equal ones of a lower index, four a step
#pragma unroll 8
    for (int i = 0; i < E; i += 4) {
      const v4i l = *reinterpret_cast<const v4i*>(lengths + i);
#pragma unroll
      for (int j = 0; j < 4; ++j) before += l[j] > mine.length || (l[j] == mine.length && i + j < e) ? 1 : 0;
    }
    segment[before] = packed(mine);
    expert[before] = (uint8_t)e;
  }
  lds_barrier();
  o.expert = 0;
#pragma unroll
  for (int j = 0; j < kOrderE / 64; ++j) {
    const uint32_t at = j * 64 + (threadIdx.x & 63);
    o.segment[j] = segment[at];
    o.expert |= (uint32_t)expert[at] << (8 * j);
  }
  lds_barrier();  // the loads may come
}

// The workgroup's nth tile.
struct Found {
  bool any;  // there is one (and, if so, there may be another behind it)
  uint32_t first, length, expert;  // in blocks
  uint32_t i0, j0;
};
__device__ __forceinline__ Found find_tile(const Order& o, const int32_t* __restrict__ offsets, int32_t rows,
                                           uint32_t nth, uint32_t E, uint32_t tiles_m, uint32_t tiles_n) {
  const uint32_t v = nth * gridDim.x + blockIdx.x, xcd = v % 8, in = v / 8, turn = in / RUN;
  const uint32_t t = (turn * 8 + (turn & 1 ? 7 - xcd : xcd)) * RUN + in % RUN;
  const uint32_t tiles = tiles_m * tiles_n, at = __builtin_amdgcn_readfirstlane(t / tiles);
  if (at >= E) return {false, 0, 0, 0, 0, 0};
  const TileAt tile = tile_at<4>(t - at * tiles, tiles_m, tiles_n);
  uint32_t seg, expert = at;
  if (E <= (uint32_t)kOrderE) {
    const uint32_t j = at / 64, lane = at % 64;
    uint32_t all[kOrderE / 64];
#pragma unroll
    for (int i = 0; i < kOrderE / 64; ++i) all[i] = __builtin_amdgcn_readlane(o.segment[i], lane);
    static_assert(kOrderE / 64 == 4, "a choice of four");
    seg = j < 2 ? (j == 0 ? all[0] : all[1]) : (j == 2 ? all[2] : all[3]);
    expert = __builtin_amdgcn_readlane(o.expert, lane) >> (8 * j) & 0xFF;
  } else {
    seg = __builtin_amdgcn_readfirstlane(packed(segment_of(offsets, (int)at, rows)));
  }
  return {true, seg & 0xFFFF, seg >> 16, expert, tile.m * TILE, tile.n * TILE};
}

// 16-byte chunk c of row r of an operand's pair sits at chunk c ^ swz(r): fragment
// reads, of 8 or 16 consecutive rows at one chunk, then touch every bank once.
__device__ __forceinline__ uint32_t swz(uint32_t row) { return ((row & 31) ^ ((row & 31) >> 3)) & 7; }

// A tile of zeros; what accumulates stays as it is.
__device__ __forceinline__ void store_zeros(const GemmArgs& g, void* out, uint32_t i0, uint32_t j0) {
  if (g.accumulate) return;
  const int64_t bytes = g.out_f32 ? 4 : 2, per = 16 / bytes;
  const int64_t cols = g.J - j0 < TILE ? g.J - j0 : TILE, rows = g.I - i0 < TILE ? g.I - i0 : TILE;
  for (int64_t k = threadIdx.x; k < rows * (cols / per); k += THREADS) {
    const int64_t i = i0 + k / (cols / per), j = j0 + k % (cols / per) * per;
    *reinterpret_cast<u32x4*>(static_cast<char*>(out) + (i * g.J + j) * bytes) = u32x4{0, 0, 0, 0};
  }
}

// An accumulator where it is used: the compiler would move all of them out of the
// matrix registers at once, for which there are no others.
__device__ __forceinline__ v16f from_here(v16f v) {
  asm volatile("" : "+a"(v));
  return v;
}

// The wave's 128 x 128 of a finished tile.  acc[a][b] lane l, element e holds row
// 32a + l%32, column 32b + 8*(e/4) + 4*(l/32) + e%4.  Through the wave's own staging
// area, 32 rows of 128 bytes at a time, so that whole lines are stored; the unit (4
// columns) is XORed with the pair of rows, which spreads writes and reads over all
// banks.  The direct loads of the tiles to come were issued before: they have landed
// when the first store is issued, so that nobody has to count them among the stores.
__device__ __forceinline__ void store_wave(const GemmArgs& g, void* out, uint8_t* staging, int64_t row0, int64_t col0,
                                           const v16f (&acc)[TM][TN]) {
  uint32_t lane = threadIdx.x & 63;
  int64_t ld = g.J;
  asm volatile("" : "+v"(lane), "+s"(ld));  // no address is to stay in registers from one tile to the next
  const uint32_t l32 = lane & 31, g2 = lane >> 5, k = lane & 7;
  // (128 columns are all in or all out)
  const int64_t rows = col0 < g.J ? g.I - row0 : 0;
  if (!g.out_f32) {
    uint16_t* p = static_cast<uint16_t*>(out) + (row0 + (lane >> 3)) * ld + col0 + 8 * k;
#pragma unroll
    for (int a = 0; a < TM; ++a, p += 32 * ld)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
#pragma unroll
        for (int b = 0; b < 2; ++b) {
          const v16f v = from_here(acc[a][2 * h + b]);
#pragma unroll
          for (int q = 0; q < 4; ++q)
            *reinterpret_cast<uint2*>(staging + l32 * 128 + ((8 * b + 2 * q + g2) ^ (l32 >> 1)) * 8) =
                make_uint2(bf16x2_rne(v[4 * q], v[4 * q + 1]), bf16x2_rne(v[4 * q + 2], v[4 * q + 3]));
        }
        u32x4 o[4];
#pragma unroll
        for (int s = 0; s < 4; ++s) {
          const uint32_t row = 8 * s + (lane >> 3), pu = (2 * k) ^ (row >> 1);
          o[s] = *reinterpret_cast<const u32x4*>(staging + row * 128 + (pu & ~1u) * 8);
          if ((row >> 1) & 1) o[s] = u32x4{o[s][2], o[s][3], o[s][0], o[s][1]};  // the pair is stored swapped
        }
        if (a == 0 && h == 0) wait_vmcnt<0>();
#pragma unroll
        for (int s = 0; s < 4; ++s) {
          const uint32_t row = 32 * a + 8 * s + (lane >> 3);
          if (row < rows) __builtin_nontemporal_store(o[s], reinterpret_cast<u32x4*>(p + (8 * s) * ld + 64 * h));
        }
        __builtin_amdgcn_sched_barrier(0);
      }
  } else {
    float* p = static_cast<float*>(out) + (row0 + (lane >> 3)) * ld + col0 + 4 * k;
#pragma unroll
    for (int a = 0; a < TM; ++a, p += 32 * ld)
#pragma unroll
      for (int b = 0; b < TN; ++b) {
        const v16f v = from_here(acc[a][b]);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          *reinterpret_cast<v4f*>(staging + l32 * 128 + ((2 * q + g2) ^ ((l32 >> 1) & 7)) * 16) =
              v4f{v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]};
        }
        v4f o[4];
#pragma unroll
        for (int s = 0; s < 4; ++s) {
          const uint32_t row = 8 * s + (lane >> 3);
          o[s] = *reinterpret_cast<const v4f*>(staging + row * 128 + (k ^ ((row >> 1) & 7)) * 16);
        }
        if (a == 0 && b == 0) wait_vmcnt<0>();
        if (g.accumulate) {
          v4f was[4];
#pragma unroll
          for (int s = 0; s < 4; ++s) {
            const uint32_t row = 32 * a + 8 * s + (lane >> 3);
            if (row < rows) was[s] = *reinterpret_cast<const v4f*>(p + (8 * s) * ld + 32 * b);
          }
#pragma unroll
          for (int s = 0; s < 4; ++s)
            o[s] = v4f{was[s][0] + o[s][0], was[s][1] + o[s][1], was[s][2] + o[s][2], was[s][3] + o[s][3]};
        }
#pragma unroll
        for (int s = 0; s < 4; ++s) {
          const uint32_t row = 32 * a + 8 * s + (lane >> 3);
          if (row < rows) __builtin_nontemporal_store(o[s], reinterpret_cast<v4f*>(p + (8 * s) * ld + 32 * b));
        }
        __builtin_amdgcn_sched_barrier(0);
      }
  }
}

template <int V>
struct IntC {
  static constexpr int value = V;
};

__global__ __launch_bounds__(THREADS) void grouped_mx_wgrad_kernel(GroupedArgs ga, uint32_t tiles_m, uint32_t tiles_n,
                                                                   uint32_t each) {
  extern __shared__ __attribute__((aligned(1024))) uint8_t lds[];
  const GemmArgs& g = ga.g;
  const uint32_t R = (uint32_t)g.R, nkb = R / 128;
  Order order;
  make_order(order, lds, ga.offsets, (int)ga.E, (int32_t)R);
  const auto find = [&](uint32_t nth) {
    return find_tile(order, ga.offsets, (int32_t)R, nth, (uint32_t)ga.E, tiles_m, tiles_n);
  };

  const uint32_t lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const uint32_t l32 = lane & 31, g2 = lane >> 5, lds0 = lds_offset(lds);

  // ---- the pair that is loaded next: of the tile before l_nth, l_left with the
  // pairs behind it.  Behind the workgroup's last pair that one is loaded again, into
  // a slot that is never read again.  Rows past the edge of the result read the last
  // one (and are not stored).
  uint32_t l_nth = 0, l_left = 0, l_block = 0, l_last_a = 0, l_last_b = 0;
  bool l_group = false;     // its scales have to be loaded: a tile's first pair or the first of four
  const uint8_t *l_a = nullptr, *l_b = nullptr, *l_sa = nullptr, *l_sb = nullptr;
  const auto next_pair = [&]() {
    if (l_left > 1) {
      --l_left;
      ++l_block;
      l_group = (l_block & 3) == 0;
      return;
    }
    while (l_nth < each) {
      const Found f = find(l_nth);
      l_nth = f.any ? l_nth + 1 : each;
      if (!f.any || f.length == 0) continue;
      l_left = f.length;
      l_block = f.first;
      l_group = true;
      l_last_a = (uint32_t)(g.I - f.i0 < TILE ? g.I - f.i0 : TILE) - 1;
      l_last_b = (uint32_t)(g.J - f.j0 < TILE ? g.J - f.j0 : TILE) - 1;
      l_a = g.a + (int64_t)f.i0 * R;
      l_b = g.b + (int64_t)f.j0 * R;
      l_sa = reinterpret_cast<const uint8_t*>(g.sa + (int64_t)f.i0 * nkb);
      l_sb = reinterpret_cast<const uint8_t*>(g.sb + (int64_t)f.j0 * nkb);
      return;
    }
  };
  // The wave's u-th load of an operand of the pair: 8 rows of 128 bytes; lane p
  // writes bytes 16 p .. of that KiB, row p / 8's chunk p % 8.
  uint32_t row_at = (wave * LOADS * 8 + (lane >> 3)) * R, chunk = ((lane & 7) ^ (lane >> 3)) << 4;
  const auto load_rows = [&](int u, uint32_t slot, bool b) {
    asm volatile("" : "+v"(row_at), "+v"(chunk));  // the offsets of 16 loads are not to be kept
    const uint32_t at = row_at + 8 * u * R, last = (b ? l_last_b : l_last_a) * R;
    dma16((b ? l_b : l_a) + (int64_t)l_block * PK, (at < last ? at : last) + (chunk ^ ((u & 3) << 4)),
          lds0 + slot * SLOT + (b ? OPERAND : 0) + (wave * LOADS + u) * 1024);
  };
  // The scales of its group of four blocks go to the slot that the group before does
  // not have: pairs of at most two groups are yet to be read.  Returns where in LDS the
  // pair's are.
  uint32_t l_scales = 0;
  const auto load_scales = [&]() {
    if (l_group) {
      l_scales ^= SCALES;
      uint32_t row = wave * 64 + lane;
      asm volatile("" : "+v"(row));
      const uint32_t to = lds0 + AT_SCALES + l_scales + wave * 1024;
      const int64_t at = (int64_t)(l_block & ~3u) * 4;
      dma16(l_sa + at, (row < l_last_a ? row : l_last_a) * nkb * 4, to);
      dma16(l_sb + at, (row < l_last_b ? row : l_last_b) * nkb * 4, to + TILE * 16);
    }
    return AT_SCALES + l_scales + (l_block & 3) * 4;
  };

  // ---- fragments: lane l holds row l%32 of a 32-row MFMA tile and, of half h of
  // its pair, logical chunks 4h + 2*(l/32) and the next one.
  const uint32_t wm0 = (wave >> 1) * 128, wn0 = (wave & 1) * 128;
  const uint32_t sw = swz(l32);
  const uint32_t c0 = ((0 + 2 * g2) ^ sw) << 4, c1 = ((4 + 2 * g2) ^ sw) << 4;
  const uint32_t rowA = (wm0 + l32) * PK, rowB = OPERAND + (wn0 + l32) * PK;
  const int32_t second = (sw & 1) ? -16 : 16;
  const auto read_frag = [&](uint32_t slot, int half, uint32_t row) {
    const uint8_t* p = lds + slot * SLOT + row + (half ? c1 : c0);
    const u32x4 lo = *reinterpret_cast<const u32x4*>(p);
    const u32x4 hi = *reinterpret_cast<const u32x4*>(p + second);
    return v8i{(int)lo[0], (int)lo[1], (int)lo[2], (int)lo[3], (int)hi[0], (int)hi[1], (int)hi[2], (int)hi[3]};
  };
  // a scale's exponent field is its E8M0 byte (scales are positive)
  const auto read_scale = [&](uint32_t at, uint32_t row) {
    return *reinterpret_cast<const uint32_t*>(lds + at + row * 16) >> 23;
  };

  v16f acc[TM][TN];
  v8i fa[2][TM], fb[2][TN];
  uint32_t sa[TM], sb[TN];
  uint32_t slot = 0;                           // the pair at hand is in it, the next one in the other
  uint32_t scales = 0, scales_behind = 0;      // where their scales are

  // prologue: pairs 0 and 1
  next_pair();
  if (l_left > 0) {
#pragma unroll
    for (uint32_t s = 0; s < 2; ++s) {
      (s ? scales_behind : scales) = load_scales();
#pragma unroll
      for (int u = 0; u < LOADS; ++u) {
        load_rows(u, s, false);
        load_rows(u, s, true);
      }
      next_pair();
    }
  }
  wait_vmcnt<0>();
  lds_barrier();
  const auto read_first = [&]() {  // of a tile: the first stage's fragments, the scales
#pragma unroll
    for (int t = 0; t < TM; ++t) fa[0][t] = read_frag(slot, 0, rowA + t * 32 * PK);
#pragma unroll
    for (int t = 0; t < TN; ++t) fb[0][t] = read_frag(slot, 0, rowB + t * 32 * PK);
#pragma unroll
    for (int t = 0; t < TM; ++t) sa[t] = read_scale(scales, wm0 + t * 32 + l32);
#pragma unroll
    for (int t = 0; t < TN; ++t) sb[t] = read_scale(scales, TILE + wn0 + t * 32 + l32);
  };

  // One 64-deep stage.  Entry: its fragments are in registers (set HALF).  Its 16
  // MFMAs go in pairs, between which the wave reads a fragment of the next stage.
  // The second half of a pair first waits for the next pair (unless it is known to
  // have landed) and passes a barrier, behind which nobody reads this pair's slot any
  // more; it reads the next pair's scales and refills the slot, two loads a step.
  const auto stage = [&](auto half_tag, auto zero_tag, auto wait_tag) {
    constexpr int HALF = decltype(half_tag)::value, NEXT = HALF ^ 1;
    constexpr bool ZERO = decltype(zero_tag)::value, WAIT = decltype(wait_tag)::value;
    const uint32_t from = HALF ? slot ^ 1 : slot;
    uint32_t na[TM], nb[TN], loading = 0;
    if constexpr (HALF == 1) {
      if constexpr (WAIT) wait_vmcnt<0>();
      lds_barrier();
      loading = load_scales();
    }
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int p = 0; p < 2 * TM; ++p) {
      const int a = p >> 1, b0 = 2 * (p & 1);
#pragma unroll
      for (int b = b0; b < b0 + 2; ++b)
        acc[a][b] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
            fb[HALF][b], fa[HALF][a], ZERO ? v16f{} : acc[a][b], 0, 0, 0, (int)sb[b], 0, (int)sa[a]);
      if (p == 0) fa[NEXT][0] = read_frag(from, NEXT, rowA);
      else if (p <= 4) fb[NEXT][p - 1] = read_frag(from, NEXT, rowB + (p - 1) * 32 * PK);
      else fa[NEXT][p - 4] = read_frag(from, NEXT, rowA + (p - 4) * 32 * PK);
      if constexpr (HALF == 1) {
        if (p < 4) na[p] = read_scale(scales_behind, wm0 + p * 32 + l32);
        else nb[p - 4] = read_scale(scales_behind, TILE + wn0 + (p - 4) * 32 + l32);
        load_rows(p, slot, false);
        load_rows(p, slot, true);
      }
      __builtin_amdgcn_sched_barrier(0);
    }
    // (the compiler would move all of the MFMAs behind the next branch)
#pragma unroll
    for (int a = 0; a < TM; ++a)
#pragma unroll
      for (int b = 0; b < TN; ++b) asm volatile("" ::"a"(acc[a][b]));
    if constexpr (HALF == 1) {
#pragma unroll
      for (int t = 0; t < TM; ++t) sa[t] = na[t];
#pragma unroll
      for (int t = 0; t < TN; ++t) sb[t] = nb[t];
      next_pair();
      slot ^= 1;
      scales = scales_behind;
      scales_behind = loading;
    }
  };

  for (uint32_t nth = 0; nth < each; ++nth) {
    const Found f = find(nth);
    if (!f.any) break;
    void* const out = element(g.out, f.expert * ga.out_stride, g.out_f32);
    if (f.length == 0) {
      store_zeros(g, out, f.i0, f.j0);
      continue;
    }
    // (read again behind a store, which they would not fit in the registers beside)
    read_first();
    stage(IntC<0>{}, IntC<1>{}, IntC<0>{});
    stage(IntC<1>{}, IntC<0>{}, IntC<0>{});  // the next pair landed before the store, or in the prologue
    for (uint32_t k = 1; k < f.length; ++k) {
      stage(IntC<0>{}, IntC<0>{}, IntC<0>{});
      stage(IntC<1>{}, IntC<0>{}, IntC<1>{});
    }
    store_wave(g, out, lds + AT_STAGING + wave * STAGING, f.i0 + wm0, f.j0 + wn0, acc);
  }
  wait_vmcnt<0>();  // no direct load may still target this workgroup's LDS at exit
}

}  // namespace

hipError_t launch_grouped_wgrad_mx(const GroupedArgs& a, hipStream_t stream) {
  const int64_t tiles_m = (a.g.I + TILE - 1) / TILE, tiles_n = (a.g.J + TILE - 1) / TILE, tiles = a.E * tiles_m * tiles_n;
  const int64_t each = wgrad_plan(a).each;
  constexpr int64_t kWhole = 8 * RUN;
  const int64_t workgroups = ((tiles + each - 1) / each + kWhole - 1) / kWhole * kWhole;
  static std::atomic<uint64_t> attr_set{0};
  if (hipError_t e = ensure_lds_limit(reinterpret_cast<const void*>(&grouped_mx_wgrad_kernel), LDS_BYTES, &attr_set))
    return e;
  hipLaunchKernelGGL(grouped_mx_wgrad_kernel, dim3((uint32_t)workgroups), dim3(THREADS), LDS_BYTES, stream, a,
                     (uint32_t)tiles_m, (uint32_t)tiles_n, (uint32_t)each);
  return hipGetLastError();
}

}  // namespace fp8blk
