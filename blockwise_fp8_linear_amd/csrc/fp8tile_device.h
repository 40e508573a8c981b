// A 128 x 128 tile of bf16 values held in the registers of a 256-thread
// workgroup, quantized in row groups, in column groups (written transposed), or
// both: the core of the one-pass quantizer (quant.hip) and of the kernels that
// make such a tile on the way (sorted.hip, gated.hip).
//
// Thread t owns rows 8 * (t / 16) .. +7 and columns 8 * (t % 16) .. +7; v[i]
// holds row i's eight values, two per word.  Row groups: the 16 lanes of a DPP
// row share the rows, so the row amax is a DPP reduction and each lane stores 8
// codes per row.  Column groups: a packed per-column max over the thread's rows,
// then over the 16 row blocks (wave shuffles, then LDS across the 4 waves); the
// thread's 8x8 codes are formed column by column (each pair of rows gathered
// into one word by a byte permute, then converted) and staged in LDS, from where
// whole 128-byte lines of the transposed output are stored.
#pragma once

#include "fp8blk_device.h"
#include "fp8quotient.h"
#include "fp8tile_order.h"

namespace fp8blk {

constexpr int kTileThreads = 256;

// What the column groups of one tile need of LDS.
struct TileLds {
  uint32_t red[kTileThreads / 64][16][4];
  __attribute__((aligned(16))) uint2 tq[128][16];  // column codes: [column][8-row block]
};

// Codes are stored past the caches (NT) where a call writes more of them than the
// Infinity Cache keeps for the next one: what the call reads again -- a token's row
// for each of its experts -- stays in the caches then.  Gather of 135296 rows of
// 2048 in both orientations, weighted: 219 us with plain stores, 163 past the caches.
constexpr int64_t kStoreNt = int64_t(128) << 20;  // bytes of codes
typedef uint32_t tile_u32x2 __attribute__((ext_vector_type(2)));
template <bool NT, class V>
__device__ __forceinline__ void store_codes(uint8_t* p, V v) {
  if constexpr (NT) __builtin_nontemporal_store(v, reinterpret_cast<V*>(p));
  else *reinterpret_cast<V*>(p) = v;
}

// The amax / 448 rule with fewer instructions, for scales in [kQuotientLeast,
// kQuotientMost) of fp8quotient.h.  The scale: a product with 1 / 448 and one
// correction, which gives the correctly rounded quotient of every such bf16 amax.  A
// value's quotient: Fp32Scale's without its factor, its clamp and its sign, from a
// reciprocal in two parts, x r + x r2, in one rounding of what is then 2^-44 off.  r2 is
// not negative, so both terms of a zero have its sign.  The amax's own quotient may
// exceed 448 by an ulp and rounds to 448 without the clamp.  A thread of a tile has 16
// scales and 128 quotients, which bind the kernels of this rule.
struct Fp32Quotient {
  static constexpr bool kScaledCvt = false;
  float s, r, r2;
  __device__ __forceinline__ explicit Fp32Quotient(uint32_t amax_bits) {
    const float a = __uint_as_float(amax_bits << 16), c = 1.0f / 448.0f, y = a * c;
    s = amax_bits == 0 ? 1.0f : __builtin_fmaf(__builtin_fmaf(-448.0f, y, a), c, y);
    const ReciprocalParts p = reciprocal_parts(s, __builtin_amdgcn_rcpf(s));  // an ulp off at most
    r = p.r;
    r2 = p.r2;
  }
  // (s is not negative: written so, the gather has a value less in scratch memory and takes
  // 184 us for 135296 rows of 2048 in both orientations, without the absolute value 189)
  __device__ __forceinline__ bool fits() const { return __builtin_fabsf(s) < kQuotientMost && s >= kQuotientLeast; }
  __device__ __forceinline__ float operator()(float x) const { return __builtin_fmaf(x, r, x * r2); }
};

// f(scale) for the group of this amax: under the amax / 448 rule with the short
// quotient where the whole wave's groups fit it.  Returns the scale that is stored.
template <class S, class F>
__device__ __forceinline__ float with_scale(uint32_t amax_bits, F f) {
  if constexpr (!S::kScaledCvt) {
    const Fp32Quotient sc(amax_bits);
    if (__builtin_amdgcn_ballot_w64(!sc.fits()) == 0) {
      f(sc);
      return sc.s;
    }
  }
  const S sc(amax_bits);
  f(sc);
  return sc.s;
}

// Eight values of a group of 128 that 16 lanes hold -> their codes and the scale.
template <class S>
__device__ __forceinline__ float quant_group(u32x4 v, tile_u32x2& o) {
  uint32_t m = pk_max_u16(pk_max_u16(abs2(v.x), abs2(v.y)), pk_max_u16(abs2(v.z), abs2(v.w)));
  m = row16_max(max(m & 0xFFFFu, m >> 16));
  return with_scale<S>(m, [&](const auto& sc) { o = tile_u32x2{quant4(v.x, v.y, sc), quant4(v.z, v.w, sc)}; });
}

// Row groups.  q: the tile's first row and the thread's first column; s: the
// tile's first row and its group; G: groups per row of s.
template <class S, bool NT = false>
__device__ __forceinline__ void tile_row_groups(const u32x4 (&v)[8], uint8_t* __restrict__ q, int64_t ld_q,
                                                float* __restrict__ s, uint32_t G, uint32_t rb, uint32_t cb) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    tile_u32x2 o;
    const float scale = quant_group<S>(v[i], o);
    store_codes<NT>(q + (int64_t)(rb * 8 + i) * ld_q, o);
    if (cb == 0) s[(int64_t)(rb * 8 + i) * G] = scale;
  }
}

// Column groups.  qT: the tile's first column (a row of qT) and first row; sT:
// the tile's first column and its row group; G: row groups per column of sT.
// Passes two barriers; the LDS may be used again after another one.
template <class S, bool NT = false>
__device__ __forceinline__ void tile_col_groups(const u32x4 (&v)[8], TileLds& lds, uint8_t* __restrict__ qT,
                                                int64_t ld_qT, float* __restrict__ sT, uint32_t G, uint32_t rb,
                                                uint32_t cb) {
  const uint32_t t = threadIdx.x, lane = t & 63, wave = t >> 6;
  // packed (two columns per word) max over the 128 rows
  uint32_t cm[4] = {0, 0, 0, 0};
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    cm[0] = pk_max_u16(cm[0], abs2(v[i].x));
    cm[1] = pk_max_u16(cm[1], abs2(v[i].y));
    cm[2] = pk_max_u16(cm[2], abs2(v[i].z));
    cm[3] = pk_max_u16(cm[3], abs2(v[i].w));
  }
#pragma unroll
  for (int w = 0; w < 4; ++w) {  // the wave's 4 row blocks of this column block: lanes cb, cb+16, +32, +48
    cm[w] = pk_max_u16(cm[w], (uint32_t)__shfl_xor((int)cm[w], 16, 64));
    cm[w] = pk_max_u16(cm[w], (uint32_t)__shfl_xor((int)cm[w], 32, 64));
  }
  if (lane < 16) {
#pragma unroll
    for (int w = 0; w < 4; ++w) lds.red[wave][cb][w] = cm[w];
  }
  __syncthreads();
#pragma unroll
  for (int w = 0; w < 4; ++w)
    cm[w] = pk_max_u16(pk_max_u16(lds.red[0][cb][w], lds.red[1][cb][w]),
                       pk_max_u16(lds.red[2][cb][w], lds.red[3][cb][w]));
  // column j's amax is half j % 2 of cm[j / 2]
  const auto amax = [&](int j) { return j & 1 ? cm[j >> 1] >> 16 : cm[j >> 1] & 0xFFFFu; };
  // The thread's 8x8 codes, one column at a time (rows 0..3 and 4..7 of
  // column j, each with the column's scale: word j / 2 of each row, half
  // j % 2), go through LDS as tq[column][row block], the 8-byte unit
  // XOR-swizzled by the column block cb, and leave as whole 128-byte lines of
  // qT: 8 lanes per column, 16 bytes (two row blocks) each.
  const auto column = [&](int j, const auto& sc) {
    const int m = j >> 1;
    uint32_t a, b;
    if (j & 1) {
      a = quant4_col<1>(v[0][m], v[1][m], v[2][m], v[3][m], sc);
      b = quant4_col<1>(v[4][m], v[5][m], v[6][m], v[7][m], sc);
    } else {
      a = quant4_col<0>(v[0][m], v[1][m], v[2][m], v[3][m], sc);
      b = quant4_col<0>(v[4][m], v[5][m], v[6][m], v[7][m], sc);
    }
    lds.tq[cb * 8 + j][rb ^ cb] = make_uint2(a, b);
  };
  float scale[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) scale[j] = with_scale<S>(amax(j), [&](const auto& sc) { column(j, sc); });
  __syncthreads();
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const uint32_t c = k * 32 + (t >> 3), p = t & 7;
    const uint32_t pu = (2 * p) ^ (c >> 3);  // physical unit of row block 2p
    u32x4 w = *reinterpret_cast<const u32x4*>(&lds.tq[c][pu & ~1u]);
    if (pu & 1) w = u32x4{w[2], w[3], w[0], w[1]};  // the pair is stored swapped
    store_codes<NT>(qT + (int64_t)c * ld_qT + 16 * p, w);
  }
  if (rb == 0) {
#pragma unroll
    for (int j = 0; j < 8; ++j) sT[(int64_t)(cb * 8 + j) * G] = scale[j];
  }
}

}  // namespace fp8blk
