// Device-side core shared by the kernels that multiply a few rows (tokens)
// with E4M3 weights in 128x128 blocks: rows.hip (one linear) and moe.hip
// (the experts of a mixture).
//
// The contraction is the library's:
//   out[t][n] = sum over 128-deep blocks b of sx(t, b) * sw(n / 128, b) *
//               sum_{k in b} dec(qx[t][k]) * dec(qw[n][k]),
// with x quantized as by fp8_quantize_rowgroup (the same codes and scales).
//
// For few rows it is bound by reading the weights once, so it is laid out for
// that: a wave takes 16 weight rows x 128 reduction values per step, straight
// from memory into registers (no LDS: every weight byte is used by one wave
// only), and the waves of a workgroup split the reduction and add their sums
// through LDS in wave order, so results are deterministic.
//
// The products run on the bf16 matrix instructions, not the fp8 ones: an E4M3
// value is a bf16 value exactly, a product of two is exact in fp32, and the
// bf16 instructions keep the sum to fp32 rounding (the fp8 ones were measured
// at 1.5e-5 of the result's norm).  The extra conversions (16 per 2 KiB of
// weights and wave) stay far below the time to read the weights.
#pragma once

#include "fp8blk_device.h"

namespace fp8blk {

typedef __bf16 v8bf_t __attribute__((ext_vector_type(8)));

// A lane's part of one 128-deep block of one operand row.  Lane l of a wave
// holds row l % 16 of a 16-row tile and, with c = l / 16, the reduction values
// 16 c .. +15 and 64 + 16 c .. +15: two 16-byte pieces of codes, so that four
// lanes read 64 contiguous bytes of a row.  The matrix instruction's own
// order of reduction values does not matter as long as both operands use the
// same one.
struct CodeFrag {
  u32x4 lo, hi;
};
// The same values in bf16, as four operands of v_mfma_f32_16x16x32_bf16.
struct BfFrag {
  v8bf_t v[4];
};

__device__ __forceinline__ v8bf_t decode8(uint32_t w0, uint32_t w1) {
  // v_cvt_scalef32_pk_bf16_fp8 with scale 1: two codes to bf16, exactly
  typedef __bf16 v2 __attribute__((ext_vector_type(2)));
  const v2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w0, 1.0f, false);
  const v2 b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w0, 1.0f, true);
  const v2 c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w1, 1.0f, false);
  const v2 d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w1, 1.0f, true);
  return v8bf_t{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

__device__ __forceinline__ BfFrag decode(const CodeFrag& q) {
  BfFrag f;
  f.v[0] = decode8(q.lo[0], q.lo[1]);
  f.v[1] = decode8(q.lo[2], q.lo[3]);
  f.v[2] = decode8(q.hi[0], q.hi[1]);
  f.v[3] = decode8(q.hi[2], q.hi[3]);
  return f;
}

// acc += A B^T over one 128-deep block, from zero: lane l gets, as element i,
// the product of A's row 4 (l / 16) + i with B's row l % 16.
__device__ __forceinline__ v4f block_product(const BfFrag& a, const BfFrag& b) {
  v4f p{};
#pragma unroll
  for (int j = 0; j < 4; ++j) p = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a.v[j], b.v[j], p, 0, 0, 0);
  return p;
}

// Largest of the four lanes l, l ^ 16, l ^ 32, l ^ 48 (those that share an
// operand row), in every lane.  v_permlane*_swap exchanges whole 16- or
// 32-lane halves between its two operands; given the same value twice, the
// two results hold, lane by lane, the two values to compare.
__device__ __forceinline__ uint32_t quarter_max(uint32_t v) {
  const auto a = __builtin_amdgcn_permlane16_swap(v, v, false, false);
  v = max((uint32_t)a[0], (uint32_t)a[1]);
  const auto b = __builtin_amdgcn_permlane32_swap(v, v, false, false);
  return max((uint32_t)b[0], (uint32_t)b[1]);
}

// A lane's 32 bf16 values of one 128-group, as loaded: the pieces 16 c .. +7,
// 16 c + 8 .. +15, 64 + 16 c .. +7 and 64 + 16 c + 8 .. +15.
struct RawFrag {
  u32x4 w[4];
};

__device__ __forceinline__ RawFrag load_raw(const uint16_t* p) {
  RawFrag r;
  r.w[0] = *reinterpret_cast<const u32x4*>(p);
  r.w[1] = *reinterpret_cast<const u32x4*>(p + 8);
  r.w[2] = *reinterpret_cast<const u32x4*>(p + 64);
  r.w[3] = *reinterpret_cast<const u32x4*>(p + 72);
  return r;
}

// The group's codes (this lane's part) and its scale, exactly as the row-group
// quantizer forms them: amax over the group, scale rule S, round to nearest
// even.
template <class S>
__device__ __forceinline__ CodeFrag quantize_group(const RawFrag& r, float& scale) {
  uint32_t m = 0;
#pragma unroll
  for (int j = 0; j < 4; ++j)
    m = pk_max_u16(m, pk_max_u16(pk_max_u16(abs2(r.w[j][0]), abs2(r.w[j][1])),
                                 pk_max_u16(abs2(r.w[j][2]), abs2(r.w[j][3]))));
  m = quarter_max(max(m & 0xFFFFu, m >> 16));
  const S sc(m);
  scale = sc.s;
  CodeFrag q;
  q.lo = u32x4{quant4(r.w[0][0], r.w[0][1], sc), quant4(r.w[0][2], r.w[0][3], sc), quant4(r.w[1][0], r.w[1][1], sc),
               quant4(r.w[1][2], r.w[1][3], sc)};
  q.hi = u32x4{quant4(r.w[2][0], r.w[2][1], sc), quant4(r.w[2][2], r.w[2][3], sc), quant4(r.w[3][0], r.w[3][1], sc),
               quant4(r.w[3][2], r.w[3][3], sc)};
  return q;
}

__device__ __forceinline__ CodeFrag load_codes(const uint8_t* p) {
  CodeFrag q;
  q.lo = *reinterpret_cast<const u32x4*>(p);
  q.hi = *reinterpret_cast<const u32x4*>(p + 64);
  return q;
}

// Weights: read once by one wave; each line of 128 bytes is taken by two
// adjacent loads of the same wave.
__device__ __forceinline__ CodeFrag load_weights(const uint8_t* p) { return load_codes(p); }

// acc[rt][tt] += the blocks [b0, b1) of RT 16-row weight tiles times TT
// 16-token tiles.  Per lane: wp[rt] is its piece of its weight row at block
// 0, xp[tt] its piece of its token's row; sw[rt] points at the scales of the
// weight blocks that hold the tile (wave-uniform).  A lane without a token of
// its own points at some other row that may be read: the tokens are columns of
// the matrix instruction and do not mix, and its sums are not for use (leaving
// such loads out by a mask measured slower).  All loads of D blocks are issued
// before the first is used.
template <int RT, int TT, int D, class S>
__device__ __forceinline__ void rows_product(const uint8_t* const (&wp)[RT], const float* const (&sw)[RT],
                                             const uint16_t* const (&xp)[TT], int b0, int b1, v4f (&acc)[RT][TT]) {
  for (int b = b0; b < b1; b += D) {
    CodeFrag w[D][RT];
    RawFrag x[D][TT];
    float s[D][RT];
#pragma unroll
    for (int d = 0; d < D; ++d) {
      const int i = min(b + d, b1 - 1);
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) w[d][rt] = load_weights(wp[rt] + (int64_t)i * 128);
#pragma unroll
      for (int tt = 0; tt < TT; ++tt) x[d][tt] = load_raw(xp[tt] + (int64_t)i * 128);
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) s[d][rt] = sw[rt][i];
    }
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int d = 0; d < D; ++d) {
      if (d > 0 && b + d >= b1) break;
      BfFrag xf[TT];
      float m[TT];
#pragma unroll
      for (int tt = 0; tt < TT; ++tt) xf[tt] = decode(quantize_group<S>(x[d][tt], m[tt]));
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) {
        const BfFrag wf = decode(w[d][rt]);
#pragma unroll
        for (int tt = 0; tt < TT; ++tt) {
          const v4f p = block_product(wf, xf[tt]);
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[rt][tt][i] = __builtin_fmaf(p[i], m[tt] * s[d][rt], acc[rt][tt][i]);
        }
      }
    }
  }
}

// The same for x that is quantized already, and for a wave that owns its
// weight rows over the whole reduction: xp[tt] points at the lane's piece of
// its token's codes, xs[tt] at its token's scales.  Two stages are in
// registers, one being multiplied while the next one loads; past the end the
// last block is loaded again and not used, so that the loads of a stage stay
// one run without branches and the compiler can wait for one stage while the
// other is in flight.  Only the first `tiles` of the TT token tiles are read.
template <int RT, int TT>
struct RowsStage {
  CodeFrag w[RT], x[TT];
  float sx[TT], s[RT];

  __device__ __forceinline__ void load(const uint8_t* const (&wp)[RT], const float* const (&sw)[RT],
                                       const uint8_t* const (&xp)[TT], const float* const (&xs)[TT], int tiles,
                                       int b) {
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) w[rt] = load_weights(wp[rt] + (int64_t)b * 128);
#pragma unroll
    for (int tt = 0; tt < TT; ++tt) {
      if (tt < tiles) {
        x[tt] = load_codes(xp[tt] + b * 128);
        sx[tt] = xs[tt][b];
      }
    }
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) s[rt] = sw[rt][b];
  }

  __device__ __forceinline__ void multiply(int tiles, v4f (&acc)[RT][TT]) const {
    BfFrag wf[RT];
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) wf[rt] = decode(w[rt]);
#pragma unroll
    for (int tt = 0; tt < TT; ++tt) {
      if (tt < tiles) {
        const BfFrag xf = decode(x[tt]);
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) {
          const v4f p = block_product(wf[rt], xf);
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[rt][tt][i] = __builtin_fmaf(p[i], sx[tt] * s[rt], acc[rt][tt][i]);
        }
      }
    }
  }
};

template <int RT, int TT>
__device__ __forceinline__ void rows_stream(const uint8_t* const (&wp)[RT], const float* const (&sw)[RT],
                                            const uint8_t* const (&xp)[TT], const float* const (&xs)[TT], int tiles,
                                            int nkb, v4f (&acc)[RT][TT]) {
  RowsStage<RT, TT> even, odd;
  even.load(wp, sw, xp, xs, tiles, 0);
  for (int b = 0; b < nkb; b += 2) {
    odd.load(wp, sw, xp, xs, tiles, min(b + 1, nkb - 1));
    __builtin_amdgcn_sched_barrier(0);
    even.multiply(tiles, acc);
    if (b + 1 >= nkb) break;
    even.load(wp, sw, xp, xs, tiles, min(b + 2, nkb - 1));
    __builtin_amdgcn_sched_barrier(0);
    odd.multiply(tiles, acc);
  }
}

}  // namespace fp8blk
