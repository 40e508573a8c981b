// Device-side core shared by the kernels that multiply a few rows (tokens)
// with E4M3 weights in 128x128 blocks: rows.hip (one linear) and moe.hip
// (the experts of a mixture).
//
// The contraction is the library's:
//   out[t][n] = sum over 128-deep blocks b of sx(t, b) * sw(n / 128, b) *
//               sum_{k in b} dec(qx[t][k]) * dec(qw[n][k]),
// with x quantized as by fp8_quantize_rowgroup (the same codes and scales).
//
// For few rows it is bound by reading the weights once, and laid out for that:
// a wave takes tiles of 16 weight rows x 128 reduction values, loaded by whole
// lines into LDS that only it uses, and the waves of a workgroup split the
// reduction (adding their sums in wave order at the end) or the weight rows;
// either way the order of every sum is fixed.
//
// The products run on the bf16 matrix instructions, not the fp8 ones: an E4M3
// value is a bf16 value exactly, a product of two is exact in fp32, and the
// bf16 instructions keep the sum to fp32 rounding (the fp8 ones were measured
// at 1.5e-5 to 4.5e-5 of the result's norm).  The extra conversions (16 per 2 KiB of
// weights and wave) stay far below the time to read the weights.
#pragma once

#include "fp8blk_device.h"
#include "fp8moe_launch.h"

namespace fp8blk {

// Four neighbouring elements of the result; ACCUM: a call may ask to add them.
template <bool ACCUM>
__device__ __forceinline__ void store_rows(const RowsOut& out, int64_t at, const v4f& v) {
  if (out.f32) {
    v4f* y = reinterpret_cast<v4f*>(static_cast<float*>(out.y) + at);
    *y = ACCUM && out.accumulate ? *y + v : v;
  } else {
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(out.y) + at) =
        make_uint2(bf16x2_rne(v[0], v[1]), bf16x2_rne(v[2], v[3]));
  }
}

// A group of 128 bf16 values on 16 neighbouring lanes, 8 each: this lane's codes
// and the group's scale, as the row-group quantizer gives them (amax over the
// group, scale rule S, round to nearest even).
template <class S>
__device__ __forceinline__ uint2 quantize8(const u32x4& v, float* scale) {
  const uint32_t m = pk_max_u16(pk_max_u16(abs2(v[0]), abs2(v[1])), pk_max_u16(abs2(v[2]), abs2(v[3])));
  const S sc(row16_max(max(m & 0xFFFFu, m >> 16)));
  *scale = sc.s;
  return make_uint2(quant4(v[0], v[1], sc), quant4(v[2], v[3], sc));
}

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

// The same on the fp8 matrix instruction, straight from the codes: a quarter of
// the instructions and no conversions, for where the fp8 GEMMs' accuracy does:
// the instruction adds a block's 128 products with fewer bits than fp32 has
// (1.5e-5 to 4.5e-5 of the result's norm, the more the wider the codes' range;
// the blocks are then added in fp32).  Each operand's own scale is 2^0.
__device__ __forceinline__ v4f block_product_fp8(const CodeFrag& a, const CodeFrag& b) {
  typedef int v8i_t __attribute__((ext_vector_type(8)));
  const auto join = [](const CodeFrag& q) {
    return v8i_t{(int)q.lo[0], (int)q.lo[1], (int)q.lo[2], (int)q.lo[3],
                 (int)q.hi[0], (int)q.hi[1], (int)q.hi[2], (int)q.hi[3]};
  };
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(join(a), join(b), v4f{}, 0, 0, 0, 0x7F7F7F7F, 0,
                                                          0x7F7F7F7F);
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

// ---------------------------------------------------------------------------
// Operand tiles in LDS, filled by direct 16-byte global->LDS loads.
//
// Loading a fragment straight into registers would put neighbouring lanes on
// different rows, and the address unit then takes one lane at a time: 16
// bytes per clock and CU, measured as 57 cache accesses per load and the bound
// of the first form of these kernels.  In a direct load neighbouring lanes take
// neighbouring 16-byte chunks of one row (a whole 128-byte line per row of
// codes), and the fragments are then read from LDS.
//
// Chunk i of row r of a tile lies at place i ^ (r & 7) of the row, so that
// eight rows read at one chunk touch different banks.
// ---------------------------------------------------------------------------
constexpr int kCodeTile = 16 * 128;  // bytes of a tile of codes: 16 rows x 128

// The row of the tile that lane p of direct load `load` brings a chunk of, and
// the chunk's byte offset in that row: a load covers 8 rows.
__device__ __forceinline__ uint32_t code_row(uint32_t p, int load) { return load * 8 + (p >> 3); }
__device__ __forceinline__ uint32_t code_chunk(uint32_t p, int load) {
  return ((p & 7) ^ (code_row(p, load) & 7)) << 4;
}
__device__ __forceinline__ CodeFrag read_codes(const uint8_t* tile, uint32_t r, uint32_t c) {
  const uint32_t at = r * 128 + ((c ^ (r & 7)) << 4);
  CodeFrag q;
  q.lo = *reinterpret_cast<const u32x4*>(tile + at);
  q.hi = *reinterpret_cast<const u32x4*>(tile + (at ^ 64));
  return q;
}

// Rows that are still bf16 come through registers, 4 to a load: lane p has the
// chunk p % 16 (8 values) of row 4 load + p / 16, sixteen neighbouring lanes a
// whole group.  They are quantized on the way into the tile of codes, and each
// row's scale goes to scale[row].
__device__ __forceinline__ uint32_t raw_row(uint32_t p, int load) { return load * 4 + (p >> 4); }

template <class S>
__device__ __forceinline__ void quantize_into(uint8_t* tile, float* scale, const u32x4& v, uint32_t p, int load) {
  const uint32_t row = raw_row(p, load), l16 = p & 15;
  float s;
  *reinterpret_cast<uint2*>(tile + row * 128 + (((l16 >> 1) ^ (row & 7)) << 4) + (l16 & 1) * 8) = quantize8<S>(v, &s);
  if (l16 == 0) scale[row] = s;
}

// The wave's direct loads have landed / its LDS reads have returned.  (Written
// out because the compiler does not know of the direct loads.)
__device__ __forceinline__ void loads_landed() { asm volatile("s_waitcnt vmcnt(0)" ::: "memory"); }
__device__ __forceinline__ void reads_returned() { asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory"); }

// ---------------------------------------------------------------------------
// acc[rt][tt] += the blocks [b0, b1) of RT 16-row weight tiles times TT
// 16-token tiles, by one wave on its own: `lds` is its own area of
// D * rows_stage_bytes<RT, TT, RAW, XL>() bytes and no barrier is passed.  The
// loads of up to D blocks are issued together and then waited for; what hides
// them is the other waves of the CU, each at its own place.
//   w[rt]: the tile's first row at block 0 (wave-uniform), rows K bytes apart
//   sw[rt]: the scales of the weight blocks that hold the tile
//   RAW: the tokens' rows are bf16 and quantized here by rule S; otherwise they
//     are codes, and xs[tt] points at the scales of token l % 16 of the tile,
//     xs_b apart from block to block
//   XL: loads per token tile, 4 rows each (codes: 8); with fewer than the
//     tile has, the rows beyond repeat the last one (the tokens are columns of
//     the matrix instruction and do not mix, and nobody wants theirs)
//   x: base of the tokens' rows (wave-uniform), xoff[tt][u]: for this lane the
//     byte offset of its chunk of the row that load u of tile tt brings
// ---------------------------------------------------------------------------
template <int RT, int TT, bool RAW, int XL>
__device__ __host__ constexpr int rows_stage_bytes() {
  return RT * kCodeTile + TT * XL * (RAW ? 512 + 16 : 1024);
}

template <int RT, int TT, int XL, int D, bool RAW, class S>
__device__ __forceinline__ void rows_product(uint8_t* lds, const uint8_t* const (&w)[RT], const float* const (&sw)[RT],
                                             int64_t K, const uint8_t* x, const uint32_t (&xoff)[TT][XL],
                                             const float* const (&xs)[TT], int64_t xs_b, int b0, int b1,
                                             v4f (&acc)[RT][TT]) {
  constexpr int SB = rows_stage_bytes<RT, TT, RAW, XL>(), ROWS = XL * (RAW ? 4 : 8);
  constexpr int TILE = ROWS * 128, SCALES = RT * kCodeTile + TT * TILE;  // (raw) the rows' scales behind the tiles
  const uint32_t lane = threadIdx.x & 63, r = lane & 15, c = lane >> 4, xr = min(r, (uint32_t)ROWS - 1);
  const uint32_t at = lds_offset(lds);
  const uint32_t woff[2] = {(uint32_t)(code_row(lane, 0) * K) + code_chunk(lane, 0),
                            (uint32_t)(code_row(lane, 1) * K) + code_chunk(lane, 1)};
  for (int b = b0; b < b1; b += D) {
    float s[D][RT], m[D][TT];
    u32x4 v[D][TT][RAW ? XL : 1];
#pragma unroll
    for (int d = 0; d < D; ++d) {
      if (b + d >= b1) break;
      const int i = b + d;
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) {
        dma16(w[rt] + (int64_t)i * 128, woff[0], at + d * SB + rt * kCodeTile);
        dma16(w[rt] + (int64_t)i * 128, woff[1], at + d * SB + rt * kCodeTile + 1024);
        s[d][rt] = sw[rt][i];
      }
#pragma unroll
      for (int tt = 0; tt < TT; ++tt) {
#pragma unroll
        for (int u = 0; u < XL; ++u) {
          if constexpr (RAW)
            v[d][tt][u] = *reinterpret_cast<const u32x4*>(x + (int64_t)i * 256 + xoff[tt][u]);
          else
            dma16(x + (int64_t)i * 128, xoff[tt][u], at + d * SB + RT * kCodeTile + tt * TILE + u * 1024);
        }
        if constexpr (!RAW) m[d][tt] = xs[tt][i * xs_b];
      }
    }
    if constexpr (RAW) {
#pragma unroll
      for (int d = 0; d < D; ++d) {
        if (b + d >= b1) break;
#pragma unroll
        for (int tt = 0; tt < TT; ++tt)
#pragma unroll
          for (int u = 0; u < XL; ++u)
            quantize_into<S>(lds + d * SB + RT * kCodeTile + tt * TILE,
                             reinterpret_cast<float*>(lds + d * SB + SCALES) + tt * ROWS, v[d][tt][u], lane, u);
      }
    }
    loads_landed();
#pragma unroll
    for (int d = 0; d < D; ++d) {
      if (b + d >= b1) break;
      const uint8_t* st = lds + d * SB;
      BfFrag xf[TT];
#pragma unroll
      for (int tt = 0; tt < TT; ++tt) {
        if constexpr (RAW) m[d][tt] = reinterpret_cast<const float*>(st + SCALES)[tt * ROWS + xr];
        xf[tt] = decode(read_codes(st + RT * kCodeTile + tt * TILE, xr, c));
      }
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) {
        const BfFrag wf = decode(read_codes(st + rt * kCodeTile, r, c));
#pragma unroll
        for (int tt = 0; tt < TT; ++tt) {
          const v4f p = block_product(wf, xf[tt]);
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[rt][tt][i] = __builtin_fmaf(p[i], m[d][tt] * s[d][rt], acc[rt][tt][i]);
        }
      }
    }
    reads_returned();  // before the next loads overwrite what was read
  }
}

// ---------------------------------------------------------------------------
// acc[rt][tt] += all blocks of RT 16-row weight tiles (each wave its own) times
// the TT 16-token tiles that the workgroup's eight waves share.  Every thread
// of the workgroup calls it, with the same x, xs and nkb.
//   The blocks go through SLOTS slots in LDS, one multiplied while the others
// fill: each wave loads its own weight tiles and an eighth of the tokens' codes
// (some twice where there are fewer loads than waves).  One barrier per block
// says that the block has landed for everyone and that the slot before it may be
// filled again.  (More than two slots pay where a CU has one workgroup anyway:
// the launchers' choice.)
//   FP8: on the fp8 matrix instruction instead of the bf16 one.
//   Scales, for kPanel blocks at a time: the weights' in registers, lane i
// holding block i's; the tokens' in LDS, [block][token], by direct loads that
// the first block's wait covers.  (For 64 blocks at a time two tiles of tokens
// would not fit a CU twice: 150 tokens, 64 experts of 1024 101 us, so 94.)
//   xoff: the byte offset, from x, of the chunk that this lane's load brings:
// load wave % (2 TT) of the tokens' codes, two of them to a tile;
//   xs: the tokens' scales in memory, that of token i of the tiles in block b at
// b xs_b + xrow(i), which for kPanel blocks stays within 2^29.
// ---------------------------------------------------------------------------
constexpr int kPanel = 32;

template <int RT, int TT, int SLOTS>
__device__ __host__ constexpr int rows_ring_bytes() {
  return SLOTS * (8 * RT + TT) * kCodeTile + kPanel * 16 * TT * 4;
}

template <int RT, int TT, int SLOTS, bool FP8 = false, class XRow>
__device__ __forceinline__ void rows_ring(uint8_t* lds, const uint8_t* const (&w)[RT], const float* const (&sw)[RT],
                                          int64_t K, const uint8_t* x, uint32_t xoff, const float* xs,
                                          int64_t xs_b, XRow xrow, int nkb,
                                          v4f (&acc)[RT][TT]) {
  constexpr int SLOT = (8 * RT + TT) * kCodeTile, LOADS = 2 * RT + 1;  // of a block and wave
  const uint32_t lane = threadIdx.x & 63, r = lane & 15, c = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), xload = wave % (2 * TT);
  const uint32_t at = lds_offset(lds);
  float* const scales = reinterpret_cast<float*>(lds + SLOTS * SLOT);
  const uint32_t woff[2] = {(uint32_t)(code_row(lane, 0) * K) + code_chunk(lane, 0),
                            (uint32_t)(code_row(lane, 1) * K) + code_chunk(lane, 1)};
  for (int p0 = 0; p0 < nkb; p0 += kPanel) {
    const int nb = min(kPanel, nkb - p0);
    float s[RT];
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) s[rt] = sw[rt][p0 + min((int)lane, nb - 1)];
    const auto issue = [&](int b) {
      const uint32_t slot = at + b % SLOTS * SLOT;
      const int64_t k = (int64_t)(p0 + b) * 128;
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) {
        dma16(w[rt] + k, woff[0], slot + (wave * RT + rt) * kCodeTile);
        dma16(w[rt] + k, woff[1], slot + (wave * RT + rt) * kCodeTile + 1024);
      }
      dma16(x + k, xoff, slot + 8 * RT * kCodeTile + xload * 1024);
    };
    __syncthreads();  // the scales and slots before have been read, stores are done
    issue(0);
    // the tokens' scales come with the first block
    const uint8_t* const panel = reinterpret_cast<const uint8_t*>(xs + p0 * xs_b);
    for (int i = wave * 64; i < nb * 16 * TT; i += 512) {
      const int l = min(i + (int)lane, nb * 16 * TT - 1);
      dma4(panel, (uint32_t)(l / (16 * TT) * xs_b + xrow(l % (16 * TT))) * 4, lds_offset(scales) + i * 4);
    }
#pragma unroll
    for (int b = 1; b < SLOTS - 1; ++b)
      if (b < nb) issue(b);
    // the weights' scales are there before the loop, where the compiler's wait
    // for them would be one for every load in flight
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) asm volatile("" ::"v"(s[rt]));
    for (int b = 0; b < nb; ++b) {
      if (SLOTS > 2 && b + SLOTS - 2 < nb)
        wait_vmcnt<(SLOTS - 2) * LOADS>();  // the blocks after this one may still be on their way
      else
        wait_vmcnt<0>();
      lds_barrier();
      if (b + SLOTS - 1 < nb) issue(b + SLOTS - 1);
      const uint8_t* slot = lds + b % SLOTS * SLOT;
      const auto operand = [&](const uint8_t* tile) {
        if constexpr (FP8) return read_codes(tile, r, c);
        else return decode(read_codes(tile, r, c));
      };
      decltype(operand(slot)) wf[RT];
      float sb[RT];
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) {
        wf[rt] = operand(slot + (wave * RT + rt) * kCodeTile);
        sb[rt] = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(s[rt]), b));
      }
#pragma unroll
      for (int tt = 0; tt < TT; ++tt) {
        const auto xf = operand(slot + (8 * RT + tt) * kCodeTile);
        const float m = scales[b * 16 * TT + tt * 16 + r];
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) {
          v4f p;
          if constexpr (FP8) p = block_product_fp8(wf[rt], xf);
          else p = block_product(wf[rt], xf);
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[rt][tt][i] = __builtin_fmaf(p[i], m * sb[rt], acc[rt][tt][i]);
        }
      }
    }
  }
}

// f(tag) for the number of 16-row tiles that hold `rows` rows, at most MAX.
template <int V>
struct Tiles {
  static constexpr int value = V;
};
template <int MAX, class F>
__device__ __forceinline__ void with_tiles(int rows, F f) {
  if constexpr (MAX > 1) {
    if (rows <= 16 * (MAX - 1)) return with_tiles<MAX - 1>(rows, f);
  }
  f(Tiles<MAX>{});
}

}  // namespace fp8blk
