// The gated unit between two linears with its inputs kept in 8 bits, its
// gradient from them, and row groups turned into column groups
// (include/fp8train.h).
//
//   sig = 1 / (1 + e^-g),  h = g sig u,
//   du = dh g sig,  dg = dh u sig (1 + g (1 - sig)).
//
// All are bound by memory: per element of h the forward pass moves 4 bytes in
// and 3 out, the backward pass 4 in and 5 out, the turn 1 in and 1 out (and a
// thirty-second more for scales).  Under power-of-two scales 8192 rows of 6144 take 66
// and 103 us, 5.4 and 4.5 TB/s, and under the amax / 448 rule, whose quotients bind the
// backward pass, 68 and 114; the turn of 69632 rows of 2048 63 us.
#include "fp8blk_device.h"
#include "fp8tile_device.h"
#include "fp8train_launch.h"
#include "fp8used_device.h"

namespace fp8blk {

namespace {

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

constexpr int kThreads = 256;

// sigmoid(g).  e^-g is 2^(-g log2 e), off by about |g| 2^-24 of itself: for a
// large g it vanishes beside 1, and for a very negative one the result, which is
// then as far off, stays within 2^-17, well inside the bf16 rounding (2^-9) that
// follows.  The quotient is the hardware's reciprocal r with one correction, r + (1
// - d r) r, as near as a division in a third of the instructions (the backward pass
// on 8192 rows of 6144: 103.5 us, 106 with a division; amax / 448: 115 and 118).  The hardware's
// power of two gives 0 below fp32's normal range, which vanishes beside 1, and
// infinity beyond it, whose reciprocal is 0 and needs no correction.  A sigmoid below
// 2^-126 is not a normal number and comes out as 0: below kFarBelow see far_sigmoid.
__device__ __forceinline__ float sigmoid(float g) {
  const float d = 1.0f + __builtin_amdgcn_exp2f(g * -1.4426950408889634f);
  const float r = __builtin_amdgcn_rcpf(d);
  return d < INFINITY ? __builtin_fmaf(__builtin_fmaf(-d, r, 1.0f), r, r) : r;
}

__device__ __forceinline__ float gated(float g, float u) {
#pragma clang fp contract(off)
  return g * sigmoid(g) * u;
}

// The sigmoid of a g below -87, e^g there (1 + e^g is 1 in fp64 too), in 64 bits: times
// a u, or a dh and a u, near fp32's limit it leaves a result that is not small.  e^g is
// the fourth power of e^(g / 4), which is a normal number down to g = -349, where no
// product with two bf16 values is left.  Few waves ever come here, by a test of all that
// a wave holds, and the results of its other values are those without it.
constexpr float kFarBelow = -87.0f;
constexpr uint32_t kFarBelowBits = 0xC2AE;  // as bf16; the patterns above it are of lower values and of NaN
__device__ __forceinline__ double far_sigmoid(float g) {
  const double e = (double)__builtin_amdgcn_exp2f(g * (1.4426950408889634f / 4));
  return (e * e) * (e * e);
}

// Whether the wave holds a g below kFarBelow among eight of its lanes' values.
__device__ __forceinline__ bool any_far_below(u32x4 g) {
  const uint32_t m = pk_max_u16(pk_max_u16(g.x, g.y), pk_max_u16(g.z, g.w));
  return __builtin_amdgcn_ballot_w64(max(m & 0xFFFFu, m >> 16) > kFarBelowBits) != 0;
}

// Two elements of h (the word was) with those of a g below kFarBelow put right.
__device__ __forceinline__ uint32_t far_gated2(uint32_t g, uint32_t u, uint32_t was) {
  float h[2] = {bf16_lo(was), bf16_hi(was)};
#pragma unroll
  for (int b = 0; b < 2; ++b) {
    const float gv = b ? bf16_hi(g) : bf16_lo(g), uv = b ? bf16_hi(u) : bf16_lo(u);
    if (gv < kFarBelow) h[b] = (float)(gv * far_sigmoid(gv) * uv);
  }
  return bf16x2_rne(h[0], h[1]);
}

// ---------------------------------------------------------------------------
// Forward: 16 lanes to a group of 128 columns of g and of u, and of h.
// ---------------------------------------------------------------------------
constexpr int kUnroll = 2;
constexpr int kGroupsPerWave = 4 * kUnroll;

template <class S, bool KEEP>
__global__ __launch_bounds__(kThreads) void gated_forward_kernel(int64_t M, uint32_t G, const uint16_t* __restrict__ gu,
                                                                 int64_t ld_gu, const int32_t* __restrict__ used,
                                                                 CodesOut q, CodesOut qc) {
  const uint32_t lane = threadIdx.x & 63, sub = lane >> 4, l16 = lane & 15;
  const uint32_t total = (uint32_t)used_rows(used, M) * G;
  const uint32_t g0 = (blockIdx.x * (kThreads / 64) + (threadIdx.x >> 6)) * kGroupsPerWave;
  if (g0 >= total) return;
  const int64_t I = (int64_t)G * 128;
  u32x4 g[kUnroll], u[kUnroll];
  uint32_t row[kUnroll], grp[kUnroll];
#pragma unroll
  for (int i = 0; i < kUnroll; ++i) {
    const uint32_t at = g0 + i * 4 + sub, a = at < total ? at : 0;
    row[i] = a / G;
    grp[i] = a - row[i] * G;
    const uint16_t* p = gu + (int64_t)row[i] * ld_gu + grp[i] * 128 + l16 * 8;
    g[i] = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(p));
    u[i] = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(p + I));
  }
#pragma unroll
  for (int i = 0; i < kUnroll; ++i) {
    u32x4 h;
#pragma unroll
    for (int j = 0; j < 4; ++j)
      h[j] = bf16x2_rne(gated(bf16_lo(g[i][j]), bf16_lo(u[i][j])), gated(bf16_hi(g[i][j]), bf16_hi(u[i][j])));
    if (any_far_below(g[i])) {
#pragma unroll
      for (int j = 0; j < 4; ++j) h[j] = far_gated2(g[i][j], u[i][j], h[j]);
    }
    u32x2 oh, og, ou;
    const float sh = quant_group<S>(h, oh);
    const bool live = g0 + i * 4 + sub < total;
    const int64_t r = row[i];
    const int64_t c = grp[i] * 128 + l16 * 8;
    if (live) {
      *reinterpret_cast<u32x2*>(q.q + r * q.ld + c) = oh;
      if (l16 == 0) q.s[r * G + grp[i]] = sh;
    }
    if constexpr (KEEP) {
      const float sg = quant_group<S>(g[i], og);
      const float su = quant_group<S>(u[i], ou);
      if (live) {
        *reinterpret_cast<u32x2*>(qc.q + r * qc.ld + c) = og;
        *reinterpret_cast<u32x2*>(qc.q + r * qc.ld + I + c) = ou;
        if (l16 == 0) {
          qc.s[r * 2 * G + grp[i]] = sg;
          qc.s[r * 2 * G + G + grp[i]] = su;
        }
      }
    }
  }
}

// Two E4M3 codes (the low or high half of a word) times a power of two, exact in
// fp32, in one instruction.
template <bool HI>
__device__ __forceinline__ v2f_t decode2_pow2(uint32_t codes, float s) {
  return __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(codes, s, HI);
}

// Four E4M3 codes times their scale, rounded to bf16 (exact for power-of-two
// scales from 2^-124 on), two to a word.
__device__ __forceinline__ u32x2 decode4(uint32_t codes, float s) {
  const auto a = __builtin_amdgcn_cvt_pk_f32_fp8((int)codes, false);
  const auto b = __builtin_amdgcn_cvt_pk_f32_fp8((int)codes, true);
  return u32x2{bf16x2_rne(a[0] * s, a[1] * s), bf16x2_rne(b[0] * s, b[1] * s)};
}

// Lane I of each 16, to all of them (DPP row_newbcast).
template <int I>
__device__ __forceinline__ float from_lane(float v) {
  return __uint_as_float(dpp<0x150 + I>(__float_as_uint(v)));
}

// A thread's eight codes of each of its 8 rows of a 128 x 128 tile.  q: the tile's
// first row, the thread's first column.  The rows' scales are one load for the 16
// lanes that share the rows: lane i (or 8 + i) has row i's.
__device__ __forceinline__ void load_codes(u32x2 (&c)[8], const uint8_t* __restrict__ q, int64_t ld_q, uint32_t rb) {
#pragma unroll
  for (int i = 0; i < 8; ++i)
    c[i] = __builtin_nontemporal_load(reinterpret_cast<const u32x2*>(q + (int64_t)(rb * 8 + i) * ld_q));
}
__device__ __forceinline__ u32x4 decode8(u32x2 c, float s) {
  const u32x2 a = decode4(c.x, s), b = decode4(c.y, s);
  return u32x4{a.x, a.y, b.x, b.y};
}
// In fp32: exact under power-of-two scales, else rounded to bf16.
struct Eight {
  v2f_t v[4];
};
template <class S>
__device__ __forceinline__ Eight values8(u32x2 c, float s) {
  if constexpr (S::kScaledCvt) {
    return {decode2_pow2<false>(c.x, s), decode2_pow2<true>(c.x, s), decode2_pow2<false>(c.y, s),
            decode2_pow2<true>(c.y, s)};
  } else {
    const u32x4 w = decode8(c, s);
    Eight e;
#pragma unroll
    for (int j = 0; j < 4; ++j) e.v[j] = v2f_t{bf16_lo(w[j]), bf16_hi(w[j])};
    return e;
  }
}

// ---------------------------------------------------------------------------
// Backward: a 128 x 128 tile of h, with the tiles of g and u that it comes from.
// ---------------------------------------------------------------------------
struct GatedBackward {
  const uint16_t* dh;
  int64_t ld_dh;
  const uint8_t* qc;
  int64_t ld_qc;
  const float* sc;
  const int32_t* used;
  int64_t M;
  CodesOut q, qT, qhT;
};

// Two values rounded to bf16, now: the compiler would put the rounding off to where
// the word is used and keep both values until then.
__device__ __forceinline__ uint32_t rounded_here(float lo, float hi) {
  uint32_t w = bf16x2_rne(lo, hi);
  asm volatile("" : "+v"(w));
  return w;
}

// A code of the largest scale of the power-of-two rule may stand for 2^128, which fp32
// does not hold (255 is rounded to 256): then, and only then, a g or u is infinite.
constexpr float kTopScale = 0x1p120f;
__device__ __forceinline__ double code_value(float v) {
  return __builtin_fabsf(v) == INFINITY ? __builtin_copysign(0x1p128, (double)v) : (double)v;
}

// Word j of dg, du and h: puts those of its two elements right that are not right in 32
// bits: a g below kFarBelow, a g or u of 2^128, and a dh u past fp32's range, whose dg
// need not be.
__device__ __forceinline__ void far_row2(int j, v2f_t g, v2f_t u, uint32_t dh, u32x4& dg, u32x4& du, u32x4& h) {
  float o[3][2] = {{bf16_lo(dg[j]), bf16_hi(dg[j])}, {bf16_lo(du[j]), bf16_hi(du[j])}, {bf16_lo(h[j]), bf16_hi(h[j])}};
#pragma unroll
  for (int b = 0; b < 2; ++b) {
    const float dv = b ? bf16_hi(dh) : bf16_lo(dh);
    const bool all = g[b] < kFarBelow || __builtin_fabsf(g[b]) == INFINITY || __builtin_fabsf(u[b]) == INFINITY;
    if (!all && __builtin_fabsf(dv * u[b]) != INFINITY) continue;
    const double gv = code_value(g[b]), uv = code_value(u[b]);
    const double sig = g[b] < kFarBelow ? far_sigmoid(g[b]) : (double)sigmoid(g[b]), silu = gv * sig;
    o[0][b] = (float)(dv * uv * (sig * (1.0 + gv * (1.0 - sig))));
    if (all) {
      o[1][b] = (float)(dv * silu);
      o[2][b] = (float)(silu * uv);
    }
  }
  dg[j] = bf16x2_rne(o[0][0], o[0][1]);
  du[j] = bf16x2_rne(o[1][0], o[1][1]);
  h[j] = bf16x2_rne(o[2][0], o[2][1]);
}

// What a thread has seen that may need far_row2: the lowest g (as bits, where a lower
// negative number is a larger one; floats would be quieted first), the largest |dh u|.
struct FarSeen {
  uint32_t lowest = 0;
  float most = 0.0f;
  __device__ __forceinline__ bool any(float top_scale) const {
    return lowest > __float_as_uint(kFarBelow) || most == INFINITY || top_scale >= kTopScale;
  }
};

// dg, du and h of eight elements, two to a word.
__device__ __forceinline__ void gated_row(const Eight& g, const Eight& u, u32x4 dh, u32x4& dg, u32x4& du, u32x4& h,
                                          FarSeen& seen) {
#pragma clang fp contract(off)
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    float o[3][2];
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      const float gv = g.v[j][b], uv = u.v[j][b], dv = b ? bf16_hi(dh[j]) : bf16_lo(dh[j]);
      const float sig = sigmoid(gv), silu = gv * sig, dhu = dv * uv;
      o[0][b] = dhu * (sig * (1.0f + gv * (1.0f - sig)));
      o[1][b] = dv * silu;
      o[2][b] = silu * uv;
      seen.lowest = max(seen.lowest, __float_as_uint(gv));
      seen.most = __builtin_fmaxf(seen.most, __builtin_fabsf(dhu));
    }
    dg[j] = rounded_here(o[0][0], o[0][1]);
    du[j] = rounded_here(o[1][0], o[1][1]);
    h[j] = rounded_here(o[2][0], o[2][1]);
  }
}

template <class S, bool NT>
__global__ __launch_bounds__(kTileThreads, S::kScaledCvt ? 3 : 2) void gated_backward_kernel(GatedBackward a, TileGrid grid) {
  __shared__ TileLds lds;
  const uint32_t row_tiles = grid.row_tiles, col_tiles = grid.col_tiles;
  uint32_t rt, ct;
  tile_of(blockIdx.x, col_tiles, grid.blocked, rt, ct);
  if (ct >= col_tiles || rt >= used_tiles(a.used, a.M)) return;
  const uint32_t rb = threadIdx.x >> 4, cb = threadIdx.x & 15;
  const int64_t m0 = (int64_t)rt * 128, c0 = (int64_t)ct * 128, I = (int64_t)col_tiles * 128;
  const uint32_t G = 2 * col_tiles;
  u32x4 dh[8], g[8], u[8];
  u32x2 cg[8], cu[8];
  // lanes 0 .. 7: the rows' scales of g, 8 .. 15: of u
  const float sc = a.sc[(m0 + rb * 8 + (cb & 7)) * G + (cb < 8 ? ct : col_tiles + ct)];
  load_codes(cg, a.qc + m0 * a.ld_qc + c0 + cb * 8, a.ld_qc, rb);
  load_codes(cu, a.qc + m0 * a.ld_qc + I + c0 + cb * 8, a.ld_qc, rb);
#pragma unroll
  for (int i = 0; i < 8; ++i)
    dh[i] = __builtin_nontemporal_load(
        reinterpret_cast<const u32x4*>(a.dh + (m0 + rb * 8 + i) * a.ld_dh + c0 + cb * 8));
  // dg, du, and h in dh's place, row by row: the fence keeps the compiler from
  // working on all rows at once, which takes 372 registers (one wave a SIMD)
  FarSeen seen;
#define FP8BLK_ROW(R)                                                                                           \
  __builtin_amdgcn_sched_barrier(0);                                                                            \
  gated_row(values8<S>(cg[R], from_lane<R>(sc)), values8<S>(cu[R], from_lane<8 + R>(sc)), dh[R], g[R], u[R], dh[R], \
            seen)
  FP8BLK_ROW(0);
  FP8BLK_ROW(1);
  FP8BLK_ROW(2);
  FP8BLK_ROW(3);
  FP8BLK_ROW(4);
  FP8BLK_ROW(5);
  FP8BLK_ROW(6);
  FP8BLK_ROW(7);
#undef FP8BLK_ROW
  __builtin_amdgcn_sched_barrier(0);
  if (__builtin_amdgcn_ballot_w64(seen.any(sc)) != 0) {
    // a row at a time, its operands once more: their registers hold the results
#pragma unroll 1
    for (uint32_t i = 0; i < 8; ++i) {
      const int64_t r = m0 + rb * 8 + i;
      const uint8_t* const c = a.qc + r * a.ld_qc + c0 + cb * 8;
      const Eight gv = values8<S>(*reinterpret_cast<const u32x2*>(c), __shfl(sc, (threadIdx.x & 48) | i, 64));
      const Eight uv = values8<S>(*reinterpret_cast<const u32x2*>(c + I), __shfl(sc, (threadIdx.x & 48) | 8 | i, 64));
      const u32x4 d = *reinterpret_cast<const u32x4*>(a.dh + r * a.ld_dh + c0 + cb * 8);
      u32x4 o[3] = {g[0], u[0], dh[0]};
#pragma unroll
      for (uint32_t k = 1; k < 8; ++k)
        if (i == k) o[0] = g[k], o[1] = u[k], o[2] = dh[k];
#pragma unroll
      for (int j = 0; j < 4; ++j) far_row2(j, gv.v[j], uv.v[j], d[j], o[0], o[1], o[2]);
#pragma unroll
      for (uint32_t k = 0; k < 8; ++k)
        if (i == k) g[k] = o[0], u[k] = o[1], dh[k] = o[2];
    }
  }
  // one tensor after the other, each in both orientations: its registers are free
  // for the next
  tile_row_groups<S, NT>(g, a.q.q + m0 * a.q.ld + c0 + cb * 8, a.q.ld, a.q.s + m0 * G + ct, G, rb, cb);
  __builtin_amdgcn_sched_barrier(0);
  tile_col_groups<S, NT>(g, lds, a.qT.q + c0 * a.qT.ld + m0, a.qT.ld, a.qT.s + c0 * row_tiles + rt, row_tiles, rb, cb);
  __builtin_amdgcn_sched_barrier(0);
  tile_row_groups<S, NT>(u, a.q.q + m0 * a.q.ld + I + c0 + cb * 8, a.q.ld, a.q.s + m0 * G + col_tiles + ct, G, rb, cb);
  __syncthreads();
  __builtin_amdgcn_sched_barrier(0);
  tile_col_groups<S, NT>(u, lds, a.qT.q + (I + c0) * a.qT.ld + m0, a.qT.ld, a.qT.s + (I + c0) * row_tiles + rt,
                         row_tiles, rb, cb);
  __syncthreads();
  __builtin_amdgcn_sched_barrier(0);
  tile_col_groups<S, NT>(dh, lds, a.qhT.q + c0 * a.qhT.ld + m0, a.qhT.ld, a.qhT.s + c0 * row_tiles + rt, row_tiles, rb,
                         cb);
}

template <class S, bool NT>
__global__ __launch_bounds__(kTileThreads, 8) void requantize_kernel(const uint8_t* __restrict__ q, int64_t rows,
                                                                  int64_t ld_q, const float* __restrict__ s,
                                                                  const int32_t* __restrict__ used, CodesOut qT,
                                                                  TileGrid grid) {
  __shared__ TileLds lds;
  const uint32_t row_tiles = grid.row_tiles, col_tiles = grid.col_tiles;
  uint32_t rt, ct;
  tile_of(blockIdx.x, col_tiles, grid.blocked, rt, ct);
  if (ct >= col_tiles || rt >= used_tiles(used, rows)) return;
  const uint32_t rb = threadIdx.x >> 4, cb = threadIdx.x & 15;
  const int64_t m0 = (int64_t)rt * 128, c0 = (int64_t)ct * 128;
  u32x2 c[8];
  const float sc = s[(m0 + rb * 8 + (cb & 7)) * col_tiles + ct];
  load_codes(c, q + m0 * ld_q + c0 + cb * 8, ld_q, rb);
  const u32x4 v[8] = {decode8(c[0], from_lane<0>(sc)), decode8(c[1], from_lane<1>(sc)), decode8(c[2], from_lane<2>(sc)),
                      decode8(c[3], from_lane<3>(sc)), decode8(c[4], from_lane<4>(sc)), decode8(c[5], from_lane<5>(sc)),
                      decode8(c[6], from_lane<6>(sc)), decode8(c[7], from_lane<7>(sc))};
  tile_col_groups<S, NT>(v, lds, qT.q + c0 * qT.ld + m0, qT.ld, qT.s + c0 * row_tiles + rt, row_tiles, rb, cb);
}

template <class S>
hipError_t forward(int64_t M, int64_t I, const uint16_t* gu, int64_t ld_gu, const int32_t* used, CodesOut q,
                   CodesOut qc, hipStream_t stream) {
  const uint32_t G = (uint32_t)(I / 128);
  const uint32_t groups = (uint32_t)M * G, per = kGroupsPerWave * (kThreads / 64);
  const dim3 grid((groups + per - 1) / per), block(kThreads);
  if (qc.q)
    hipLaunchKernelGGL((gated_forward_kernel<S, true>), grid, block, 0, stream, M, G, gu, ld_gu, used, q, qc);
  else
    hipLaunchKernelGGL((gated_forward_kernel<S, false>), grid, block, 0, stream, M, G, gu, ld_gu, used, q, qc);
  return hipGetLastError();
}

template <class S, bool NT>
void backward(const GatedBackward& a, const TileGrid& g, hipStream_t stream) {
  hipLaunchKernelGGL((gated_backward_kernel<S, NT>), dim3(g.workgroups), dim3(kTileThreads), 0, stream, a, g);
}

template <class S, bool NT>
void requantize(const uint8_t* q, int64_t rows, int64_t ld_q, const float* s, const int32_t* used, CodesOut qT,
                const TileGrid& g, hipStream_t stream) {
  hipLaunchKernelGGL((requantize_kernel<S, NT>), dim3(g.workgroups), dim3(kTileThreads), 0, stream, q, rows, ld_q, s,
                     used, qT, g);
}

}  // namespace

hipError_t launch_gated_forward(int64_t M, int64_t I, const uint16_t* gu, int64_t ld_gu, const int32_t* used,
                                CodesOut q, CodesOut qc, bool fp32_scale, hipStream_t stream) {
  return fp32_scale ? forward<Fp32Scale>(M, I, gu, ld_gu, used, q, qc, stream)
                    : forward<Pow2Scale>(M, I, gu, ld_gu, used, q, qc, stream);
}

hipError_t launch_gated_backward(int64_t M, int64_t I, const uint16_t* dh, int64_t ld_dh, const uint8_t* qc,
                                 int64_t ld_qc, const float* sc, const int32_t* used, CodesOut q, CodesOut qT,
                                 CodesOut qhT, bool fp32_scale, hipStream_t stream) {
  const TileGrid g = tile_grid(M, I);
  const GatedBackward a{dh, ld_dh, qc, ld_qc, sc, used, M, q, qT, qhT};
  const bool nt = 5 * M * I > kStoreNt;
  if (fp32_scale)
    nt ? backward<Fp32Scale, true>(a, g, stream) : backward<Fp32Scale, false>(a, g, stream);
  else
    nt ? backward<Pow2Scale, true>(a, g, stream) : backward<Pow2Scale, false>(a, g, stream);
  return hipGetLastError();
}

hipError_t launch_requantize_colgroup(const uint8_t* q, int64_t rows, int64_t cols, int64_t ld_q, const float* s,
                                      const int32_t* used, CodesOut qT, bool fp32_scale, hipStream_t stream) {
  const TileGrid g = tile_grid(rows, cols);
  const bool nt = rows * cols > kStoreNt;
  if (fp32_scale)
    nt ? requantize<Fp32Scale, true>(q, rows, ld_q, s, used, qT, g, stream)
       : requantize<Fp32Scale, false>(q, rows, ld_q, s, used, qT, g, stream);
  else
    nt ? requantize<Pow2Scale, true>(q, rows, ld_q, s, used, qT, g, stream)
       : requantize<Pow2Scale, false>(q, rows, ld_q, s, used, qT, g, stream);
  return hipGetLastError();
}

}  // namespace fp8blk
