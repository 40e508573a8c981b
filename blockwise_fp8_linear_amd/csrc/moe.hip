// A mixture-of-experts layer for a few tokens (include/fp8moe.h), gfx950:
//   y[t] = sum_i w[t][i] Wd[e] q(bf16(silu(G[e] x) * (U[e] x))), e = ids[t][i],
// q the quantizer in groups of 128.  Bound by reading the weights of the
// experts reached, 3 H I bytes each; everything else is small beside it, or
// (for one token) a chain of short launches.  A few tokens: the logits (and,
// of a small router, the choice), gate/up with the choice, down, and the sum of
// its parts where there are several.  More: the logits, the choice with x's
// codes (a small router: all three in one launch), gate/up, down, the sum over a
// token's choices.
#include "fp8blk_launch.h"
#include "fp8moe_launch.h"
#include "fp8route_device.h"
#include "fp8rows_device.h"

namespace fp8blk {

namespace {

// ---------------------------------------------------------------------------
// Router logits x wr^T, fp32: 16 experts x 16 tokens per workgroup, the waves
// split H.  Bound by the latency of its loads (64 experts x 2048: 4.3 us for one
// token, 5.6 for 256; 8 waves instead of 16 0.8 us more).
// ---------------------------------------------------------------------------
constexpr int kLogitsWaves = 16;
__global__ __launch_bounds__(64 * kLogitsWaves) void logits_kernel(int T, int E, int H, const uint16_t* __restrict__ x,
                                                                   int64_t ld_x, const uint16_t* __restrict__ wr,
                                                                   float* __restrict__ logits) {
  __shared__ v4f red[kLogitsWaves][64];
  const int lane = threadIdx.x & 63, r = lane & 15, c = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int e0 = blockIdx.x * 16, t0 = blockIdx.y * 16, nkb = H / 128;
  const uint16_t* wp = wr + (int64_t)min(e0 + r, E - 1) * H + c * 16;
  const uint16_t* xp = x + (int64_t)min(t0 + r, T - 1) * ld_x + c * 16;
  v4f acc{};
  for (int b = wave; b < nkb; b += kLogitsWaves) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int at = b * 128 + (j >> 1) * 64 + (j & 1) * 8;
      acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(*reinterpret_cast<const v8bf_t*>(wp + at),
                                                    *reinterpret_cast<const v8bf_t*>(xp + at), acc, 0, 0, 0);
    }
  }
  red[wave][lane] = acc;
  __syncthreads();
  if (wave == 0) {
#pragma unroll
    for (int w = 1; w < kLogitsWaves; ++w) acc += red[w][lane];
    const int t = t0 + r;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (t < T && e0 + 4 * c + i < E) logits[(int64_t)t * E + e0 + 4 * c + i] = acc[i];
  }
}

// The choice of one token by one wave, from its logits.
template <int NI>
__device__ __forceinline__ RouteChoice choose(const float* __restrict__ row, int E, int k, bool renorm, int lane) {
  float v[NI];
#pragma unroll
  for (int i = 0; i < NI; ++i) v[i] = lane + i * 64 < E ? row[lane + i * 64] : -INFINITY;
  return route_choose<64, NI>(v, k, renorm, lane);
}
__device__ __forceinline__ RouteChoice choose(const float* __restrict__ row, int E, int k, bool renorm, int lane) {
  if (E <= 64) return choose<1>(row, E, k, renorm, lane);
  if (E <= 128) return choose<2>(row, E, k, renorm, lane);
  if (E <= 256) return choose<4>(row, E, k, renorm, lane);
  return choose<16>(row, E, k, renorm, lane);
}

// ---------------------------------------------------------------------------
// One workgroup per token: its choice, and (where qx is given) its row of x
// quantized, 16 lanes per group of 128, the scales transposed, [H / 128][T].
//   WR: the logits are found here too, a wave taking four experts at a time,
// each lane 8 neighbouring values of every 512: whole lines, fp32 sums of exact
// products.  One CU reads all of wr for its token: faster than a launch of its
// own for the logits while wr is small (40 tokens, 32 experts x 1024: 28.2
// instead of 29.2 us for a layer, and one launch of the host's less), slower
// when it is not (512 tokens, 64 x 2048: 95.7 and 88.9; one token: 27.5 and
// 25.1).  Otherwise the choice is from `logits`, if there are any.
//   Bound by latency: 4 us for 256 tokens of 2048 with 64 logits.
// ---------------------------------------------------------------------------
constexpr int64_t kTokenLogits = 64 * 1024;  // E H, at most

template <bool WR>
constexpr int kTokenThreads = WR ? 1024 : 256;

template <bool WR, class S>
__global__ __launch_bounds__(kTokenThreads<WR>) void token_kernel(MoeArgs a, const float* __restrict__ logits,
                                                                  uint8_t* __restrict__ qx, float* __restrict__ sx) {
  __shared__ float row[WR ? 1024 : 1];
  const int t = blockIdx.x, l16 = threadIdx.x & 15, lane = threadIdx.x & 63;
  const uint16_t* x = a.x + t * a.ld_x;
  if constexpr (WR) {
    const int wave = threadIdx.x >> 6;
    for (int e0 = wave * 4; e0 < a.E; e0 += 64) {
      float sum[4] = {};
#pragma unroll 4
      for (int h = lane * 8; h < a.H; h += 512) {
        const u32x4 v = *reinterpret_cast<const u32x4*>(x + h);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const u32x4 w = *reinterpret_cast<const u32x4*>(a.wr + (int64_t)min(e0 + i, a.E - 1) * a.H + h);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            sum[i] = __builtin_fmaf(bf16_lo(w[j]), bf16_lo(v[j]), sum[i]);
            sum[i] = __builtin_fmaf(bf16_hi(w[j]), bf16_hi(v[j]), sum[i]);
          }
        }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float s = lanes_sum<64>(sum[i]);
        if (lane == 0 && e0 + i < a.E) row[e0 + i] = s;
      }
    }
  }
  if (qx) {
    for (int g = threadIdx.x >> 4; g < a.H / 128; g += kTokenThreads<WR> / 16) {
      const u32x4 v = *reinterpret_cast<const u32x4*>(x + g * 128 + l16 * 8);
      float scale;
      *reinterpret_cast<uint2*>(qx + (int64_t)t * a.H + g * 128 + l16 * 8) = quantize8<S>(v, &scale);
      if (l16 == 0) sx[(int64_t)g * a.T + t] = scale;
    }
  }
  if constexpr (WR) __syncthreads();
  if ((WR || logits) && threadIdx.x < 64) {
    const RouteChoice c = choose(WR ? row : logits + (int64_t)t * a.E, a.E, a.k, a.renorm, lane);
    if (lane < a.k) {
      a.ids[t * a.k + lane] = c.id;
      a.weights[t * a.k + lane] = c.weight;
    }
  }
}

// The rows t k + j (j-th choice of token t) that chose expert e, in order, into
// `list`; their number.  Every thread of a workgroup of 512 calls it.
__device__ __forceinline__ int rows_of_expert(const int32_t* __restrict__ ids, int n, int e, uint16_t* list,
                                              int* scratch) {
  constexpr int N = 4;  // places per thread and round, loaded together
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  int found = 0;
  for (int s0 = 0; s0 < n; s0 += 512 * N) {
    uint64_t mask[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int s = s0 + i * 512 + threadIdx.x;
      mask[i] = __ballot(ids[min(s, n - 1)] == e && s < n);
    }
    if (lane < N) {
      int count = 0;
#pragma unroll
      for (int i = 0; i < N; ++i) count = lane == i ? __popcll(mask[i]) : count;
      scratch[lane * 8 + wave] = count;
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) {
      int before = found;
      for (int w = 0; w < 8; ++w) {
        const int count = scratch[i * 8 + w];
        before += w < wave ? count : 0;
        found += count;
      }
      if ((mask[i] >> lane) & 1)
        list[before + __popcll(mask[i] & ((1ull << lane) - 1))] = (uint16_t)(s0 + i * 512 + threadIdx.x);
    }
    __syncthreads();
  }
  return found;
}

// Whether the layer's own choice for a token, whose first id is `first`, found
// no expert.  That is where every logit is NaN or -infinity, so x[t], wr or
// their product is not finite: the result is NaN, where the zeros of a token
// that the caller gives no expert (a padded one) would hide it.
__device__ __forceinline__ bool none_chosen(const MoeArgs& a, int first) { return a.wr && first < 0; }
__device__ __forceinline__ v4f none() {
  const float nan = __uint_as_float(0x7FC00000u);
  return v4f{nan, nan, nan, nan};
}

__device__ __forceinline__ float silu(float g) { return g / (1.0f + expf(-g)); }

// ---------------------------------------------------------------------------
// Up to 16 tokens: the tokens themselves are the columns of the matrix
// instruction, whichever expert is multiplied, and the waves of a workgroup
// split the reduction, so that a few experts of one token fill the chip: 8 of
// 64 experts of 1024 are 512 workgroups of gate/up, where the wide kernel below
// has 64 (20 and 27 us for both products).
// ---------------------------------------------------------------------------
constexpr int kParts = 16;  // workgroups that share a column of y, at most

// The choice of the whole call in LDS, and the experts it reaches, in the order
// of their first mention.
struct FewChoice {
  int32_t ids[kFew * 16];    // -1 where there is none
  float weights[kFew * 16];
  int32_t first[1024];       // by expert: the first place that names it
};

// Fills it: from the logits (ROUTE), or from a.ids and a.weights.  Every
// thread of the workgroup calls it.
template <bool ROUTE>
__device__ __forceinline__ void few_choice(const MoeArgs& a, const float* __restrict__ logits, FewChoice& f) {
  const int n = a.T * a.k, lane = threadIdx.x & 63, wave = threadIdx.x >> 6, waves = blockDim.x >> 6;
  for (int i = threadIdx.x; i < a.E; i += blockDim.x) f.first[i] = n;
  if constexpr (ROUTE) {
    for (int t = wave; t < a.T; t += waves) {
      const RouteChoice c = choose(logits + (int64_t)t * a.E, a.E, a.k, a.renorm, lane);
      if (lane < a.k) {
        f.ids[t * a.k + lane] = c.id;
        f.weights[t * a.k + lane] = c.weight;
      }
    }
  } else {
    for (int s = threadIdx.x; s < n; s += blockDim.x) {
      const int id = a.ids[s];
      f.ids[s] = id >= 0 && id < a.E ? id : -1;
      f.weights[s] = a.weights[s];
    }
  }
  __syncthreads();
  for (int s = threadIdx.x; s < n; s += blockDim.x)
    if (f.ids[s] >= 0) atomicMin(&f.first[f.ids[s]], s);  // a minimum: the order does not matter
  __syncthreads();
}

// The `want`-th expert reached, -1 if there are fewer; by one wave.
__device__ __forceinline__ int few_expert(const FewChoice& f, int n, int want) {
  const int lane = threadIdx.x & 63;
  int before = 0;
  for (int s0 = 0; s0 < n; s0 += 64) {
    const int s = s0 + lane, id = s < n ? f.ids[s] : -1;
    const uint64_t mask = __ballot(id >= 0 && f.first[max(id, 0)] == s);
    const int rank = before + __popcll(mask & ((1ull << lane) - 1));
    const uint64_t found = __ballot(((mask >> lane) & 1) && rank == want);
    if (found) return __builtin_amdgcn_readlane(id, __builtin_ctzll(found));
    before += __popcll(mask);
  }
  return -1;
}

// The first place of token t that names expert e, -1 if there is none.
__device__ __forceinline__ int few_place(const FewChoice& f, int t, int k, int e) {
  for (int j = 0; j < k; ++j)
    if (f.ids[t * k + j] == e) return t * k + j;
  return -1;
}

// h[place] = bf16(silu(G x) * (U x)): 16 columns of I of the blockIdx.y-th
// expert reached.  XL loads bring x's rows of a block, 4 each.  H 2048, I 1024:
// 9.7 us for one token's 8 experts (3.5 TB/s, a launch's start and two
// latencies), 20.7 for the 28 experts of four (5.6 TB/s).
template <int W, int XL, int D, bool ROUTE, class S>
__global__ __launch_bounds__(64 * W) void gate_up_few_kernel(MoeArgs a, const float* __restrict__ logits,
                                                             uint16_t* __restrict__ h) {
  extern __shared__ uint8_t lds[];  // the waves' areas; then their sums, [W][2][64] v4f
  __shared__ FewChoice f;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int nkb = a.H / 128, n = a.T * a.k;
  few_choice<ROUTE>(a, logits, f);
  if (ROUTE && blockIdx.x == 0 && blockIdx.y == 0) {
    for (int s = threadIdx.x; s < n; s += 64 * W) {
      a.ids[s] = f.ids[s];
      a.weights[s] = f.weights[s];
    }
  }
  const int e = few_expert(f, n, blockIdx.y);
  if (e < 0) return;

  const uint8_t* base = a.qw1 + (int64_t)e * 2 * a.I * a.H;
  const float* sbase = a.sw1 + (int64_t)e * (2 * a.I / 128) * nkb;
  const float* const none[1] = {nullptr};
  uint32_t xoff[1][XL];
#pragma unroll
  for (int u = 0; u < XL; ++u)
    xoff[0][u] = (uint32_t)(min((int)raw_row(lane, u), a.T - 1) * a.ld_x * 2) + (lane & 15) * 16;
  v4f* red = reinterpret_cast<v4f*>(lds);
  const int place = wave == 0 && (lane & 15) < a.T ? few_place(f, lane & 15, a.k, e) : -1;
  for (int n0 = blockIdx.x * 16; n0 < a.I; n0 += gridDim.x * 16) {
    const uint8_t* const wp[2] = {base + (int64_t)n0 * a.H, base + (int64_t)(a.I + n0) * a.H};
    const float* const sp[2] = {sbase + n0 / 128 * nkb, sbase + (a.I + n0) / 128 * nkb};
    v4f acc[2][1] = {};
    rows_product<2, 1, XL, D, true, S>(lds + wave * D * rows_stage_bytes<2, 1, true, XL>(), wp, sp, a.H,
                                       reinterpret_cast<const uint8_t*>(a.x), xoff, none, 0, wave * nkb / W,
                                       (wave + 1) * nkb / W, acc);
    __syncthreads();
    red[(wave * 2) * 64 + lane] = acc[0][0];
    red[(wave * 2 + 1) * 64 + lane] = acc[1][0];
    __syncthreads();
    if (place >= 0) {
      v4f g = red[lane], u = red[64 + lane];
      for (int w = 1; w < W; ++w) {
        g += red[w * 128 + lane];
        u += red[w * 128 + 64 + lane];
      }
      *reinterpret_cast<uint2*>(h + (int64_t)place * a.I + n0 + 4 * (lane >> 4)) =
          make_uint2(bf16x2_rne(silu(g[0]) * u[0], silu(g[1]) * u[1]),
                     bf16x2_rne(silu(g[2]) * u[2], silu(g[3]) * u[3]));
    }
    __syncthreads();  // before the sums are overwritten
  }
}

// y, 16 columns of H per workgroup: the blocks of all experts reached are one
// long reduction, which the workgroups of a column (gridDim.y) and their waves
// split; a term's routing weight goes into its block's scale.  RAW: h is bf16
// [place][I] and quantized here; otherwise it is codes, with the scales
// sh[I / 128][place].  With several workgroups per column their sums go to
// partial[blockIdx.y][t][H] instead of y: H / 16 workgroups are too few to read
// many blocks (9 tokens, 7 experts of 6144: 40 us, in three parts 22.6 or 4.2
// TB/s, and 3.9 for the sum).
template <int W, int XL, int D, bool RAW, class S>
__global__ __launch_bounds__(64 * W) void down_few_kernel(MoeArgs a, const uint8_t* __restrict__ h,
                                                          const float* __restrict__ sh, float* __restrict__ partial) {
  extern __shared__ uint8_t lds[];  // the waves' areas; then their sums, [W][64] v4f
  __shared__ FewChoice f;
  __shared__ int16_t place[kFew * 16][kFew];  // by expert reached and token: the place whose h it is, -1 none
  __shared__ float weight[kFew * 16];         // by place: of the expert named there, all of its token's mentions
  __shared__ int16_t expert[kFew * 16];
  constexpr int SB = rows_stage_bytes<1, 1, RAW, XL>(), ROWS = XL * (RAW ? 4 : 8), TILE = ROWS * 128;
  const int lane = threadIdx.x & 63, r = lane & 15, c = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int n0 = blockIdx.x * 16, nkb = a.I / 128, n = a.T * a.k;
  few_choice<false>(a, nullptr, f);
  int reached = 0;
  for (int s0 = 0; s0 < n; s0 += 64) {  // every wave finds the same list
    const int s = s0 + lane, id = s < n ? f.ids[s] : -1;
    const bool is = id >= 0 && f.first[max(id, 0)] == s;
    const uint64_t mask = __ballot(is);
    if (is) expert[reached + __popcll(mask & ((1ull << lane) - 1))] = (int16_t)id;
    reached += __popcll(mask);
  }
  __syncthreads();
  for (int i = threadIdx.x; i < reached * kFew; i += 64 * W) {
    const int at = i / kFew, t = i % kFew, e = expert[at];
    int p = -1;
    float w = 0.0f;
    if (t < a.T) {
      for (int j = a.k - 1; j >= 0; --j) {
        if (f.ids[t * a.k + j] == e) {
          p = t * a.k + j;
          w += f.weights[p];
        }
      }
    }
    place[at][t] = (int16_t)p;
    if (p >= 0) weight[p] = w;
  }
  __syncthreads();

  v4f acc{};
  uint8_t* const area = lds + wave * D * SB;
  const uint32_t at0 = lds_offset(area), xr = min(r, ROWS - 1);
  const uint32_t woff[2] = {(uint32_t)(code_row(lane, 0) * a.I) + code_chunk(lane, 0),
                            (uint32_t)(code_row(lane, 1) * a.I) + code_chunk(lane, 1)};
  const int64_t total = (int64_t)reached * nkb, parts = (int64_t)gridDim.y * W, part = (int64_t)blockIdx.y * W + wave;
  const int end = (int)((part + 1) * total / parts);
  for (int b = (int)(part * total / parts); b < end; b += D) {
    float s[D], m[D];
    u32x4 v[D][RAW ? XL : 1];
#pragma unroll
    for (int d = 0; d < D; ++d) {
      if (b + d >= end) break;
      const int which = (b + d) / nkb, i = b + d - which * nkb;
      const int e = __builtin_amdgcn_readfirstlane(expert[which]);
      const uint8_t* w = a.qw2 + ((int64_t)e * a.H + n0) * a.I + (int64_t)i * 128;
      dma16(w, woff[0], at0 + d * SB);
      dma16(w, woff[1], at0 + d * SB + 1024);
      s[d] = a.sw2[((int64_t)e * (a.H / 128) + n0 / 128) * nkb + i];
#pragma unroll
      for (int u = 0; u < XL; ++u) {
        const int64_t p = max((int)place[which][RAW ? raw_row(lane, u) : code_row(lane, u)], 0);
        if constexpr (RAW)
          v[d][u] = *reinterpret_cast<const u32x4*>(h + (p * a.I + i * 128) * 2 + (lane & 15) * 16);
        else
          dma16(h + (int64_t)i * 128, (uint32_t)(p * a.I) + code_chunk(lane, u), at0 + d * SB + kCodeTile + u * 1024);
      }
      if constexpr (!RAW) m[d] = sh[(int64_t)i * n + max((int)place[which][r], 0)];
    }
    if constexpr (RAW) {
#pragma unroll
      for (int d = 0; d < D; ++d) {
        if (b + d >= end) break;
#pragma unroll
        for (int u = 0; u < XL; ++u)
          quantize_into<S>(area + d * SB + kCodeTile, reinterpret_cast<float*>(area + d * SB + kCodeTile + TILE),
                           v[d][u], lane, u);
      }
    }
    loads_landed();
#pragma unroll
    for (int d = 0; d < D; ++d) {
      if (b + d >= end) break;
      const int which = (b + d) / nkb, p = place[which][r];
      const uint8_t* st = area + d * SB;
      if constexpr (RAW) m[d] = reinterpret_cast<const float*>(st + kCodeTile + TILE)[xr];
      const v4f prod = block_product(decode(read_codes(st, r, c)), decode(read_codes(st + kCodeTile, xr, c)));
      const float scale = m[d] * weight[max(p, 0)] * s[d];
#pragma unroll
      for (int i = 0; i < 4; ++i)  // others' values do not come near (they may not even be finite)
        acc[i] = p >= 0 ? __builtin_fmaf(prod[i], scale, acc[i]) : acc[i];
    }
    reads_returned();
  }
  v4f* red = reinterpret_cast<v4f*>(lds);
  __syncthreads();
  red[wave * 64 + lane] = acc;
  __syncthreads();
  if (wave == 0 && r < a.T) {
    v4f v = red[lane];
    for (int w = 1; w < W; ++w) v += red[w * 64 + lane];
    if (none_chosen(a, f.ids[r * a.k])) v = none();
    const int64_t at = (int64_t)r * a.H + n0 + 4 * c;
    if (gridDim.y > 1)
      *reinterpret_cast<v4f*>(partial + (int64_t)blockIdx.y * a.T * a.H + at) = v;
    else
      store_rows<false>(a.out, at, v);
  }
}

// y = the sum of `parts` partial results, in their order.
__global__ __launch_bounds__(256) void sum_parts_kernel(MoeArgs a, const float* __restrict__ partial, int parts) {
  const int64_t at = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4, size = (int64_t)a.T * a.H;
  if (at >= size) return;
  v4f v{};
  for (int p = 0; p < parts; ++p) v += *reinterpret_cast<const v4f*>(partial + p * size + at);
  store_rows<false>(a.out, at, v);
}

// ---------------------------------------------------------------------------
// The same two products for more tokens: each wave owns 16 columns of I (their
// G and their U rows), or 16 RT columns of H, over the whole reduction, and the
// eight waves of a workgroup share the tokens' codes in LDS.  128 columns of I
// in one workgroup are one group of h, so h leaves quantized.  TMAX tiles of 16
// rows at once; an expert with more rows is read again (from L2 or the
// memory-side cache) for the rest, by the same workgroup or (gridDim.z) another.
//   40 tokens, 121 of 128 experts of 768 reached: gate/up 69 us (5.5 TB/s),
//   down 35 (5.4); 256 tokens, 64 experts of 1024: 59 (4.5) and 35 (3.8).
// ---------------------------------------------------------------------------
// Dynamic LDS: the slots for the most tiles, then the list of rows.
constexpr int kMostRows = 8192;  // T k
template <int RT, int TMAX, int SLOTS>
constexpr int kRing = rows_ring_bytes<RT, TMAX, SLOTS>();

template <int TMAX, int SLOTS, class S>
__global__ __launch_bounds__(512) void gate_up_wide_kernel(MoeArgs a, const uint8_t* __restrict__ qx,
                                                           const float* __restrict__ sx, uint8_t* __restrict__ qh,
                                                           float* __restrict__ sh) {
  extern __shared__ uint8_t lds[];
  __shared__ int scratch[4 * 8];
  __shared__ uint32_t amax[8][16 * TMAX];
  uint16_t* const list = reinterpret_cast<uint16_t*>(lds + kRing<2, TMAX, SLOTS>);
  const int lane = threadIdx.x & 63, r = lane & 15, c = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int e = blockIdx.y, n0 = blockIdx.x * 128 + wave * 16, nkb = a.H / 128;
  const int rows = rows_of_expert(a.ids, a.T * a.k, e, list, scratch);

  const uint8_t* base = a.qw1 + (int64_t)e * 2 * a.I * a.H;
  const float* sbase = a.sw1 + (int64_t)e * (2 * a.I / 128) * nkb;
  const uint8_t* const wp[2] = {base + (int64_t)n0 * a.H, base + (int64_t)(a.I + n0) * a.H};
  const float* const sp[2] = {sbase + n0 / 128 * nkb, sbase + (a.I + n0) / 128 * nkb};
  for (int r0 = blockIdx.z * 16 * TMAX; r0 < rows; r0 += gridDim.z * 16 * TMAX) {
    with_tiles<TMAX>(rows - r0, [&](auto tag) {
      constexpr int TT = decltype(tag)::value;
      const int load = wave % (2 * TT), row = r0 + (load >> 1) * 16 + code_row(lane, load & 1);
      const uint32_t xoff = (uint32_t)(list[min(row, rows - 1)] / a.k) * a.H + code_chunk(lane, load & 1);
      v4f acc[2][TT];
#pragma unroll
      for (int tt = 0; tt < TT; ++tt) acc[0][tt] = acc[1][tt] = v4f{};
      rows_ring<2, TT, SLOTS>(
          lds, wp, sp, a.H, qx, xoff, sx, a.T, [&](int i) { return list[min(r0 + i, rows - 1)] / a.k; }, nkb, acc);
      uint32_t h[TT][2];
#pragma unroll
      for (int tt = 0; tt < TT; ++tt) {
        const v4f g = acc[0][tt], u = acc[1][tt];
        h[tt][0] = bf16x2_rne(silu(g[0]) * u[0], silu(g[1]) * u[1]);
        h[tt][1] = bf16x2_rne(silu(g[2]) * u[2], silu(g[3]) * u[3]);
        const uint32_t m = pk_max_u16(abs2(h[tt][0]), abs2(h[tt][1]));
        amax[wave][tt * 16 + r] = quarter_max(max(m & 0xFFFFu, m >> 16));
      }
      __syncthreads();
#pragma unroll
      for (int tt = 0; tt < TT; ++tt) {
        uint32_t m = 0;
#pragma unroll
        for (int w = 0; w < 8; ++w) m = max(m, amax[w][tt * 16 + r]);
        const S sc(m);
        const int row = r0 + tt * 16 + r;
        if (row < rows) {
          const int64_t s = list[row];
          *reinterpret_cast<uint32_t*>(qh + s * a.I + n0 + 4 * c) = quant4(h[tt][0], h[tt][1], sc);
          if (wave == 0 && c == 0) sh[(int64_t)blockIdx.x * (a.T * a.k) + s] = sc.s;
        }
      }
      // (the next rows' maxima are written behind rows_ring's barriers)
    });
  }
}

template <int RT, int TMAX, int SLOTS>
__global__ __launch_bounds__(512) void down_wide_kernel(MoeArgs a, const uint8_t* __restrict__ qh,
                                                        const float* __restrict__ sh, float* __restrict__ partial) {
  extern __shared__ uint8_t lds[];
  __shared__ int scratch[4 * 8];
  uint16_t* const list = reinterpret_cast<uint16_t*>(lds + kRing<RT, TMAX, SLOTS>);
  const int lane = threadIdx.x & 63, r = lane & 15, c = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int e = blockIdx.y, n0 = (blockIdx.x * 8 + wave) * 16 * RT, nkb = a.I / 128;
  // waves past the last column (H may be an odd number of 128s) repeat it: they
  // pass the barriers and store nothing
  const int n = min(n0, a.H - 16 * RT);
  const int rows = rows_of_expert(a.ids, a.T * a.k, e, list, scratch);

  const uint8_t* base = a.qw2 + ((int64_t)e * a.H + n) * a.I;
  const float* s = a.sw2 + ((int64_t)e * (a.H / 128) + n / 128) * nkb;
  const uint8_t* wp[RT];
  const float* sp[RT];
#pragma unroll
  for (int rt = 0; rt < RT; ++rt) {
    wp[rt] = base + (int64_t)rt * 16 * a.I;
    sp[rt] = s;
  }
  for (int r0 = blockIdx.z * 16 * TMAX; r0 < rows; r0 += gridDim.z * 16 * TMAX) {
    with_tiles<TMAX>(rows - r0, [&](auto tag) {
      constexpr int TT = decltype(tag)::value;
      const int load = wave % (2 * TT), row = r0 + (load >> 1) * 16 + code_row(lane, load & 1);
      const uint32_t xoff = (uint32_t)list[min(row, rows - 1)] * a.I + code_chunk(lane, load & 1);
      v4f acc[RT][TT];
#pragma unroll
      for (int rt = 0; rt < RT; ++rt)
#pragma unroll
        for (int tt = 0; tt < TT; ++tt) acc[rt][tt] = v4f{};
      rows_ring<RT, TT, SLOTS>(
          lds, wp, sp, a.I, qh, xoff, sh, a.T * a.k, [&](int i) { return (int)list[min(r0 + i, rows - 1)]; }, nkb,
          acc);
#pragma unroll
      for (int tt = 0; tt < TT; ++tt) {
        const int row = r0 + tt * 16 + r;
        if (row < rows && n0 < a.H) {
          const int64_t s = list[row];
          const float w = a.weights[s];
#pragma unroll
          for (int rt = 0; rt < RT; ++rt)
            *reinterpret_cast<v4f*>(partial + s * a.H + n0 + rt * 16 + 4 * c) = acc[rt][tt] * w;
        }
      }
    });
  }
}

// y[t] = the sum of the token's terms in the order of its choice; ids that are
// none have no term.
__global__ __launch_bounds__(256) void combine_kernel(MoeArgs a, const float* __restrict__ partial) {
  const int u = blockIdx.x * 256 + threadIdx.x, per = a.H / 4;
  const int t = u / per, n = (u - t * per) * 4;
  if (t >= a.T) return;
  v4f v = none_chosen(a, a.ids[t * a.k]) ? none() : v4f{};
  for (int j0 = 0; j0 < a.k; j0 += 4) {  // the terms of four choices are loaded together
    v4f term[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int s = t * a.k + min(j0 + j, a.k - 1), id = a.ids[s];
      const bool is = j0 + j < a.k && id >= 0 && id < a.E;
      term[j] = is ? *reinterpret_cast<const v4f*>(partial + (int64_t)s * a.H + n) : v4f{};
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) v += term[j];
  }
  store_rows<false>(a.out, (int64_t)t * a.H + n, v);
}

// The launches of up to kFew tokens, and of more.
struct MoeBuffers {
  float* logits;  // null where ids and weights are there already
  uint8_t *qx, *h;
  float *sx, *sh, *partial;
};

// `reached`: about how many experts the tokens reach.
template <int XL, bool RAW, class S>
hipError_t down_few(const MoeArgs& a, const MoeBuffers& b, double reached, hipStream_t stream) {
  constexpr int W = RAW && XL <= 2 ? 16 : 8, D = RAW && XL != 2 ? 2 : 1;
  constexpr int lds = W * D * rows_stage_bytes<1, 1, RAW, XL>();
  static_assert(lds >= W * 1024, "the waves' sums fit");
  static std::atomic<uint64_t> raised{0};
  const auto k = &down_few_kernel<W, XL, D, RAW, S>;
  if (hipError_t e = ensure_lds_limit(reinterpret_cast<const void*>(k), lds, &raised)) return e;
  // as many parts as leave a wave a few rounds of loads, up to one workgroup per
  // CU where only one fits, else two (four tokens, 28 experts of 1024: 2 parts 42
  // us, 3 parts 47; 16 tokens, 56 experts: 4 parts 80, 5 parts 84, 6 parts 82)
  const int columns = a.H / 16, most = (RAW && XL == 1 ? 256 : 512) / columns;
  int parts = (int)(reached * (a.I / 128) / (W * D * (W == 16 ? 2 : 4)));
  if (parts > most) parts = most;
  parts = parts < 1 ? 1 : parts > kParts ? kParts : parts;
  hipLaunchKernelGGL(k, dim3(a.H / 16, parts), dim3(64 * W), lds, stream, a, b.h, b.sh, b.partial);
  if (parts == 1) return hipGetLastError();
  if (hipError_t e = hipGetLastError()) return e;
  hipLaunchKernelGGL(sum_parts_kernel, dim3((a.T * (a.H / 4) + 255) / 256), dim3(256), 0, stream, a, b.partial, parts);
  return hipGetLastError();
}

template <int XL, class S>
hipError_t moe_few(const MoeArgs& a, const MoeBuffers& b, double reached, hipStream_t stream) {
  constexpr int W = 8, D = 1, lds = W * D * rows_stage_bytes<2, 1, true, XL>();
  static_assert(lds >= W * 2 * 1024, "the waves' sums fit");
  static std::atomic<uint64_t> raised[2];
  const auto k = b.logits ? &gate_up_few_kernel<W, XL, D, true, S> : &gate_up_few_kernel<W, XL, D, false, S>;
  if (hipError_t e = ensure_lds_limit(reinterpret_cast<const void*>(k), lds, &raised[b.logits != nullptr])) return e;
  const int most = a.T * a.k < a.E ? a.T * a.k : a.E;  // experts reached
  hipLaunchKernelGGL(k, dim3(few_columns(a.T, a.I, a.E, a.k), most), dim3(64 * W), lds, stream, a, b.logits,
                     reinterpret_cast<uint16_t*>(b.h));
  if (hipError_t e = hipGetLastError()) return e;
  return down_few<XL, true, S>(a, b, reached, stream);
}

template <int TT, int SLOTS, class S>
hipError_t gate_up_launch(const MoeArgs& a, const MoeBuffers& b, int parts, hipStream_t stream) {
  static std::atomic<uint64_t> raised{0};
  const auto k = &gate_up_wide_kernel<TT, SLOTS, S>;
  constexpr int ring = kRing<2, TT, SLOTS>;
  if (hipError_t e = ensure_lds_limit(reinterpret_cast<const void*>(k), ring + kMostRows * 2, &raised)) return e;
  hipLaunchKernelGGL(k, dim3(a.I / 128, a.E, parts), dim3(512), ring + a.T * a.k * 2, stream, a, b.qx, b.sx, b.h, b.sh);
  return hipGetLastError();
}

template <int TT, class S>
hipError_t gate_up_wide(const MoeArgs& a, const MoeBuffers& b, const WidePlan& p, hipStream_t stream) {
  return p.slots == 2 ? gate_up_launch<TT, 2, S>(a, b, p.parts, stream)
                      : gate_up_launch<TT, gate_up_slots(TT), S>(a, b, p.parts, stream);
}

template <int RT, int TT, int SLOTS>
hipError_t down_launch(const MoeArgs& a, const MoeBuffers& b, int parts, hipStream_t stream) {
  static std::atomic<uint64_t> raised{0};
  const auto k = &down_wide_kernel<RT, TT, SLOTS>;
  constexpr int ring = kRing<RT, TT, SLOTS>;
  if (hipError_t e = ensure_lds_limit(reinterpret_cast<const void*>(k), ring + kMostRows * 2, &raised)) return e;
  hipLaunchKernelGGL(k, dim3((a.H + 128 * RT - 1) / (128 * RT), a.E, parts), dim3(512), ring + a.T * a.k * 2, stream, a,
                     b.h, b.sh, b.partial);
  return hipGetLastError();
}

template <int TT>
hipError_t down_wide(const MoeArgs& a, const MoeBuffers& b, const WidePlan& p, hipStream_t stream) {
  constexpr int RT = down_columns(TT);
  return p.slots == 2 ? down_launch<RT, TT, 2>(a, b, p.parts, stream)
                      : down_launch<RT, TT, down_slots(TT)>(a, b, p.parts, stream);
}

template <class S>
hipError_t moe_wide(const MoeArgs& a, const MoeBuffers& b, hipStream_t stream) {
  const WidePlan g = gate_up_plan(a.T, a.I, a.E, a.k), d = down_plan(a.T, a.H, a.E, a.k);
  if (hipError_t e = g.tiles == 1   ? gate_up_wide<1, S>(a, b, g, stream)
                     : g.tiles == 2 ? gate_up_wide<2, S>(a, b, g, stream)
                                    : gate_up_wide<4, S>(a, b, g, stream))
    return e;
  if (hipError_t e = d.tiles == 1   ? down_wide<1>(a, b, d, stream)
                     : d.tiles == 2 ? down_wide<2>(a, b, d, stream)
                                    : down_wide<4>(a, b, d, stream))
    return e;
  hipLaunchKernelGGL(combine_kernel, dim3((a.T * (a.H / 4) + 255) / 256), dim3(256), 0, stream, a, b.partial);
  return hipGetLastError();
}

template <class S>
hipError_t moe(const MoeArgs& a, MoeBuffers b, hipStream_t stream) {
  const double reached = experts_reached(a.T, a.E, a.k);
  const bool few = few_plan(a.T, a.I, a.E, a.k, a.fp32_scale);
  // the choice: with its logits where wr is small, else from the logits' own launch, by the narrow gate/up itself or
  // with x's codes
  if (a.wr && a.E * (int64_t)a.H <= kTokenLogits) {
    hipLaunchKernelGGL((token_kernel<true, S>), dim3(a.T), dim3(kTokenThreads<true>), 0, stream, a, nullptr,
                       few ? nullptr : b.qx, b.sx);
    if (hipError_t e = hipGetLastError()) return e;
    b.logits = nullptr;
  } else {
    if (a.wr) {
      hipLaunchKernelGGL(logits_kernel, dim3((a.E + 15) / 16, (a.T + 15) / 16), dim3(64 * kLogitsWaves), 0, stream, a.T,
                         a.E, a.H, a.x, a.ld_x, a.wr, b.logits);
      if (hipError_t e = hipGetLastError()) return e;
    }
    if (!few) {
      hipLaunchKernelGGL((token_kernel<false, S>), dim3(a.T), dim3(kTokenThreads<false>), 0, stream, a, b.logits, b.qx,
                         b.sx);
      if (hipError_t e = hipGetLastError()) return e;
    }
  }
  if (few) {
    if (a.T <= 4) return moe_few<1, S>(a, b, reached, stream);
    return a.T <= 8 ? moe_few<2, S>(a, b, reached, stream) : moe_few<4, S>(a, b, reached, stream);
  }
  if (a.T <= kFew) {
    if (hipError_t e = gate_up_wide<1, S>(a, b, gate_up_plan(a.T, a.I, a.E, a.k), stream)) return e;
    return a.T <= 8 ? down_few<1, false, S>(a, b, reached, stream) : down_few<2, false, S>(a, b, reached, stream);
  }
  return moe_wide<S>(a, b, stream);
}

}  // namespace

hipError_t launch_moe(const MoeArgs& a, hipStream_t stream) {
  const MoeWorkspace w = moe_workspace(a.T, a.H, a.I, a.E, a.k);
  char* ws = static_cast<char*>(a.ws);
  const auto f32 = [ws](size_t at) { return reinterpret_cast<float*>(ws + at); };
  const MoeBuffers b{a.wr ? f32(w.logits) : nullptr, reinterpret_cast<uint8_t*>(ws + w.qx),
                     reinterpret_cast<uint8_t*>(ws + w.h), f32(w.sx), f32(w.sh), f32(w.partial)};
  return a.fp32_scale ? moe<Fp32Scale>(a, b, stream) : moe<Pow2Scale>(a, b, stream);
}

}  // namespace fp8blk
