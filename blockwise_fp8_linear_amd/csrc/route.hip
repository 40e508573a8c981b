// The router of a mixture of experts: top-k and softmax weights of each
// token's logits, and their gradient (include/fp8moe.h).
//
//   chosen = the k largest logits (equal ones by lower index)
//   w_i = exp(l_i - m) / sum_j exp(l_j - m),  j over the chosen or over all,
//   dl_j = p_j (g_j [j chosen] - sum_i g_i w_i).
//
// Bound by latency for a few tokens and by vector instructions for many.
// LANES lanes share a token (16 up to 256 experts, so that a wave takes four
// tokens and its reductions stay within a DPP row; the whole wave beyond), each
// with NI logits in registers: the logits are read once, in one pass, and the k
// rounds of the selection run on registers: a maximum of the lane's logits, one
// across the lanes, and the same again for the lowest index that has it.
//   16384 x 128 fp32, k 8: 8.0 us forward (1.1 TB/s), 10.1 backward; 4095 x 60
//   bf16, k 4: 3.2 and 4.0.  At 16384 tokens a SIMD has four waves of 851
//   (forward) and 969 (backward) vector instructions, 4 clocks each: 5.7 and 6.5
//   us of issue at 2.4 GHz, beside 8 and 10 loads a wave.  Most of the forward's
//   are the k rounds; the backward's are k times NI comparisons, which bring the
//   choices' gradients to their logits, and the exponentials.
#include "fp8blk_device.h"
#include "fp8moe_launch.h"
#include "fp8route_device.h"

namespace fp8blk {

namespace {

constexpr int kThreads = 256;
constexpr int64_t kLaunch = int64_t(1) << 24;  // tokens of one launch, which has fewer than 2^32 threads

template <class T>
__device__ __forceinline__ float to_f32(T v);
template <>
__device__ __forceinline__ float to_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ float to_f32<uint16_t>(uint16_t v) { return __uint_as_float((uint32_t)v << 16); }
__device__ __forceinline__ void store_as(float* p, float v) { *p = v; }
__device__ __forceinline__ void store_as(uint16_t* p, float v) { *p = (uint16_t)bf16x2_rne(v, 0.0f); }

template <int LANES, int NI, class L>
__global__ __launch_bounds__(kThreads) void route_kernel(int64_t T, int E, int k, const L* __restrict__ logits,
                                                         int64_t ld, bool renorm, int32_t* __restrict__ ids,
                                                         float* __restrict__ weights) {
  const int64_t t = (int64_t)blockIdx.x * (kThreads / LANES) + threadIdx.x / LANES;
  const int lane = threadIdx.x % LANES;
  const bool live = t < T;
  const L* row = logits + (live ? t : T - 1) * ld;
  float v[NI];
#pragma unroll
  for (int i = 0; i < NI; ++i) v[i] = lane + i * LANES < E ? to_f32(row[lane + i * LANES]) : -INFINITY;
  const RouteChoice c = route_choose<LANES, NI>(v, k, renorm, lane);
  if (live && lane < k) {
    ids[t * k + lane] = c.id;
    weights[t * k + lane] = c.weight;
  }
}

template <int LANES, int NI, class L>
__global__ __launch_bounds__(kThreads) void route_backward_kernel(int64_t T, int E, int k, const L* __restrict__ logits,
                                                                  int64_t ld, const int32_t* __restrict__ ids,
                                                                  const float* __restrict__ g, bool renorm,
                                                                  L* __restrict__ dlogits, int64_t ld_d) {
  const int64_t t = (int64_t)blockIdx.x * (kThreads / LANES) + threadIdx.x / LANES;
  const int lane = threadIdx.x % LANES;
  const bool live = t < T;
  const int64_t tt = live ? t : T - 1;
  const L* row = logits + tt * ld;
  float v[NI], gs[NI];
  bool chosen[NI];
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    v[i] = lane + i * LANES < E ? to_f32(row[lane + i * LANES]) : -INFINITY;
    gs[i] = 0.0f;
    chosen[i] = false;
  }
  // lane j brings the j-th choice; the others get it from there
  const int mine = lane < k ? ids[tt * k + lane] : -1;
  const float gmine = lane < k ? g[tt * k + lane] : 0.0f;
  for (int j = 0; j < k; ++j) {
    const int id = __shfl(mine, j, LANES);
    const float gj = __shfl(gmine, j, LANES);
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      if (id == lane + i * LANES && id < E && v[i] > -INFINITY) {
        gs[i] += gj;
        chosen[i] = true;
      }
    }
  }
  // the softmax over the chosen or over all; masked-out ones (not > -inf) are in neither
  float top = -INFINITY;
#pragma unroll
  for (int i = 0; i < NI; ++i)
    if (v[i] > -INFINITY && (chosen[i] || !renorm)) top = fmaxf(top, v[i]);
  top = lanes_max<LANES>(top);
  float sum = 0.0f, mean = 0.0f;
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    const bool in = v[i] > -INFINITY && (chosen[i] || !renorm);
    v[i] = in ? exp_from(v[i], top) : 0.0f;
    sum += v[i];
    mean += chosen[i] ? v[i] * gs[i] : 0.0f;
  }
  sum = lanes_sum<LANES>(sum);
  mean = lanes_sum<LANES>(mean);
  const float inv = sum > 0.0f ? 1.0f / sum : 0.0f;
  mean *= inv;
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    const int e = lane + i * LANES;
    if (live && e < E) store_as(dlogits + t * ld_d + e, v[i] > 0.0f ? v[i] * inv * (gs[i] - mean) : 0.0f);
  }
}

template <int LANES, int NI, class L>
hipError_t forward(int64_t T, int E, int k, const void* logits, int64_t ld, bool renorm, int32_t* ids, float* weights,
                   hipStream_t stream) {
  constexpr int per = kThreads / LANES;
  for (int64_t t = 0; t < T; t += kLaunch) {
    const int64_t n = T - t < kLaunch ? T - t : kLaunch;
    hipLaunchKernelGGL((route_kernel<LANES, NI, L>), dim3((uint32_t)((n + per - 1) / per)), dim3(kThreads), 0, stream,
                       n, E, k, static_cast<const L*>(logits) + t * ld, ld, renorm, ids + t * k, weights + t * k);
    if (hipError_t e = hipGetLastError()) return e;
  }
  return hipSuccess;
}

template <int LANES, int NI, class L>
hipError_t backward(int64_t T, int E, int k, const void* logits, int64_t ld, const int32_t* ids, const float* g,
                    bool renorm, void* dlogits, int64_t ld_d, hipStream_t stream) {
  constexpr int per = kThreads / LANES;
  for (int64_t t = 0; t < T; t += kLaunch) {
    const int64_t n = T - t < kLaunch ? T - t : kLaunch;
    hipLaunchKernelGGL((route_backward_kernel<LANES, NI, L>), dim3((uint32_t)((n + per - 1) / per)), dim3(kThreads), 0,
                       stream, n, E, k, static_cast<const L*>(logits) + t * ld, ld, ids + t * k, g + t * k, renorm,
                       static_cast<L*>(dlogits) + t * ld_d, ld_d);
    if (hipError_t e = hipGetLastError()) return e;
  }
  return hipSuccess;
}

}  // namespace

hipError_t launch_moe_route(int64_t T, int E, int k, const void* logits, bool f32, int64_t ld, bool renorm,
                            int32_t* ids, float* weights, hipStream_t stream) {
#define FP8MOE_ROUTE(LANES, NI)                                                                             \
  (f32 ? forward<LANES, NI, float>(T, E, k, logits, ld, renorm, ids, weights, stream)                       \
       : forward<LANES, NI, uint16_t>(T, E, k, logits, ld, renorm, ids, weights, stream))
  if (E <= 64) return FP8MOE_ROUTE(16, 4);
  if (E <= 128) return FP8MOE_ROUTE(16, 8);
  if (E <= 256) return FP8MOE_ROUTE(16, 16);
  return E <= 512 ? FP8MOE_ROUTE(64, 8) : FP8MOE_ROUTE(64, 16);
#undef FP8MOE_ROUTE
}

hipError_t launch_moe_route_backward(int64_t T, int E, int k, const void* logits, bool f32, int64_t ld,
                                     const int32_t* ids, const float* g, bool renorm, void* dlogits, int64_t ld_d,
                                     hipStream_t stream) {
#define FP8MOE_ROUTE(LANES, NI)                                                                             \
  (f32 ? backward<LANES, NI, float>(T, E, k, logits, ld, ids, g, renorm, dlogits, ld_d, stream)             \
       : backward<LANES, NI, uint16_t>(T, E, k, logits, ld, ids, g, renorm, dlogits, ld_d, stream))
  if (E <= 64) return FP8MOE_ROUTE(16, 4);
  if (E <= 128) return FP8MOE_ROUTE(16, 8);
  if (E <= 256) return FP8MOE_ROUTE(16, 16);
  return E <= 512 ? FP8MOE_ROUTE(64, 8) : FP8MOE_ROUTE(64, 16);
#undef FP8MOE_ROUTE
}

}  // namespace fp8blk
