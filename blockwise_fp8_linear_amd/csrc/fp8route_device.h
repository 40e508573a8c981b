// The router's selection on the lanes of a wave, shared by route.hip (many
// tokens) and moe.hip (the few tokens of a whole layer).
#pragma once

#include "fp8blk_device.h"

namespace fp8blk {

// Reductions over the LANES lanes (a DPP row of 16, or the wave) that share a
// token; every one of them gets the result.  Sums are added in the same tree
// whatever the values, so they do not depend on the launch.
template <int LANES>
__device__ __forceinline__ uint32_t lanes_max_u(uint32_t v) {
  v = row16_max(v);
  if constexpr (LANES == 64) {
    const auto a = __builtin_amdgcn_permlane16_swap(v, v, false, false);
    v = max((uint32_t)a[0], (uint32_t)a[1]);
    const auto b = __builtin_amdgcn_permlane32_swap(v, v, false, false);
    v = max((uint32_t)b[0], (uint32_t)b[1]);
  }
  return v;
}

template <int LANES>
__device__ __forceinline__ float lanes_max(float v) {
#define FP8MOE_STEP(CTRL) v = fmaxf(v, __uint_as_float(dpp<CTRL>(__float_as_uint(v))))
  FP8MOE_STEP(kDppRowRor8);
  FP8MOE_STEP(kDppRowRor4);
  FP8MOE_STEP(kDppRowRor2);
  FP8MOE_STEP(kDppRowRor1);
#undef FP8MOE_STEP
  if constexpr (LANES == 64) {
    v = fmaxf(v, __shfl_xor(v, 16, 64));
    v = fmaxf(v, __shfl_xor(v, 32, 64));
  }
  return v;
}

template <int LANES>
__device__ __forceinline__ float lanes_sum(float v) {
#define FP8MOE_STEP(CTRL) v += __uint_as_float(dpp<CTRL>(__float_as_uint(v)))
  FP8MOE_STEP(kDppRowRor8);
  FP8MOE_STEP(kDppRowRor4);
  FP8MOE_STEP(kDppRowRor2);
  FP8MOE_STEP(kDppRowRor1);
#undef FP8MOE_STEP
  if constexpr (LANES == 64) {
    v += __shfl_xor(v, 16, 64);
    v += __shfl_xor(v, 32, 64);
  }
  return v;
}

// exp(v - top) for v <= top.  Equal ones give 1 without the difference, which
// infinity minus infinity would turn into NaN.
__device__ __forceinline__ float exp_from(float v, float top) { return v == top ? 1.0f : expf(v - top); }

// A logit as an unsigned number of the same order, 0 for the ones that cannot
// be chosen (-infinity, NaN).  Adding 0 makes one zero of the two.
__device__ __forceinline__ uint32_t route_key(float v) {
  const uint32_t u = __float_as_uint(v + 0.0f);
  return v > -INFINITY ? u ^ ((u >> 31) ? 0xFFFFFFFFu : 0x80000000u) : 0u;
}

__device__ __forceinline__ float route_value(uint32_t key) {
  return __uint_as_float(key ^ ((key >> 31) ? 0x80000000u : 0xFFFFFFFFu));
}

// The choice of one token, whose logits its LANES lanes hold: v[i] is expert
// lane + i LANES (-infinity past the last).  Lane j gets the j-th choice and
// its weight, j < k <= 16; the other lanes' results are not for use.
struct RouteChoice {
  int id;
  float weight;
};

template <int LANES, int NI>
__device__ __forceinline__ RouteChoice route_choose(const float (&v)[NI], int k, bool renorm, int lane) {
  uint32_t key[NI];
#pragma unroll
  for (int i = 0; i < NI; ++i) key[i] = route_key(v[i]);
  RouteChoice mine{-1, 0.0f};
  float top = 0.0f, sum = 0.0f;
  for (int j = 0; j < k; ++j) {
    uint32_t best = 0;
#pragma unroll
    for (int i = 0; i < NI; ++i) best = max(best, key[i]);
    best = lanes_max_u<LANES>(best);
    // the lowest expert among those with that key (as the largest complement)
    uint32_t at = 0;
#pragma unroll
    for (int i = NI - 1; i >= 0; --i)
      if (key[i] == best) at = 0xFFFFu - (uint32_t)(lane + i * LANES);
    at = 0xFFFFu - lanes_max_u<LANES>(at);
#pragma unroll
    for (int i = 0; i < NI; ++i)
      if (lane + i * LANES == (int)at) key[i] = 0;
    const float value = route_value(best);
    if (j == 0) top = value;
    const float w = best ? exp_from(value, top) : 0.0f;
    sum += w;
    if (lane == j) mine = RouteChoice{best ? (int)at : -1, w};
  }
  if (!renorm) {
    sum = 0.0f;
#pragma unroll
    for (int i = 0; i < NI; ++i) sum += v[i] > -INFINITY ? exp_from(v[i], top) : 0.0f;
    sum = lanes_sum<LANES>(sum);
  }
  mine.weight = sum > 0.0f ? mine.weight / sum : 0.0f;
  return mine;
}

}  // namespace fp8blk
