// A quotient x / s by a reciprocal in two parts, for fp8tile_device.h and the test of
// its range.
#pragma once

#include <hip/hip_runtime.h>
#include <math.h>

namespace fp8blk {

// The scales it is for.  The second part is some 2^-24 / s: from 2^106 on what it loses
// by being no normal number would be more than the rest of the error, which is below
// 2^-44 of 1 / s; and x times a reciprocal has to stay finite.
constexpr float kQuotientLeast = 0x1p-64f, kQuotientMost = 0x1p100f;

// 1 / s = r + r2, from q, an ulp off 1 / s at most: r is at most 1 / s and r2 = (1 - s r) r.
struct ReciprocalParts {
  float r, r2;
};
__host__ __device__ inline ReciprocalParts reciprocal_parts(float s, float q) {
  const float e = __builtin_fmaf(-s, q, 1.0f);
  uint32_t bits;
  __builtin_memcpy(&bits, &q, 4);
  bits -= e < 0.0f ? 1 : 0;
  float r;
  __builtin_memcpy(&r, &bits, 4);
  return {r, __builtin_fmaf(-s, r, 1.0f) * r};
}

}  // namespace fp8blk
