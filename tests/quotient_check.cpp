// How far the reciprocal of csrc/fp8quotient.h is off, for tests/test_quotient.py: over the amax / 448 scales of all
// bf16 values that it is for, from all reciprocals that are an ulp off at most, prints how many scales there were, the
// largest error in units of 2^-60, and how many second parts were negative or parts not finite.
#include <cstdint>
#include <cstdio>
#include <cstring>

#include "../blockwise_fp8_linear_amd/csrc/fp8quotient.h"

using namespace fp8blk;

int main() {
  long long scales = 0, bad = 0;
  long double worst = 0;
  for (uint32_t amax = 1; amax < 0x7F80; ++amax) {
    const uint32_t bits = amax << 16;
    float a;
    std::memcpy(&a, &bits, 4);
    const float s = a / 448.0f;
    if (!(s >= kQuotientLeast && s < kQuotientMost)) continue;
    ++scales;
    // the largest float that is at most 1 / s: it and the next one are an ulp off at most, and the one before where
    // it is 1 / s itself
    const float rounded = (float)(1.0L / s);
    uint32_t below;
    std::memcpy(&below, &rounded, 4);
    const __float128 over = (__float128)s * rounded - 1;
    below -= over > 0 ? 1 : 0;
    for (int off = over == 0 ? -1 : 0; off <= 1; ++off) {
      const uint32_t q = below + off;
      float near;
      std::memcpy(&near, &q, 4);
      const ReciprocalParts p = reciprocal_parts(s, near);
      bad += !(p.r2 >= 0.0f) || !std::isfinite(p.r) || !std::isfinite(p.r2);
      // s (r + r2) is exact in 113 bits
      const __float128 e = (__float128)s * ((__float128)p.r + (__float128)p.r2) - 1;
      const long double x = (long double)(e < 0 ? -e : e);
      worst = x > worst ? x : worst;
    }
  }
  std::printf("%lld %.0Lf %lld\n", scales, worst * 0x1p60L, bad);
  return 0;
}
