// quotient.cuh -- codes of a row under its scale, as the step's append makes
// them, for the appends of prompts.
#pragma once
#include <stdint.h>

#include "fp8.cuh"

namespace wave {

// The codes of v / sc, the quotient rounded to fp32 first (an IEEE division),
// as the step's append makes them.  v (1 / sc) is within 3 units in the last
// place of that quotient, which decides the code only next to a value midway
// between two codes (mantissa bits 1000... below the three of a code) or below
// the codes' normal range: those, and scales whose reciprocal is not an
// ordinary number, take the division.
__device__ __forceinline__ uint32_t encode4(const float* v, float sc) {
  const float r = __frcp_rn(sc);
  float q[4];
  bool exact = !(sc >= 0x1p-100f && sc <= 0x1.fffffep127f);
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    q[e] = v[e] * r;
    const uint32_t b = __float_as_uint(q[e]);
    exact |= ((b - 0x7FFFDu) & 0xFFFFFu) <= 6u || (b & 0x7FFFFFFFu) - 1u < 0x3C800000u - 1u;  // next to midway; below 2^-6, but not 0
  }
  if (exact) {
    if (sc == 0.f) return 0;
#pragma unroll
    for (int e = 0; e < 4; ++e) q[e] = __fdiv_rn(v[e], sc);
  }
  return (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(q[0], q[1]), __NV_SATFINITE, __NV_E4M3) |
         (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(q[2], q[3]), __NV_SATFINITE, __NV_E4M3) << 16;
}

}  // namespace wave
