// divide.h -- fp32 quotients of many numbers by one divisor, with a reciprocal
// and two fused steps in place of a division each. Also built for the host,
// where a test compares them with the division.
#pragma once

#include <math.h>

#include "segments.h"   // NVFP4_HD

namespace nvfp4 {

// Where quotient() may stand for the division: the reciprocal is normal, no
// product overflows, and the remainder of a quotient of 2^-12 or more is a
// multiple of 2^-122, so that it is exact. top: the largest |v|.
NVFP4_HD inline bool divides_fast(float d, float top) {
  return d >= 0x1p-64f && d <= 0x1p96f && top <= d * 0x1p20f;
}

// v / d with r = 1 / d correctly rounded: q = v r is within an ulp and a half,
// and q + (v - q d) r rounds to the quotient. Quotients below 2^-12 may be off
// in their last bit; to E4M3 and E2M1 they are zero.
NVFP4_HD inline float quotient(float v, float d, float r) {
  const float q = v * r;
  return fmaf(fmaf(-q, d, v), r, q);
}

}  // namespace nvfp4
