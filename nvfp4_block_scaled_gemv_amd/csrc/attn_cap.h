// attn_cap.h -- the cap of attention's scores, z -> cap tanh(z / cap). Also built
// for the host, where a test compares it with the definition.
#pragma once

#include <math.h>

#include "segments.h"   // NVFP4_HD

namespace nvfp4 {

// inv = 1 / cap. With x = z inv, up to |x| = 1.25 a quotient of tanh's continued
// fraction, z (10395 + 1260 s + 21 s^2) / (10395 + 4725 s + 210 s^2 + s^3) with s =
// x^2, off by 2^-27 at most; beyond, cap (1 - 2 / (exp(2 x) + 1)), which is cap where
// the exponential overflows (below, its rounding, 2^-24 of one, would show). z itself
// enters the quotient, not cap x: nothing of it is lost however large the cap, and
// however small x, is. Within 2^-21 of the capped score, with Op::rcp and Op::exp2
// off by one unit in the last place.
constexpr float kCapNear = 1.25f;
template <class Op>
NVFP4_HD inline float capped_near(float z, float inv) {
  const float x = z * inv, s = x * x;
  const float n = fmaf(fmaf(s, 21.0f, 1260.0f), s, 10395.0f);
  const float d = fmaf(fmaf(s + 210.0f, s, 4725.0f), s, 10395.0f);
  return z * n * Op::rcp(d);
}
template <class Op>
NVFP4_HD inline float capped(float z, float cap, float inv) {
  const float y = fabsf(z * inv);
  const float e = Op::exp2(y * 2.885390081777927f);   // 2 log2(e)
  const float far = cap * fmaf(-2.0f, Op::rcp(e + 1.0f), 1.0f);
  return y <= kCapNear ? capped_near<Op>(z, inv) : copysignf(far, z);
}

}  // namespace nvfp4
