// Host check of attn_cap.h against tanh in 64 bits: scores from far below the cap to
// far above it, caps over their whole range, every number around the border of the
// two parts, the reciprocal and the exponential exact and one unit in the last place
// off to either side. Prints "ok <scores>" or the first difference.
#include <cmath>
#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <initializer_list>

#include "attn_cap.h"

static long scores = 0;

template <int RCP, int EXP>   // units in the last place
struct Ops {
  static float moved(float x, int by) {
    return by == 0 || !std::isfinite(x) ? x : std::nextafterf(x, by > 0 ? INFINITY : -INFINITY);
  }
  static float rcp(float x) { return moved(1.0f / x, RCP); }
  static float exp2(float x) { return moved(std::exp2(x), EXP); }
};

template <class Op>
static void check(float z, float cap) {
  const float inv = Op::rcp(cap);
  const float got = nvfp4::capped<Op>(z, cap, inv);
  const double want = (double)cap * std::tanh((double)z / (double)cap);
  ++scores;
  // below the normal numbers a step of fp32 more
  if (!(std::fabs((double)got - want) <= std::fabs(want) * 0x1p-21 + 0x1p-149)) {
    std::printf("z %a cap %a: %a, tanh gives %a\n", (double)z, (double)cap, (double)got, want);
    std::exit(1);
  }
  if (std::fabs(z * inv) <= nvfp4::kCapNear) {   // what tiles without a far score take
    const float near = nvfp4::capped_near<Op>(z, inv);
    if (near != got) {
      std::printf("z %a cap %a: %a and %a\n", (double)z, (double)cap, (double)near, (double)got);
      std::exit(1);
    }
  }
}

template <class Op>
static void all() {
  const float log2e = 1.4426950408889634f;
  for (float c : {1e-6f, 3.3e-5f, 0.01f, 0.5f, 1.0f, 2.0f, 7.3f, 30.0f, 50.0f, 500.0f, 65504.0f,
                  1e9f, 1e20f, 1e28f, 3e29f, 1e30f}) {
    const float cap = c * log2e;   // as the kernels have it
    for (float sign : {1.0f, -1.0f}) {
      for (int e = -90; e <= 60; ++e)               // shares of the cap
        for (int i = 0; i < 64; ++i) {
          const float z = sign * std::ldexp(cap * (1.0f + (float)i * 0x1.04p-6f), e);
          if (std::isfinite(z) && std::fabs(z) >= 0x1p-126f) check<Op>(z, cap);
        }
      for (int i = 0; i < 40000; ++i) check<Op>(sign * cap * ((float)i * 0x1.01p-12f), cap);
      float z = sign * 1.25f * cap;
      for (int i = 0; i < 2000; ++i) z = std::nextafterf(z, 0.0f);
      for (int i = 0; i < 4000; ++i) {
        check<Op>(z, cap);
        z = std::nextafterf(z, sign * INFINITY);
      }
    }
    check<Op>(0.0f, cap);
    check<Op>(INFINITY, cap);
    check<Op>(-INFINITY, cap);
    if (!std::isnan(nvfp4::capped<Op>(NAN, cap, Op::rcp(cap)))) {
      std::printf("NaN at cap %a\n", (double)cap);
      std::exit(1);
    }
  }
}

int main() {
  all<Ops<0, 0>>();
  all<Ops<1, 1>>();
  all<Ops<1, -1>>();
  all<Ops<-1, 1>>();
  all<Ops<-1, -1>>();
  std::printf("ok %ld\n", scores);
  return 0;
}
