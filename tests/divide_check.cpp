// Host check of the quotients of divide.h against the division: random
// dividends and divisors over the whole range of the rule, divisors and
// dividends next to powers of two, quotients next to the middle between two
// numbers. Prints "ok <quotients>" or the first difference.
#include <cmath>
#include <cstdint>
#include <cstdio>
#include <cstring>

#include "divide.h"

static uint64_t rng = 0x9E3779B97F4A7C15ull;
static uint32_t next_u32() {
  rng = rng * 6364136223846793005ull + 1442695040888963407ull;
  return (uint32_t)(rng >> 32);
}

static float make(uint32_t mantissa, int exponent) {
  return std::ldexp(1.0f + (float)(mantissa & 0x7FFFFFu) * 0x1p-23f, exponent);
}

// a mantissa: any, or within 8 steps of a power of two
static uint32_t mantissa() {
  const uint32_t u = next_u32();
  return u & 1u ? u >> 9 : u & 2u ? (u >> 9) & 7u : 0x7FFFFFu - ((u >> 9) & 7u);
}

int main() {
  long n = 0;
  for (long i = 0; i < 20000000; ++i) {
    const int de = (int)(next_u32() % 160) - 64;                  // d in 2^-64 .. 2^96
    const float d = make(mantissa(), de);
    if (!nvfp4::divides_fast(d, d)) continue;
    float v;
    const uint32_t how = next_u32();
    if (how & 1u) {
      v = make(mantissa(), de - 11 + (int)(next_u32() % 31));     // quotients 2^-12 .. 2^20
    } else {
      // a dividend next to d times the middle of two numbers, or a number
      const int qe = (int)(next_u32() % 30) - 11;
      const double q = std::ldexp(1.0 + (double)(mantissa() * 2u + (how >> 1 & 1u)) * 0x1p-24, qe);
      v = (float)(q * (double)d);
    }
    if (!(v <= d * 0x1p20f) || v < d * 0x1p-12f) continue;
    if (how & 4u) v = -v;
    const float a = nvfp4::quotient(v, d, 1.0f / d), b = v / d;
    ++n;
    if (std::memcmp(&a, &b, 4) != 0) {
      std::printf("v %a d %a: %a, the division gives %a\n", (double)v, (double)d, (double)a, (double)b);
      return 1;
    }
  }
  // outside the rule
  const float out[][2] = {{0x1p-65f, 0x1p-65f}, {0x1p97f, 1.0f}, {1.0f, 0x1.2p20f}, {0.0f, 0.0f},
                          {-1.0f, 1.0f}, {NAN, 1.0f}, {1.0f, NAN}, {1.0f, INFINITY}};
  for (const auto& o : out)
    if (nvfp4::divides_fast(o[0], o[1])) {
      std::printf("d %a top %a is taken\n", (double)o[0], (double)o[1]);
      return 1;
    }
  std::printf("ok %ld\n", n);
  return 0;
}
