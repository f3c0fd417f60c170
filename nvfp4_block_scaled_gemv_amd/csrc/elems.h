// elems.h -- loads, conversions and stores of groups of 8 and 16 activation
// elements (bf16, fp32, E4M3), shared by the kernels of the decode step that
// stand between the GEMVs (norm, rotation and append, paged attention).
#pragma once

#include "device.h"

namespace nvfp4 {

typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));

// Two fp32 to packed bf16, round to nearest even (NaN stays NaN).
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const bf16x2_t v = {(__bf16)lo, (__bf16)hi};
  return __builtin_bit_cast(uint32_t, v);
}
__device__ __forceinline__ float bf16_lo(uint32_t u) { return __uint_as_float(u << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t u) { return __uint_as_float(u & 0xFFFF0000u); }

// Into E4M3's range. The conversion instruction turns a value past 448 into
// NaN; a stored activation saturates instead, and NaN stays NaN.
__device__ __forceinline__ float e4m3_clamp(float v) {
  return v != v ? v : fminf(fmaxf(v, -448.0f), 448.0f);
}
// Four fp32 to four E4M3 bytes, round to nearest even, saturating.
__device__ __forceinline__ uint32_t pack_e4m3(float a, float b, float c, float d) {
  int w = __builtin_amdgcn_cvt_pk_fp8_f32(e4m3_clamp(a), e4m3_clamp(b), 0, false);
  w = __builtin_amdgcn_cvt_pk_fp8_f32(e4m3_clamp(c), e4m3_clamp(d), w, true);
  return (uint32_t)w;
}

// Eight consecutive elements as loaded (Raw8<T>) and as fp32.
template <typename T>
struct Raw8;
template <>
struct Raw8<uint16_t> {   // bf16 bits
  u32x4_t r;
  __device__ __forceinline__ void load(const uint16_t* p) {
    r = *reinterpret_cast<const u32x4_t*>(p);
  }
  __device__ __forceinline__ void get(float (&v)[8]) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = bf16_lo(r[i]);
      v[2 * i + 1] = bf16_hi(r[i]);
    }
  }
};
template <>
struct Raw8<float> {
  f32x4_t a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = *reinterpret_cast<const f32x4_t*>(p);
    b = *reinterpret_cast<const f32x4_t*>(p + 4);
  }
  __device__ __forceinline__ void get(float (&v)[8]) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[i] = a[i];
      v[4 + i] = b[i];
    }
  }
};

__device__ __forceinline__ void store8(uint16_t* p, const float (&v)[8]) {
  u32x4_t o;
#pragma unroll
  for (int i = 0; i < 4; ++i) o[i] = pack_bf16(v[2 * i], v[2 * i + 1]);
  *reinterpret_cast<u32x4_t*>(p) = o;
}
__device__ __forceinline__ void store8(float* p, const float (&v)[8]) {
  *reinterpret_cast<f32x4_t*>(p) = f32x4_t{v[0], v[1], v[2], v[3]};
  *reinterpret_cast<f32x4_t*>(p + 4) = f32x4_t{v[4], v[5], v[6], v[7]};
}
__device__ __forceinline__ void store8(uint8_t* p, const float (&v)[8]) {   // E4M3
  *reinterpret_cast<u32x2_t*>(p) = u32x2_t{pack_e4m3(v[0], v[1], v[2], v[3]),
                                           pack_e4m3(v[4], v[5], v[6], v[7])};
}

}  // namespace nvfp4
