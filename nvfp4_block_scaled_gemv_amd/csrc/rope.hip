// rope.hip -- rotary positions of q and k, and the append of k and v to a
// paged key-value cache, in one pass over the projections' outputs.
//
// Pair i of a head's first R elements turns by the angle a = position *
// inv_freq[i]:
//   (x0, x1) -> (x0 cos a - x1 sin a, x1 cos a + x0 sin a) * rope_scale
// with x0, x1 at i and i + R/2 (half layout) or at 2i and 2i + 1
// (interleaved); the rest of the head passes through. The product is formed
// in 64 bits and reduced to a fraction of a turn there (at position 10^6 a
// 32-bit product would be off by up to 0.03 rad), then sine and cosine are
// 32-bit.
//
// Bound: bytes for a prompt, latency for a token. A workgroup takes one token
// (several when their heads are few): it computes each of the R/2 angles once
// into LDS while the element loads are in flight, then every thread turns 8
// pairs (16 elements) at a time. Both layouts give a thread two 8-element
// groups: i and i + R/2, or 16 consecutive elements. Measured, 32 / 8 heads of
// 128: 5 tokens fp32 3.2 us (a launch and two dependent loads), 4096 tokens
// fp32 30.6 us, 4.9 TB/s of reads and writes, a copy's rate (23.9 where the
// arrays are found in the last cache). To an NVFP4 cache a thread takes a block of 16
// elements of k or v whole, for its scale: 5 tokens 4.2 us, 4099 tokens bf16, half of
// each head turned, 21.4 us, 4.2 TB/s (28.1 with codes by comparisons).
#include "elems.h"
#include "divide.h"
#include "internal.h"

namespace nvfp4 {

namespace {

constexpr int kThreads = 256;
constexpr int kMaxTokens = 8;   // tokens per workgroup

struct RopeShape {
  int Hq, Hkv, D, R;
  int J;        // jobs (16 elements) per token: (Hq + 2 Hkv) * D / 16
  int tpb;      // tokens per workgroup
  int parts;    // workgroups per token (tpb == 1 where parts > 1)
};

struct Nvfp4 {};   // a cache of E2M1 codes and E4M3 block scales

// Eight E2M1 codes, nibble i of x[i], as e2m1_encode gives them (compared on the
// card for every fp32 but NaN): the conversion rounds to the nearest even code, the
// rest is its saturation and the sign of zero. A chain of comparisons for each
// instead: 4099 tokens of 8 heads of 128 28.1 -> 21.2 us.
__device__ __forceinline__ uint32_t e2m1x8(const float (&x)[16], int at) {
  float c[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) c[i] = fminf(fmaxf(x[at + i], -6.0f), 6.0f);
  uint32_t w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(0u, c[0], c[1], 1.0f, 0);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, c[2], c[3], 1.0f, 1);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, c[4], c[5], 1.0f, 2);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, c[6], c[7], 1.0f, 3);
  const uint32_t mag = w & 0x77777777u;
  const uint32_t some = (mag | (mag >> 1) | (mag >> 2)) & 0x11111111u;   // not zero
  return mag | (w & (some << 3));
}

// Block b (16 elements) of a head of k (turned where it lies in the first R) or
// v to the NVFP4 cache, by one thread: the half layout's partners are read a
// second time, from the cache, by their own block's thread. The encoders are
// pack's and quantize_act's; a block that holds a NaN gets the scale NaN.
template <typename TX, bool INTER>
__device__ __forceinline__ void append_block(const TX* src, int b, bool turn, int half,
                                             const float2* trig, float g, uint8_t* codes,
                                             uint8_t* scale) {
  Raw8<TX> raw[2], other[2];
  const int e0 = b * 16;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int e = e0 + i * 8;
    raw[i].load(src + e);
    if (!INTER && turn) other[i].load(src + (e < half ? e + half : e - half));
  }
  float x[16];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int e = e0 + i * 8;
    float v[8];
    raw[i].get(v);
    if (turn && INTER) {
#pragma unroll
      for (int p = 0; p < 4; ++p) {
        const float2 u = trig[e / 2 + p];
        const float p0 = v[2 * p], p1 = v[2 * p + 1];
        v[2 * p] = fmaf(p0, u.x, -(p1 * u.y));
        v[2 * p + 1] = fmaf(p1, u.x, p0 * u.y);
      }
    } else if (turn) {
      float w[8];
      other[i].get(w);
      const bool first = e < half;
      const float2* tr = trig + (first ? e : e - half);
#pragma unroll
      for (int p = 0; p < 8; ++p) {
        const float2 u = tr[p];
        v[p] = fmaf(v[p], u.x, first ? -(w[p] * u.y) : w[p] * u.y);
      }
    }
#pragma unroll
    for (int p = 0; p < 8; ++p) x[i * 8 + p] = v[p];
  }
  uint32_t top = 0u;   // the largest magnitude's bits; a NaN's are above infinity's
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const uint32_t u = __float_as_uint(x[i]) & 0x7FFFFFFFu;
    top = top > u ? top : u;
  }
  const float amax = __uint_as_float(top);
  uint32_t lo = 0u, hi = 0u;
  uint32_t sc = 0x7Fu;
  if (top <= 0x7F800000u) {
    sc = e4m3_encode(amax / (6.0f * g));
    const float s = e4m3_to_f32<0>(sc);
    if (s != 0.0f) {
      const float d = s * g;
      if (divides_fast(d, amax)) {
        const float inv = 1.0f / d;
#pragma unroll
        for (int i = 0; i < 16; ++i) x[i] = quotient(x[i], d, inv);
      } else {
#pragma unroll
        for (int i = 0; i < 16; ++i) x[i] = x[i] / d;
      }
      lo = e2m1x8(x, 0);
      hi = e2m1x8(x, 8);
    }
  }
  *reinterpret_cast<u32x2_t*>(codes) = u32x2_t{lo, hi};
  *scale = (uint8_t)sc;
}

template <typename TX, typename TC, bool INTER>
__global__ __launch_bounds__(kThreads) void k_rope_append(const RopeArgs a, const RopeShape sh) {
  extern __shared__ float2 trig[];   // [tpb][R / 2] cos, sin
  const int half = sh.R / 2;
  const int64_t t0 = (int64_t)(blockIdx.x / sh.parts) * sh.tpb;
  const int part = blockIdx.x % sh.parts;
  const int ntok = (int)(a.T - t0 < sh.tpb ? a.T - t0 : sh.tpb);
  for (int i = threadIdx.x; i < ntok * half; i += kThreads) {
    const int tk = i / half, f = i - tk * half;
    double turns = (double)a.positions[t0 + tk] * (double)a.inv_freq[f] * 0.15915494309189535;
    turns -= rint(turns);
    float s, c;
    sincospif(2.0f * (float)turns, &s, &c);
    trig[i] = float2{c * a.rope_scale, s * a.rope_scale};
  }
  __syncthreads();
  constexpr bool kFour = __is_same(TC, Nvfp4);
  float ks = 1.0f, vs = 1.0f;
  if ((kFour || sizeof(TC) == 1) && sh.Hkv) {
    ks = *a.k_scale;
    vs = *a.v_scale;
  }
  const int chunks = sh.D / 16, nq = sh.Hq * chunks, nk = sh.Hkv * chunks;
  for (int job = part * kThreads + threadIdx.x; job < ntok * sh.J; job += sh.parts * kThreads) {
    const int tk = sh.tpb == 1 ? 0 : job / sh.J;
    int j = job - tk * sh.J;
    const int64_t t = t0 + tk;
    // which tensor: 0 q, 1 k, 2 v
    const int kind = j < nq ? 0 : j < nq + nk ? 1 : 2;
    j -= kind == 0 ? 0 : kind == 1 ? nq : nq + nk;
    const int head = j / chunks, c = j - head * chunks;
    const TX* src = (const TX*)(kind == 0 ? a.q : kind == 1 ? a.k : a.v) +
                    t * (kind == 0 ? a.q_stride : kind == 1 ? a.k_stride : a.v_stride) +
                    (int64_t)head * sh.D;
    if constexpr (kFour) {
      if (kind != 0) {
        const int64_t slot = a.slots[t];
        const int64_t block = slot / a.page;
        if (slot < 0 || block >= a.num_blocks) continue;
        const int64_t place = slot - block * a.page;
        append_block<TX, INTER>(
            src, c, kind == 1 && c * 16 < sh.R, half, trig + tk * half, kind == 1 ? ks : vs,
            (uint8_t*)(kind == 1 ? a.k_cache : a.v_cache) + block * a.sb + place * a.st +
                head * a.sh + c * 8,
            (kind == 1 ? a.k_blocks : a.v_blocks) + block * a.block_sb + place * a.block_st +
                head * a.block_sh + c);
        continue;
      }
    }
    // the two groups of 8: the chunk's pairs, or 16 elements as they are
    const bool turn = kind != 2 && c * 16 < sh.R;
    const int e0 = turn && !INTER ? c * 8 : c * 16;
    const int e1 = turn && !INTER ? c * 8 + half : c * 16 + 8;
    Raw8<TX> r0, r1;
    r0.load(src + e0);
    r1.load(src + e1);
    float x0[8], x1[8];
    r0.get(x0);
    r1.get(x1);
    if (turn) {
      const float2* tr = trig + tk * half + c * 8;
      if (INTER) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 u = tr[i], w = tr[4 + i];
          const float p0 = x0[2 * i], p1 = x0[2 * i + 1];
          x0[2 * i] = fmaf(p0, u.x, -(p1 * u.y));
          x0[2 * i + 1] = fmaf(p1, u.x, p0 * u.y);
          const float q0 = x1[2 * i], q1 = x1[2 * i + 1];
          x1[2 * i] = fmaf(q0, w.x, -(q1 * w.y));
          x1[2 * i + 1] = fmaf(q1, w.x, q0 * w.y);
        }
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float2 u = tr[i];
          const float p0 = x0[i], p1 = x1[i];
          x0[i] = fmaf(p0, u.x, -(p1 * u.y));
          x1[i] = fmaf(p1, u.x, p0 * u.y);
        }
      }
    }
    if (kind == 0) {
      uint16_t* o = a.q_out + (t * sh.Hq + head) * sh.D;
      store8(o + e0, x0);
      store8(o + e1, x1);
    } else if constexpr (!kFour) {
      const int64_t slot = a.slots[t];
      const int64_t block = slot / a.page;
      if (slot >= 0 && block < a.num_blocks) {
        if (sizeof(TC) == 1) {
          const float sc = kind == 1 ? ks : vs;
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            x0[i] = x0[i] / sc;
            x1[i] = x1[i] / sc;
          }
        }
        TC* o = (TC*)(kind == 1 ? a.k_cache : a.v_cache) + block * a.sb +
                (slot - block * a.page) * a.st + head * a.sh;
        store8(o + e0, x0);
        store8(o + e1, x1);
      }
    }
  }
}

template <typename TX, typename TC>
hipError_t launch_c(const RopeArgs& a, hipStream_t stream) {
  RopeShape sh;
  sh.Hq = (int)a.Hq;
  sh.Hkv = (int)a.Hkv;
  sh.D = (int)a.D;
  sh.R = (int)a.R;
  sh.J = (int)((a.Hq + 2 * a.Hkv) * (a.D / 16));
  // few tokens: a workgroup per 256 jobs of a token; many: one token each, or
  // as many as fill the threads. In graphs, 32 / 8 heads of 128 from fp32, the
  // first against the second: 64 tokens 3.0 us / 3.6, 256 3.9 / 4.2, 1024 8.6 /
  // 8.2; 16 / 16 heads from bf16 to E4M3: 128 3.7 / 4.0, 256 4.6 / 4.3; 8 / 1
  // heads: 256 3.0 / 3.3, 1024 3.7 / 3.8.
  const bool few = a.T <= 256;
  sh.parts = few ? (sh.J + kThreads - 1) / kThreads : 1;
  sh.tpb = few || sh.J >= kThreads ? 1 : kThreads / sh.J;
  if (sh.tpb > kMaxTokens) sh.tpb = kMaxTokens;
  const int64_t grid = (a.T + sh.tpb - 1) / sh.tpb * sh.parts;
  const size_t lds = (size_t)sh.tpb * (size_t)(sh.R / 2) * sizeof(float2);
  if (a.interleaved)
    hipLaunchKernelGGL((k_rope_append<TX, TC, true>), dim3((uint32_t)grid), dim3(kThreads), lds,
                       stream, a, sh);
  else
    hipLaunchKernelGGL((k_rope_append<TX, TC, false>), dim3((uint32_t)grid), dim3(kThreads), lds,
                       stream, a, sh);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_rope_append(const RopeArgs& a, hipStream_t stream) {
  if (a.cache_nvfp4)
    return a.x_f32 ? launch_c<float, Nvfp4>(a, stream) : launch_c<uint16_t, Nvfp4>(a, stream);
  if (a.x_f32)
    return a.cache_e4m3 ? launch_c<float, uint8_t>(a, stream)
                        : launch_c<float, uint16_t>(a, stream);
  return a.cache_e4m3 ? launch_c<uint16_t, uint8_t>(a, stream)
                      : launch_c<uint16_t, uint16_t>(a, stream);
}

}  // namespace nvfp4
