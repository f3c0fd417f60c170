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
// arrays are found in the last cache).
#include "elems.h"
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
  float ks = 1.0f, vs = 1.0f;
  if (sizeof(TC) == 1 && sh.Hkv) {
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
    } else {
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
  if (a.x_f32)
    return a.cache_e4m3 ? launch_c<float, uint8_t>(a, stream)
                        : launch_c<float, uint16_t>(a, stream);
  return a.cache_e4m3 ? launch_c<uint16_t, uint8_t>(a, stream)
                      : launch_c<uint16_t, uint16_t>(a, stream);
}

}  // namespace nvfp4
