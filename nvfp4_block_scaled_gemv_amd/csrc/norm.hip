// norm.hip -- RMS norm with the residual's addition, in front of the GEMVs.
//
//   s[m, i] = x[m, i] + residual[m, i]            (fp32; stored, rounded once)
//   y[m, i] = s[m, i] * rsqrt(mean_i s^2 + eps) * w[i]
//
// y leaves as bf16 (a GEMV's x), as E4M3 with fp32 scales, or as NVFP4 with a
// static scale (the W4A4 GEMV's x); the 8- and 4-bit forms are rounded from
// the fp32 y, not from its bf16 rounding.
//
// Bound: bytes for a prompt's rows, the latency of one load, one reduction and
// one store for a token. The row stays in registers between the sum of
// squares and the scaling, so every byte moves once: W wavefronts hold one
// row, VPT groups of 8 elements per lane, and all loads of a lane are issued
// before the first use. Rows of at most 512 elements take one wavefront each,
// four rows to a workgroup, and no LDS.
#include "elems.h"
#include "internal.h"

namespace nvfp4 {

namespace {

constexpr int kOutBf16 = 0, kOutE4m3 = 1, kOutNvfp4 = 2;

struct None {};

template <typename TR>
struct Residual {
  Raw8<TR> raw;
};
template <>
struct Residual<None> {};

// Sum (MAX: largest value) over the W wavefronts of a row; every thread gets
// it. Fixed order. The two uses in a kernel take different LDS words, so one
// barrier each is enough.
template <bool MAX>
__device__ __forceinline__ float row_reduce(float v, int W, float* lds) {
  if (MAX) {
    v = fmaxf(v, dpp_f32<0xB1>(v));
    v = fmaxf(v, dpp_f32<0x4E>(v));
    v = fmaxf(v, dpp_f32<0x141>(v));
    v = fmaxf(v, dpp_f32<0x140>(v));
    float r[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      r[i] = __builtin_bit_cast(float,
                                __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), 16 * i));
    v = fmaxf(fmaxf(r[0], r[1]), fmaxf(r[2], r[3]));
  } else {
    v = wave_sum(v);
  }
  if (W == 1) return v;
  if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
  __syncthreads();
  v = lds[0];
  for (int w = 1; w < W; ++w) v = MAX ? fmaxf(v, lds[w]) : v + lds[w];
  return v;
}

template <typename TX, typename TR, int OUT, int VPT>
__global__ __launch_bounds__(1024) void k_add_rmsnorm(
    const TX* __restrict__ x, const TR* residual, TR* residual_out,   // may be one array
    const uint16_t* __restrict__ weight, float eps, int64_t M, int H, int W, int group,
    const float* __restrict__ gscale, void* __restrict__ out, void* __restrict__ out_scales) {
  constexpr bool kRes = !__is_same(TR, None);
  __shared__ float lds[32];
  // W == 1: one row per wavefront; otherwise one row per workgroup
  const int64_t row =
      W == 1 ? (int64_t)blockIdx.x * (blockDim.x >> 6) + (threadIdx.x >> 6) : (int64_t)blockIdx.x;
  if (row >= M) return;   // whole wavefronts, and only where no barrier follows
  const int lane = W == 1 ? (int)(threadIdx.x & 63) : (int)threadIdx.x;
  const int lanes = W * 64;
  const int64_t at = row * H;
  Raw8<TX> rx[VPT];
  Residual<TR> rr[VPT];
  Raw8<uint16_t> rw[VPT];
#pragma unroll
  for (int v = 0; v < VPT; ++v) {
    const int i = (v * lanes + lane) * 8;
    if (i < H) {
      rx[v].load(x + at + i);
      if constexpr (kRes) rr[v].raw.load(residual + at + i);
      rw[v].load(weight + i);
    }
  }
  float s[VPT][8];
  float sq = 0.0f;
#pragma unroll
  for (int v = 0; v < VPT; ++v) {
    const int i = (v * lanes + lane) * 8;
    if (i < H) {
      rx[v].get(s[v]);
      if constexpr (kRes) {
        float r[8];
        rr[v].raw.get(r);
#pragma unroll
        for (int e = 0; e < 8; ++e) s[v][e] += r[e];
        store8(residual_out + at + i, s[v]);
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) sq = fmaf(s[v][e], s[v][e], sq);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) s[v][e] = 0.0f;
    }
  }
  sq = row_reduce<false>(sq, W, lds);
  const float rstd = 1.0f / sqrtf(sq / (float)H + eps);
#pragma unroll
  for (int v = 0; v < VPT; ++v) {
    const int i = (v * lanes + lane) * 8;
    if (i < H) {
      float w[8];
      rw[v].get(w);
#pragma unroll
      for (int e = 0; e < 8; ++e) s[v][e] = s[v][e] * rstd * w[e];
    }
  }
  if (OUT == kOutBf16) {
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      const int i = (v * lanes + lane) * 8;
      if (i < H) store8((uint16_t*)out + at + i, s[v]);
    }
    return;
  }
  if (OUT == kOutE4m3) {
    float am[VPT];
    float all = 0.0f;
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      am[v] = 0.0f;
#pragma unroll
      for (int e = 0; e < 8; ++e) am[v] = fmaxf(am[v], fabsf(s[v][e]));
      all = fmaxf(all, am[v]);
    }
    // a group of 32, 64 or 128 elements is 4, 8 or 16 lanes of one DPP row;
    // H is a multiple of the group, so its lanes are all inside the row
    if (group == 0) {
      all = row_reduce<true>(all, W, lds + 16);
#pragma unroll
      for (int v = 0; v < VPT; ++v) am[v] = all;
    } else {
#pragma unroll
      for (int v = 0; v < VPT; ++v) {
        am[v] = fmaxf(am[v], dpp_f32<0xB1>(am[v]));
        am[v] = fmaxf(am[v], dpp_f32<0x4E>(am[v]));
        if (group > 32) am[v] = fmaxf(am[v], dpp_f32<0x141>(am[v]));
        if (group > 64) am[v] = fmaxf(am[v], dpp_f32<0x140>(am[v]));
      }
    }
    const int gsize = group == 0 ? H : group;
    float* sc = (float*)out_scales + row * (H / gsize);
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      const int i = (v * lanes + lane) * 8;
      if (i < H) {
        const float scale = am[v] > 0.0f ? am[v] / 448.0f : 1.0f;
        float q[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) q[e] = s[v][e] / scale;
        store8((uint8_t*)out + at + i, q);
        if (i % gsize == 0) sc[i / gsize] = scale;
      }
    }
    return;
  }
  // NVFP4: a 16-element block is two neighbouring lanes; the encoders of pack
  const float g = *gscale;
#pragma unroll
  for (int v = 0; v < VPT; ++v) {
    const int i = (v * lanes + lane) * 8;
    float ab = 0.0f;
#pragma unroll
    for (int e = 0; e < 8; ++e) ab = fmaxf(ab, fabsf(s[v][e]));
    ab = fmaxf(ab, dpp_f32<0xB1>(ab));
    const uint32_t code = e4m3_encode(ab / (6.0f * g));
    const float sv = e4m3_to_f32<0>(code);
    uint32_t word = 0u;
    if (sv != 0.0f) {
      const float dn = sv * g;
#pragma unroll
      for (int e = 0; e < 8; ++e) word |= e2m1_encode(s[v][e] / dn) << (4 * e);
    }
    if (i < H) {
      reinterpret_cast<uint32_t*>(out)[(at + i) >> 3] = word;
      if ((i & 15) == 0) ((uint8_t*)out_scales)[(at + i) >> 4] = (uint8_t)code;
    }
  }
}

template <typename TX, typename TR, int OUT, int VPT>
hipError_t launch_v(const NormArgs& a, int W, hipStream_t stream) {
  const int rows = W == 1 ? 4 : 1;   // rows per workgroup
  const int64_t grid = (a.M + rows - 1) / rows;
  hipLaunchKernelGGL((k_add_rmsnorm<TX, TR, OUT, VPT>), dim3((uint32_t)grid), dim3(64 * W * rows),
                     0, stream, (const TX*)a.x, (const TR*)a.residual, (TR*)a.residual_out,
                     a.weight, a.eps, a.M, (int)a.H, W, a.group, a.gscale, a.out, a.out_scales);
  return hipGetLastError();
}

template <typename TX, typename TR, int OUT>
hipError_t launch_o(const NormArgs& a, hipStream_t stream) {
  // groups of 8 per lane: one while the row fits 1024 threads that way
  const int64_t vecs = a.H / 8;
  const int VPT = vecs <= 1024 ? 1 : vecs <= 2048 ? 2 : 4;
  const int W = (int)((vecs + 64 * VPT - 1) / (64 * VPT));
  return VPT == 1   ? launch_v<TX, TR, OUT, 1>(a, W, stream)
         : VPT == 2 ? launch_v<TX, TR, OUT, 2>(a, W, stream)
                    : launch_v<TX, TR, OUT, 4>(a, W, stream);
}

template <typename TX, typename TR>
hipError_t launch_r(const NormArgs& a, hipStream_t stream) {
  return a.form == NormForm::bf16   ? launch_o<TX, TR, kOutBf16>(a, stream)
         : a.form == NormForm::e4m3 ? launch_o<TX, TR, kOutE4m3>(a, stream)
                                    : launch_o<TX, TR, kOutNvfp4>(a, stream);
}

template <typename TX>
hipError_t launch_x(const NormArgs& a, hipStream_t stream) {
  if (!a.residual) return launch_r<TX, None>(a, stream);
  return a.residual_f32 ? launch_r<TX, float>(a, stream) : launch_r<TX, uint16_t>(a, stream);
}

}  // namespace

hipError_t launch_add_rmsnorm(const NormArgs& a, hipStream_t stream) {
  return a.x_f32 ? launch_x<float>(a, stream) : launch_x<uint16_t>(a, stream);
}

}  // namespace nvfp4
