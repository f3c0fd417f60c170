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
// before the first use. Rows of at most 512 elements take one wavefront (of at
// most 128 a quarter of one) and no LDS. Measured: one token of 7168, bf16 with
// residual, 2.2 us; 2048 rows of 7168 to E4M3 with an fp32 residual 34 us, 162 MB at the
// rate of a copy.
#include "elems.h"
#include "divide.h"
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

// Sum (MAX: largest value) over a row's threads; each of them gets it. Fixed
// order. lpr 16: the row is a DPP row; otherwise W wavefronts. The two uses in
// a kernel take different LDS words, so one barrier each is enough.
template <bool MAX>
__device__ __forceinline__ float row_reduce(float v, int lpr, int W, float* lds) {
  auto join = [](float a, float b) { return MAX ? fmaxf(a, b) : a + b; };
  v = join(v, dpp_f32<0xB1>(v));    // quad_perm [1,0,3,2]
  v = join(v, dpp_f32<0x4E>(v));    // quad_perm [2,3,0,1]
  v = join(v, dpp_f32<0x141>(v));   // row_half_mirror
  v = join(v, dpp_f32<0x140>(v));   // row_mirror
  if (lpr == 16) return v;
  float r[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    r[i] = __builtin_bit_cast(float,
                              __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), 16 * i));
  v = join(join(r[0], r[1]), join(r[2], r[3]));
  if (W == 1) return v;
  if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
  __syncthreads();
  v = lds[0];
  for (int w = 1; w < W; ++w) v = join(v, lds[w]);
  return v;
}

// v[i] / d for 8 numbers, two fused steps in place of a division each: E4M3 rows
// of 7168 fp32 values were bound by the divisions, 86.6 us for 8192 of them.
// The division itself where d or the largest |v[i]|, top, could take a step out
// of the normal numbers (a saturated block scale leaves quotients as large as
// fp32 holds).
__device__ __forceinline__ void divide8(float (&v)[8], float d, float top) {
  if (divides_fast(d, top)) {
    const float r = 1.0f / d;
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = quotient(v[e], d, r);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = v[e] / d;
  }
}

template <typename TX, typename TR, int OUT, int VPT>
__global__ __launch_bounds__(1024) void k_add_rmsnorm(
    const TX* __restrict__ x, const TR* residual, TR* residual_out,   // may be one array
    const uint16_t* __restrict__ weight, float eps, int64_t M, int H, int lpr, int W, int group,
    const float* __restrict__ gscale, void* __restrict__ out, void* __restrict__ out_scales) {
  constexpr bool kRes = !__is_same(TR, None);
  __shared__ float lds[32];
  // W == 1: 64 / lpr rows per wavefront; otherwise one row per workgroup
  const int64_t row = W == 1 ? ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) / lpr
                             : (int64_t)blockIdx.x;
  if (row >= M) return;   // whole DPP rows or wavefronts, and no barrier follows
  const int lane = W == 1 ? (int)threadIdx.x & (lpr - 1) : (int)threadIdx.x;
  const int lanes = W == 1 ? lpr : W * 64;
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
  sq = row_reduce<false>(sq, lpr, W, lds);
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
      all = row_reduce<true>(all, lpr, W, lds + 16);
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
        float scale = am[v] / 448.0f;
        if (!(scale > 0.0f)) scale = 1.0f;   // zeros, or too small for a scale
        divide8(s[v], scale, am[v]);
        store8((uint8_t*)out + at + i, s[v]);
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
      divide8(s[v], sv * g, ab);
#pragma unroll
      for (int e = 0; e < 8; ++e) word |= e2m1_encode(s[v][e]) << (4 * e);
    }
    if (i < H) {
      reinterpret_cast<uint32_t*>(out)[(at + i) >> 3] = word;
      if ((i & 15) == 0) ((uint8_t*)out_scales)[(at + i) >> 4] = (uint8_t)code;
    }
  }
}

template <typename TX, typename TR, int OUT, int VPT>
hipError_t launch_v(const NormArgs& a, int W, hipStream_t stream) {
  // rows of at most 128: 16 lanes each (163840 rows of 128, bf16 with a
  // residual, the same arrays: 25.5 us, 37.6 with a wavefront each)
  const int lpr = a.H <= 128 ? 16 : 64;
  const int rows = W == 1 ? 256 / lpr : 1;   // rows per workgroup
  const int64_t grid = (a.M + rows - 1) / rows;
  hipLaunchKernelGGL((k_add_rmsnorm<TX, TR, OUT, VPT>), dim3((uint32_t)grid),
                     dim3(W == 1 ? 256 : 64 * W), 0, stream, (const TX*)a.x, (const TR*)a.residual,
                     (TR*)a.residual_out, a.weight, a.eps, a.M, (int)a.H, lpr, W, a.group,
                     a.gscale, a.out, a.out_scales);
  return hipGetLastError();
}

template <typename TX, typename TR, int OUT>
hipError_t launch_o(const NormArgs& a, hipStream_t stream) {
  // Groups of 8 per lane: one while the row fits 1024 threads that way, which
  // is the shortest way through few rows. With many, fewer threads per row, so
  // that more rows are in flight where one reduces and encodes. A residual's
  // stores keep enough in flight without, so there only NVFP4 gains, later. Rows
  // of 7168 with fewer threads against one group, us, other arrays each time:
  //   fp32 to E4M3            1024 rows 11.0 / 12.2, 2048 17.0 / 21.1, 8192 54 / 69
  //   bf16 to bf16            1024 7.4 / 8.2, 8192 44 / 53
  //   bf16 + fp32 to E4M3     1024 21.5 / 20.9, 8192 120 / 117
  //   bf16 to NVFP4           1024 13.1 / 12.6, 2048 19.9 / 21.3, 8192 56 / 76
  //   fp32 + bf16 to NVFP4    1024 21.2 / 18.4, 2048 32.6 / 30.4, 4096 53.7 / 55.4
  constexpr bool kRes = !__is_same(TR, None);
  constexpr int64_t many = OUT == kOutNvfp4 ? (kRes ? 4096 : 2048) : kRes ? INT64_MAX : 1024;
  const int64_t vecs = a.H / 8, one = a.M >= many ? 256 : 1024;
  const int VPT = vecs <= one ? 1 : vecs <= 2 * one ? 2 : 4;
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
