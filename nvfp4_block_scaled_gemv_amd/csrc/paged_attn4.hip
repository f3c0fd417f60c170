// paged_attn4.hip -- attention of the new tokens of each sequence over a paged
// key-value cache in NVFP4: E2M1 codes, an E4M3 scale for each 16 elements of a
// head and one fp32 scale for all keys (values). The split of the work, the
// pass and the join are those of the other caches (attn_wave.h).
//
// Bound: the bytes of K and V, 9/16 of one per element, and next to it the
// vector ALU, which turns each element into a number: a tile of 32 keys of 128
// is 4.6 KB, which the card reads in 390 clocks per CU, and some 270 vector
// instructions of 4 clocks on each of four SIMDs.
//
// A code times its block's scale has 6 significant bits and lies between 2^-10
// and 2688: it is exact in fp16 (and in bf16, which has no packed product). So
// the products with the matrix cores are fp16:
//   S^T[key, row] = K Q^T    O^T[dim, row] += V^T P^T
// - K: a lane takes one key's D / 4 consecutive dims (16 bytes of codes at 128)
//   and their scales; two codes a conversion, two elements a packed product.
// - Q: a row of bf16 is multiplied by a power of two that takes its largest
//   element to 2^14 .. 2^15; fp16 then holds every element down to 2^-31 of that
//   one whole, and the smaller ones to 2^-40 of it. The scores' factor
//   takes the power back.
// - V^T wants pairs of keys where a byte holds a pair of dims: the nibbles of
//   two keys' words change places first, 4 instructions for 16 elements, and
//   each conversion gives one dim of two keys. The pair's two scales multiply it.
// - P enters as the sum of two fp16, each rounded to nearest: 2^-24 of it at
//   most is lost, or 2^-36 of the largest weight at small ones. The exponents
//   are raised by 11 to use fp16's range.
#include "attn_wave.h"

namespace nvfp4 {

namespace {

typedef _Float16 f16x2_t __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8_t __attribute__((ext_vector_type(8)));

// The reference of the exponentials is moved only when a score passes it by
// more than kSlack (in powers of two); a weight is at most 2^(kRaise + kSlack),
// which fp16 holds.
constexpr float kSlack = 4.0f;
constexpr float kRaise = 11.0f;

// Wavefronts per SIMD of the split form.
constexpr int waves_per_simd(int RT, int D) { return RT == 1 && D < 256 ? 2 : 1; }
static_assert(waves_per_simd(1, 64) * kCus * 4 <= kMaxRuns, "the join's weights");

template <int SEL>
__device__ __forceinline__ f16x2_t e2m1x2_to_f16(uint32_t w) {   // byte SEL, exact
  return __builtin_bit_cast(f16x2_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, SEL));
}
template <int HALF>
__device__ __forceinline__ f16x2_t e4m3x2_to_f16(uint32_t w) {   // bytes 2 HALF, + 1, exact
  return __builtin_bit_cast(f16x2_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, 1.0f, HALF));
}
__device__ __forceinline__ uint32_t bits(f16x2_t v) { return __builtin_bit_cast(uint32_t, v); }
// Eight elements of one block: a word's codes times s (twice).
__device__ __forceinline__ u32x4_t scaled8(uint32_t w, f16x2_t s) {
  return u32x4_t{bits(e2m1x2_to_f16<0>(w) * s), bits(e2m1x2_to_f16<1>(w) * s),
                 bits(e2m1x2_to_f16<2>(w) * s), bits(e2m1x2_to_f16<3>(w) * s)};
}
__device__ __forceinline__ f32x4_t mma(u32x4_t a, u32x4_t b, f32x4_t acc) {
  return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8_t, a),
                                                __builtin_bit_cast(f16x8_t, b), acc, 0, 0, 0);
}

template <int D, int RT, bool PG, bool MOD>
struct Attn4Wave : AttnPass<Attn4Wave<D, RT, PG, MOD>, RT, PG, MOD> {
  using Pass = AttnPass<Attn4Wave, RT, PG, MOD>;
  using Pass::a, Pass::sh, Pass::n, Pass::g, Pass::h, Pass::Q, Pass::G, Pass::row0, Pass::c,
      Pass::tok, Pass::m, Pass::l, Pass::NU, Pass::NO;
  static constexpr int kD = D;
  static constexpr bool kScaled = true;
  static constexpr int kPerSimd = waves_per_simd(RT, D);
  static constexpr int NP = TK / 32;           // products over the keys
  static constexpr int NJ = D / 32;            // products over the dims: words of K per lane and key
  static constexpr int NV = D / 16;            // dims per lane of V
  static constexpr int VW = NV > 8 ? 2 : 1;    // words of V per lane and key
  static constexpr int kParts = 2;             // fp16 numbers that hold a probability
  typedef u32x4_t Weights[kParts][RT][NP];

  const int64_t head_off, head_boff;
  const uint32_t st, bst, v_sel;
  u32x4_t qf[RT][NJ];
  float qs[RT];                                // scale of a row's scores
  f32x4_t O[RT][NV];
  uint32_t kr[NU][NJ], kb[NU];                 // K: codes, scales
  uint32_t vr[TK / 4][VW], vb[TK / 4];         // V: codes, the 4 scales that hold the lane's
  int64_t off[NO], boff[NO];                   // bytes, from place()

  __device__ __forceinline__ Attn4Wave(const AttnArgs& a_, const AttnShape& sh_, int h_, int row0_,
                                       float k_scale)
      : Pass(a_, sh_, h_, row0_, k_scale), head_off((int64_t)h_ * a_.sh),
        head_boff((int64_t)h_ * a_.block_sh), st((uint32_t)a_.st), bst((uint32_t)a_.block_st),
        // the byte of the lane's block in two keys' words
        v_sel(0x0C0C0400u + (uint32_t)((n * NV / 16) & 3) * 0x0101u) {
    clear();
  }
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
#pragma unroll
      for (int t = 0; t < NV; ++t) O[rt][t] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
      m[rt] = -INFINITY;
      l[rt] = 0.0f;
    }
  }
  __device__ __forceinline__ void load_q(int b) {
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      const int r = row0 + rt * 16 + n;
      const bool live = tok[rt] >= 0;
      // rows that do not exist read another's: nothing of them is written
      const uint16_t* qp = a.q + ((int64_t)(b * (int64_t)Q + (live ? tok[rt] : 0)) * a.Hq + h * G +
                                  (live ? r - tok[rt] * G : 0)) * D + g * (D / 4);
      u32x4_t raw[NJ];
      uint32_t top = 0u;                       // the row's largest, as bits
#pragma unroll
      for (int j = 0; j < NJ; ++j) {
        raw[j] = *reinterpret_cast<const u32x4_t*>(qp + j * 8);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const uint32_t lo = (raw[j][e] << 16) & 0x7FFFFFFFu, hi = raw[j][e] & 0x7FFF0000u;
          top = top > lo ? top : lo;
          top = top > hi ? top : hi;
        }
      }
      uint32_t o = __shfl_xor(top, 16, 64);
      top = top > o ? top : o;
      o = __shfl_xor(top, 32, 64);
      top = top > o ? top : o;
      // 2^up takes it to 2^14 .. (2^126 at most: such rows' scores are nothing)
      int up = 14 + 127 - (int)(top >> 23);
      up = up > 126 ? 126 : up;
      const float f = __uint_as_float((uint32_t)(127 + up) << 23);
      qs[rt] = c * __uint_as_float((uint32_t)(127 - up) << 23);
#pragma unroll
      for (int j = 0; j < NJ; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const f16x2_t v = {(_Float16)(bf16_lo(raw[j][e]) * f), (_Float16)(bf16_hi(raw[j][e]) * f)};
          qf[rt][j][e] = bits(v);
        }
    }
  }
  __device__ __forceinline__ void place(int u, int id, int in) {
    off[u] = (int64_t)id * a.sb + (int64_t)in * a.st + head_off;
    boff[u] = (int64_t)id * a.block_sb + (int64_t)in * a.block_st + head_boff;
  }
  // the key of the tile that a lane has as the e-th (of TK / 4) of V, S^T and P:
  // four neighbours per e and run, so that a load of V takes whole stretches
  static __device__ __forceinline__ int key_of(int e, int g) {
    return (e >> 2) * 16 + (e & 3) * 4 + g;
  }
  // want: false where no tile follows. The loads are issued all the same, all
  // lanes from one address: a branch around them would make the waits on both
  // sides drain everything in flight.
  __device__ __forceinline__ void load_k(bool want) {
    const uint8_t *const kc = (const uint8_t*)a.k_cache, *const bc = a.k_blocks;
    const int key = (n & 3) * 4 + (n >> 2);    // row n of S^T
#pragma unroll
    for (int u = 0; u < NU; ++u) {
      const uint8_t *p, *b;
      if constexpr (PG) {
        p = kc + off[u] + (want ? (uint32_t)key * st + (uint32_t)g * (D / 8) : 0u);
        b = bc + boff[u] + (want ? (uint32_t)key * bst + (uint32_t)g * (D / 64) : 0u);
      } else {
        p = want ? kc + this->from_lane(off[0], 16 * u + key) + g * (D / 8) : kc;
        b = want ? bc + this->from_lane(boff[0], 16 * u + key) + g * (D / 64) : bc;
      }
      if constexpr (D == 64) {
        const u32x2_t v = *reinterpret_cast<const u32x2_t*>(p);
        kr[u][0] = v[0];
        kr[u][1] = v[1];
        kb[u] = *b;
      } else {
#pragma unroll
        for (int j = 0; j < NJ; j += 4) {
          const u32x4_t v = *reinterpret_cast<const u32x4_t*>(p + j * 4);
#pragma unroll
          for (int e = 0; e < 4; ++e) kr[u][j + e] = v[e];
        }
        kb[u] = D == 128 ? *reinterpret_cast<const uint16_t*>(b)
                         : *reinterpret_cast<const uint32_t*>(b);
      }
    }
  }
  __device__ __forceinline__ void load_v(bool want) {
    const uint8_t *const vc = (const uint8_t*)a.v_cache, *const bc = a.v_blocks;
    const uint32_t dim = (uint32_t)n * (NV / 2), blk = (uint32_t)(n * NV / 64) * 4;
#pragma unroll
    for (int e = 0; e < TK / 4; ++e) {
      const uint8_t *p, *b;
      if constexpr (PG) {
        const uint32_t key = want ? (uint32_t)((e & 3) * 4 + g) : 0u;
        p = vc + off[e >> 2] + (key * st + (want ? dim : 0u));
        b = bc + boff[e >> 2] + (key * bst + (want ? blk : 0u));
      } else {
        p = want ? vc + this->from_lane(off[0], key_of(e, g)) + dim : vc;
        b = want ? bc + this->from_lane(boff[0], key_of(e, g)) + blk : bc;
      }
      if constexpr (NV == 4) {
        vr[e][0] = *reinterpret_cast<const uint16_t*>(p);
      } else if constexpr (NV == 8) {
        vr[e][0] = *reinterpret_cast<const uint32_t*>(p);
      } else {
        const u32x2_t v = *reinterpret_cast<const u32x2_t*>(p);
        vr[e][0] = v[0];
        vr[e][VW - 1] = v[1];
      }
      vb[e] = *reinterpret_cast<const uint32_t*>(b);
    }
  }

  // S^T of the loaded tile, scaled
  __device__ __forceinline__ void scores(f32x4_t (&S)[RT][NU]) {
#pragma unroll
    for (int u = 0; u < NU; ++u) {
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) S[rt][u] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
      const f16x2_t s01 = e4m3x2_to_f16<0>(kb[u]), s23 = e4m3x2_to_f16<1>(kb[u]);
#pragma unroll
      for (int j = 0; j < NJ; ++j) {
        const f16x2_t s = j >> 2 ? s23 : s01;
        const _Float16 one = (j >> 1) & 1 ? s[1] : s[0];
        const u32x4_t kv = scaled8(kr[u][j], f16x2_t{one, one});
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) S[rt][u] = mma(kv, qf[rt][j], S[rt][u]);
      }
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) S[rt][u] *= qs[rt];
    }
  }
  // The running maximum and sum, and P (times 2^kRaise) as the sum of two fp16.
  __device__ __forceinline__ void softmax(const f32x4_t (&S)[RT][NU], Weights& pf) {
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      float mx = -INFINITY;
#pragma unroll
      for (int e = 0; e < 4 * NU; ++e) mx = fmaxf(mx, S[rt][e >> 2][e & 3]);
      if (__any(mx > m[rt] + kSlack)) {
        mx = fmaxf(mx, __shfl_xor(mx, 16, 64));
        mx = fmaxf(mx, __shfl_xor(mx, 32, 64));
        const float m_new = fmaxf(m[rt], mx);
        const float f = m_new == -INFINITY ? 1.0f : __builtin_amdgcn_exp2f(m[rt] - m_new);
        m[rt] = m_new;
        l[rt] *= f;
#pragma unroll
        for (int t = 0; t < NV; ++t) O[rt][t] *= f;
      }
      const float m_use = m[rt] == -INFINITY ? 0.0f : m[rt] - kRaise;
#pragma unroll
      for (int e = 0; e < 2 * NU; ++e) {
        const float p0 = __builtin_amdgcn_exp2f(S[rt][e >> 1][(e & 1) * 2] - m_use);
        const float p1 = __builtin_amdgcn_exp2f(S[rt][e >> 1][(e & 1) * 2 + 1] - m_use);
        l[rt] += p0 + p1;
        const f16x2_t hi = {(_Float16)p0, (_Float16)p1};
        // what is left is exact in fp32
        const f16x2_t lo = {(_Float16)fmaf((float)hi[0], -1.0f, p0),
                            (_Float16)fmaf((float)hi[1], -1.0f, p1)};
        pf[0][rt][e >> 2][e & 3] = bits(hi);
        pf[1][rt][e >> 2][e & 3] = bits(lo);
      }
    }
  }
  // O += V^T P^T, the smaller part first
  __device__ __forceinline__ void values(const Weights& pf) {
#pragma unroll
    for (int q = 0; q < NP; ++q) {
      f16x2_t s[4];                            // of four pairs of keys
#pragma unroll
      for (int i = 0; i < 4; ++i)
        s[i] = e4m3x2_to_f16<0>(
            __builtin_amdgcn_perm(vb[q * 8 + 2 * i + 1], vb[q * 8 + 2 * i], v_sel));
#pragma unroll
      for (int w = 0; w < VW; ++w) {
        uint32_t even[4], odd[4];              // two keys' dims 0 2 4 6, and 1 3 5 7
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t x = vr[q * 8 + 2 * i][w], y = vr[q * 8 + 2 * i + 1][w];
          even[i] = (x & 0x0F0F0F0Fu) | ((y << 4) & 0xF0F0F0F0u);
          odd[i] = ((x >> 4) & 0x0F0F0F0Fu) | (y & 0xF0F0F0F0u);
        }
        two<0>(even, odd, s, pf, q, w * 8);
        two<1>(even, odd, s, pf, q, w * 8);
        if constexpr (NV > 4) {
          two<2>(even, odd, s, pf, q, w * 8);
          two<3>(even, odd, s, pf, q, w * 8);
        }
      }
    }
  }
  // products t0 + 2 B and + 1: byte B of the pairs' words
  template <int B>
  __device__ __forceinline__ void two(const uint32_t (&even)[4], const uint32_t (&odd)[4],
                                      const f16x2_t (&s)[4], const Weights& pf, int q, int t0) {
    const u32x4_t v0 = {bits(e2m1x2_to_f16<B>(even[0]) * s[0]), bits(e2m1x2_to_f16<B>(even[1]) * s[1]),
                        bits(e2m1x2_to_f16<B>(even[2]) * s[2]), bits(e2m1x2_to_f16<B>(even[3]) * s[3])};
    const u32x4_t v1 = {bits(e2m1x2_to_f16<B>(odd[0]) * s[0]), bits(e2m1x2_to_f16<B>(odd[1]) * s[1]),
                        bits(e2m1x2_to_f16<B>(odd[2]) * s[2]), bits(e2m1x2_to_f16<B>(odd[3]) * s[3])};
#pragma unroll
    for (int rt = 0; rt < RT; ++rt)
#pragma unroll
      for (int i = kParts - 1; i >= 0; --i) {
        O[rt][t0 + 2 * B] = mma(v0, pf[i][rt][q], O[rt][t0 + 2 * B]);
        O[rt][t0 + 2 * B + 1] = mma(v1, pf[i][rt][q], O[rt][t0 + 2 * B + 1]);
      }
  }

  // the lane's e-th key of V becomes zero where it is not seen: codes are
  // finite, so its scales do
  __device__ __forceinline__ void keep(int e, bool see) { vb[e] = see ? vb[e] : 0u; }
  __device__ __forceinline__ bool not_finite(int e) const {   // E4M3's NaN
    return ((vb[e] >> (8 * (v_sel & 3u))) & 0x7Fu) == 0x7Fu;
  }

  // Row g * 4 + i of the products is dims (g * 4 + i) * NV .. + NV - 1. f(d0,
  // v): 4 consecutive dims of row rt * 16 + n.
  template <typename F>
  __device__ __forceinline__ void each4(int rt, F f) const {
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int t = 0; t < NV; t += 4)
        f((g * 4 + i) * NV + t,
          f32x4_t{O[rt][t][i], O[rt][t + 1][i], O[rt][t + 2][i], O[rt][t + 3][i]});
  }
};

int row_tiles(int64_t rows) { return rows <= 16 ? 1 : 2; }

AttnLayout layout(int64_t rows, int64_t Hkv, int64_t D) {
  const int RT = row_tiles(rows);
  return attn_layout(rows, Hkv, D, RT, waves_per_simd(RT, (int)D));
}

int64_t whole_keys(const AttnArgs&, const AttnShape&) { return 512; }

template <int D, bool MOD>
hipError_t launch_d(const AttnArgs& a, hipStream_t stream) {
  const bool pg = a.page % 16 == 0;
  const AttnLayout L = layout(a.Hq / a.Hkv * a.Q, a.Hkv, D);
  const AttnShape sh = attn_shape(a, L);
  const int64_t whole = whole_keys(a, sh);
  if (L.RT == 2)
    return pg ? launch_forms<Attn4Wave<D, 2, true, MOD>>(a, sh, whole, stream)
              : launch_forms<Attn4Wave<D, 2, false, MOD>>(a, sh, whole, stream);
  return pg ? launch_forms<Attn4Wave<D, 1, true, MOD>>(a, sh, whole, stream)
            : launch_forms<Attn4Wave<D, 1, false, MOD>>(a, sh, whole, stream);
}

template <bool MOD>
hipError_t launch_scored(const AttnArgs& a, hipStream_t stream) {
  return a.D == 64    ? launch_d<64, MOD>(a, stream)
         : a.D == 128 ? launch_d<128, MOD>(a, stream)
                      : launch_d<256, MOD>(a, stream);
}

}  // namespace

int attn4_row_units(int64_t rows, int64_t Hkv, int64_t D) { return layout(rows, Hkv, D).NHV; }

size_t attn4_workspace_bytes(int64_t rows, int64_t Hkv, int64_t D) {
  return layout(rows, Hkv, D).total;
}

hipError_t launch_paged_attention4(const AttnArgs& a, hipStream_t stream) {
  return a.softcap > 0.0f || a.slopes ? launch_scored<true>(a, stream)
                                      : launch_scored<false>(a, stream);
}

}  // namespace nvfp4
