// paged_attn.hip -- attention of the new tokens of each sequence over a paged
// key-value cache: one token per sequence (decode) or a few (verification of
// drafts).
//
// Row r of a (sequence, key-value head) is one query: token i = r / G of the
// Q new ones, query head h G + r % G, with G = Hq / Hkv. It sits at position
// len - Q + i and sees the keys up to there (with a window: the last `window`
// of them):
//   o = sum_k exp(s_k - m) v_k / sum_k exp(s_k - m),  s_k = scale q . k
// in one pass over the cache with a running maximum m and sum.
//
// Bound: the bytes of K and V, each read once for all rows of its head. The
// rows of a head (up to 16, or two tiles of 16) fill the columns of the matrix
// instructions, so one pass serves them all:
//   S^T[key, row] = K Q^T     A = K (16 keys x 32 dims), B = Q^T
//   O^T[dim, row] += V^T P^T  A = V^T (16 dims x 32 keys), B = P^T
// A lane ends S^T with 4 keys of one row per 16 keys. The order of the keys in
// the second product is free as long as V follows, so those registers are its
// B operand as they stand: P never leaves the registers. V^T's operand needs 8
// keys of one dim per lane: a lane loads 8 dims of 8 keys (whole rows of V per
// load) and pairs halves with one v_perm_b32 per dword. K, V and P pass no LDS.
//
// Split: the lengths are on the device, so the grid is fixed (a multiple of
// the CUs) and the kernel itself divides the work. The 128-key steps of all
// (sequence, head) pairs are numbered in one row; workgroup w takes an equal
// run of them, whatever the lengths are. A pair that lies inside one run is
// finished there; others leave partial (m, sum, O) records, at most two per
// workgroup, that k_attn_join adds in a fixed order. No atomics.
#include "elems.h"
#include "internal.h"

namespace nvfp4 {

namespace {

constexpr int kWaves = 4;
constexpr int kTile = 32;                 // keys per wavefront and turn
constexpr int kStep = kWaves * kTile;     // keys per workgroup and turn
constexpr int kCus = 256;
constexpr float kLog2e = 1.4426950408889634f;
// The reference of the exponentials is moved only when a score passes it by
// more than this (in powers of two): exp2 of at most 2^8 loses nothing in fp32
// or bf16, and most turns need no maximum across lanes and no rescaling.
constexpr float kSlack = 8.0f;

struct AttnShape {
  int rows;        // G * Q
  int G;
  int NRT;         // row tiles (of RT * 16 rows) per key-value head
  int NHV;         // Hkv * NRT
  int nwg;
  int page_shift;  // log2(page), or -1
  int cap;         // keys that a row of the table can name
  int slot_rows;   // rows of one partial record
  float* ml;       // [slots][slot_rows][2]
  float* o;        // [slots][slot_rows][D]
};

typedef const __attribute__((address_space(4))) int32_t* const_i32;

// The run of steps of one sequence and head: keys base .. len - 1.
struct Span {
  int len, base, n;   // n >= 1: an empty sequence has one step that writes zeros
};
__device__ __forceinline__ Span span_of(const AttnArgs& a, const AttnShape& sh, int len) {
  Span s;
  s.len = len < 0 ? 0 : len > sh.cap ? sh.cap : len;
  int64_t lo = a.window ? (int64_t)s.len - a.Q - a.window + 1 : 0;
  s.base = lo <= 0 ? 0 : (int)lo & ~(kTile - 1);
  s.n = s.len > s.base ? (s.len - s.base + kStep - 1) / kStep : 1;
  return s;
}

__device__ __forceinline__ int wave_sum_i32(int v) {
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) v += __shfl_xor(v, off, 64);
  return __builtin_amdgcn_readfirstlane(v);
}

// Steps of all sequences (per head), by every wavefront for itself.
__device__ __forceinline__ int total_steps(const AttnArgs& a, const AttnShape& sh) {
  const int lane = threadIdx.x & 63, B = (int)a.B;
  int t = 0;
  for (int b = lane; b < B; b += 64) t += span_of(a, sh, a.lens[b]).n;
  return wave_sum_i32(t);
}
// The sequence that holds step u (of one head's row), and the steps before it.
__device__ __forceinline__ int find_sequence(const AttnArgs& a, const AttnShape& sh, int u,
                                             int& before) {
  const int lane = threadIdx.x & 63, B = (int)a.B;
  int run = 0;
  for (int b0 = 0; b0 < B; b0 += 64) {
    const int n = b0 + lane < B ? span_of(a, sh, a.lens[b0 + lane]).n : 0;
    int incl = n;
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
      const int o = __shfl_up(incl, off, 64);
      if (lane >= off) incl += o;
    }
    const uint64_t past = __ballot(run + incl > u);
    if (past) {
      const int l = __builtin_ctzll(past);
      before = run + __builtin_amdgcn_readlane(incl - n, l);
      return b0 + l;
    }
    run += __builtin_amdgcn_readlane(incl, 63);
  }
  before = 0;
  return 0;   // not reached for u below the total
}
// Workgroup w's run starts at step run_start(w); the first r runs have q + 1
// steps and the others q (total = nw * q + r). run_of(s): who has step s.
struct Runs {
  int q, r;
  __device__ __forceinline__ Runs(int total, int nw) : q(total / nw), r(total % nw) {}
  __device__ __forceinline__ int start(int w) const { return w * q + (w < r ? w : r); }
  __device__ __forceinline__ int of(int s) const {
    const int big = r * (q + 1);
    return s < big ? s / (q + 1) : r + (s - big) / q;
  }
};

__device__ __forceinline__ uint32_t perm_lo(uint32_t a, uint32_t b) {   // halves 0 of a, b
  return __builtin_amdgcn_perm(b, a, 0x05040100u);
}
__device__ __forceinline__ uint32_t perm_hi(uint32_t a, uint32_t b) {   // halves 1 of a, b
  return __builtin_amdgcn_perm(b, a, 0x07060302u);
}
template <int SEL>
__device__ __forceinline__ uint32_t e4m3x2_to_bf16(uint32_t w) {   // exact
  return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.0f, SEL));
}

// One key's elements as a lane holds them: V dwords of NV dims (bf16: NV / 2,
// E4M3: NV / 4), as bf16 pairs through get().
template <int NV, bool FP8>
struct VRow {
  static constexpr int kDw = FP8 ? NV / 4 : NV / 2;
  uint32_t w[kDw];
  // p: the key's row at this lane's first dim; a head of 256 has a second
  // group of 8 dims, half a row further
  __device__ __forceinline__ void load(const uint8_t* p) {
    constexpr int kPiece = kDw > 4 ? 4 : NV == 16 && FP8 ? 2 : kDw;   // dwords per load
#pragma unroll
    for (int i = 0; i < kDw; i += kPiece) {
      const uint8_t* q = p + (i ? 128 * (FP8 ? 1 : 2) : 0);
      if constexpr (kPiece == 4) {
        const u32x4_t v = *reinterpret_cast<const u32x4_t*>(q);
#pragma unroll
        for (int e = 0; e < 4; ++e) w[i + e] = v[e];
      } else if constexpr (kPiece == 2) {
        const u32x2_t v = *reinterpret_cast<const u32x2_t*>(q);
        w[i] = v[0];
        w[i + 1] = v[1];
      } else {
        w[i] = *reinterpret_cast<const uint32_t*>(q);
      }
    }
  }
  __device__ __forceinline__ uint32_t get(int d) const {   // dims 2 d, 2 d + 1
    if constexpr (FP8)
      return (d & 1) ? e4m3x2_to_bf16<1>(w[d >> 1]) : e4m3x2_to_bf16<0>(w[d >> 1]);
    else
      return w[d];
  }
};

template <int D, bool FP8, int RT, bool PG>
__global__ __launch_bounds__(kWaves * 64) void k_paged_attn(const AttnArgs a, const AttnShape sh) {
  constexpr int NJ = D / 32;            // products over the dims
  constexpr int NV = D / 16;            // dims per lane of V = products over them
  constexpr int ES = FP8 ? 1 : 2;
  constexpr int KL = D * ES / 64;       // 16-byte loads of K per lane and 16 keys
  constexpr int LD = D + 4;             // LDS row, padded
  __shared__ float lds_o[kWaves][RT * 16][LD];
  __shared__ float lds_ml[kWaves][RT * 16][2];

  const int lane = threadIdx.x & 63;
  const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int n = lane & 15, g = lane >> 4;
  const int Q = (int)a.Q, G = sh.G;
  const int total = total_steps(a, sh) * sh.NHV;
  const int nw = sh.nwg < total ? sh.nwg : total;
  const int w = blockIdx.x;
  if (w >= nw) return;
  const Runs runs(total, nw);
  int s = runs.start(w);
  const int s_end = runs.start(w + 1);
  int before;
  int b = find_sequence(a, sh, s / sh.NHV, before);
  const const_i32 lens = (const_i32)(uintptr_t)a.lens;
  Span sp = span_of(a, sh, lens[b]);
  int hv = (s - before * sh.NHV) / sp.n;
  int s_in = s - before * sh.NHV - hv * sp.n;
  const float ks = FP8 ? *a.k_scale : 1.0f, vs = FP8 ? *a.v_scale : 1.0f;
  const float c = a.scale * ks * kLog2e;
  const uint8_t* const kc = (const uint8_t*)a.k_cache;
  const uint8_t* const vc = (const uint8_t*)a.v_cache;
  const uint32_t stb = (uint32_t)a.st * ES;                  // bytes between tokens of a page
  const uint32_t k_lane = (uint32_t)n * stb + (uint32_t)g * 16;
  const uint32_t v_dim = (uint32_t)n * (NV > 8 ? 8 : NV) * ES;
  bool first = true;

  while (s < s_end) {
    const int e_in = sp.n - s_in < s_end - s ? sp.n : s_in + (s_end - s);
    const int h = hv / sh.NRT;
    const int row0 = (hv - h * sh.NRT) * (RT * 16);
    const int rows = sh.rows - row0 < RT * 16 ? sh.rows - row0 : RT * 16;
    const int64_t head_off = (int64_t)h * a.sh;
    // the queries, and each row's keys lo .. hi
    bf16x8_t qf[RT][NJ];
    int tok[RT];
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      const int r = row0 + rt * 16 + n;
      const bool live = r < sh.rows;
      tok[rt] = live ? r / G : -1;
      const uint16_t* qp =
          a.q + ((int64_t)(b * (int64_t)Q + (live ? tok[rt] : 0)) * a.Hq + h * G +
                 (live ? r - tok[rt] * G : 0)) * D;
#pragma unroll
      for (int j = 0; j < NJ; ++j) {
        const int d0 = FP8 ? (j >> 1) * 64 + g * 16 + (j & 1) * 8 : j * 32 + g * 8;
        u32x4_t v = *reinterpret_cast<const u32x4_t*>(qp + d0);
        if (!live) v = u32x4_t{0, 0, 0, 0};
        qf[rt][j] = __builtin_bit_cast(bf16x8_t, v);
      }
    }
    const int pos0 = sp.len - Q;
    // keys that every row of this sequence sees
    const int64_t full_lo = a.window ? (int64_t)sp.len - a.window : 0;
    const int full_hi = pos0;
    const const_i32 table = (const_i32)(uintptr_t)(a.table + (int64_t)b * a.max_blocks);

    f32x4_t O[RT][NV];
    float m[RT], l[RT];
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
#pragma unroll
      for (int t = 0; t < NV; ++t) O[rt][t] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
      m[rt] = -INFINITY;
      l[rt] = 0.0f;
    }

    u32x4_t kr[2][KL];
    VRow<NV, FP8> vr[8];
    // where a tile's keys lie: PG, two runs of 16 keys inside one page each
    // (off in elements, uniform); otherwise one offset per lane, for key
    // lane % 32. ok: bit per key, its page exists.
    int64_t off[2] = {0, 0};
    uint32_t ok = 0;
    auto locate = [&](int key0) {
      if (PG) {
        ok = 0;
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const int key = key0 + 16 * u;
          int pi = sh.page_shift >= 0 ? key >> sh.page_shift : key / (int)a.page;
          const int in = key - pi * (int)a.page;
          pi = pi < (int)a.max_blocks ? pi : (int)a.max_blocks - 1;
          const int id = table[pi];
          const bool fine = id >= 0 && id < a.num_blocks;
          off[u] = (int64_t)(fine ? id : 0) * a.sb + (int64_t)in * a.st + head_off;
          ok |= fine ? 0xFFFFu << (16 * u) : 0u;
        }
      } else {
        const int key = key0 + (lane & 31);
        int pi = key / (int)a.page;
        const int in = key - pi * (int)a.page;
        pi = pi < (int)a.max_blocks ? pi : (int)a.max_blocks - 1;
        const int id = a.table[(int64_t)b * a.max_blocks + pi];
        const bool fine = id >= 0 && id < a.num_blocks;
        off[0] = (int64_t)(fine ? id : 0) * a.sb + (int64_t)in * a.st + head_off;
        ok = (uint32_t)__ballot(fine);
      }
    };
    auto at_key = [&](int src) {   // byte offset of the key that lane src holds
      const int lo = __shfl((int)off[0], src, 64);
      const int hi = __shfl((int)(off[0] >> 32), src, 64);
      return (int64_t)(((uint64_t)(uint32_t)hi << 32) | (uint32_t)lo) * ES;
    };
    auto load_k = [&]() {
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        if (PG) {
          const uint8_t* p = kc + off[u] * ES;
#pragma unroll
          for (int j = 0; j < KL; ++j)
            kr[u][j] = *reinterpret_cast<const u32x4_t*>(p + (k_lane + j * 64));
        } else {
          const uint8_t* p = kc + at_key(16 * u + n) + g * 16;
#pragma unroll
          for (int j = 0; j < KL; ++j) kr[u][j] = *reinterpret_cast<const u32x4_t*>(p + j * 64);
        }
      }
    };
    auto load_v = [&](const int64_t (&o2)[2]) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if (PG) {
          const uint8_t* p = vc + o2[i >> 2] * ES;
          vr[i].load(p + ((uint32_t)(g * 4 + (i & 3)) * stb + v_dim));
        } else {
          const int src = (i >> 2) * 16 + g * 4 + (i & 3);
          vr[i].load(vc + at_key(src) + v_dim);
        }
      }
    };

    int key0 = sp.base + s_in * kStep + wv * kTile;
    const int key_end = sp.base + e_in * kStep < sp.len ? sp.base + e_in * kStep : sp.len;
    if (key0 < key_end) {
      locate(key0);
      load_k();
      load_v(off);
    }
    while (key0 < key_end) {
      const int next = key0 + kStep;
      // S^T for 32 keys
      f32x4_t S[RT][2];
#pragma unroll
      for (int u = 0; u < 2; ++u) {
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) S[rt][u] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
          u32x4_t kv;
          if (FP8) {
            const uint32_t x = kr[u][j >> 1][(j & 1) * 2], y = kr[u][j >> 1][(j & 1) * 2 + 1];
            kv = u32x4_t{e4m3x2_to_bf16<0>(x), e4m3x2_to_bf16<1>(x), e4m3x2_to_bf16<0>(y),
                         e4m3x2_to_bf16<1>(y)};
          } else {
            kv = kr[u][j];
          }
#pragma unroll
          for (int rt = 0; rt < RT; ++rt)
            S[rt][u] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                __builtin_bit_cast(bf16x8_t, kv), qf[rt][j], S[rt][u], 0, 0, 0);
        }
      }
      const uint32_t ok_now = ok;
      if (next < key_end) {
        locate(next);
        load_k();
      }
      const bool all = ok_now == 0xFFFFFFFFu && key0 >= full_lo && key0 + kTile - 1 <= full_hi;
      uint32_t pf[RT][4];   // P as bf16 pairs: keys u * 16 + g * 4 + i
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) {
        float mx = -INFINITY;
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int i = 0; i < 4; ++i) S[rt][u][i] *= c;
        if (!all) {
          const int hi = tok[rt] < 0 ? -1 : pos0 + tok[rt];
          const int64_t lo = a.window ? (int64_t)hi - a.window + 1 : 0;
#pragma unroll
          for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int kk = u * 16 + g * 4 + i, key = key0 + kk;
              const bool see = key <= hi && key >= lo && ((ok_now >> kk) & 1u);
              S[rt][u][i] = see ? S[rt][u][i] : -INFINITY;
            }
        }
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int i = 0; i < 4; ++i) mx = fmaxf(mx, S[rt][u][i]);
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
        const float m_use = m[rt] == -INFINITY ? 0.0f : m[rt];
        float p[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          p[e] = __builtin_amdgcn_exp2f(S[rt][e >> 2][e & 3] - m_use);
          l[rt] += p[e];
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) pf[rt][e] = pack_bf16(p[2 * e], p[2 * e + 1]);
      }
      // O^T += V^T P^T
      if (all) {
#pragma unroll
        for (int d = 0; d < NV / 2; ++d) {
          uint32_t x[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) x[i] = vr[i].get(d);
          const u32x4_t lo = {perm_lo(x[0], x[1]), perm_lo(x[2], x[3]), perm_lo(x[4], x[5]),
                              perm_lo(x[6], x[7])};
          const u32x4_t hi = {perm_hi(x[0], x[1]), perm_hi(x[2], x[3]), perm_hi(x[4], x[5]),
                              perm_hi(x[6], x[7])};
#pragma unroll
          for (int rt = 0; rt < RT; ++rt) {
            const u32x4_t pv = {pf[rt][0], pf[rt][1], pf[rt][2], pf[rt][3]};
            O[rt][2 * d] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                __builtin_bit_cast(bf16x8_t, lo), __builtin_bit_cast(bf16x8_t, pv), O[rt][2 * d],
                0, 0, 0);
            O[rt][2 * d + 1] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                __builtin_bit_cast(bf16x8_t, hi), __builtin_bit_cast(bf16x8_t, pv),
                O[rt][2 * d + 1], 0, 0, 0);
          }
        }
      } else {
        // A value that no row sees, or that another token sees, may be anything
        // (0 * inf would reach every row): one product per token, on the
        // values that it sees, kept by that token's rows.
        const int t0 = row0 / G, t1 = (row0 + rows - 1) / G;
        for (int i0 = t0; i0 <= t1; ++i0) {
          const int hi_key = pos0 + i0;
          const int64_t lo_key = a.window ? (int64_t)hi_key - a.window + 1 : 0;
          bool see[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int kk = (i >> 2) * 16 + g * 4 + (i & 3), key = key0 + kk;
            see[i] = key <= hi_key && key >= lo_key && ((ok_now >> kk) & 1u);
          }
#pragma unroll
          for (int d = 0; d < NV / 2; ++d) {
            uint32_t x[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = see[i] ? vr[i].get(d) : 0u;
            const u32x4_t lo = {perm_lo(x[0], x[1]), perm_lo(x[2], x[3]), perm_lo(x[4], x[5]),
                                perm_lo(x[6], x[7])};
            const u32x4_t hi = {perm_hi(x[0], x[1]), perm_hi(x[2], x[3]), perm_hi(x[4], x[5]),
                                perm_hi(x[6], x[7])};
#pragma unroll
            for (int rt = 0; rt < RT; ++rt) {
              const u32x4_t pv = {pf[rt][0], pf[rt][1], pf[rt][2], pf[rt][3]};
              const f32x4_t o0 = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                  __builtin_bit_cast(bf16x8_t, lo), __builtin_bit_cast(bf16x8_t, pv),
                  O[rt][2 * d], 0, 0, 0);
              const f32x4_t o1 = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                  __builtin_bit_cast(bf16x8_t, hi), __builtin_bit_cast(bf16x8_t, pv),
                  O[rt][2 * d + 1], 0, 0, 0);
              const bool mine = tok[rt] == i0;
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                O[rt][2 * d][i] = mine ? o0[i] : O[rt][2 * d][i];
                O[rt][2 * d + 1][i] = mine ? o1[i] : O[rt][2 * d + 1][i];
              }
            }
          }
        }
      }
      if (next < key_end) load_v(off);
      key0 = next;
    }

    // join the wavefronts
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      l[rt] += __shfl_xor(l[rt], 16, 64);
      l[rt] += __shfl_xor(l[rt], 32, 64);
      if (g == 0) {
        lds_ml[wv][rt * 16 + n][0] = m[rt];
        lds_ml[wv][rt * 16 + n][1] = l[rt];
      }
#pragma unroll
      for (int t = 0; t < NV; t += 4)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          // O^T row g * 4 + i of product t is dim (g * 4 + i) * 8 + t (heads of
          // 64: * 4; of 256: products 8.. are the second half)
          constexpr int kRun = NV > 8 ? 8 : NV;
          const int d = (t / kRun) * 128 + (g * 4 + i) * kRun + t % kRun;
          *reinterpret_cast<f32x4_t*>(&lds_o[wv][rt * 16 + n][d]) =
              f32x4_t{O[rt][t][i], O[rt][t + 1][i], O[rt][t + 2][i], O[rt][t + 3][i]};
        }
    }
    __syncthreads();
    const bool whole = s_in == 0 && e_in == sp.n;
    const int slot = first ? 2 * w : 2 * w + 1;
    for (int it = threadIdx.x; it < rows * (D / 8); it += kWaves * 64) {
      const int r = it / (D / 8), d0 = (it % (D / 8)) * 8;
      float mm = -INFINITY;
#pragma unroll
      for (int v = 0; v < kWaves; ++v) mm = fmaxf(mm, lds_ml[v][r][0]);
      const float m_use = mm == -INFINITY ? 0.0f : mm;
      float ll = 0.0f, o[8] = {0, 0, 0, 0, 0, 0, 0, 0};
#pragma unroll
      for (int v = 0; v < kWaves; ++v) {
        const float f = __builtin_amdgcn_exp2f(lds_ml[v][r][0] - m_use);
        ll = fmaf(lds_ml[v][r][1], f, ll);
#pragma unroll
        for (int e = 0; e < 8; ++e) o[e] = fmaf(lds_o[v][r][d0 + e], f, o[e]);
      }
      if (whole) {
        const float f = ll == 0.0f ? 0.0f : vs / ll;
#pragma unroll
        for (int e = 0; e < 8; ++e) o[e] *= f;
        const int rr = row0 + r, t = rr / G;
        store8(a.out + ((int64_t)(b * (int64_t)Q + t) * a.Hq + h * G + (rr - t * G)) * D + d0, o);
      } else {
        store8(sh.o + ((int64_t)slot * sh.slot_rows + r) * D + d0, o);
        if (d0 == 0) {
          sh.ml[((int64_t)slot * sh.slot_rows + r) * 2] = mm;
          sh.ml[((int64_t)slot * sh.slot_rows + r) * 2 + 1] = ll;
        }
      }
    }
    first = false;
    s += e_in - s_in;
    s_in = 0;
    if (e_in == sp.n && ++hv == sh.NHV) {
      hv = 0;
      if (++b < (int)a.B) sp = span_of(a, sh, lens[b]);
    }
    if (s < s_end) __syncthreads();   // the records in LDS are read: the next part may write
  }
}

// One workgroup per (sequence, head tile, row) of a pair that several
// workgroups share: groups of D / 4 threads take its partial records in turn,
// then meet in LDS.
template <int D>
__global__ __launch_bounds__(256) void k_attn_join(const AttnArgs a, const AttnShape sh) {
  constexpr int TD = D / 4, NG = 256 / TD;
  __shared__ float lds[NG][D + 4];
  __shared__ float lds_ml[NG][2];
  const int b = blockIdx.x / sh.NHV, hv = blockIdx.x % sh.NHV, r = blockIdx.y;
  const int lane = threadIdx.x & 63;
  // steps before this sequence, and all of them
  int bef = 0, tot = 0;
  for (int i = lane; i < (int)a.B; i += 64) {
    const int n = span_of(a, sh, a.lens[i]).n;
    tot += n;
    bef += i < b ? n : 0;
  }
  const int total = wave_sum_i32(tot) * sh.NHV;
  const int nb = span_of(a, sh, a.lens[b]).n;
  const int s0 = wave_sum_i32(bef) * sh.NHV + hv * nb;
  const int nw = sh.nwg < total ? sh.nwg : total;
  const Runs runs(total, nw);
  const int w0 = runs.of(s0), w1 = runs.of(s0 + nb - 1);
  if (w0 == w1) return;   // finished by its one workgroup
  const int h = hv / sh.NRT, rr = (hv - h * sh.NRT) * sh.slot_rows + r;
  if (rr >= sh.rows) return;
  const int grp = threadIdx.x / TD, d0 = (threadIdx.x % TD) * 4;
  float m = -INFINITY, l = 0.0f;
  f32x4_t o = {0.0f, 0.0f, 0.0f, 0.0f};
  for (int w = w0 + grp; w <= w1; w += NG) {
    // a run that starts inside this pair, or with it, has it as its first part
    const int64_t slot = w > w0 || runs.start(w) == s0 ? 2 * w : 2 * w + 1;
    const int64_t rec = slot * sh.slot_rows + r;
    const float mw = sh.ml[rec * 2], lw = sh.ml[rec * 2 + 1];
    const f32x4_t ow = *reinterpret_cast<const f32x4_t*>(sh.o + rec * D + d0);
    const float mn = fmaxf(m, mw);
    const float use = mn == -INFINITY ? 0.0f : mn;
    const float f0 = __builtin_amdgcn_exp2f(m - use), f1 = __builtin_amdgcn_exp2f(mw - use);
    l = l * f0 + lw * f1;
#pragma unroll
    for (int e = 0; e < 4; ++e) o[e] = o[e] * f0 + ow[e] * f1;
    m = mn;
  }
  *reinterpret_cast<f32x4_t*>(&lds[grp][d0]) = o;
  if (d0 == 0) {
    lds_ml[grp][0] = m;
    lds_ml[grp][1] = l;
  }
  __syncthreads();
  if (threadIdx.x >= D / 8) return;
  const int d = threadIdx.x * 8;
  float mm = -INFINITY;
#pragma unroll
  for (int v = 0; v < NG; ++v) mm = fmaxf(mm, lds_ml[v][0]);
  const float use = mm == -INFINITY ? 0.0f : mm;
  float ll = 0.0f, out[8] = {0, 0, 0, 0, 0, 0, 0, 0};
#pragma unroll
  for (int v = 0; v < NG; ++v) {
    const float f = __builtin_amdgcn_exp2f(lds_ml[v][0] - use);
    ll = fmaf(lds_ml[v][1], f, ll);
#pragma unroll
    for (int e = 0; e < 8; ++e) out[e] = fmaf(lds[v][d + e], f, out[e]);
  }
  const float f = ll == 0.0f ? 0.0f : (a.cache_e4m3 ? *a.v_scale : 1.0f) / ll;
#pragma unroll
  for (int e = 0; e < 8; ++e) out[e] *= f;
  const int t = rr / sh.G;
  store8(a.out + ((int64_t)(b * a.Q + t) * a.Hq + h * sh.G + (rr - t * sh.G)) * D + d, out);
}

// Row tiles of 16, or of 32 where a head has more rows (heads of 256 keep 16:
// their registers are full).
int row_tiles(int64_t rows, int64_t D) { return rows <= 16 || D == 256 ? 1 : 2; }
// Workgroups of 4 wavefronts that a CU holds at once.
int per_cu(int RT, int64_t D) { return D == 256 ? 1 : RT == 2 ? 2 : 3; }

struct AttnLayout {
  size_t ml, o, total;
  int slot_rows;
};
AttnLayout attn_layout(int64_t rows, int64_t D) {
  const int RT = row_tiles(rows, D);
  AttnLayout L;
  L.slot_rows = (int)(rows < RT * 16 ? rows : RT * 16);
  const size_t slots = (size_t)2 * kCus * per_cu(RT, D);
  L.ml = 0;
  L.o = (slots * L.slot_rows * 2 * sizeof(float) + 255) & ~(size_t)255;
  L.total = (L.o + slots * L.slot_rows * (size_t)D * sizeof(float) + 255) & ~(size_t)255;
  return L;
}

// Keys that a row of the table can name (none where there is no page).
int capacity(const AttnArgs& a) {
  const int64_t cap = a.num_blocks ? a.max_blocks * a.page : 0;
  return (int)(cap < 0x7FFFFF00 ? cap : 0x7FFFFF00);
}
// Steps that a sequence has at most: by its table row, or by its window (which
// starts at most a tile early).
int64_t most_steps(const AttnArgs& a) {
  int64_t keys = capacity(a);
  if (a.window && a.window + a.Q + kTile < keys) keys = a.window + a.Q + kTile;
  return keys <= kStep ? 1 : (keys + kStep - 1) / kStep;
}

template <int D, bool FP8>
hipError_t launch_d(const AttnArgs& a, hipStream_t stream) {
  AttnShape sh;
  sh.G = (int)(a.Hq / a.Hkv);
  sh.rows = sh.G * (int)a.Q;
  const int RT = row_tiles(sh.rows, D);
  sh.NRT = (sh.rows + RT * 16 - 1) / (RT * 16);
  sh.NHV = (int)a.Hkv * sh.NRT;
  sh.cap = capacity(a);
  sh.page_shift = (a.page & (a.page - 1)) == 0 ? __builtin_ctzll((uint64_t)a.page) : -1;
  const AttnLayout L = attn_layout(sh.rows, D);
  sh.slot_rows = L.slot_rows;
  sh.ml = (float*)((char*)a.workspace + L.ml);
  sh.o = (float*)((char*)a.workspace + L.o);
  const int64_t steps = most_steps(a);
  const int64_t most = steps * sh.NHV * a.B;
  const int64_t fit = (int64_t)kCus * per_cu(RT, D);
  sh.nwg = (int)(most < fit ? most : fit);
  const bool pg = a.page % 16 == 0;
  const dim3 grid(sh.nwg), block(kWaves * 64);
#define NVFP4_ATTN(RT_)                                                                        \
  if (pg)                                                                                      \
    hipLaunchKernelGGL((k_paged_attn<D, FP8, RT_, true>), grid, block, 0, stream, a, sh);      \
  else                                                                                         \
    hipLaunchKernelGGL((k_paged_attn<D, FP8, RT_, false>), grid, block, 0, stream, a, sh)
  if constexpr (D == 256) {
    NVFP4_ATTN(1);
  } else {
    if (RT == 1) {
      NVFP4_ATTN(1);
    } else {
      NVFP4_ATTN(2);
    }
  }
#undef NVFP4_ATTN
  hipError_t e = hipGetLastError();
  // a pair of one step is never shared
  if (e != hipSuccess || steps == 1) return e;
  hipLaunchKernelGGL((k_attn_join<D>), dim3((uint32_t)(a.B * sh.NHV), (uint32_t)sh.slot_rows),
                     dim3(256), 0, stream, a, sh);
  return hipGetLastError();
}

}  // namespace

bool attn_fits(const AttnArgs& a) {
  const int64_t rows = a.Hq / a.Hkv * a.Q;   // one row tile per 16 rows at most
  return (__int128)most_steps(a) * a.B * a.Hkv * ((rows + 15) / 16) < 0x7FFFFFFF;
}

size_t attn_workspace_bytes(int64_t B, int64_t Q, int64_t Hq, int64_t Hkv, int64_t D) {
  if (B == 0 || Q == 0) return 0;
  return attn_layout(Hq / Hkv * Q, D).total;
}

hipError_t launch_paged_attention(const AttnArgs& a, hipStream_t stream) {
  if (a.cache_e4m3)
    return a.D == 64    ? launch_d<64, true>(a, stream)
           : a.D == 128 ? launch_d<128, true>(a, stream)
                        : launch_d<256, true>(a, stream);
  return a.D == 64    ? launch_d<64, false>(a, stream)
         : a.D == 128 ? launch_d<128, false>(a, stream)
                      : launch_d<256, false>(a, stream);
}

}  // namespace nvfp4
