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
// rows of a head (one or two tiles of 16) fill the columns of the matrix
// instructions, so one pass serves them all:
//   S^T[key, row] = K Q^T     A = K (16 keys x 32 dims), B = Q^T
//   O^T[dim, row] += V^T P^T  A = V^T (16 dims x 32 keys), B = P^T
// A lane ends S^T with 4 keys of one row per 16 keys. The order of the keys in
// the second product is free as long as V follows, so those registers are its
// B operand as they stand: P never leaves the registers. V^T's operand needs 8
// keys of one dim per lane: a lane loads 8 dims of 8 keys (whole rows of V per
// load) and pairs halves with one v_perm_b32 per dword. K, V and P pass no LDS.
//
// Split: a wavefront takes one head and a run of tiles by itself; neighbouring
// wavefronts take the other heads of the same tokens, so that a workgroup
// reads whole stretches of memory in the [page, heads, D] order. The lengths
// are on the device, so the grid is fixed and the kernel divides the work: the
// tiles of all sequences are numbered in one row, and run j of every head is
// the j-th equal part of them, whatever the lengths are. A sequence that lies
// inside one run is finished there; others leave partial (m, sum, O) records,
// at most two per wavefront, that k_attn_join adds in a fixed order. No
// atomics. Where the table's rows are short (whole_keys), one workgroup of
// eight wavefronts takes a sequence and head whole and joins them in LDS.
#include "attn_wave.h"

namespace nvfp4 {

namespace {

// The reference of the exponentials is moved only when a score passes it by
// more than this (in powers of two): exp2 of at most 2^8 loses nothing in fp32
// or bf16, and most turns need no maximum across lanes and no rescaling.
constexpr float kSlack = 8.0f;
// Wavefronts per SIMD of the split form. Few long streams read memory best:
// heads of 256 bytes and more keep 16 KB and more in flight per wavefront with
// one; smaller heads need two.
constexpr int waves_per_simd(int RT, int D, bool FP8) {
  return RT == 1 && D * (FP8 ? 1 : 2) < 256 ? 2 : 1;
}
static_assert(waves_per_simd(1, 64, true) * kCus * 4 <= kMaxRuns, "the join's weights");

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
        const u32x4_t v = load_stream(q);
#pragma unroll
        for (int e = 0; e < 4; ++e) w[i + e] = v[e];
      } else if constexpr (kPiece == 2) {
        const u32x2_t v = __builtin_nontemporal_load(reinterpret_cast<const u32x2_t*>(q));
        w[i] = v[0];
        w[i + 1] = v[1];
      } else {
        w[i] = __builtin_nontemporal_load(reinterpret_cast<const uint32_t*>(q));
      }
    }
  }
  // some element is infinite or NaN (E4M3: NaN): a half, or byte, with all
  // exponent bits (and E4M3's mantissa) set
  __device__ __forceinline__ bool not_finite() const {
    constexpr uint32_t kSet = FP8 ? 0x7F7F7F7Fu : 0x7F807F80u;
    constexpr uint32_t kOnes = FP8 ? 0x01010101u : 0x00010001u;
    constexpr uint32_t kTops = FP8 ? 0x80808080u : 0x80008000u;
    uint32_t hit = 0u;
#pragma unroll
    for (int d = 0; d < kDw; ++d) {
      const uint32_t x = (w[d] & kSet) ^ kSet;   // a field of zeros
      hit |= (x - kOnes) & ~x & kTops;
    }
    return hit != 0u;
  }
  __device__ __forceinline__ uint32_t get(int d) const {   // dims 2 d, 2 d + 1
    if constexpr (FP8)
      return (d & 1) ? e4m3x2_to_bf16<1>(w[d >> 1]) : e4m3x2_to_bf16<0>(w[d >> 1]);
    else
      return w[d];
  }
};

// K, V and O of one wavefront's pass over tiles of one head, or of two side by
// side (E4M3): of a tile's 32 rows of K and V, slots, those of quads 0 and 2 of
// each 16 are then the first head's, of 1 and 3 the second's, at the same keys. A
// load takes both heads of a key, and a lane's scores are all of one head.
template <int D, bool FP8, int RT, bool PG, bool MOD, int HEADS = 1>
struct AttnWave : AttnPass<AttnWave<D, FP8, RT, PG, MOD, HEADS>, TK / HEADS, RT, PG ? 16 : 0, MOD,
                           HEADS, TK / 16> {
  using Pass = AttnPass<AttnWave, TK / HEADS, RT, PG ? 16 : 0, MOD, HEADS, TK / 16>;
  using Pass::a, Pass::sh, Pass::n, Pass::g, Pass::h, Pass::Q, Pass::G, Pass::row0, Pass::c,
      Pass::head_off, Pass::tok, Pass::m, Pass::l, Pass::hl, Pass::col, Pass::NU, Pass::NO;
  static_assert(HEADS == 1 || (FP8 && RT == 1 && D == 64), "any_nan, load_v");
  static constexpr bool kOthers = HEADS > 1;
  using Args = AttnArgs;
  static constexpr int kD = D;
  static constexpr bool kScaled = FP8;
  static constexpr int kPerSimd = waves_per_simd(RT, D, FP8);
  static constexpr int kStage = 0;
  static constexpr bool kCapInv = false;
  static constexpr int NP = TK / 32;           // products over the keys
  static constexpr int NJ = D / 32;            // products over the dims
  static constexpr int NV = D / 16;            // dims per lane of V
  static constexpr int ES = FP8 ? 1 : 2;
  static constexpr int KL = D * ES / 64;       // 16-byte loads of K per lane and 16 keys
  static constexpr int kParts = 3;             // bf16 numbers that hold a probability
  typedef u32x4_t Weights[kParts][RT][NP];

  const uint32_t stb, shb, k_in, k_lane, v_dim, v_lane;   // bytes
  bf16x8_t qf[RT][NJ];
  f32x4_t O[RT][NV];
  u32x4_t kr[NU][KL];
  VRow<NV, FP8> vr[TK / 4];
  int64_t off[NO];                             // elements, from place()

  __device__ __forceinline__ AttnWave(const AttnArgs& a_, const AttnShape& sh_, int h_, int row0_,
                                      float k_scale, uint8_t*)
      : Pass(a_, sh_, h_, row0_, k_scale),
        stb((uint32_t)a_.st * ES), shb(HEADS == 1 ? 0u : (uint32_t)a_.sh * ES),
        k_in(head_of(n >> 2) * shb + (uint32_t)g * 16),
        k_lane((uint32_t)key_at(0, n >> 2, n & 3) * stb + k_in),
        v_dim(head_of(g) * shb + (uint32_t)n * (NV > 8 ? 8 : NV) * ES),
        v_lane((uint32_t)key_at(0, g, 0) * stb + v_dim) {
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
      const int r = row0 + rt * 16 + col;
      const bool live = tok[rt] >= 0;
      const uint16_t* qp = a.q + ((int64_t)(b * (int64_t)Q + (live ? tok[rt] : 0)) * a.Hq +
                                  (h + hl) * G + (live ? r - tok[rt] * G : 0)) * D;
#pragma unroll
      for (int j = 0; j < NJ; ++j) {
        const int d0 = FP8 ? (j >> 1) * 64 + g * 16 + (j & 1) * 8 : j * 32 + g * 8;
        // rows that do not exist read another's: nothing of them is written
        qf[rt][j] = *reinterpret_cast<const bf16x8_t*>(qp + d0);
      }
    }
  }
  __device__ __forceinline__ void place(int u, int id, int in) {
    off[u] = (int64_t)id * a.sb + (int64_t)in * a.st + head_off;
  }
  // byte offset of lane src's key
  __device__ __forceinline__ int64_t at_key(int src) const {
    return this->from_lane(off[0], src) * ES;
  }
  // slot i of quad `quad` of run u: its key in the tile, and its head from h on
  static __device__ __forceinline__ int key_at(int u, int quad, int i) {
    return u * (16 / HEADS) + quad / HEADS * 4 + i;
  }
  static __device__ __forceinline__ uint32_t head_of(int quad) {
    return HEADS == 1 ? 0u : (uint32_t)quad & 1u;
  }
  // the key of the tile that a lane has as the e-th (of TK / 4) of V, S^T and P
  static __device__ __forceinline__ int key_of(int e, int g) { return key_at(e >> 2, g, e & 3); }
  // run u of 16 slots in its page: two heads' runs share one
  __device__ __forceinline__ uint32_t run(int u, bool want) const {
    return HEADS > 1 && want ? (uint32_t)(u * (16 / HEADS)) * stb : 0u;
  }
  // want: false where no tile follows. The loads are issued all the same, all
  // lanes from one address: a branch around them would make the waits on both
  // sides drain everything in flight.
  __device__ __forceinline__ void load_k(bool want) {
    const uint8_t* const kc = (const uint8_t*)a.k_cache;
    const uint32_t lane_off = want ? k_lane : 0u;
#pragma unroll
    for (int u = 0; u < NU; ++u) {
      const uint8_t* p = PG ? kc + off[NO > 1 ? u : 0] * ES + run(u, want) + lane_off
                            : want ? kc + at_key(key_at(u, n >> 2, n & 3)) + k_in : kc;
#pragma unroll
      for (int j = 0; j < KL; ++j)
        // a load takes 64 bytes of a key: half of an E4M3 head of 128, whose
        // other half the hint would read again (6.1 against 5.9 TB/s); wider
        // rows want the hint (bf16: 6.6 against 6.4)
        kr[u][j] = FP8 ? *reinterpret_cast<const u32x4_t*>(p + j * 64) : load_stream(p + j * 64);
    }
  }
  __device__ __forceinline__ void load_v(bool want) {
    const uint8_t* const vc = (const uint8_t*)a.v_cache;
    const uint32_t lane_off = want ? v_lane : 0u, st = want ? stb : 0u;
    if constexpr (HEADS > 1 && !PG) {   // pages hold whole quads of keys
#pragma unroll
      for (int u = 0; u < NU; ++u) {
        const uint8_t* p = want ? vc + at_key(key_at(u, g, 0)) + v_dim : vc;
#pragma unroll
        for (int i = 0; i < 4; ++i) vr[u * 4 + i].load(p + (uint32_t)i * st);
      }
      return;
    }
#pragma unroll
    for (int i = 0; i < TK / 4; ++i)
      vr[i].load(PG ? vc + off[NO > 1 ? i >> 2 : 0] * ES + run(i >> 2, want) +
                          (uint32_t)(i & 3) * st + lane_off
                    : want ? vc + at_key(key_of(i, g)) + v_dim : vc);
  }

  __device__ __forceinline__ void take_v() {}

  // S^T of the loaded tile, scaled
  __device__ __forceinline__ void scores(f32x4_t (&S)[RT][NU]) {
#pragma unroll
    for (int u = 0; u < NU; ++u) {
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
          S[rt][u] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, kv),
                                                             qf[rt][j], S[rt][u], 0, 0, 0);
      }
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) S[rt][u] *= c;
    }
  }
  // The running maximum and sum, and P as the sum of three bf16, which hold all
  // 24 bits of it: each takes the upper half of what the ones before it leave.
  // Two would hold 16 bits, and where the values of a head cancel their
  // rounding (2^-18 of each weight) would stand above the output's: of 8192
  // outputs over 1277 keys 20 rounded the other way, 2 with three. The third
  // takes a half more of these products: 5 tokens on 32773 keys 27.8 -> 28.3 us,
  // 700 keys 6.2 -> 6.3, a short batch with two row tiles 16.3 -> 17.3.
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
      const float m_use = m[rt] == -INFINITY ? 0.0f : m[rt];
#pragma unroll
      for (int e = 0; e < 2 * NU; ++e) {
        const float p0 = __builtin_amdgcn_exp2f(S[rt][e >> 1][(e & 1) * 2] - m_use);
        const float p1 = __builtin_amdgcn_exp2f(S[rt][e >> 1][(e & 1) * 2 + 1] - m_use);
        l[rt] += p0 + p1;
        uint32_t u0 = __float_as_uint(p0), u1 = __float_as_uint(p1);
#pragma unroll
        for (int i = 0; i < kParts; ++i) {
          pf[i][rt][e >> 2][e & 3] = perm_hi(u0, u1);
          u0 = __float_as_uint(__uint_as_float(u0) - bf16_hi(u0));   // exact
          u1 = __float_as_uint(__uint_as_float(u1) - bf16_hi(u1));
        }
      }
    }
  }
  __device__ __forceinline__ f32x4_t product(u32x4_t v, u32x4_t pf, f32x4_t acc) const {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, v),
                                                   __builtin_bit_cast(bf16x8_t, pf), acc, 0, 0, 0);
  }
  // O += V^T P^T, the smallest parts first
  __device__ __forceinline__ void values(const Weights& pf) {
#pragma unroll
    for (int d = 0; d < NV / 2; ++d) {
#pragma unroll
      for (int q = 0; q < NP; ++q) {
        uint32_t x[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = vr[q * 8 + i].get(d);
        const u32x4_t lo = {perm_lo(x[0], x[1]), perm_lo(x[2], x[3]), perm_lo(x[4], x[5]),
                            perm_lo(x[6], x[7])};
        const u32x4_t hi = {perm_hi(x[0], x[1]), perm_hi(x[2], x[3]), perm_hi(x[4], x[5]),
                            perm_hi(x[6], x[7])};
#pragma unroll
        for (int rt = 0; rt < RT; ++rt)
#pragma unroll
          for (int i = kParts - 1; i >= 0; --i) {
            O[rt][2 * d] = product(lo, pf[i][rt][q], O[rt][2 * d]);
            O[rt][2 * d + 1] = product(hi, pf[i][rt][q], O[rt][2 * d + 1]);
          }
      }
    }
  }

  // the lane's e-th key of V becomes zero where it is not seen
  __device__ __forceinline__ void keep(int e, bool see) {
#pragma unroll
    for (int d = 0; d < VRow<NV, FP8>::kDw; ++d) vr[e].w[d] = see ? vr[e].w[d] : 0u;
  }
  // some value of the tile is NaN (E4M3)
  __device__ __forceinline__ bool any_nan() const {
    uint32_t hit = 0u;
#pragma unroll
    for (int e = 0; e < TK / 4; ++e)
#pragma unroll
      for (int d = 0; d < VRow<NV, FP8>::kDw; ++d) hit |= (vr[e].w[d] & 0x7F7F7F7Fu) + 0x01010101u;
    return __any((hit & 0x80808080u) != 0u);
  }
  // A key that some rows see and others do not has weight 0 for these, which is
  // enough unless its value is infinite or NaN (0 * inf would reach them). Such
  // a value becomes zero, and the sum of the rows that see it NaN. weightless:
  // bit e, this lane's row does not see key e.
  __device__ __forceinline__ void settle(const uint32_t (&weightless)[RT]) {
#pragma unroll
    for (int e = 0; e < TK / 4; ++e) {
      const bool bad = vr[e].not_finite();
      keep(e, !bad);
      const bool any = (__ballot(bad) >> (16 * g)) & 0xFFFFu;   // of the key's 16 lanes
#pragma unroll
      for (int rt = 0; rt < RT; ++rt)
        if (any && !((weightless[rt] >> e) & 1u)) l[rt] = __builtin_nanf("");
    }
  }

  // O^T row g * 4 + i of the products is dims (g * 4 + i) * 8 .. + 7 (heads of
  // 64: * 4 .. + 3; of 256: products 8 .. 15 are the second half). f(d0, v): 4
  // consecutive dims of row rt * 16 + n.
  template <typename F>
  __device__ __forceinline__ void each4(int rt, F f) const {
    constexpr int kRun = NV > 8 ? 8 : NV;
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int t = 0; t < NV; t += 4)
          f((t / kRun) * 128 + (g * 4 + i) * kRun + t % kRun,
            f32x4_t{O[rt][t][i], O[rt][t + 1][i], O[rt][t + 2][i], O[rt][t + 3][i]});
  }
};

// Row tiles of 16 in one pass; a head with more rows is read again for the
// others. One against two, 8 sequences, bf16: 20000 keys, 8 heads of 128 with 20
// rows 210 / 114 us, 8192 keys with 64 rows 186 / 103, with 256 rows 557 / 336 (the
// row tiles of a head are neighbouring wavefronts, but their loads carry the
// streaming hint all the same). Heads of 256 take two where pages hold whole
// runs of 16 keys (pg): 20000 keys, 8 heads with 20 rows 387 / 241, 2 heads with 32
// rows 112 / 102, though the bf16 form spills 45 VGPRs. Without, one offset per
// lane and key spills more than it saves (40 rows, pages of 20: 108 / 163 us).
int row_tiles(int64_t rows, int64_t D, bool pg) { return rows <= 16 || (D == 256 && !pg) ? 1 : 2; }

// The whole form takes tables of at most this many keys (a row's, or a
// window's). It saves the join, but a wavefront reads 32 of every 256 keys one
// after the other: about 4 us a turn in bf16 at heads of 128, half of it in E4M3
// or at heads of 64. So few sequences take it for one such turn (2^16 bytes of a
// head's keys); from 256 rows on, where the join's own work is more, for two;
// where the workgroups fill the CUs, or half of them with 16 rows each, up to 1024
// keys. More than 256 workgroups run one after the other (their registers allow
// one per CU, or two), which only a long join pays for: with less than four rows
// each they take tables of one turn, and past 768 none. Whole against split in
// us, in graphs of 20 calls, 8 key-value heads of 128 if not said otherwise:
//   1 token, G 4, bf16:   1 sequence 256 keys 7.1 / 9.5, 512 11.2 / 10.0;
//                         8: 512 13.0 / 12.1, 1024 21.8 / 14.0; 16: 512 13.7 /
//                         13.9, 1024 23.2 / 19.5; 32: 1024 27.2 / 30.1
//   the same, E4M3:       1: 512 7.5 / 9.3, 1024 11.9 / 9.7; 8: 1024 13.1 / 14.3
//   5 tokens, bf16:       1: 256 11.0 / 12.7, 512 15.7 / 13.4; 8: 512 17.5 / 21.2,
//                         1024 25.8 / 23.0; 16: 1024 28.4 / 29.6
//   pages of 20, 5 tokens: 1: 256 12.9 / 13.4, 512 22.3 / 14.2
//   16 heads of 64, G 1:  1: 512 9.4 / 9.3; 8: 1024 15.9 / 13.9; 16: 17.6 / 19.8;
//                         24: 512 18.2 / 17.2, 1024 31.1 / 25.3; 64: 128 16.4 / 15.3,
//                         512 36.3 / 30.4
int64_t whole_keys(const AttnArgs& a, const AttnShape& sh) {
  const int64_t wgs = a.B * sh.NHV, one = (1 << 16) / (a.D * (a.cache_e4m3 ? 1 : 2));
  if (wgs > kCus && sh.rows < 4) return wgs > 3 * kCus ? 0 : one;
  if (wgs >= kCus || (wgs >= kCus / 2 && sh.rows >= 16)) return 1024;
  return a.B * a.Q * a.Hq >= 256 && one < 1024 ? 2 * one : one;
}
AttnLayout layout(int64_t rows, int64_t Hkv, int64_t D, bool e4m3, bool pg, int heads = 1) {
  const int RT = row_tiles(rows, D, pg);
  return attn_layout(rows, Hkv, D, RT, waves_per_simd(RT, (int)D, e4m3), heads);
}

// Two heads of 64 in E4M3 side by side, for scores that are capped or biased (plain
// ones keep the order of sums that they had): a load then takes whole lines of 128
// bytes, where each head's 64 come at half of memory's rate, but a wavefront leaves
// twice the rows to the join. From 2^19 keys of all heads on (by the tables, as
// the lengths are on the device), and for pages of whole quads of keys, whose places
// a lane looks up once (with one look-up a key pages of 20 gain nothing). One head
// against two, us: 16 heads, G 1, pages of 16: 1 sequence of 16384 keys 17.4 /
// 17.9; 4 of 8192 23.0 / 22.4; 16 of 20000 151 / 119, pages of 20 202 / 161; 8
// heads, G 4: 4 of 8192 18.1 / 18.3; 16 of 20000 78 / 68; 2 heads, G 8: 16 of 20000
// 27.4 / 28.5, pages of 20 34.4 / 33.1. A load's bytes have to be counted in 32 bits.
bool pairs(int64_t rows, int64_t Hkv, int64_t D) { return D == 64 && rows <= 8 && Hkv % 2 == 0; }
bool side_by_side(const AttnArgs& a, const AttnShape& sh) {
  return pairs(sh.rows, a.Hkv, a.D) && a.page % 4 == 0 &&
         a.B * most_keys(a) * a.Hkv >= 1 << 19 && a.sh < 1 << 28 &&
         most_keys(a) > whole_keys(a, sh) &&
         (most_keys(a) + 15) / 16 * a.B < 0x7FFFFFFF;   // tiles, as in attn_fits
}

template <int D, bool FP8, int RT, bool PG, bool MOD>
hipError_t launch_rt(const AttnArgs& a, const AttnShape& sh, hipStream_t stream) {
  return launch_forms<AttnWave<D, FP8, RT, PG, MOD>>(a, sh, whole_keys(a, sh), stream);
}

template <int D, bool FP8, bool MOD>
hipError_t launch_d(const AttnArgs& a, hipStream_t stream) {
  const bool pg = a.page % 16 == 0;
  const AttnLayout L = layout(a.Hq / a.Hkv * a.Q, a.Hkv, D, FP8, pg);
  const AttnShape sh = attn_shape(a, L);
  if constexpr (D == 64 && FP8 && MOD) {
    if (side_by_side(a, sh)) {
      const AttnShape two = attn_shape(a, layout(sh.rows, a.Hkv, D, FP8, pg, 2));
      return pg ? launch_forms<AttnWave<D, FP8, 1, true, MOD, 2>>(a, two, 0, stream)
                : launch_forms<AttnWave<D, FP8, 1, false, MOD, 2>>(a, two, 0, stream);
    }
  }
  if (L.RT == 2) {
    if (pg) return launch_rt<D, FP8, 2, true, MOD>(a, sh, stream);
    if constexpr (D < 256) return launch_rt<D, FP8, 2, false, MOD>(a, sh, stream);
  }
  return pg ? launch_rt<D, FP8, 1, true, MOD>(a, sh, stream)
            : launch_rt<D, FP8, 1, false, MOD>(a, sh, stream);
}

template <bool MOD>
hipError_t launch_scored(const AttnArgs& a, hipStream_t stream) {
  if (a.cache_e4m3)
    return a.D == 64    ? launch_d<64, true, MOD>(a, stream)
           : a.D == 128 ? launch_d<128, true, MOD>(a, stream)
                        : launch_d<256, true, MOD>(a, stream);
  return a.D == 64    ? launch_d<64, false, MOD>(a, stream)
         : a.D == 128 ? launch_d<128, false, MOD>(a, stream)
                      : launch_d<256, false, MOD>(a, stream);
}

}  // namespace

bool attn_fits(const AttnCommon& a) {
  const int64_t rows = a.Hq / a.Hkv * a.Q;
  const int NHV = a.cache_nvfp4 ? attn4_row_units(rows, a.Hkv, a.D)
                                : layout(rows, a.Hkv, a.D, a.cache_e4m3, a.page % 16 == 0).NHV;
  // tiles are numbered in 31 bits, a launch's work-items in 32
  return (most_keys(a) + TK - 1) / TK * a.B < 0x7FFFFFFF && a.B * NHV <= 1 << 22;
}

size_t attn_workspace_bytes(int64_t B, int64_t Q, int64_t Hq, int64_t Hkv, int64_t D) {
  if (B == 0 || Q == 0) return 0;
  // the call's cache type and page are not known here: the largest of all
  size_t most = attn4_workspace_bytes(Hq / Hkv * Q, Hkv, D);
  for (int i = 0; i < 4; ++i) {
    const size_t n = layout(Hq / Hkv * Q, Hkv, D, i & 1, i & 2).total;
    most = n > most ? n : most;
  }
  if (pairs(Hq / Hkv * Q, Hkv, D)) {
    const size_t n = layout(Hq / Hkv * Q, Hkv, D, true, true, 2).total;
    most = n > most ? n : most;
  }
  return most;
}

size_t attn_workspace_need(const AttnArgs& a) {
  const int64_t rows = a.Hq / a.Hkv * a.Q;
  const bool pg = a.page % 16 == 0;
  const size_t one = layout(rows, a.Hkv, a.D, a.cache_e4m3, pg).total;
  if (!a.cache_e4m3 || !scored(a) || !pairs(rows, a.Hkv, a.D)) return one;
  const size_t two = layout(rows, a.Hkv, a.D, true, pg, 2).total;
  return one > two ? one : two;
}

hipError_t launch_paged_attention(const AttnArgs& a, hipStream_t stream) {
  return scored(a) ? launch_scored<true>(a, stream) : launch_scored<false>(a, stream);
}

}  // namespace nvfp4
