// paged_attn4.hip -- attention of the new tokens of each sequence over a paged
// key-value cache in NVFP4: E2M1 codes, an E4M3 scale for each 16 elements of a
// head and one fp32 scale for all keys (values). The split of the work, the
// pass and the join are those of the other caches (attn_wave.h).
//
// Bound: the bytes of K and V, 9/16 of one per element, and next to it the
// vector ALU, which turns each element into a number. A tile of 64 rows of K and V
// of 128 is 9.2 KB, of which the card reads one per CU in 780 clocks, one per SIMD
// in 3100; a wavefront issues some 450 vector and 48 matrix instructions for it, 2300
// clocks. So the long batch (16 sequences of 20000 to 65536 keys, 8 heads of 128, 713
// MB) takes 131 us in the first ten calls of a row, 150 to 200 in the next hundred and
// 140 from then on, whatever the inputs, and 6 to 8 for the join: 5.1 TB/s, where a
// plain read takes 99. The arithmetic of one wavefront has to run beside the loads of
// another, at the rate that the card keeps under it. Tiles of 64 rows (one page
// look-up, one maximum and one branch for each 64, not 32) and V through LDS brought
// most of it: 165 -> 131 us on one set of inputs.
//
// A code times its block's scale has 6 significant bits and lies between 2^-10
// and 2688: it is exact in fp16 (and in bf16, which has no packed product). So
// the products with the matrix cores are fp16:
//   S^T[key, row] = K Q^T    O^T[dim, row] += V^T P^T
// - K: a lane takes one key's D / 4 consecutive dims (16 bytes of codes at 128)
//   and their scales; two codes a conversion, two elements a packed product.
// - Q: a row of bf16 is multiplied by a power of two that takes its largest
//   element to 2^14 .. 2^15; fp16 then holds every element down to 2^-31 of that
//   one whole, and the smaller ones to 2^-39 of it. The scores' factor takes the
//   power back.
// - V is loaded in whole rows, 16 bytes a lane, and goes through LDS of the wavefront's
//   own (5 KB with both's scales at 128), as the lanes need other stretches of it.
// - V^T wants pairs of keys where a byte holds a pair of dims: the nibbles of
//   two keys' words change places first, 4 instructions for 16 elements, and
//   each conversion gives one dim of two keys. The pair's two scales multiply it.
// - P enters as the sum of two fp16, each rounded to nearest: 2^-23 of it at most is
//   lost (of what the first leaves 12 bits, the last of them set), or 2^-36 of the
//   largest weight at small ones. The exponents are raised by 11 to use fp16's range.
#include "attn_wave.h"

namespace nvfp4 {

namespace {

typedef _Float16 f16x2_t __attribute__((ext_vector_type(2)));
typedef float f32x2_t __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8_t __attribute__((ext_vector_type(8)));

// The reference of the exponentials is moved only when a score passes it by
// more than kSlack (in powers of two); a weight is at most 2^(kRaise + kSlack),
// which fp16 holds.
constexpr float kSlack = 4.0f;
constexpr float kRaise = 11.0f;

// Wavefronts per SIMD of the split form: the second one's arithmetic runs while
// the first waits. Two against one, us, 8 sequences of 20000 keys, 8 heads: of 128, 4
// rows, pages of 16, 20 and 64 48 / 55, 54 / 70, 49 / 56; of 64, 20 rows (two tiles)
// 59 / 73, 55 / 66, 52 / 64; of 256 160 / 151 (there the registers are too few: one).
// Two tiles at heads of 128 fit into half of the registers only where a tile is
// one page's (74 / 83 on pages of 64, 14 VGPRs spilled, 26 where scored): with a place for
// each run of 16 or each key 91 to 106 spill, and one wavefront would be faster there
// (pages of 16 190 / 90, of 20 216 / 106; capped 185 / 128, 210 / 143). Open.
constexpr int waves_per_simd(int D) { return D < 256 ? 2 : 1; }
static_assert(waves_per_simd(64) * kCus * 4 <= kMaxRuns, "the join's weights");

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

// A tile is 64 rows of K and V, slots: 64 / HEADS keys of HEADS neighbouring
// heads, slot = key * HEADS + head, which is how they lie in memory where a
// token's heads are neighbours.
template <int D, int RT, int RUN, bool MOD, int HEADS>
struct Attn4Wave
    : AttnPass<Attn4Wave<D, RT, RUN, MOD, HEADS>, 64 / HEADS, RT, RUN, MOD, HEADS> {
  using Pass = AttnPass<Attn4Wave, 64 / HEADS, RT, RUN, MOD, HEADS>;
  using Pass::a, Pass::sh, Pass::lane, Pass::n, Pass::g, Pass::h, Pass::Q, Pass::G, Pass::row0,
      Pass::c, Pass::head_off, Pass::tok, Pass::m, Pass::l, Pass::hl, Pass::col, Pass::NO;
  using Args = Attn4Args;
  static constexpr int kD = D;
  static constexpr bool kScaled = true;
  static constexpr bool kOthers = false;
  static constexpr bool kCapInv = true;
  static constexpr int kPerSimd = waves_per_simd(D);
  static constexpr int NU = 4;                 // runs of 16 slots
  static constexpr int E = 16 / HEADS;         // scores that count per lane and row tile
  static constexpr int PU = 4 / HEADS;         // of them per run of 16 slots
  static constexpr int NS = Pass::NU;          // words of four scores
  static constexpr int NP = 2;                 // products over the slots
  static constexpr int NJ = D / 32;            // products over the dims: words of K per lane and key
  static constexpr int NV = D / 16;            // dims per lane of V
  static constexpr int VW = NV > 8 ? 2 : 1;    // words of V per lane and key
  static constexpr int kParts = 2;             // fp16 numbers that hold a probability
  typedef u32x4_t Weights[kParts][RT][NP];
  // What a wavefront takes through LDS: V's codes, K's scales key by key, V's
  // scales block by block.
  static constexpr int kRow = D / 2, kBlocks = D / 16;   // bytes of a key
  static constexpr int kStage = 64 * (kRow + 2 * kBlocks);
  static constexpr int VL = D / 32;            // 16-byte loads of V per lane and tile: of 1 KB
  static constexpr int kPerV = kRow / 16, kPerB = kBlocks / 4;   // lanes per slot of a load
  static constexpr int KV = 1024 / kRow;       // slots of such a load
  static constexpr int SL = D / 64;            // 4-byte loads of scales per lane and tile
  static constexpr int KS = 256 / kBlocks;     // slots of such a load

  const Attn4Args& more;                       // a, with the block scales
  const int64_t head_boff;
  const uint32_t st, bst;
  const uint32_t sh1, bsh1;                    // from a head to the next
  const uint32_t k_in, v_in, b_in;             // the lane's bytes of K, V, scales in a load
  const bool alike;                            // scales lie as the codes, 8 bytes to one
  uint8_t* const vs;                           // LDS
  u32x4_t qf[RT][NJ];
  float qs[RT];                                // scale of a row's scores
  f32x4_t O[RT][NV];
  uint32_t kr[NU][NJ], kb[SL];                 // K: codes of the lane's slots, scales as loaded
  u32x4_t vr[VL];                              // V as loaded
  uint32_t vl[SL];
  uint32_t vb[NU];                             // V's scales of the lane's slots: 4 to a word
  int64_t off[NO], boff[NO];                   // bytes, from place()

  __device__ __forceinline__ Attn4Wave(const Attn4Args& a_, const AttnShape& sh_, int h_,
                                       int row0_, float k_scale, uint8_t* stage)
      : Pass(a_, sh_, h_, row0_, k_scale), more(a_),
        head_boff((int64_t)h_ * a_.block_sh), st((uint32_t)a_.st), bst((uint32_t)a_.block_st),
        sh1((uint32_t)a_.sh), bsh1((uint32_t)a_.block_sh),
        k_in(in_load(n, st, sh1) + (uint32_t)g * (D / 8)),
        v_in(in_load(v_slot(lane / kPerV), st, sh1) + (uint32_t)(lane % kPerV) * 16),
        b_in(in_load(lane / kPerB, bst, bsh1) + (uint32_t)(lane % kPerB) * 4),
        alike(a_.sb == 8 * a_.block_sb && a_.st == 8 * a_.block_st && a_.sh == 8 * a_.block_sh),
        vs(stage) {
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
      // rows that do not exist read another's: nothing of them is written
      const uint16_t* qp = a.q + ((int64_t)(b * (int64_t)Q + (live ? tok[rt] : 0)) * a.Hq +
                                  (h + hl) * G + (live ? r - tok[rt] * G : 0)) * D + g * (D / 4);
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
      // 2^up takes it to 2^14 .. (2^126 at most: such rows' scores are nothing).
      // The scores' factor is made positive, so that a maximum can be taken
      // before it: its sign goes to q, and a factor of zero too.
      int up = 14 + 127 - (int)(top >> 23);
      up = up > 126 ? 126 : up;
      const float f = c == 0.0f ? 0.0f
                                : copysignf(__uint_as_float((uint32_t)(127 + up) << 23), c);
      qs[rt] = fmaxf(fabsf(c) * __uint_as_float((uint32_t)(127 - up) << 23), 0x1p-126f);
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
    // a page's stride is a multiple of 16 below 2^35 (its scales' one of 4 below
    // 2^33): products of 32 bits
    off[u] = (int64_t)((uint64_t)(uint32_t)id * (uint32_t)(a.sb >> 4)) * 16 +
             (int64_t)((uint64_t)(uint32_t)in * st) + head_off;
    boff[u] = alike ? off[u] >> 3
                    : (int64_t)((uint64_t)(uint32_t)id * (uint32_t)(more.block_sb >> 2)) * 4 +
                          (int64_t)((uint64_t)(uint32_t)in * bst) + head_boff;
  }
  // The lane's e-th score (of E) is this key of the tile. Its slots of V and P
  // are u * 16 + g * 4 + i for i = 0 .. 3; slot i is of head i % HEADS, and a lane
  // (a row of head hl) has weights for those of its own head only.
  static __device__ __forceinline__ int key_of(int e, int g) {
    return e / PU * (16 / HEADS) + g * PU + e % PU;
  }
  // A slot's bytes from a load's first slot on, inside one run of keys.
  static __device__ __forceinline__ uint32_t in_load(int slot, uint32_t key, uint32_t head) {
    return (uint32_t)(slot / HEADS % (RUN ? RUN : 64)) * key + (uint32_t)(slot % HEADS) * head;
  }
  // Where the lane's slot of a load lies: the load's keys are FIRST .. FIRST +
  // COUNT - 1 of the tile, `slot` counts from FIRST's first on, `lane_in` are its
  // bytes there (in_load's and those inside the slot, `in`). want: false where no
  // tile follows. The loads are issued all the same, all lanes from one address: a
  // branch around them would make the waits on both sides drain everything in
  // flight.
  template <int FIRST, int COUNT>
  __device__ __forceinline__ const uint8_t* at(const void* base, const int64_t (&o)[NO],
                                               uint32_t stride, uint32_t head, int slot,
                                               uint32_t in, uint32_t lane_in, bool want) const {
    const uint8_t* const p = (const uint8_t*)base;
    if constexpr (RUN == 0) {
      return want ? p + this->from_lane(o[0], FIRST + slot / HEADS) +
                        ((uint32_t)(slot % HEADS) * head + in) : p;
    } else {
      // uniform, but for loads of several runs
      const uint8_t* q = p + o[FIRST / RUN];
      if constexpr (COUNT == 2 * RUN) {
        q = p + (slot / HEADS < RUN ? o[FIRST / RUN] : o[FIRST / RUN + 1]);
      } else if constexpr (COUNT == 4 * RUN) {
        const int r = slot / HEADS / RUN;
        const int64_t lo = r & 1 ? o[1] : o[0], hi = r & 1 ? o[3] : o[2];
        q = p + (r & 2 ? hi : lo);
      }
      return q + (uint32_t)(FIRST % RUN) * stride + (want ? lane_in : 0u);
    }
  }
  template <int U>
  __device__ __forceinline__ void load_k_run(bool want) {
    const uint8_t* p = at<U * 16 / HEADS, 16 / HEADS>(
        a.k_cache, off, st, sh1, n, (uint32_t)g * (D / 8), k_in, want);
    if constexpr (D == 64) {
      const u32x2_t v = *reinterpret_cast<const u32x2_t*>(p);
      kr[U][0] = v[0];
      kr[U][1] = v[1];
    } else {
#pragma unroll
      for (int j = 0; j < NJ; j += 4) {
        const u32x4_t v = *reinterpret_cast<const u32x4_t*>(p + j * 4);
#pragma unroll
        for (int e = 0; e < 4; ++e) kr[U][j + e] = v[e];
      }
    }
  }
  __device__ __forceinline__ void load_k(bool want) {
    load_k_run<0>(want);
    load_k_run<1>(want);
    load_k_run<2>(want);
    load_k_run<3>(want);
    load_scales<0>(more.k_blocks, want, kb);
  }
  // V: whole rows, 16 bytes a lane. Of each 16 slots the lanes take 0 4 8 12 1 5 ..
  // in turn, and so they lie in LDS: what the lanes' groups g read at once, slots
  // i, i + 4, i + 8, i + 12, is one stretch.
  // (A load of 8 slots is half of a 16's places: i and i + 1 of each four.)
  static __device__ __forceinline__ int v_slot(int place) {
    return KV >= 16 ? (place & ~15) + (place & 3) * 4 + ((place >> 2) & 3)
                    : (place & 3) * 4 + (place >> 2);
  }
  template <int I>
  __device__ __forceinline__ void load_v_from(bool want) {
    constexpr int kFirst = KV >= 16 ? I * KV : I / 2 * 16, kCount = KV >= 16 ? KV : 16;   // slots
    constexpr int kHalf = KV >= 16 ? 0 : (I & 1) * 2;
    // the second half's slots are two further
    const uint32_t more = kHalf == 0 ? 0u : (uint32_t)(2 / HEADS) * st;
    vr[I] = *reinterpret_cast<const u32x4_t*>(
        at<kFirst / HEADS, kCount / HEADS>(a.v_cache, off, st, sh1, v_slot(lane / kPerV) + kHalf,
                                           (uint32_t)(lane % kPerV) * 16, v_in + more, want));
    if constexpr (I + 1 < VL) load_v_from<I + 1>(want);
  }
  __device__ __forceinline__ void load_v(bool want) {
    load_v_from<0>(want);
    load_scales<0>(more.v_blocks, want, vl);
  }
  // The scales of the tile's slots, 4 bytes a lane.
  template <int I>
  __device__ __forceinline__ void load_scales(const uint8_t* blocks, bool want, uint32_t (&w)[SL]) {
    w[I] = *reinterpret_cast<const uint32_t*>(at<I * KS / HEADS, KS / HEADS>(
        blocks, boff, bst, bsh1, lane / kPerB, (uint32_t)(lane % kPerB) * 4, b_in, want));
    if constexpr (I + 1 < SL) load_scales<I + 1>(blocks, want, w);
  }
  // V's tile to LDS, and the scales of the lane's slots back: 16 of its block.
  __device__ __forceinline__ void take_v() {
    uint8_t* const to = vs + 64 * (kRow + kBlocks);
    in_order();                                // after the last tile's reads
#pragma unroll
    for (int i = 0; i < VL; ++i) *reinterpret_cast<u32x4_t*>(vs + i * 1024 + lane * 16) = vr[i];
#pragma unroll
    for (int i = 0; i < SL; ++i)
#pragma unroll
      for (int b = 0; b < 4; ++b)
        to[((lane % kPerB) * 4 + b) * 64 + i * KS + lane / kPerB] = (uint8_t)(vl[i] >> (8 * b));
    in_order();
    const uint32_t* from = reinterpret_cast<const uint32_t*>(to + (n * NV / 16) * 64 + g * 4);
#pragma unroll
    for (int u = 0; u < NU; ++u) vb[u] = from[u * 4];
  }

  // S^T of the loaded tile, times qs the scores
  __device__ __forceinline__ void scores(f32x4_t (&out)[RT][NS]) {
    uint8_t* const to = vs + 64 * kRow;
    in_order();
#pragma unroll
    for (int i = 0; i < SL; ++i) *reinterpret_cast<uint32_t*>(to + i * 256 + lane * 4) = kb[i];
    in_order();
#pragma unroll
    for (int u = 0; u < NU; ++u) {
      f32x4_t S[RT];
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) S[rt] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
      const uint8_t* b = to + (u * 16 + n) * kBlocks + g * (D / 64);
      const uint32_t w = D == 64 ? *b : D == 128 ? *reinterpret_cast<const uint16_t*>(b)
                                                 : *reinterpret_cast<const uint32_t*>(b);
      const f16x2_t s01 = e4m3x2_to_f16<0>(w), s23 = e4m3x2_to_f16<1>(w);
#pragma unroll
      for (int j = 0; j < NJ; ++j) {
        const f16x2_t s = j >> 2 ? s23 : s01;
        const _Float16 one = (j >> 1) & 1 ? s[1] : s[0];
        const u32x4_t kv = scaled8(kr[u][j], f16x2_t{one, one});
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) S[rt] = mma(kv, qf[rt][j], S[rt]);
      }
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) {
        if (MOD) S[rt] *= qs[rt];
        // those of the lane's own head
        if constexpr (HEADS == 1) {
          out[rt][u] = S[rt];
        } else {
          out[rt][u >> 1][(u & 1) * 2] = hl ? S[rt][1] : S[rt][0];
          out[rt][u >> 1][(u & 1) * 2 + 1] = hl ? S[rt][3] : S[rt][2];
        }
      }
    }
  }
  // The running maximum and sum, and P (times 2^kRaise) as the sum of two fp16.
  __device__ __forceinline__ void softmax(const f32x4_t (&S)[RT][NS], Weights& pf) {
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      const float q = MOD ? 1.0f : qs[rt];
      float mx = -INFINITY;
#pragma unroll
      for (int e = 0; e < E; ++e) mx = fmaxf(mx, S[rt][e >> 2][e & 3]);
      mx *= q;
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
      const float m_use = m[rt] == -INFINITY ? 0.0f : kRaise - m[rt];
      float minus = -1.0f;   // not to be seen: one mixed fma takes each half
      asm("" : "+s"(minus));
#pragma unroll
      for (int e = 0; e < E / 2; ++e) {
        const float p0 = __builtin_amdgcn_exp2f(fmaf(S[rt][e >> 1][(e & 1) * 2], q, m_use));
        const float p1 = __builtin_amdgcn_exp2f(fmaf(S[rt][e >> 1][(e & 1) * 2 + 1], q, m_use));
        l[rt] += p0 + p1;
        const f16x2_t hi = __builtin_convertvector((f32x2_t{p0, p1}), f16x2_t);
        // what is left is exact in fp32
        const f16x2_t lo = __builtin_convertvector(
            (f32x2_t{fmaf((float)hi[0], minus, p0), fmaf((float)hi[1], minus, p1)}), f16x2_t);
        put(pf[0][rt], e, bits(hi));
        put(pf[1][rt], e, bits(lo));
      }
    }
  }
  // The weights of the lane's scores 2 e and 2 e + 1 (halves of w) to their slots,
  // with zeros for other heads' slots.
  __device__ __forceinline__ void put(u32x4_t (&p)[NP], int e, uint32_t w) const {
    if constexpr (HEADS == 1) {                // slots as scores
      p[e >> 2][e & 3] = w;
    } else {                                   // a score: half hl of its word
      p[e >> 1][(e & 1) * 2] = hl ? w << 16 : w & 0xFFFFu;
      p[e >> 1][(e & 1) * 2 + 1] = hl ? w & 0xFFFF0000u : w >> 16;
    }
  }
  // O += V^T P^T, the smaller part first
  __device__ __forceinline__ void values(const Weights& pf) {
#pragma unroll
    for (int q = 0; q < NP; ++q) {
      const f16x2_t s[4] = {e4m3x2_to_f16<0>(vb[2 * q]), e4m3x2_to_f16<1>(vb[2 * q]),
                            e4m3x2_to_f16<0>(vb[2 * q + 1]), e4m3x2_to_f16<1>(vb[2 * q + 1])};
      uint32_t x[8][VW];                       // the lane's slots' dims
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const uint8_t* p =
            vs + ((2 * q + (e >> 2)) * 16 + (e & 3) * 4 + g) * kRow + n * (NV / 2);
        if constexpr (NV == 4) {
          x[e][0] = *reinterpret_cast<const uint16_t*>(p);
        } else {
#pragma unroll
          for (int w = 0; w < VW; ++w) x[e][w] = reinterpret_cast<const uint32_t*>(p)[w];
        }
      }
#pragma unroll
      for (int w = 0; w < VW; ++w) {
        uint32_t even[4], odd[4];              // two slots' dims 0 2 4 6, and 1 3 5 7
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t k0 = x[2 * i][w], k1 = x[2 * i + 1][w];
          even[i] = (k0 & 0x0F0F0F0Fu) | ((k1 << 4) & 0xF0F0F0F0u);
          odd[i] = ((k0 >> 4) & 0x0F0F0F0Fu) | (k1 & 0xF0F0F0F0u);
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
    u32x4_t v0, v1;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v0[i] = bits(e2m1x2_to_f16<B>(even[i]) * s[i]);
      v1[i] = bits(e2m1x2_to_f16<B>(odd[i]) * s[i]);
    }
#pragma unroll
    for (int rt = 0; rt < RT; ++rt)
#pragma unroll
      for (int i = kParts - 1; i >= 0; --i) {
        O[rt][t0 + 2 * B] = mma(v0, pf[i][rt][q], O[rt][t0 + 2 * B]);
        O[rt][t0 + 2 * B + 1] = mma(v1, pf[i][rt][q], O[rt][t0 + 2 * B + 1]);
      }
  }

  // the lane's e-th key's slots of V become zero where it is not seen: codes are
  // finite, so their scales do
  __device__ __forceinline__ void keep(int e, bool see) {
    constexpr uint32_t kKey = 0xFFFFFFFFu >> (32 - 8 * HEADS);
    vb[e / PU] &= see ? 0xFFFFFFFFu : ~(kKey << (e % PU * 8 * HEADS));
  }
  // Some scale of V's tile is NaN: a byte whose lower 7 bits are set.
  __device__ __forceinline__ bool any_nan() const {
    uint32_t hit = 0u;
#pragma unroll
    for (int u = 0; u < NU; ++u) hit |= (vb[u] & 0x7F7F7F7Fu) + 0x01010101u;
    return __any((hit & 0x80808080u) != 0u);
  }
  // A key that some rows see and others do not (and, of two heads, the other's
  // rows never) has weight 0 for these, which is enough unless its value is NaN
  // (0 times it would reach them). Such a value becomes zero, and the sum of the
  // rows that see it NaN. weightless: bit e, this lane's row does not see key e.
  __device__ __forceinline__ void settle(const uint32_t (&weightless)[RT]) {
#pragma unroll
    for (int s = 0; s < 16; ++s) {
      const bool bad = ((vb[s >> 2] >> (8 * (s & 3))) & 0x7Fu) == 0x7Fu;   // E4M3's NaN
      if (bad) vb[s >> 2] &= ~(0xFFu << (8 * (s & 3)));
      const bool any = (__ballot(bad) >> (16 * g)) & 0xFFFFu;   // of the slot's 16 lanes
      const int e = (s >> 2) * PU + (s & 3) / HEADS;
#pragma unroll
      for (int rt = 0; rt < RT; ++rt)
        if (any && (s & 3) % HEADS == hl && !((weightless[rt] >> e) & 1u)) l[rt] = __builtin_nanf("");
    }
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

// Row tiles of 16 in one pass; a head with more rows is read again for the others.
// Heads of 256 take one: two spill some 130 VGPRs (8 sequences of 20000 keys, 8
// heads, 20 rows: 163 us against 159).
constexpr int row_tiles(int64_t rows, int64_t D) { return rows <= 16 || D == 256 ? 1 : 2; }

// Heads side by side.
int heads_of(int64_t rows, int64_t Hkv) { return rows <= 8 && Hkv % 2 == 0 ? 2 : 1; }

AttnLayout layout(int64_t rows, int64_t Hkv, int64_t D, int heads) {
  return attn_layout(rows, Hkv, D, row_tiles(rows, D), waves_per_simd((int)D), heads);
}

// Two heads side by side from 2^18 keys of all sequences' heads on (by the
// tables, as the lengths are on the device): a load then takes whole lines of 128
// bytes, where each head's 64 come at half of memory's rate, and half of the
// columns' scores drop out, but a wavefront leaves twice the rows to the join. One
// head against two, 8 heads of 128, G 4, us: 1 sequence of 4096 keys 14.0 / 14.2,
// 8192 15.8 / 17.0; 4 of 8192 21.6 / 21.2; 16 of 4096 28.6 / 27.1, 8192 48.1 /
// 41.9; 16 heads of 64, G 1, 16 of 20000 141 / 97. (Four heads: the long batch of
// 713 MB 136 + 9.1 for the join against 131 + 6.8 with two and 161 + 6 with one.)
// A load's bytes have to be counted in 32 bits.
bool side_by_side(const Attn4Args& a) {
  return a.B * most_keys(a) * a.Hkv >= 1 << 18 && a.sh < 1 << 28 && a.block_sh < 1 << 28;
}

// The whole form takes tables of at most this many keys: two turns of its eight
// wavefronts, or half of one where its workgroups are more than the CUs. Whole
// against split, us, 8 heads of 128, G 4: 1 sequence of 256 keys 7.7 / 12.1, 512 9.6 / 12.2, 1024 12.7 / 12.5; 4: 512 10.0 /
// 12.4, 1024 14.0 / 13.5; 16: 512 12.4 / 14.9, 1024 16.4 / 18.8, 2048 22.9 / 21.8;
// 64: 256 18.6 / 20.2, 512 26.6 / 21.8.
int64_t whole_keys(const Attn4Args& a, int NHV) {
  return a.B * NHV > kCus ? 256 : 1024;
}

template <int D, int RT, bool MOD, int HEADS>
hipError_t launch_run(const Attn4Args& a, const AttnShape& sh, hipStream_t stream) {
  const int64_t whole = HEADS == 1 ? whole_keys(a, sh.NHV) : 0;
  if (HEADS == 1 && a.page % 64 == 0)
    return launch_forms<Attn4Wave<D, RT, HEADS == 1 ? 64 : 16, MOD, HEADS>>(a, sh, whole, stream);
  return a.page % 16 == 0 ? launch_forms<Attn4Wave<D, RT, 16, MOD, HEADS>>(a, sh, whole, stream)
                          : launch_forms<Attn4Wave<D, RT, 0, MOD, HEADS>>(a, sh, whole, stream);
}

template <int D, bool MOD>
hipError_t launch_d(const Attn4Args& a, hipStream_t stream) {
  const int64_t rows = a.Hq / a.Hkv * a.Q;
  // (short tables take the whole form, which has one head a wavefront)
  const bool whole = D < 256 && most_keys(a) <= whole_keys(a, layout(rows, a.Hkv, D, 1).NHV);
  const int heads = !whole && side_by_side(a) ? heads_of(rows, a.Hkv) : 1;
  const AttnLayout L = layout(rows, a.Hkv, D, heads);
  const AttnShape sh = attn_shape(a, L);
  if constexpr (D < 256)
    if (L.RT == 2) return launch_run<D, 2, MOD, 1>(a, sh, stream);
  return heads == 2 ? launch_run<D, 1, MOD, 2>(a, sh, stream)
                    : launch_run<D, 1, MOD, 1>(a, sh, stream);
}

template <bool MOD>
hipError_t launch_scored(const Attn4Args& a, hipStream_t stream) {
  return a.D == 64    ? launch_d<64, MOD>(a, stream)
         : a.D == 128 ? launch_d<128, MOD>(a, stream)
                      : launch_d<256, MOD>(a, stream);
}

}  // namespace

int attn4_row_units(int64_t rows, int64_t Hkv, int64_t D) { return layout(rows, Hkv, D, 1).NHV; }

size_t attn4_workspace_bytes(int64_t rows, int64_t Hkv, int64_t D) {
  const size_t one = layout(rows, Hkv, D, 1).total;
  const size_t more = layout(rows, Hkv, D, heads_of(rows, Hkv)).total;
  return one > more ? one : more;
}

hipError_t launch_paged_attention4(const Attn4Args& a, hipStream_t stream) {
  return scored(a) ? launch_scored<true>(a, stream) : launch_scored<false>(a, stream);
}

}  // namespace nvfp4
