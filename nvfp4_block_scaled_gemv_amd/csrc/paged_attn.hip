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
#include "elems.h"
#include "attn_span.h"
#include "internal.h"

namespace nvfp4 {

namespace {

constexpr int kCus = 256;
constexpr int kWholeWaves = 8;   // wavefronts per workgroup of the whole form
constexpr float kLog2e = 1.4426950408889634f;
// The reference of the exponentials is moved only when a score passes it by
// more than this (in powers of two): exp2 of at most 2^8 loses nothing in fp32
// or bf16, and most turns need no maximum across lanes and no rescaling.
constexpr float kSlack = 8.0f;
// s_waitcnt vmcnt(0), no other counter.
constexpr int kVmcnt0 = 0x0F70;
// Wavefronts per SIMD of the split form. Few long streams read memory best:
// heads of 256 bytes and more keep 16 KB and more in flight per wavefront with
// one; smaller heads need two.
constexpr int waves_per_simd(int RT, int D, bool FP8) {
  return RT == 1 && D * (FP8 ? 1 : 2) < 256 ? 2 : 1;
}
// Runs of one head at most: all its wavefronts on the chip, where there is but
// one head (attn_layout).
constexpr int kMaxRuns = kCus * 4 * 2;
static_assert(waves_per_simd(1, 64, true) * kCus * 4 <= kMaxRuns, "the join's weights");

struct AttnShape {
  int rows;        // G * Q
  int G;
  int NHV;         // heads as the wavefronts see them: Hkv * row tiles
  int groups;      // runs
  int page_shift;  // log2(page), or -1
  int cap;         // keys that a row of the table can name
  int slot_rows;   // rows of one partial record
  float* ml;       // [slots][slot_rows][2]
  float* o;        // [slots][slot_rows][D]
};

typedef const __attribute__((address_space(4))) int32_t* const_i32;

__device__ __forceinline__ Span span_of(const AttnArgs& a, const AttnShape& sh, int len) {
  return nvfp4::span_of(len, sh.cap, a.Q, a.window);
}

// Inclusive sums over the 64 lanes, by DPP: within rows of 16, then from each
// row's last lane to the rows after it.
__device__ __forceinline__ int scan64(int v) {
  v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xF, 0xF, true);   // row_shr:1
  v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xF, 0xF, true);   // row_shr:2
  v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xF, 0xF, true);   // row_shr:4
  v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xF, 0xF, true);   // row_shr:8
  v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xA, 0xF, true);   // row_bcast:15
  v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xC, 0xF, true);   // row_bcast:31
  return v;
}

// The tiles of all sequences, by every wavefront for itself (all 64 lanes).
struct Tiles {
  const AttnArgs& a;
  const AttnShape& sh;
  const int lane;
  int len, n, incl;   // of sequence `lane`, and the tiles up to it (of the first 64)
  int total;
  __device__ __forceinline__ Tiles(const AttnArgs& a_, const AttnShape& sh_)
      : a(a_), sh(sh_), lane(threadIdx.x & 63) {
    len = lane < (int)a.B ? a.lens[lane] : 0;
    n = lane < (int)a.B ? span_of(a, sh, len).n : 0;
    incl = scan64(n);
    total = __builtin_amdgcn_readlane(incl, 63);
    for (int b0 = 64; b0 < (int)a.B; b0 += 64) {
      const int b = b0 + lane;
      const int m = b < (int)a.B ? span_of(a, sh, a.lens[b]).n : 0;
      total += __builtin_amdgcn_readlane(scan64(m), 63);
    }
  }
  // The sequence that holds tile u, its length, and the tiles before it.
  __device__ __forceinline__ int find(int u, int& before, int& its_len) const {
    int run = 0, len_l = len, n_l = n, incl_l = incl;
    for (int b0 = 0;;) {
      const uint64_t past = __ballot(run + incl_l > u);
      if (past) {
        const int l = __builtin_ctzll(past);
        before = run + __builtin_amdgcn_readlane(incl_l - n_l, l);
        its_len = __builtin_amdgcn_readlane(len_l, l);
        return b0 + l;
      }
      run += __builtin_amdgcn_readlane(incl_l, 63);
      b0 += 64;
      if (b0 >= (int)a.B) break;   // not reached for u below the total
      len_l = b0 + lane < (int)a.B ? a.lens[b0 + lane] : 0;
      n_l = b0 + lane < (int)a.B ? span_of(a, sh, len_l).n : 0;
      incl_l = scan64(n_l);
    }
    before = its_len = 0;
    return 0;
  }
  // The tiles before sequence b.
  __device__ __forceinline__ int before(int b) const {
    int run = 0, n_l = n, incl_l = incl;
    for (int b0 = 0; b - b0 >= 64;) {
      run += __builtin_amdgcn_readlane(incl_l, 63);
      b0 += 64;
      n_l = b0 + lane < (int)a.B ? span_of(a, sh, a.lens[b0 + lane]).n : 0;
      incl_l = scan64(n_l);
    }
    return run + __builtin_amdgcn_readlane(incl_l - n_l, b & 63);
  }
};
// Run w starts at tile start(w); the first r runs have q + 1 tiles and the
// others q (nw * q + r in all). of(s): the run that has tile s.
struct Runs {
  int nw, q, r;
  __device__ __forceinline__ Runs(int total, int groups) {
    nw = total < groups ? total : groups;
    q = total / nw;
    r = total % nw;
  }
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

// A tile of a wavefront's run.
struct Cursor {
  int b, len;   // its sequence
  int key;      // its first key
  int left;     // tiles of the sequence from it on
};

// One wavefront's pass over tiles of one head.
template <int D, bool FP8, int RT, bool PG>
struct AttnWave {
  static constexpr int NU = TK / 16;           // runs of 16 keys
  static constexpr int NP = TK / 32;           // products over the keys
  static constexpr int NJ = D / 32;            // products over the dims
  static constexpr int NV = D / 16;            // dims per lane of V
  static constexpr int ES = FP8 ? 1 : 2;
  static constexpr int KL = D * ES / 64;       // 16-byte loads of K per lane and 16 keys
  static constexpr int NO = PG ? NU : 1;
  static constexpr uint32_t kAll = 0xFFFFFFFFu;
  static constexpr int kParts = 3;             // bf16 numbers that hold a probability

  const AttnArgs& a;
  const AttnShape& sh;
  const int lane, n, g;
  const int h, Q, G, row0, rows;
  const float c;                               // scale of the scores, log2
  const int64_t head_off;
  const uint32_t stb, k_lane, v_dim, v_lane;
  const const_i32 lens;
  int len_after;                               // of the sequence after the last cursor's
  bf16x8_t qf[RT][NJ];
  int tok[RT];
  f32x4_t O[RT][NV];
  float m[RT], l[RT];
  u32x4_t kr[NU][KL];
  VRow<NV, FP8> vr[TK / 4];
  // Where a tile's keys lie. fetch() reads the page numbers, a tile ahead of
  // resolve(), which turns them into offsets: PG, runs of 16 keys inside one
  // page each (uniform); otherwise one offset per lane, for key lane % TK. ok:
  // bit per key, its page exists (page 0 is read in its place).
  int ids[NO], in_page[NO];
  int64_t off[NO];
  uint32_t ok;

  __device__ __forceinline__ AttnWave(const AttnArgs& a_, const AttnShape& sh_, int h_, int row0_,
                                      float c_)
      : a(a_), sh(sh_), lane(threadIdx.x & 63), n(lane & 15), g(lane >> 4), h(h_), Q((int)a_.Q),
        G(sh_.G), row0(row0_), rows(sh_.rows - row0_ < RT * 16 ? sh_.rows - row0_ : RT * 16),
        c(c_), head_off((int64_t)h_ * a_.sh), stb((uint32_t)a_.st * ES),
        k_lane((uint32_t)n * stb + (uint32_t)g * 16),
        v_dim((uint32_t)n * (NV > 8 ? 8 : NV) * ES), v_lane((uint32_t)(g * 4) * stb + v_dim),
        lens((const_i32)(uintptr_t)a_.lens) {
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      const int r = row0 + rt * 16 + n;
      tok[rt] = r < sh.rows ? r / G : -1;
    }
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
      const uint16_t* qp = a.q + ((int64_t)(b * (int64_t)Q + (live ? tok[rt] : 0)) * a.Hq + h * G +
                                  (live ? r - tok[rt] * G : 0)) * D;
#pragma unroll
      for (int j = 0; j < NJ; ++j) {
        const int d0 = FP8 ? (j >> 1) * 64 + g * 16 + (j & 1) * 8 : j * 32 + g * 8;
        // rows that do not exist read another's: nothing of them is written
        qf[rt][j] = *reinterpret_cast<const bf16x8_t*>(qp + d0);
      }
    }
  }
  __device__ __forceinline__ Cursor first_of(int b, int len, int idx) {
    const Span s = span_of(a, sh, len);
    len_after = lens[b + 1 < (int)a.B ? b + 1 : b];
    return Cursor{b, s.len, s.base + idx * TK, s.n - idx};
  }
  // The tile `step` further in c's sequence, or the next one's first (past the
  // last sequence: any tile, it is not computed).
  __device__ __forceinline__ Cursor after(const Cursor& c, int step) {
    if (c.left <= step && c.b + 1 < (int)a.B) return first_of(c.b + 1, len_after, 0);
    return Cursor{c.b, c.len, tile_after(c.key, step), c.left - step};
  }

  __device__ __forceinline__ int page_of(int key, int ahead, int& in) const {
    return nvfp4::page_of(key, ahead, (int)a.page, sh.page_shift, (int)a.max_blocks, in);
  }
  // Only for tiles that hold a key: an empty sequence's table has no row.
  __device__ __forceinline__ void fetch(const Cursor& c) {
    if constexpr (PG) {
      const const_i32 table = (const_i32)(uintptr_t)(a.table + (int64_t)c.b * a.max_blocks);
#pragma unroll
      for (int u = 0; u < NU; ++u) ids[u] = table[page_of(c.key, 16 * u, in_page[u])];
    } else {
      const int pi = page_of(c.key, lane & (TK - 1), in_page[0]);
      ids[0] = a.table[(int64_t)c.b * a.max_blocks + pi];
    }
  }
  __device__ __forceinline__ void resolve() {
    ok = 0;
#pragma unroll
    for (int u = 0; u < NO; ++u) {
      const bool fine = (uint32_t)ids[u] < (uint32_t)a.num_blocks;
      off[u] = (int64_t)(fine ? ids[u] : 0) * a.sb + (int64_t)in_page[u] * a.st + head_off;
      if (PG)
        ok |= fine ? 0xFFFFu << (16 * u) : 0u;
      else
        ok = (uint32_t)__ballot(fine);
    }
  }
  // byte offset of lane src's key
  __device__ __forceinline__ int64_t at_key(const int64_t (&off)[NO], int src) const {
    const int lo = __shfl((int)off[0], src, 64);
    const int hi = __shfl((int)(off[0] >> 32), src, 64);
    return (int64_t)(((uint64_t)(uint32_t)hi << 32) | (uint32_t)lo) * ES;
  }
  // lane's key of V, and of S^T and P: i-th of the tile (of TK / 4)
  __device__ __forceinline__ int key_of(int i) const { return (i >> 2) * 16 + g * 4 + (i & 3); }
  // want: false where no tile follows. The loads are issued all the same, all
  // lanes from one address: a branch around them would make the waits on both
  // sides drain everything in flight.
  __device__ __forceinline__ void load_k(bool want) {
    const uint8_t* const kc = (const uint8_t*)a.k_cache;
    const uint32_t lane_off = want ? k_lane : 0u;
#pragma unroll
    for (int u = 0; u < NU; ++u) {
      const uint8_t* p = PG ? kc + off[PG ? u : 0] * ES + lane_off
                            : want ? kc + at_key(off, 16 * u + n) + g * 16 : kc;
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
#pragma unroll
    for (int i = 0; i < TK / 4; ++i)
      vr[i].load(PG ? vc + off[PG ? i >> 2 : 0] * ES + (uint32_t)(i & 3) * st + lane_off
                    : want ? vc + at_key(off, key_of(i)) + v_dim : vc);
  }

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
  __device__ __forceinline__ void softmax(const f32x4_t (&S)[RT][NU],
                                          u32x4_t (&pf)[kParts][RT][NP]) {
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
  __device__ __forceinline__ void values(const u32x4_t (&pf)[kParts][RT][NP]) {
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

  // Values that no row sees may be anything: they become zero.
  __device__ __forceinline__ void drop(const Cursor& cur, uint32_t ok_now, int t0, int t1) {
    const int last = cur.len - Q + t1;
    const int64_t firsts = a.window ? (int64_t)cur.len - Q + t0 - a.window + 1 : 0;
#pragma unroll
    for (int i = 0; i < TK / 4; ++i) {
      const int key = cur.key + key_of(i);
      const bool see = key <= last && key >= firsts && ((ok_now >> key_of(i)) & 1u);
#pragma unroll
      for (int d = 0; d < VRow<NV, FP8>::kDw; ++d) vr[i].w[d] = see ? vr[i].w[d] : 0u;
    }
  }
  // A key that some rows see and others do not has weight 0 for these, which is
  // enough unless its value is infinite or NaN (0 * inf would reach them). Such
  // a value becomes zero, and the sum of the rows that see it NaN. weightless:
  // bit i, this lane's row does not see key i.
  __device__ __forceinline__ void settle(const uint32_t (&weightless)[RT]) {
#pragma unroll
    for (int i = 0; i < TK / 4; ++i) {
      const bool bad = vr[i].not_finite();
#pragma unroll
      for (int d = 0; d < VRow<NV, FP8>::kDw; ++d) vr[i].w[d] = bad ? 0u : vr[i].w[d];
      const bool any = (__ballot(bad) >> (16 * g)) & 0xFFFFu;   // of the key's 16 lanes
#pragma unroll
      for (int rt = 0; rt < RT; ++rt)
        if (any && !((weightless[rt] >> i) & 1u)) l[rt] = __builtin_nanf("");
    }
  }

  // `count` (>= 1) tiles from cur on, `step` apart. While a tile is computed
  // the next one is loaded (K while the values are multiplied, V while the
  // next scores are), also across sequences. finish(cursor) where a
  // sequence or the run ends, with O, m and l (summed over a row's lanes) of
  // the tiles since the last one. One body for every kind of tile: code that
  // runs once is paid for in instruction fetches.
  template <typename F>
  __device__ __forceinline__ void pass(Cursor cur, int count, int step, F finish) {
    load_q(cur.b);
    fetch(cur);
    resolve();
    load_k(true);
    load_v(true);
    Cursor nxt = after(cur, step);
    fetch(nxt);
    const int t0 = row0 / G, t1 = (row0 + rows - 1) / G;   // the rows' tokens
    for (;;) {
      const bool more = --count > 0;
      f32x4_t S[RT][NU];
      u32x4_t pf[kParts][RT][NP];
      scores(S);
      const uint32_t ok_now = ok;
      resolve();
      load_k(more);
      const Cursor nxt2 = after(nxt, step);
      fetch(nxt2);
      // every row sees the whole tile
      const int pos0 = cur.len - Q;
      const bool all = ok_now == kAll && cur.key + TK - 1 <= pos0 &&
                       (!a.window || cur.key >= (int64_t)cur.len - a.window);
      uint32_t weightless[RT];
      if (!all) {
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) {
          const int hi = tok[rt] < 0 ? -1 : pos0 + tok[rt];
          const int64_t lo = a.window ? (int64_t)hi - a.window + 1 : 0;
          weightless[rt] = 0u;
#pragma unroll
          for (int e = 0; e < 4 * NU; ++e) {
            const int key = cur.key + key_of(e);
            if (key > hi || key < lo || !((ok_now >> key_of(e)) & 1u)) {
              S[rt][e >> 2][e & 3] = -INFINITY;
              weightless[rt] |= 1u << e;
            }
          }
        }
      }
      softmax(S, pf);
      if (!all) {
        drop(cur, ok_now, t0, t1);
        if (t1 > t0) settle(weightless);
      }
      values(pf);
      load_v(more);
      if (!more || nxt.b != cur.b) {
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) {   // a row's four lanes (their maxima are the same)
          l[rt] += __shfl_xor(l[rt], 16, 64);
          l[rt] += __shfl_xor(l[rt], 32, 64);
        }
        finish(cur);
        if (!more) break;
        clear();
        load_q(nxt.b);
        // here, on the rare path: otherwise every tile would wait for queries
        // that may be in flight, and with them for its successor
        __builtin_amdgcn_s_waitcnt(kVmcnt0);
      }
      cur = nxt;
      nxt = nxt2;
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

__device__ __forceinline__ void store4(uint16_t* p, f32x4_t v) {
  *reinterpret_cast<u32x2_t*>(p) = u32x2_t{pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3])};
}

// The split form: a wavefront per (run, head).
template <int D, bool FP8, int RT, bool PG>
__global__ __launch_bounds__(256, waves_per_simd(RT, D, FP8)) void k_attn_runs(const AttnArgs a,
                                                                          const AttnShape sh) {
  const Tiles tiles(a, sh);
  const Runs runs(tiles.total, sh.groups);
  const int unit = blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int w = unit / sh.NHV, hv = unit - w * sh.NHV;
  if (w >= runs.nw) return;
  const int rt_tile = hv / (int)a.Hkv, h = hv - rt_tile * (int)a.Hkv;
  const int s = runs.start(w), count = runs.start(w + 1) - s;
  int before, len;
  const int b = tiles.find(s, before, len);
  const float ks = FP8 ? *a.k_scale : 1.0f, vs = FP8 ? *a.v_scale : 1.0f;
  AttnWave<D, FP8, RT, PG> wave(a, sh, h, rt_tile * (RT * 16), a.scale * ks * kLog2e);
  bool from_start = s == before;
  int64_t rec = (int64_t)(w * sh.NHV + hv) * 2 * sh.slot_rows;
  wave.pass(wave.first_of(b, len, s - before), count, 1, [&](const Cursor& c) {
    const bool whole = from_start && c.left == 1;
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      if (wave.tok[rt] < 0) continue;
      const int r = rt * 16 + wave.n;
      if (whole) {
        const float f = wave.l[rt] == 0.0f ? 0.0f : vs / wave.l[rt];
        uint16_t* o = a.out + ((int64_t)(c.b * a.Q + wave.tok[rt]) * a.Hq + h * sh.G +
                               (wave.row0 + r - wave.tok[rt] * sh.G)) * D;
        wave.each4(rt, [&](int d, f32x4_t v) { store4(o + d, v * f); });
      } else {
        if (wave.g == 0) {
          sh.ml[(rec + r) * 2] = wave.m[rt];
          sh.ml[(rec + r) * 2 + 1] = wave.l[rt];
        }
        float* o = sh.o + (rec + r) * D;
        wave.each4(rt, [&](int d, f32x4_t v) { *reinterpret_cast<f32x4_t*>(o + d) = v; });
      }
    }
    // only a run's first and last parts can be records
    rec = ((int64_t)(w * sh.NHV + hv) * 2 + 1) * sh.slot_rows;
    from_start = true;
  });
}

// The whole form: a workgroup per (sequence, head); its wavefronts take the
// tiles in turn and meet in LDS.
template <int D, bool FP8, int RT, bool PG>
__global__ __launch_bounds__(kWholeWaves * 64, 2) void k_attn_whole(const AttnArgs a,
                                                                    const AttnShape sh) {
  __shared__ float lds_o[kWholeWaves][RT * 16][D + 4];
  __shared__ float lds_ml[kWholeWaves][RT * 16][2];
  const int b = blockIdx.x / sh.NHV, hv = blockIdx.x - b * sh.NHV;
  const int rt_tile = hv / (int)a.Hkv, h = hv - rt_tile * (int)a.Hkv;
  const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const float ks = FP8 ? *a.k_scale : 1.0f, vs = FP8 ? *a.v_scale : 1.0f;
  const int len = ((const_i32)(uintptr_t)a.lens)[b];
  AttnWave<D, FP8, RT, PG> wave(a, sh, h, rt_tile * (RT * 16), a.scale * ks * kLog2e);
  const int count = (span_of(a, sh, len).n - wv + kWholeWaves - 1) / kWholeWaves;
  if (count > 0) wave.pass(wave.first_of(b, len, wv), count, kWholeWaves, [](const Cursor&) {});
#pragma unroll
  for (int rt = 0; rt < RT; ++rt)
    if (wave.g == 0) {
      lds_ml[wv][rt * 16 + wave.n][0] = wave.m[rt];
      lds_ml[wv][rt * 16 + wave.n][1] = wave.l[rt];
    }
#pragma unroll
  for (int rt = 0; rt < RT; ++rt)
    wave.each4(rt, [&](int d, f32x4_t v) {
      *reinterpret_cast<f32x4_t*>(&lds_o[wv][rt * 16 + wave.n][d]) = v;
    });
  __syncthreads();
  for (int it = threadIdx.x; it < wave.rows * (D / 8); it += kWholeWaves * 64) {
    const int r = it / (D / 8), d0 = (it % (D / 8)) * 8;
    float mm = -INFINITY;
#pragma unroll
    for (int v = 0; v < kWholeWaves; ++v) mm = fmaxf(mm, lds_ml[v][r][0]);
    const float m_use = mm == -INFINITY ? 0.0f : mm;
    float ll = 0.0f, o[8] = {0, 0, 0, 0, 0, 0, 0, 0};
#pragma unroll
    for (int v = 0; v < kWholeWaves; ++v) {
      const float f = __builtin_amdgcn_exp2f(lds_ml[v][r][0] - m_use);
      ll = fmaf(lds_ml[v][r][1], f, ll);
#pragma unroll
      for (int e = 0; e < 8; ++e) o[e] = fmaf(lds_o[v][r][d0 + e], f, o[e]);
    }
    const float f = ll == 0.0f ? 0.0f : vs / ll;
#pragma unroll
    for (int e = 0; e < 8; ++e) o[e] *= f;
    const int rr = wave.row0 + r, t = rr / sh.G;
    store8(a.out + ((int64_t)(b * a.Q + t) * a.Hq + h * sh.G + (rr - t * sh.G)) * D + d0, o);
  }
}

// One workgroup per (sequence, head, row) of a sequence that several runs
// share: the records' weights first, then groups of D / 4 threads add the
// records in turn and meet in LDS.
template <int D>
__global__ __launch_bounds__(256) void k_attn_join(const AttnArgs a, const AttnShape sh) {
  constexpr int TD = D / 4, NG = 256 / TD;
  __shared__ float lds[NG][D + 4];
  __shared__ float lds_f[kMaxRuns];
  __shared__ float lds_red[2][4];
  const int b = blockIdx.x / sh.NHV, hv = blockIdx.x % sh.NHV, r = blockIdx.y;
  const int rt_tile = hv / (int)a.Hkv, h = hv - rt_tile * (int)a.Hkv;
  const int rr = rt_tile * sh.slot_rows + r;
  if (rr >= sh.rows) return;
  const Tiles tiles(a, sh);
  const Runs runs(tiles.total, sh.groups);
  const int s0 = tiles.before(b), nb = span_of(a, sh, a.lens[b]).n;
  const int lane = threadIdx.x & 63;
  const int w0 = runs.of(s0), w1 = runs.of(s0 + nb - 1);
  if (w0 == w1) return;   // finished by its one wavefront
  // a run that starts inside this sequence, or with it, has it as its first
  // part
  const int odd = runs.start(w0) == s0 ? 0 : 1;
  auto record = [&](int i) {
    return (((int64_t)(w0 + i) * sh.NHV + hv) * 2 + (i == 0 ? odd : 0)) * sh.slot_rows + r;
  };
  const int np = w1 - w0 + 1, wv = threadIdx.x >> 6;
  // the first records' values are on their way while the weights are made
  constexpr int kEarly = 8;
  const int grp = threadIdx.x / TD, d0 = (threadIdx.x % TD) * 4;
  f32x4_t early[kEarly];
#pragma unroll
  for (int k = 0; k < kEarly; ++k)
    if (grp + k * NG < np)
      early[k] = *reinterpret_cast<const f32x4_t*>(sh.o + record(grp + k * NG) * D + d0);
  // the records' weights against their largest maximum, and the sum
  float mx = -INFINITY;
  for (int i = threadIdx.x; i < np; i += 256) {
    const float m = sh.ml[record(i) * 2];
    lds_f[i] = m;
    mx = fmaxf(mx, m);
  }
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) mx = fmaxf(mx, __shfl_xor(mx, o, 64));
  if (lane == 0) lds_red[0][wv] = mx;
  __syncthreads();
  mx = fmaxf(fmaxf(lds_red[0][0], lds_red[0][1]), fmaxf(lds_red[0][2], lds_red[0][3]));
  const float use = mx == -INFINITY ? 0.0f : mx;
  float l = 0.0f;
  for (int i = threadIdx.x; i < np; i += 256) {
    const float f = __builtin_amdgcn_exp2f(lds_f[i] - use);
    lds_f[i] = f;
    l = fmaf(sh.ml[record(i) * 2 + 1], f, l);
  }
  l = wave_sum(l);
  if (lane == 0) lds_red[1][wv] = l;
  __syncthreads();
  l = (lds_red[1][0] + lds_red[1][1]) + (lds_red[1][2] + lds_red[1][3]);
  f32x4_t o = {0.0f, 0.0f, 0.0f, 0.0f};
  auto add = [&](f32x4_t ow, float f) {
#pragma unroll
    for (int e = 0; e < 4; ++e) o[e] = fmaf(ow[e], f, o[e]);
  };
#pragma unroll
  for (int k = 0; k < kEarly; ++k)
    if (grp + k * NG < np) add(early[k], lds_f[grp + k * NG]);
#pragma unroll 8
  for (int i = grp + kEarly * NG; i < np; i += NG)
    add(*reinterpret_cast<const f32x4_t*>(sh.o + record(i) * D + d0), lds_f[i]);
  *reinterpret_cast<f32x4_t*>(&lds[grp][d0]) = o;
  __syncthreads();
  if (threadIdx.x >= D / 8) return;
  const int d = threadIdx.x * 8;
  const float f = l == 0.0f ? 0.0f : (a.cache_e4m3 ? *a.v_scale : 1.0f) / l;
  float out[8] = {0, 0, 0, 0, 0, 0, 0, 0};
#pragma unroll
  for (int v = 0; v < NG; ++v)
#pragma unroll
    for (int e = 0; e < 8; ++e) out[e] += lds[v][d + e];
#pragma unroll
  for (int e = 0; e < 8; ++e) out[e] *= f;
  const int t = rr / sh.G;
  store8(a.out + ((int64_t)(b * a.Q + t) * a.Hq + h * sh.G + (rr - t * sh.G)) * D + d, out);
}

// Row tiles of 16 in one pass; a head with more rows is read again for the
// others. One against two, 8 sequences, bf16: 20000 keys, 8 heads of 128 with 20
// rows 210 / 114 us, 8192 keys with 64 rows 186 / 103, with 256 rows 557 / 336 (the
// row tiles of a head are neighbouring wavefronts, but their loads carry the
// streaming hint all the same). Heads of 256 take two where pages hold whole
// runs of 16 keys (pg): 20000 keys, 8 heads with 20 rows 387 / 241, 2 heads with 32
// rows 112 / 102, though the bf16 form spills 45 VGPRs. Without, one offset per
// lane and key spills more than it saves (40 rows, pages of 20: 108 / 163 us).
int row_tiles(int64_t rows, int64_t D, bool pg) { return rows <= 16 || (D == 256 && !pg) ? 1 : 2; }

// The most runs per head (all heads' together fill the SIMDs), and where their
// records lie in the workspace.
struct AttnLayout {
  size_t ml, o, total;
  int RT, slot_rows, NHV, groups;
};
AttnLayout attn_layout(int64_t rows, int64_t Hkv, int64_t D, bool e4m3, bool pg) {
  AttnLayout L;
  L.RT = row_tiles(rows, D, pg);
  L.NHV = (int)(Hkv * ((rows + L.RT * 16 - 1) / (L.RT * 16)));
  L.slot_rows = (int)(rows < L.RT * 16 ? rows : L.RT * 16);
  L.groups = kCus * 4 * waves_per_simd(L.RT, (int)D, e4m3) / L.NHV;
  if (L.groups < 1) L.groups = 1;
  const size_t slots = (size_t)2 * L.groups * L.NHV;
  L.ml = 0;
  L.o = (slots * L.slot_rows * 2 * sizeof(float) + 255) & ~(size_t)255;
  L.total = (L.o + slots * L.slot_rows * (size_t)D * sizeof(float) + 255) & ~(size_t)255;
  return L;
}

// Keys that a row of the table can name (none where there is no page).
int capacity(const AttnArgs& a) {
  const int64_t cap = a.num_blocks ? a.max_blocks * a.page : 0;
  return (int)(cap < 0x7FFFFFFF ? cap : 0x7FFFFFFF);
}
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
// Keys that a sequence reads at most: by its table row, or by its window
// (which starts at most a tile early).
int64_t most_keys(const AttnArgs& a) {
  const int64_t keys = capacity(a);
  return a.window && a.window + a.Q + 64 < keys ? a.window + a.Q + 64 : keys;
}

template <int D, bool FP8, int RT, bool PG>
hipError_t launch_rt(const AttnArgs& a, AttnShape& sh, const AttnLayout& L, hipStream_t stream) {
  const int64_t keys = most_keys(a);
  // no page at all: every sequence is empty
  if (sh.cap == 0)
    return launch_fill_zero((float*)a.out, (size_t)(a.B * a.Q * a.Hq * D / 2), stream);
  // Heads of 256 have no whole form: eight wavefronts leave 256 registers each,
  // which two row tiles of 128 fill already (4 to 53 VGPRs spill in three of the
  // four; their times are in whole_keys).
  if constexpr (D < 256) {
    if (keys <= whole_keys(a, sh)) {
      hipLaunchKernelGGL((k_attn_whole<D, FP8, RT, PG>), dim3((uint32_t)(a.B * sh.NHV)),
                         dim3(kWholeWaves * 64), 0, stream, a, sh);
      return hipGetLastError();
    }
  }
  const int64_t most = (keys + TK - 1) / TK * a.B;   // tiles
  sh.groups = (int)(most < L.groups ? most : L.groups);
  const int64_t units = (int64_t)sh.groups * sh.NHV;
  hipLaunchKernelGGL((k_attn_runs<D, FP8, RT, PG>), dim3((uint32_t)((units + 3) / 4)), dim3(256),
                     0, stream, a, sh);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || keys <= TK) return e;   // a sequence of one tile is never shared
  hipLaunchKernelGGL((k_attn_join<D>),
                     dim3((uint32_t)(a.B * sh.NHV), (uint32_t)sh.slot_rows), dim3(256), 0, stream,
                     a, sh);
  return hipGetLastError();
}

template <int D, bool FP8>
hipError_t launch_d(const AttnArgs& a, hipStream_t stream) {
  AttnShape sh;
  sh.G = (int)(a.Hq / a.Hkv);
  sh.rows = sh.G * (int)a.Q;
  const bool pg = a.page % 16 == 0;
  const AttnLayout L = attn_layout(sh.rows, a.Hkv, D, FP8, pg);
  sh.NHV = L.NHV;
  sh.cap = capacity(a);
  sh.page_shift = (a.page & (a.page - 1)) == 0 ? __builtin_ctzll((uint64_t)a.page) : -1;
  sh.slot_rows = L.slot_rows;
  sh.ml = (float*)((char*)a.workspace + L.ml);
  sh.o = (float*)((char*)a.workspace + L.o);
  if (L.RT == 2) {
    if (pg) return launch_rt<D, FP8, 2, true>(a, sh, L, stream);
    if constexpr (D < 256) return launch_rt<D, FP8, 2, false>(a, sh, L, stream);
  }
  return pg ? launch_rt<D, FP8, 1, true>(a, sh, L, stream)
            : launch_rt<D, FP8, 1, false>(a, sh, L, stream);
}

}  // namespace

bool attn_fits(const AttnArgs& a) {
  const AttnLayout L = attn_layout(a.Hq / a.Hkv * a.Q, a.Hkv, a.D, a.cache_e4m3, a.page % 16 == 0);
  // tiles are numbered in 31 bits, a launch's work-items in 32
  return (most_keys(a) + TK - 1) / TK * a.B < 0x7FFFFFFF && a.B * L.NHV <= 1 << 22;
}

size_t attn_workspace_bytes(int64_t B, int64_t Q, int64_t Hq, int64_t Hkv, int64_t D) {
  if (B == 0 || Q == 0) return 0;
  // the call's cache type and page are not known here: the largest of all
  size_t most = 0;
  for (int i = 0; i < 4; ++i) {
    const size_t n = attn_layout(Hq / Hkv * Q, Hkv, D, i & 1, i & 2).total;
    most = n > most ? n : most;
  }
  return most;
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
