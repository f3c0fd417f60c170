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
// atomics. Where the table's rows are short (kWholeKeys), one workgroup of
// eight wavefronts takes a sequence and head whole and joins them in LDS.
#include <type_traits>

#include "elems.h"
#include "internal.h"

namespace nvfp4 {

namespace {

constexpr int kCus = 256;
constexpr int kWholeWaves = 8;
constexpr int kWholeKeys = 1024;
constexpr float kLog2e = 1.4426950408889634f;
// The reference of the exponentials is moved only when a score passes it by
// more than this (in powers of two): exp2 of at most 2^8 loses nothing in fp32
// or bf16, and most turns need no maximum across lanes and no rescaling.
constexpr float kSlack = 8.0f;
// A run has at least this many tiles: fewer records to join.
constexpr int kMinTiles = 1;

// Keys per tile: 16 KB of K and V at a time.
constexpr int tile_keys(int D, bool FP8) { return D * (FP8 ? 1 : 2) >= 256 ? 32 : 64; }
// Wavefronts per SIMD of the split form.
constexpr int waves_per_simd(int RT, int D) { return 1; }

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

// The tiles (of TK keys) of one sequence: keys base .. len - 1.
struct Span {
  int len, base, n;   // n >= 1: an empty sequence has one tile that writes zeros
};
template <int TK>
__device__ __forceinline__ Span span_of(const AttnArgs& a, const AttnShape& sh, int len) {
  Span s;
  s.len = len < 0 ? 0 : len > sh.cap ? sh.cap : len;
  const int64_t lo = a.window ? (int64_t)s.len - a.Q - a.window + 1 : 0;
  s.base = lo <= 0 ? 0 : (int)lo & ~(TK - 1);
  s.n = s.len > s.base ? (s.len - s.base + TK - 1) / TK : 1;
  return s;
}

__device__ __forceinline__ int wave_sum_i32(int v) {
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) v += __shfl_xor(v, off, 64);
  return __builtin_amdgcn_readfirstlane(v);
}

// Tiles of all sequences, by every wavefront for itself.
template <int TK>
__device__ __forceinline__ int total_tiles(const AttnArgs& a, const AttnShape& sh) {
  const int lane = threadIdx.x & 63, B = (int)a.B;
  int t = 0;
  for (int b = lane; b < B; b += 64) t += span_of<TK>(a, sh, a.lens[b]).n;
  return wave_sum_i32(t);
}
// The sequence that holds tile u, and the tiles before it.
template <int TK>
__device__ __forceinline__ int find_sequence(const AttnArgs& a, const AttnShape& sh, int u,
                                             int& before) {
  const int lane = threadIdx.x & 63, B = (int)a.B;
  int run = 0;
  for (int b0 = 0; b0 < B; b0 += 64) {
    const int n = b0 + lane < B ? span_of<TK>(a, sh, a.lens[b0 + lane]).n : 0;
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
// Run w starts at tile start(w); the first r runs have q + 1 tiles and the
// others q (total = nw * q + r). of(s): the run that has tile s.
struct Runs {
  int nw, q, r;
  __device__ __forceinline__ Runs(int total, int groups) {
    nw = (total + kMinTiles - 1) / kMinTiles;
    nw = nw < groups ? nw : groups;
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
  __device__ __forceinline__ uint32_t get(int d) const {   // dims 2 d, 2 d + 1
    if constexpr (FP8)
      return (d & 1) ? e4m3x2_to_bf16<1>(w[d >> 1]) : e4m3x2_to_bf16<0>(w[d >> 1]);
    else
      return w[d];
  }
};

// The state of one wavefront over the keys of one sequence and head, and its
// passes over tiles.
template <int D, bool FP8, int RT, bool PG, int TK>
struct AttnWave {
  static constexpr int NU = TK / 16;           // runs of 16 keys
  static constexpr int NP = TK / 32;           // products over the keys
  static constexpr int NJ = D / 32;            // products over the dims
  static constexpr int NV = D / 16;            // dims per lane of V
  static constexpr int ES = FP8 ? 1 : 2;
  static constexpr int KL = D * ES / 64;       // 16-byte loads of K per lane and 16 keys
  static constexpr uint64_t kAll = TK == 64 ? ~0ull : (1ull << (TK & 63)) - 1;

  const AttnArgs& a;
  const AttnShape& sh;
  const int lane, n, g;
  const int b, Q, G, row0, rows;
  const Span sp;
  const float c;                               // scale of the scores, log2
  const int64_t head_off;
  const uint32_t stb, k_lane, v_dim, v_lane;
  const const_i32 table;
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
  int ids[PG ? NU : 1], in_page[PG ? NU : 1];
  int64_t off[PG ? NU : 1];
  uint64_t ok;

  __device__ __forceinline__ AttnWave(const AttnArgs& a_, const AttnShape& sh_, int b_, int h,
                                      int row0_, const Span& sp_, float c_)
      : a(a_), sh(sh_), lane(threadIdx.x & 63), n(lane & 15), g(lane >> 4), b(b_), Q((int)a_.Q),
        G(sh_.G), row0(row0_), rows(sh_.rows - row0_ < RT * 16 ? sh_.rows - row0_ : RT * 16),
        sp(sp_), c(c_), head_off((int64_t)h * a_.sh), stb((uint32_t)a_.st * ES),
        k_lane((uint32_t)n * stb + (uint32_t)g * 16),
        v_dim((uint32_t)n * (NV > 8 ? 8 : NV) * ES), v_lane((uint32_t)(g * 4) * stb + v_dim),
        table((const_i32)(uintptr_t)(a_.table + (int64_t)b_ * a_.max_blocks)) {
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      const int r = row0 + rt * 16 + n;
      const bool live = r < sh.rows;
      tok[rt] = live ? r / G : -1;
      const uint16_t* qp = a.q + ((int64_t)(b * (int64_t)Q + (live ? tok[rt] : 0)) * a.Hq + h * G +
                                  (live ? r - tok[rt] * G : 0)) * D;
#pragma unroll
      for (int j = 0; j < NJ; ++j) {
        const int d0 = FP8 ? (j >> 1) * 64 + g * 16 + (j & 1) * 8 : j * 32 + g * 8;
        u32x4_t v = *reinterpret_cast<const u32x4_t*>(qp + d0);
        if (!live) v = u32x4_t{0, 0, 0, 0};
        qf[rt][j] = __builtin_bit_cast(bf16x8_t, v);
      }
#pragma unroll
      for (int t = 0; t < NV; ++t) O[rt][t] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
      m[rt] = -INFINITY;
      l[rt] = 0.0f;
    }
  }

  __device__ __forceinline__ int page_of(int key, int& in) const {
    const int pi = sh.page_shift >= 0 ? key >> sh.page_shift : key / (int)a.page;
    in = key - pi * (int)a.page;
    return pi < (int)a.max_blocks ? pi : (int)a.max_blocks - 1;
  }
  __device__ __forceinline__ void fetch(int key0) {
    if constexpr (PG) {
#pragma unroll
      for (int u = 0; u < NU; ++u) ids[u] = table[page_of(key0 + 16 * u, in_page[u])];
    } else {
      const int pi = page_of(key0 + (lane & (TK - 1)), in_page[0]);
      ids[0] = a.table[(int64_t)b * a.max_blocks + pi];
    }
  }
  __device__ __forceinline__ void resolve() {
    ok = 0;
#pragma unroll
    for (int u = 0; u < (PG ? NU : 1); ++u) {
      const bool fine = (uint32_t)ids[u] < (uint32_t)a.num_blocks;
      off[u] = (int64_t)(fine ? ids[u] : 0) * a.sb + (int64_t)in_page[u] * a.st + head_off;
      if (PG)
        ok |= fine ? 0xFFFFull << (16 * u) : 0ull;
      else
        ok = __ballot(fine) & kAll;
    }
  }
  __device__ __forceinline__ int64_t at_key(int src) const {   // byte offset of lane src's key
    const int lo = __shfl((int)off[0], src, 64);
    const int hi = __shfl((int)(off[0] >> 32), src, 64);
    return (int64_t)(((uint64_t)(uint32_t)hi << 32) | (uint32_t)lo) * ES;
  }
  // lane's key of V, and of S^T and P: i-th of the tile (of TK / 4)
  __device__ __forceinline__ int key_of(int i) const { return (i >> 2) * 16 + g * 4 + (i & 3); }
  __device__ __forceinline__ void load_k() {
    const uint8_t* const kc = (const uint8_t*)a.k_cache;
#pragma unroll
    for (int u = 0; u < NU; ++u) {
      const uint8_t* p = PG ? kc + off[PG ? u : 0] * ES + k_lane : kc + at_key(16 * u + n) + g * 16;
#pragma unroll
      for (int j = 0; j < KL; ++j) kr[u][j] = load_stream(p + j * 64);
    }
  }
  __device__ __forceinline__ void load_v() {
    const uint8_t* const vc = (const uint8_t*)a.v_cache;
#pragma unroll
    for (int i = 0; i < TK / 4; ++i)
      vr[i].load(PG ? vc + off[PG ? i >> 2 : 0] * ES + (uint32_t)(i & 3) * stb + v_lane
                    : vc + at_key(key_of(i)) + v_dim);
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
  // The running maximum and sum, and P as bf16 pairs.
  __device__ __forceinline__ void softmax(const f32x4_t (&S)[RT][NU], uint32_t (&pf)[RT][2 * NU]) {
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
        pf[rt][e] = pack_bf16(p0, p1);
      }
    }
  }
  __device__ __forceinline__ f32x4_t product(u32x4_t v, const uint32_t* pf, f32x4_t acc) const {
    const u32x4_t pv = {pf[0], pf[1], pf[2], pf[3]};
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, v),
                                                   __builtin_bit_cast(bf16x8_t, pv), acc, 0, 0, 0);
  }
  // Keys of pages that do not exist: no weight, and no value.
  __device__ __forceinline__ void hide(uint64_t ok_now, f32x4_t (&S)[RT][NU]) {
#pragma unroll
    for (int i = 0; i < TK / 4; ++i) {
      const bool there = (ok_now >> key_of(i)) & 1u;
#pragma unroll
      for (int rt = 0; rt < RT; ++rt)
        S[rt][i >> 2][i & 3] = there ? S[rt][i >> 2][i & 3] : -INFINITY;
#pragma unroll
      for (int d = 0; d < VRow<NV, FP8>::kDw; ++d) vr[i].w[d] = there ? vr[i].w[d] : 0u;
    }
  }

  // A tile that some row sees only in part.
  __device__ __forceinline__ void masked_tile(int key0) {
    fetch(key0);
    resolve();
    load_k();
    load_v();
    f32x4_t S[RT][NU];
    uint32_t pf[RT][2 * NU];
    scores(S);
    if (ok != kAll) hide(ok, S);
    const int pos0 = sp.len - Q;
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      const int hi = tok[rt] < 0 ? -1 : pos0 + tok[rt];
      const int64_t lo = a.window ? (int64_t)hi - a.window + 1 : 0;
#pragma unroll
      for (int e = 0; e < 4 * NU; ++e) {
        const int key = key0 + key_of(e);
        if (key > hi || key < lo) S[rt][e >> 2][e & 3] = -INFINITY;
      }
    }
    softmax(S, pf);
    // A value that no row sees, or that another token sees, may be anything
    // (0 * inf would reach every row): one product per token, on the values
    // that it sees, kept by that token's rows.
    const int t0 = row0 / G, t1 = (row0 + rows - 1) / G;
    for (int i0 = t0; i0 <= t1; ++i0) {
      const int hi_key = pos0 + i0;
      const int64_t lo_key = a.window ? (int64_t)hi_key - a.window + 1 : 0;
#pragma unroll
      for (int d = 0; d < NV / 2; ++d) {
#pragma unroll
        for (int q = 0; q < NP; ++q) {
          uint32_t x[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int key = key0 + key_of(q * 8 + i);
            x[i] = key <= hi_key && key >= lo_key ? vr[q * 8 + i].get(d) : 0u;
          }
          const u32x4_t lo = {perm_lo(x[0], x[1]), perm_lo(x[2], x[3]), perm_lo(x[4], x[5]),
                              perm_lo(x[6], x[7])};
          const u32x4_t hi = {perm_hi(x[0], x[1]), perm_hi(x[2], x[3]), perm_hi(x[4], x[5]),
                              perm_hi(x[6], x[7])};
#pragma unroll
          for (int rt = 0; rt < RT; ++rt) {
            const f32x4_t o0 = product(lo, &pf[rt][4 * q], O[rt][2 * d]);
            const f32x4_t o1 = product(hi, &pf[rt][4 * q], O[rt][2 * d + 1]);
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
  }
  // A tile that every row sees, loaded already. MORE: the one `ahead` keys on
  // is loaded meanwhile (K while the values are multiplied, V while the next
  // scores are). MORE is a constant, so that the loads in flight are the same
  // on every path to a wait: a branch around them would drain them all.
  template <bool MORE>
  __device__ __forceinline__ void full_tile(int key0, int ahead) {
    f32x4_t S[RT][NU];
    uint32_t pf[RT][2 * NU];
    scores(S);
    const uint64_t ok_now = ok;
    if (MORE) {
      resolve();
      load_k();
      fetch(key0 + 2 * ahead);
    }
    if (ok_now != kAll) hide(ok_now, S);
    softmax(S, pf);
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
        for (int rt = 0; rt < RT; ++rt) {
          O[rt][2 * d] = product(lo, &pf[rt][4 * q], O[rt][2 * d]);
          O[rt][2 * d + 1] = product(hi, &pf[rt][4 * q], O[rt][2 * d + 1]);
        }
      }
    }
    if (MORE) load_v();
  }

  // The tiles at key0, key0 + stride, .. below key_end. Those that some row
  // sees only in part lie before full_lo and past full_hi.
  __device__ __forceinline__ void pass(int key0, int key_end, int stride) {
    const int64_t full_lo = a.window ? (int64_t)sp.len - a.window : 0;
    const int full_hi = sp.len - Q;
    const int full_end = full_hi + 1 - TK < key_end - 1 ? full_hi + 1 - TK : key_end - 1;
    for (int part = 0; part < 2; ++part) {
      const int stop = part || full_lo >= key_end ? key_end : (int)full_lo;
      for (; key0 < stop; key0 += stride) masked_tile(key0);
      if (part || key0 > full_end) continue;
      fetch(key0);
      resolve();
      load_k();
      load_v();
      fetch(key0 + stride);
      for (; key0 + stride <= full_end; key0 += stride) full_tile<true>(key0, stride);
      full_tile<false>(key0, stride);
      key0 += stride;
    }
    // the sums over the four lane groups of a row (their maxima are the same)
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      l[rt] += __shfl_xor(l[rt], 16, 64);
      l[rt] += __shfl_xor(l[rt], 32, 64);
    }
  }

  // O^T row g * 4 + i of the products is dims (g * 4 + i) * 8 .. + 7 (heads of
  // 64: * 4 .. + 3; of 256: products 8 .. 15 are the second half). f(rt, d0,
  // v): 4 consecutive dims of row rt * 16 + n.
  template <typename F>
  __device__ __forceinline__ void each4(F f) const {
    constexpr int kRun = NV > 8 ? 8 : NV;
#pragma unroll
    for (int rt = 0; rt < RT; ++rt)
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int t = 0; t < NV; t += 4)
          f(rt, (t / kRun) * 128 + (g * 4 + i) * kRun + t % kRun,
            f32x4_t{O[rt][t][i], O[rt][t + 1][i], O[rt][t + 2][i], O[rt][t + 3][i]});
  }
};

__device__ __forceinline__ void store4(uint16_t* p, f32x4_t v) {
  *reinterpret_cast<u32x2_t*>(p) = u32x2_t{pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3])};
}

// The split form: a wavefront per (run, head).
template <int D, bool FP8, int RT, bool PG>
__global__ __launch_bounds__(256, waves_per_simd(RT, D)) void k_attn_runs(const AttnArgs a,
                                                                          const AttnShape sh) {
  constexpr int TK = tile_keys(D, FP8);
  const int total = total_tiles<TK>(a, sh);
  const Runs runs(total, sh.groups);
  const int unit = blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int w = unit / sh.NHV, hv = unit - w * sh.NHV;
  if (w >= runs.nw) return;
  const int rt_tile = hv / (int)a.Hkv, h = hv - rt_tile * (int)a.Hkv;
  int s = runs.start(w);
  const int s_end = runs.start(w + 1);
  int before;
  int b = find_sequence<TK>(a, sh, s, before);
  int s_in = s - before;
  const const_i32 lens = (const_i32)(uintptr_t)a.lens;
  const float ks = FP8 ? *a.k_scale : 1.0f, vs = FP8 ? *a.v_scale : 1.0f;
  for (bool first = true; s < s_end; first = false, ++b, s_in = 0) {
    const Span sp = span_of<TK>(a, sh, lens[b]);
    const int e_in = sp.n - s_in < s_end - s ? sp.n : s_in + (s_end - s);
    AttnWave<D, FP8, RT, PG, TK> wave(a, sh, b, h, rt_tile * (RT * 16), sp, a.scale * ks * kLog2e);
    const int end = sp.base + e_in * TK;
    wave.pass(sp.base + s_in * TK, end < sp.len ? end : sp.len, TK);
    const bool whole = s_in == 0 && e_in == sp.n;
    const int64_t rec = ((int64_t)(w * sh.NHV + hv) * 2 + (first ? 0 : 1)) * sh.slot_rows;
    float f[RT];
    uint16_t* out[RT];
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      f[rt] = wave.l[rt] == 0.0f ? 0.0f : vs / wave.l[rt];
      const int r = wave.row0 + rt * 16 + wave.n;
      out[rt] = a.out + ((int64_t)(b * a.Q + wave.tok[rt]) * a.Hq + h * sh.G +
                         (r - wave.tok[rt] * sh.G)) * D;
      if (!whole && wave.tok[rt] >= 0 && wave.g == 0) {
        sh.ml[(rec + rt * 16 + wave.n) * 2] = wave.m[rt];
        sh.ml[(rec + rt * 16 + wave.n) * 2 + 1] = wave.l[rt];
      }
    }
    wave.each4([&](int rt, int d, f32x4_t v) {
      if (wave.tok[rt] < 0) return;
      if (whole)
        store4(out[rt] + d, v * f[rt]);
      else
        *reinterpret_cast<f32x4_t*>(sh.o + (rec + rt * 16 + wave.n) * D + d) = v;
    });
    s += e_in - s_in;
  }
}

// The whole form: a workgroup per (sequence, head); its wavefronts take the
// tiles in turn and meet in LDS.
template <int D, bool FP8, int RT, bool PG>
__global__ __launch_bounds__(kWholeWaves * 64, 2) void k_attn_whole(const AttnArgs a,
                                                                    const AttnShape sh) {
  constexpr int TK = 32;
  __shared__ float lds_o[kWholeWaves][RT * 16][D + 4];
  __shared__ float lds_ml[kWholeWaves][RT * 16][2];
  const int b = blockIdx.x / sh.NHV, hv = blockIdx.x - b * sh.NHV;
  const int rt_tile = hv / (int)a.Hkv, h = hv - rt_tile * (int)a.Hkv;
  const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const float ks = FP8 ? *a.k_scale : 1.0f, vs = FP8 ? *a.v_scale : 1.0f;
  const const_i32 lens = (const_i32)(uintptr_t)a.lens;
  const Span sp = span_of<TK>(a, sh, lens[b]);
  AttnWave<D, FP8, RT, PG, TK> wave(a, sh, b, h, rt_tile * (RT * 16), sp, a.scale * ks * kLog2e);
  wave.pass(sp.base + wv * TK, sp.len, kWholeWaves * TK);
#pragma unroll
  for (int rt = 0; rt < RT; ++rt)
    if (wave.g == 0) {
      lds_ml[wv][rt * 16 + wave.n][0] = wave.m[rt];
      lds_ml[wv][rt * 16 + wave.n][1] = wave.l[rt];
    }
  wave.each4([&](int rt, int d, f32x4_t v) {
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
// share: groups of D / 4 threads take its partial records in turn,
// then meet in LDS.
template <int D, int TK>
__global__ __launch_bounds__(256) void k_attn_join(const AttnArgs a, const AttnShape sh) {
  constexpr int TD = D / 4, NG = 256 / TD;
  __shared__ float lds[NG][D + 4];
  __shared__ float lds_ml[NG][2];
  const int b = blockIdx.x / sh.NHV, hv = blockIdx.x % sh.NHV, r = blockIdx.y;
  const int rt_tile = hv / (int)a.Hkv, h = hv - rt_tile * (int)a.Hkv;
  const int rr = rt_tile * sh.slot_rows + r;
  if (rr >= sh.rows) return;
  const int lane = threadIdx.x & 63;
  // steps before this sequence, and all of them
  int bef = 0, tot = 0;
  for (int i = lane; i < (int)a.B; i += 64) {
    const int n = span_of<TK>(a, sh, a.lens[i]).n;
    tot += n;
    bef += i < b ? n : 0;
  }
  const int total = wave_sum_i32(tot), s0 = wave_sum_i32(bef);
  const int nb = span_of<TK>(a, sh, a.lens[b]).n;
  const Runs runs(total, sh.groups);
  const int w0 = runs.of(s0), w1 = runs.of(s0 + nb - 1);
  if (w0 == w1) return;   // finished by its one wavefront
  const int grp = threadIdx.x / TD, d0 = (threadIdx.x % TD) * 4;
  float m = -INFINITY, l = 0.0f;
  f32x4_t o = {0.0f, 0.0f, 0.0f, 0.0f};
  for (int w = w0 + grp; w <= w1; w += NG) {
    // a run that starts inside this sequence, or with it, has it as its first
    // part
    const int64_t slot = ((int64_t)w * sh.NHV + hv) * 2 + (w > w0 || runs.start(w) == s0 ? 0 : 1);
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

// Row tiles of 16 in one pass (heads of 256 keep one: their registers are
// full); a head with more rows is read again for the others.
int row_tiles(int64_t rows, int64_t D) { return rows <= 16 || D == 256 ? 1 : 2; }

// The most runs per head (all heads' together fill the SIMDs), and where their
// records lie in the workspace.
struct AttnLayout {
  size_t ml, o, total;
  int RT, slot_rows, NHV, groups;
};
AttnLayout attn_layout(int64_t rows, int64_t Hkv, int64_t D) {
  AttnLayout L;
  L.RT = row_tiles(rows, D);
  L.NHV = (int)(Hkv * ((rows + L.RT * 16 - 1) / (L.RT * 16)));
  L.slot_rows = (int)(rows < L.RT * 16 ? rows : L.RT * 16);
  L.groups = kCus * 4 * waves_per_simd(L.RT, (int)D) / L.NHV;
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
  return (int)(cap < 0x7FFFFF00 ? cap : 0x7FFFFF00);
}
// Keys that a sequence reads at most: by its table row, or by its window
// (which starts at most a tile early).
int64_t most_keys(const AttnArgs& a) {
  const int64_t keys = capacity(a);
  return a.window && a.window + a.Q + 64 < keys ? a.window + a.Q + 64 : keys;
}

template <int D, bool FP8, int RT, bool PG>
hipError_t launch_rt(const AttnArgs& a, AttnShape& sh, const AttnLayout& L, hipStream_t stream) {
  constexpr int TK = tile_keys(D, FP8);
  constexpr bool kFits = (size_t)kWholeWaves * RT * 16 * (D + 6) * 4 <= 160 * 1024;
  const int64_t keys = most_keys(a);
  if constexpr (kFits) {
    if (keys <= kWholeKeys) {
      hipLaunchKernelGGL((k_attn_whole<D, FP8, RT, PG>), dim3((uint32_t)(a.B * sh.NHV)),
                         dim3(kWholeWaves * 64), 0, stream, a, sh);
      return hipGetLastError();
    }
  }
  const int64_t most = (keys + TK - 1) / TK * a.B;
  sh.groups = (int)(most < a.B ? a.B : most < L.groups ? most : L.groups);
  if (sh.groups > L.groups) sh.groups = L.groups;
  const int64_t units = (int64_t)sh.groups * sh.NHV;
  hipLaunchKernelGGL((k_attn_runs<D, FP8, RT, PG>), dim3((uint32_t)((units + 3) / 4)), dim3(256),
                     0, stream, a, sh);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || keys <= TK) return e;   // a sequence of one tile is never shared
  hipLaunchKernelGGL((k_attn_join<D, TK>),
                     dim3((uint32_t)(a.B * sh.NHV), (uint32_t)sh.slot_rows), dim3(256), 0, stream,
                     a, sh);
  return hipGetLastError();
}

template <int D, bool FP8>
hipError_t launch_d(const AttnArgs& a, hipStream_t stream) {
  AttnShape sh;
  sh.G = (int)(a.Hq / a.Hkv);
  sh.rows = sh.G * (int)a.Q;
  const AttnLayout L = attn_layout(sh.rows, a.Hkv, D);
  sh.NHV = L.NHV;
  sh.cap = capacity(a);
  sh.page_shift = (a.page & (a.page - 1)) == 0 ? __builtin_ctzll((uint64_t)a.page) : -1;
  sh.slot_rows = L.slot_rows;
  sh.ml = (float*)((char*)a.workspace + L.ml);
  sh.o = (float*)((char*)a.workspace + L.o);
  const bool pg = a.page % 16 == 0;
  if constexpr (D != 256) {
    if (L.RT == 2)
      return pg ? launch_rt<D, FP8, 2, true>(a, sh, L, stream)
                : launch_rt<D, FP8, 2, false>(a, sh, L, stream);
  }
  return pg ? launch_rt<D, FP8, 1, true>(a, sh, L, stream)
            : launch_rt<D, FP8, 1, false>(a, sh, L, stream);
}

}  // namespace

bool attn_fits(const AttnArgs& a) { return (most_keys(a) + 31) / 32 * a.B < 0x7FFFFFFF; }

size_t attn_workspace_bytes(int64_t B, int64_t Q, int64_t Hq, int64_t Hkv, int64_t D) {
  if (B == 0 || Q == 0) return 0;
  return attn_layout(Hq / Hkv * Q, Hkv, D).total;
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
