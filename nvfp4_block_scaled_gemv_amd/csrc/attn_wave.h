// attn_wave.h -- what attention over a paged cache shares whatever its cache is
// held in: the split of the work, a wavefront's pass over tiles of keys, the
// scores' cap and bias, the two forms' kernels and the join of partial sums.
// The caches' own parts (paged_attn.hip: bf16 and E4M3, paged_attn4.hip: NVFP4)
// are classes derived from AttnPass.
#pragma once

#include <type_traits>

#include "elems.h"
#include "attn_cap.h"
#include "attn_span.h"
#include "internal.h"

namespace nvfp4 {

namespace {

constexpr int kCus = 256;
constexpr int kWholeWaves = 8;   // wavefronts per workgroup of the whole form
constexpr float kLog2e = 1.4426950408889634f;
// s_waitcnt vmcnt(0), no other counter.
constexpr int kVmcnt0 = 0x0F70;
// Runs of one head at most: all its wavefronts on the chip, where there is but
// one head (the layouts).
constexpr int kMaxRuns = kCus * 4 * 2;

struct AttnShape {
  int rows;        // G * Q
  int G;
  int NHV;         // heads as the wavefronts see them: Hkv / side by side * row tiles
  int groups;      // runs
  int page_shift;  // log2(page), or -1
  int cap;         // keys that a row of the table can name
  int slot_rows;   // rows of one partial record
  int by_seq;      // records of runs' last parts: by a sequence, not by the run (part_at)
  float* ml;       // [slots][slot_rows][2]
  float* o;        // [slots][slot_rows][D]
};

static_assert(sizeof(AttnArgs) + sizeof(AttnShape) <= 256, "four lines of arguments");

typedef const __attribute__((address_space(4))) int32_t* const_i32;

template <int TILE>
__device__ __forceinline__ Span span_of(const AttnCommon& a, const AttnShape& sh, int len) {
  return nvfp4::span_of<TILE>(len, sh.cap, a.Q, a.window);
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
template <int TILE>   // keys per tile
struct Tiles {
  const AttnCommon& a;
  const AttnShape& sh;
  const int lane;
  int len, n, incl;   // of sequence `lane`, and the tiles up to it (of the first 64)
  int total;
  __device__ __forceinline__ Tiles(const AttnCommon& a_, const AttnShape& sh_)
      : a(a_), sh(sh_), lane(threadIdx.x & 63) {
    len = lane < (int)a.B ? a.lens[lane] : 0;
    n = lane < (int)a.B ? span_of<TILE>(a, sh, len).n : 0;
    incl = scan64(n);
    total = __builtin_amdgcn_readlane(incl, 63);
    for (int b0 = 64; b0 < (int)a.B; b0 += 64) {
      const int b = b0 + lane;
      const int m = b < (int)a.B ? span_of<TILE>(a, sh, a.lens[b]).n : 0;
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
      n_l = b0 + lane < (int)a.B ? span_of<TILE>(a, sh, len_l).n : 0;
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
      n_l = b0 + lane < (int)a.B ? span_of<TILE>(a, sh, a.lens[b0 + lane]).n : 0;
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

struct CapOps {
  static __device__ __forceinline__ float rcp(float x) { return __builtin_amdgcn_rcpf(x); }
  static __device__ __forceinline__ float exp2(float x) { return __builtin_amdgcn_exp2f(x); }
};

// LDS is written and read by the lanes of one wavefront, in order: the compiler
// has to keep that order across lanes too.
__device__ __forceinline__ void in_order() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// A tile of a wavefront's run.
struct Cursor {
  int b, len;   // its sequence
  int key;      // its first key
  int left;     // tiles of the sequence from it on
};

// The slopes of a lane's rows, log2: none where scores are neither capped nor biased.
template <int RT, bool MOD>
struct Slopes {
  float slope[RT];
};
template <int RT>
struct Slopes<RT, false> {};

// A wavefront's pass over tiles of one head, for a class W derived from it that
// holds K and V of a tile of TILE keys and the sums O; RT tiles of 16 rows share
// it. Score e (of TILE / 4) of a lane is row rt * 16 + n and key W::key_of(e, g)
// of the tile. RUN: pages hold whole runs of that many keys (0: they do not).
// HEADS: key-value heads from h on that the wavefront takes side by side (2, where
// their rows fit): the 16 columns of a tile of rows are then HEADS blocks.
// MOD: the scores are capped or biased. W::kStage: bytes of LDS that a wavefront
// takes V through (0: none), in W::take_v().
template <class W, int TILE, int RT, int RUN, bool MOD, int HEADS = 1, int NU_ = TILE / 16>
struct AttnPass : Slopes<RT, MOD> {
  static_assert(HEADS == 1 || RT == 1, "heads side by side: one tile of rows");
  static constexpr int kTile = TILE;
  static constexpr int kHeads = HEADS;
  static constexpr int kCols = 16 / HEADS;     // columns per head
  static constexpr int kRT = RT;
  static constexpr int NU = NU_;               // a lane's scores: words of four
  static constexpr int NO = RUN ? TILE / RUN : 1;
  typedef typename std::conditional<TILE == 64, uint64_t, uint32_t>::type Mask;   // bit per key
  static constexpr Mask kAll = ~(Mask)0;

  const AttnCommon& a;
  const AttnShape& sh;
  const const_i32 lens;
  const int lane, n, g;
  const int h, Q, G, row0, rows;
  const int hl, col;                           // the lane's head from h on, and its row there
  const float c;                               // scale of the scores, log2
  const int64_t head_off;                      // of head h in the cache
  // What changes, after all that does not, and the slopes only where there are any:
  // the order of the members decides how the compiler spends the registers. With
  // the slopes always there and c among these, plain attention with two row tiles
  // took 3 to 10 % longer (8 heads of 128, 20 rows, 64 sequences of 900 keys 66.6 us
  // / 73.3; E4M3 heads of 64, 8 of 8192 36.0 / 38.5).
  int len_after;                               // of the sequence after the last cursor's
  int tok[RT];
  float m[RT], l[RT];
  // Where a tile's keys lie. fetch() reads the page numbers, a tile ahead of
  // resolve(), which turns them into places: of runs of keys inside one page
  // each (uniform), or one per lane, for key lane % TILE. ok: bit per key, its
  // page exists (page 0 is read in its place).
  int ids[NO], in_page[NO];
  Mask ok;

  __device__ __forceinline__ W& self() { return *static_cast<W*>(this); }
  __device__ __forceinline__ AttnPass(const AttnCommon& a_, const AttnShape& sh_, int h_, int row0_,
                                      float k_scale)
      : a(a_), sh(sh_), lens((const_i32)(uintptr_t)a_.lens), lane(threadIdx.x & 63),
        n(lane & 15), g(lane >> 4), h(h_), Q((int)a_.Q), G(sh_.G), row0(row0_),
        rows(sh_.rows - row0_ < RT * 16 ? sh_.rows - row0_ : RT * 16),
        hl(HEADS == 1 ? 0 : n / kCols), col(HEADS == 1 ? n : n % kCols),
        c(a_.scale * k_scale * kLog2e),
        head_off((int64_t)h_ * a_.sh) {
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      const int r = row0 + rt * 16 + col;
      tok[rt] = r < sh.rows ? r / G : -1;
      if constexpr (MOD)
        this->slope[rt] = a.slopes && tok[rt] >= 0
                              ? a.slopes[(h + hl) * G + r - tok[rt] * G] * kLog2e : 0.0f;
    }
  }
  __device__ __forceinline__ Cursor first_of(int b, int len, int idx) {
    const Span s = span_of<TILE>(a, sh, len);
    len_after = lens[b + 1 < (int)a.B ? b + 1 : b];
    return Cursor{b, s.len, s.base + idx * TILE, s.n - idx};
  }
  // The tile `step` further in c's sequence, or the next one's first (past the
  // last sequence: any tile, it is not computed).
  __device__ __forceinline__ Cursor after(const Cursor& c, int step) {
    if (c.left <= step && c.b + 1 < (int)a.B) return first_of(c.b + 1, len_after, 0);
    return Cursor{c.b, c.len, tile_after<TILE>(c.key, step), c.left - step};
  }

  __device__ __forceinline__ int page_of(int key, int ahead, int& in) const {
    return nvfp4::page_of(key, ahead, (int)a.page, sh.page_shift, (int)a.max_blocks, in);
  }
  // Only for tiles that hold a key: an empty sequence's table has no row.
  __device__ __forceinline__ void fetch(const Cursor& c) {
    if constexpr (RUN != 0) {
      const const_i32 table = (const_i32)(uintptr_t)(a.table + (int64_t)c.b * a.max_blocks);
#pragma unroll
      for (int u = 0; u < NO; ++u) ids[u] = table[page_of(c.key, RUN * u, in_page[u])];
    } else {
      const int pi = page_of(c.key, lane & (TILE - 1), in_page[0]);
      ids[0] = a.table[(int64_t)c.b * a.max_blocks + pi];
    }
  }
  __device__ __forceinline__ void resolve() {
    ok = 0;
#pragma unroll
    for (int u = 0; u < NO; ++u) {
      const bool fine = (uint32_t)ids[u] < (uint32_t)a.num_blocks;
      self().place(u, fine ? ids[u] : 0, in_page[u]);
      if (RUN != 0)
        ok |= fine ? (kAll >> (TILE - (RUN ? RUN : TILE))) << (RUN * u) : (Mask)0;
      else
        ok = (Mask)__ballot(fine);
    }
  }
  // lane src's 64 bits
  __device__ __forceinline__ int64_t from_lane(int64_t v, int src) const {
    const int lo = __shfl((int)v, src, 64);
    const int hi = __shfl((int)(v >> 32), src, 64);
    return (int64_t)(((uint64_t)(uint32_t)hi << 32) | (uint32_t)lo);
  }

  // The scores' cap, z -> cap tanh(z / cap), and the bias slope * (key - the row's
  // position). bf16, 8 sequences of two tokens, window 4096: 24.3 us without either,
  // 24.5 capped, 24.3 biased, 24.8 both; NVFP4, 713 MB: 144, 157, 153 and 164 (in one
  // run).
  __device__ __forceinline__ void modify(f32x4_t (&S)[RT][NU], const Cursor& cur) {
    if (a.cap > 0.0f) {
      // Two row tiles over NVFP4 have no lane's register left for it (8 heads of 128, 20
      // rows, pages of 20, 32773 keys: 66.3 us, 62.5 from the arguments), the other
      // caches no scalar one (E4M3 heads of 64, 8 sequences of 8192 keys: 50.7 us from
      // the arguments, 46.6).
      const float inv = W::kCapInv ? a.cap_inv : CapOps::rcp(a.cap);
      float top = 0.0f;
#pragma unroll
      for (int rt = 0; rt < RT; ++rt)
#pragma unroll
        for (int e = 0; e < 4 * NU; ++e) top = fmaxf(top, fabsf(S[rt][e >> 2][e & 3]));
      // most tiles of scores that a cap of tens is meant for hold none far out
      const bool far = __any(top * inv > kCapNear);
#pragma unroll
      for (int rt = 0; rt < RT; ++rt)
#pragma unroll
        for (int e = 0; e < 4 * NU; ++e) {
          const float z = S[rt][e >> 2][e & 3];
          S[rt][e >> 2][e & 3] = far ? capped<CapOps>(z, a.cap, inv) : capped_near<CapOps>(z, inv);
        }
    }
    if (a.slopes) {
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) {
        const int from = cur.key - (cur.len - Q + tok[rt]);
#pragma unroll
        for (int e = 0; e < 4 * NU; ++e)
          S[rt][e >> 2][e & 3] =
              fmaf(this->slope[rt], (float)(from + W::key_of(e, g)), S[rt][e >> 2][e & 3]);
      }
    }
  }

  // Values that no row sees may be anything: they become zero.
  __device__ __forceinline__ void drop(const Cursor& cur, Mask ok_now, int t0, int t1) {
    const int last = cur.len - Q + t1;
    const int64_t firsts = a.window ? (int64_t)cur.len - Q + t0 - a.window + 1 : 0;
#pragma unroll
    for (int e = 0; e < 4 * NU; ++e) {
      const int key = cur.key + W::key_of(e, g);
      self().keep(e, key <= last && key >= firsts && ((ok_now >> W::key_of(e, g)) & 1u));
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
    W& w = self();
    w.load_q(cur.b);
    fetch(cur);
    resolve();
    w.load_k(true);
    w.load_v(true);
    Cursor nxt = after(cur, step);
    fetch(nxt);
    const int t0 = row0 / G, t1 = (row0 + rows - 1) / G;   // the rows' tokens
    for (;;) {
      const bool more = --count > 0;
      f32x4_t S[RT][NU];
      typename W::Weights pf;
      w.scores(S);
      const Mask ok_now = ok;
      resolve();
      w.load_k(more);
      const Cursor nxt2 = after(nxt, step);
      fetch(nxt2);
      if constexpr (MOD) modify(S, cur);
      // every row sees the whole tile
      const int pos0 = cur.len - Q;
      const bool all = ok_now == kAll && cur.key + TILE - 1 <= pos0 &&
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
            const int key = cur.key + W::key_of(e, g);
            if (key > hi || key < lo || !((ok_now >> W::key_of(e, g)) & 1u)) {
              S[rt][e >> 2][e & 3] = -INFINITY;
              weightless[rt] |= 1u << e;
            }
          }
        }
      }
      // all of a lane's scores may be of another head than its row's
      if constexpr (W::kOthers) {
        const bool other = (g & 1) != hl;
#pragma unroll
        for (int rt = 0; rt < RT; ++rt)
#pragma unroll
          for (int e = 0; e < 4 * NU; ++e)
            S[rt][e >> 2][e & 3] = other ? -INFINITY : S[rt][e >> 2][e & 3];
      }
      w.softmax(S, pf);
      w.take_v();
      if (W::kStage) w.load_v(more);   // V is in LDS: its registers are free
      if (!all) {
        drop(cur, ok_now, t0, t1);
        if (HEADS == 1 && t1 > t0) w.settle(weightless);
      }
      // heads side by side: another head's values have weight 0 for a row, always
      if constexpr (HEADS > 1) {
        if (w.any_nan()) {
#pragma unroll
          for (int rt = 0; rt < RT; ++rt) {
            weightless[rt] = all ? 0u : weightless[rt];
            if (W::kOthers && (g & 1) != hl) weightless[rt] = ~0u;
          }
          w.settle(weightless);
        }
      }
      w.values(pf);
      if (!W::kStage) w.load_v(more);
      if (!more || nxt.b != cur.b) {
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) {   // a row's four lanes (their maxima are the same)
          l[rt] += __shfl_xor(l[rt], 16, 64);
          l[rt] += __shfl_xor(l[rt], 32, 64);
        }
        finish(cur);
        if (!more) break;
        w.clear();
        w.load_q(nxt.b);
        // here, on the rare path: otherwise every tile would wait for queries
        // that may be in flight, and with them for its successor
        __builtin_amdgcn_s_waitcnt(kVmcnt0);
      }
      cur = nxt;
      nxt = nxt2;
    }
  }
};

__device__ __forceinline__ void store4(uint16_t* p, f32x4_t v) {
  *reinterpret_cast<u32x2_t*>(p) = u32x2_t{pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3])};
}

// Workgroups go to the 8 XCDs in turn; of n the b-th becomes one of n / 8
// neighbours on its XCD.
__device__ __forceinline__ int on_one_xcd(int b, int n) {
  const int x = b & 7, q = n >> 3, r = n & 7;
  return x * q + (x < r ? x : r) + (b >> 3);
}

// Run w's partial record of head hv: of its first part, or of its last. Two a run;
// heads side by side have the last parts apart, as these may be counted by the
// sequence b of the run's first tile (attn_layout): a run with a last part ends in a
// later one, where the next run begins, so that no two such runs have the same.
template <int HEADS>
__device__ __forceinline__ int64_t part_at(const AttnShape& sh, int w, int hv, int last, int b) {
  if (HEADS == 1) return (int64_t)(w * sh.NHV + hv) * 2 + last;
  return (!last ? w : sh.groups + (sh.by_seq ? b : w)) * sh.NHV + hv;
}

// The split form: a wavefront per (run, head).
template <class Wave>
__global__ __launch_bounds__(256, Wave::kPerSimd) void k_attn_runs(const typename Wave::Args a,
                                                                   const AttnShape sh) {
  constexpr int D = Wave::kD, RT = Wave::kRT;
  __shared__ __align__(16) uint8_t stage[4][Wave::kStage ? Wave::kStage : 16];
  const Tiles<Wave::kTile> tiles(a, sh);
  const Runs runs(tiles.total, sh.groups);
  const int block = Wave::kStage ? on_one_xcd(blockIdx.x, gridDim.x) : (int)blockIdx.x;
  const int unit = block * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int w = unit / sh.NHV, hv = unit - w * sh.NHV;
  if (w >= runs.nw) return;
  const int all_heads = (int)a.Hkv / Wave::kHeads;
  const int rt_tile = hv / all_heads, h = (hv - rt_tile * all_heads) * Wave::kHeads;
  const int s = runs.start(w), count = runs.start(w + 1) - s;
  int before, len;
  const int b = tiles.find(s, before, len);
  const float ks = Wave::kScaled ? *a.k_scale : 1.0f, vs = Wave::kScaled ? *a.v_scale : 1.0f;
  Wave wave(a, sh, h, rt_tile * (RT * 16), ks, stage[threadIdx.x >> 6]);
  bool from_start = s == before;
  int64_t rec = part_at<Wave::kHeads>(sh, w, hv, 0, b) * sh.slot_rows;
  wave.pass(wave.first_of(b, len, s - before), count, 1, [&](const Cursor& c) {
    const bool whole = from_start && c.left == 1;
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      if (wave.tok[rt] < 0) continue;
      const int row = rt * 16 + wave.col, r = Wave::kHeads == 1 ? row : wave.hl * sh.rows + row;
      if (whole) {
        const float f = wave.l[rt] == 0.0f ? 0.0f : vs / wave.l[rt];
        uint16_t* o = a.out + ((int64_t)(c.b * a.Q + wave.tok[rt]) * a.Hq +
                               (h + wave.hl) * sh.G +
                               (wave.row0 + row - wave.tok[rt] * sh.G)) * D;
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
    rec = part_at<Wave::kHeads>(sh, w, hv, 1, b) * sh.slot_rows;
    from_start = true;
  });
}

// The whole form: a workgroup per (sequence, head); its wavefronts take the
// tiles in turn and meet in LDS.
template <class Wave>
__global__ __launch_bounds__(kWholeWaves * 64, 2) void k_attn_whole(const typename Wave::Args a,
                                                                    const AttnShape sh) {
  constexpr int D = Wave::kD, RT = Wave::kRT;
  // a wavefront's sums, and before them the LDS of its pass
  __shared__ __align__(16) float lds_o[kWholeWaves][RT * 16][D + 4];
  static_assert(Wave::kStage <= (int)sizeof(lds_o[0]), "the pass's LDS");
  __shared__ float lds_ml[kWholeWaves][RT * 16][2];
  const int b = blockIdx.x / sh.NHV, hv = blockIdx.x - b * sh.NHV;
  const int rt_tile = hv / (int)a.Hkv, h = hv - rt_tile * (int)a.Hkv;
  const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const float ks = Wave::kScaled ? *a.k_scale : 1.0f, vs = Wave::kScaled ? *a.v_scale : 1.0f;
  const int len = ((const_i32)(uintptr_t)a.lens)[b];
  Wave wave(a, sh, h, rt_tile * (RT * 16), ks, (uint8_t*)lds_o[wv]);
  const int count = (span_of<Wave::kTile>(a, sh, len).n - wv + kWholeWaves - 1) / kWholeWaves;
  if (count > 0) wave.pass(wave.first_of(b, len, wv), count, kWholeWaves, [](const Cursor&) {});
  if (Wave::kStage) in_order();
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
template <int D, int TILE, int HEADS, class Args>
__global__ __launch_bounds__(256) void k_attn_join(const Args a, const AttnShape sh) {
  constexpr int TD = D / 4, NG = 256 / TD;
  __shared__ float lds[NG][D + 4];
  __shared__ float lds_f[kMaxRuns];
  __shared__ float lds_red[2][4];
  const int b = blockIdx.x / sh.NHV, hv = blockIdx.x % sh.NHV, r = blockIdx.y;
  const int all_heads = (int)a.Hkv / HEADS;
  const int rt_tile = hv / all_heads, hl = HEADS == 1 ? 0 : r / sh.rows;
  const int h = (hv - rt_tile * all_heads) * HEADS + hl;
  const int rr = rt_tile * sh.slot_rows + r - hl * sh.rows;
  if (rr >= sh.rows) return;
  const Tiles<TILE> tiles(a, sh);
  const Runs runs(tiles.total, sh.groups);
  const int s0 = tiles.before(b), nb = span_of<TILE>(a, sh, a.lens[b]).n;
  const int lane = threadIdx.x & 63;
  const int w0 = runs.of(s0), w1 = runs.of(s0 + nb - 1);
  if (w0 == w1) return;   // finished by its one wavefront
  // a run that starts inside this sequence, or with it, has it as its first
  // part
  const int odd = runs.start(w0) == s0 ? 0 : 1;
  int before, len, b0 = 0;
  if (HEADS > 1 && odd && sh.by_seq) b0 = tiles.find(runs.start(w0), before, len);
  auto record = [&](int i) {
    const int last = i == 0 ? odd : 0;   // (one head: by lane, wider numbers at once)
    if (HEADS == 1) return (((int64_t)(w0 + i) * sh.NHV + hv) * 2 + last) * sh.slot_rows + r;
    return part_at<HEADS>(sh, w0 + i, hv, last, b0) * sh.slot_rows + r;
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
  const float f = l == 0.0f ? 0.0f : (a.v_scale ? *a.v_scale : 1.0f) / l;
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

// The most runs per head (all heads' together fill the SIMDs with `per_simd`
// wavefronts), and where their records lie in the workspace: two a run. One pair of
// heads side by side has as many runs as two heads have by themselves, of twice the
// rows: its records are one a run and one a sequence, in what the two heads need (or
// two of half the runs, where the sequences are more). B sequences cost B of 2048
// runs (heads of 256: 1024). Against two records a run, us: NVFP4, heads of 64, pages
// of 16, 48 sequences of 17 to 16384 keys the same, 64 of 8192 each, which 2048 runs
// divide evenly, 31.7 / 29.5; heads of 256, 64 of 4000 to 8200 56.9 / 54.8.
struct AttnLayout {
  size_t ml, o, total;
  int RT, slot_rows, NHV, groups;
  bool one;        // a record a run
};
AttnLayout attn_layout(int64_t rows, int64_t Hkv, int64_t D, int RT, int per_simd, int heads = 1) {
  AttnLayout L;
  L.RT = RT;
  L.NHV = (int)(Hkv / heads * ((rows + L.RT * 16 - 1) / (L.RT * 16)));
  L.slot_rows = (int)(heads * (rows < L.RT * 16 ? rows : L.RT * 16));
  L.groups = kCus * 4 * per_simd / L.NHV;
  if (L.groups < 1) L.groups = 1;
  L.one = heads == 2 && L.NHV == 1;
  const size_t slots = (size_t)(L.one ? 1 : 2) * L.groups * L.NHV;
  L.ml = 0;
  L.o = (slots * L.slot_rows * 2 * sizeof(float) + 255) & ~(size_t)255;
  L.total = (L.o + slots * L.slot_rows * (size_t)D * sizeof(float) + 255) & ~(size_t)255;
  return L;
}

bool scored(const AttnCommon& a) { return a.cap > 0.0f || a.slopes; }

// Keys that a row of the table can name (none where there is no page).
int capacity(const AttnCommon& a) {
  const int64_t cap = a.num_blocks ? a.max_blocks * a.page : 0;
  return (int)(cap < 0x7FFFFFFF ? cap : 0x7FFFFFFF);
}
// Keys that a sequence reads at most: by its table row, or by its window
// (which starts at most a tile early).
int64_t most_keys(const AttnCommon& a) {
  const int64_t keys = capacity(a);
  return a.window && a.window + a.Q + 64 < keys ? a.window + a.Q + 64 : keys;
}

template <class Args>
AttnShape attn_shape(const Args& a, const AttnLayout& L) {
  AttnShape sh;
  sh.G = (int)(a.Hq / a.Hkv);
  sh.rows = sh.G * (int)a.Q;
  sh.NHV = L.NHV;
  sh.by_seq = L.one && a.B <= L.groups / 2;
  sh.groups = L.one ? L.groups - (sh.by_seq ? (int)a.B : L.groups / 2) : L.groups;
  sh.cap = capacity(a);
  sh.page_shift = (a.page & (a.page - 1)) == 0 ? __builtin_ctzll((uint64_t)a.page) : -1;
  sh.slot_rows = L.slot_rows;
  sh.ml = (float*)((char*)a.workspace + L.ml);
  sh.o = (float*)((char*)a.workspace + L.o);
  return sh;
}

// The whole form for tables of at most `whole` keys, else the split form and,
// where a sequence can be shared, the join.
template <class Wave>
hipError_t launch_forms(const typename Wave::Args& a, AttnShape sh, int64_t whole,
                        hipStream_t stream) {
  constexpr int D = Wave::kD;
  const int64_t keys = most_keys(a);
  // no page at all: every sequence is empty
  if (sh.cap == 0)
    return launch_fill_zero((float*)a.out, (size_t)(a.B * a.Q * a.Hq * D / 2), stream);
  // Heads of 256 have no whole form: eight wavefronts leave 256 registers each,
  // which two row tiles of 128 fill already (4 to 53 VGPRs spill in three of the
  // four bf16 and E4M3 forms, 11 to 58 where scored, 8 to 111 in NVFP4's).
  if constexpr (D < 256 && Wave::kHeads == 1) {
    if (keys <= whole) {
      hipLaunchKernelGGL((k_attn_whole<Wave>), dim3((uint32_t)(a.B * sh.NHV)),
                         dim3(kWholeWaves * 64), 0, stream, a, sh);
      return hipGetLastError();
    }
  }
  const int64_t most = (keys + Wave::kTile - 1) / Wave::kTile * a.B;   // tiles
  if (most < sh.groups) sh.groups = (int)most;
  const int64_t units = (int64_t)sh.groups * sh.NHV;
  hipLaunchKernelGGL((k_attn_runs<Wave>), dim3((uint32_t)((units + 3) / 4)), dim3(256), 0, stream,
                     a, sh);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || keys <= Wave::kTile) return e;   // a sequence of one tile is never shared
  hipLaunchKernelGGL((k_attn_join<D, Wave::kTile, Wave::kHeads, typename Wave::Args>),
                     dim3((uint32_t)(a.B * sh.NHV), (uint32_t)sh.slot_rows), dim3(256), 0, stream,
                     a, sh);
  return hipGetLastError();
}

}  // namespace

}  // namespace nvfp4
