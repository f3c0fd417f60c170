// lora.hip -- low-rank adapters of many requests beside shared projections:
// row m of x has adapter e = ids[m], and for every projection s of x
//   y_s[m] = base_s[m] + alpha[e] B_s[e] (A_s[e] x[m])
// with A_s[e] [rank, K] and B_s[e] [N_s, rank] in bf16.
//
// Bound: the bytes of the adapters that occur, each read once for up to 16 rows
// that share it, and of y; for a few tokens the latency of loads that wait for
// each other (ids, then weights).
//
// Rows are grouped on the device: workgroups are launched for every row and each
// finds the rows of the same adapter among the ids (two ballots); it works if
// its row is the first, 17th, .. of them and takes that one and the next 15,
// which fill the 16 rows (columns) of the matrix instructions.
//   k_lora_down  t[m, r] = A x[m]: a workgroup per (row, projection, 16 ranks,
//                piece of K); its wavefronts split the piece and meet in LDS;
//                pieces leave partial sums (fp32) in the workspace.
//   k_lora_up    a workgroup per (row, 256 outputs): the pieces' sums, in a
//                fixed order, as three bf16 each (all 24 bits), times B.
//   k_lora_all   both in one launch for a few rows: a workgroup per (row, 1024
//                outputs) makes all of t for itself, in the same order.
// A's and x's products are exact in the matrix cores' fp32 sums. No atomics; a
// row's bits do not depend on the other rows.
//
// Measured, K 4096: 1 token, 6144 outputs of three projections, rank 16 9.7 us (0.7
// MB: a launch and five dependent loads); 48 rows of 39 adapters of ranks 16 to 64,
// 24576 outputs 11 + 32 us, 105 MB and 128 in whole lines: B's rows come at 4 TB/s, as
// each workgroup's wait for ids, sums and first loads is as long as its loads (more
// wavefronts, loads of whole lines or two blocks of outputs changed it by 3 %). K
// 12288, 128 rows of 16 adapters, rank 32, 4096 outputs 7.7 + 5.8 us for 24 MB.
#include "elems.h"
#include "internal.h"

namespace nvfp4 {

namespace {

constexpr int kThreads = 256;
constexpr int kStep = 32;          // inputs per matrix instruction
constexpr int kDeep = 8;           // of them per wavefront and turn
constexpr int kTurn = 4 * kDeep * kStep;   // inputs of a workgroup's turn: 1024
constexpr int kMaxChunks = 16;
// Outputs per workgroup of k_lora_up. One, two or four blocks of 256 (the next one's
// loads before one's outputs are stored), both kernels, us: 16 sequences of 8 rows,
// rank 32 13.9 / 16.5 / 16.0; 128 rows of as many adapters, 6144 outputs, rank 16 26.2 /
// 25.2 / 23.8, of one adapter 13.0 / 14.0 / 16.2; 48 rows of 39 adapters of ranks 16
// to 64, 24576 outputs 44.5 / 44.1 / 45.4.
constexpr int kOuts = 256;
constexpr int kAllOuts = 1024;     // and of k_lora_all

struct LoraShape {
  int chunks, turns;               // chunks of K, turns of a chunk
  int tiles;                       // tiles of 16 ranks
  int blocks;                      // workgroups per row of k_lora_up, k_lora_all
  float* t;                        // [chunks][segments][M][rank]
};

// The rows of a workgroup: those of row m's adapter from m on, 16 at most.
struct Rows {
  int id;      // the adapter, -1: none
  int count;   // 0: another workgroup has them
};
__device__ __forceinline__ Rows rows_of(const LoraArgs& a, int m, int (&list)[16]) {
  const int lane = threadIdx.x & 63, M = (int)a.M;
  const int E = (int)a.n_adapters;
  int i0 = lane < M ? a.ids[lane] : -2, i1 = lane + 64 < M ? a.ids[lane + 64] : -2;
  // what lies outside the adapters is none
  if (lane < M && (uint32_t)i0 >= (uint32_t)E) i0 = -1;
  if (lane + 64 < M && (uint32_t)i1 >= (uint32_t)E) i1 = -1;
  Rows r;
  r.id = __builtin_amdgcn_readlane(m < 64 ? i0 : i1, m & 63);
  uint64_t b0 = __ballot(i0 == r.id), b1 = __ballot(i1 == r.id);
  const uint64_t below = ((uint64_t)1 << (m & 63)) - 1;
  const int before = m < 64 ? __popcll(b0 & below) : __popcll(b0) + __popcll(b1 & below);
  r.count = 0;
  if (before & 15) return r;
  // from m on
  if (m < 64) {
    b0 &= ~below;
  } else {
    b0 = 0;
    b1 &= ~below;
  }
  const int n0 = __popcll(b0), n = n0 + __popcll(b1);
  r.count = n < 16 ? n : 16;
  if (threadIdx.x < 64) {
    const uint64_t mine = (uint64_t)1 << lane;
    const int p0 = __popcll(b0 & (mine - 1)), p1 = n0 + __popcll(b1 & (mine - 1));
    if ((b0 & mine) && p0 < 16) list[p0] = lane;
    if ((b1 & mine) && p1 < 16) list[p1] = lane + 64;
  }
  __syncthreads();
  return r;
}

// The row of a workgroup (M and more: none). From 16 rows on they start in the order
// 0 8 16 .., 4 12 .., 2 10 .., 6 .., 1 .., 5 .., 3 .., 7 ..: where a request has
// several rows, which are neighbours as a rule, those that begin a group start
// early, and the workgroups that have nothing to do, of 1 us each, late. It is made
// for groups of 2, 4 and 8 rows and more; those of 3 and 5, and adapters in turn over
// the rows, may lose by it. Rows in turn against this, both kernels, us, groups of
//                                       1     2     3     4     5     6     8     12    all
//   K 12288, 4096 outputs, 128 rows  now 40.0  21.2  21.1  16.0  19.3  17.5  13.8  14.7  14.0
//     rank 32                    in turn 37.7  29.4  21.1  22.8  19.2  20.0  19.3  18.0  18.5
//                          48 rows  now 16.5  14.3  16.2  12.7  14.2  13.4  10.4  12.8  11.3
//                                in turn 16.6  15.7  13.8  13.8  12.5  12.3  13.4  11.4  14.3
//   K 4096, 6144 outputs, 128 rows  now 26.8  17.8  17.5  14.2  16.7  14.2  11.8  12.3  11.3
//     rank 16                    in turn 25.7  21.9  17.4  17.0  15.9  16.2  15.7  14.3  15.6
//   16 adapters in turn over 128 rows: 18.4 / 13.8 and 15.5 / 11.8 (now / in turn); groups of
//   1 to 8 at random 19.2 / 20.4 and 16.3 / 18.3.
__device__ __forceinline__ int row_of_block() {
  const int z = blockIdx.z;
  return blockIdx.y * gridDim.z + ((z & 1) * 4 + (z & 2) + (z >> 2));
}

// A wavefront's sum over kDeep steps of K from k on: of ranks (columns g * 4 + i of
// the result) and rows (n). A, X: the lane's row of either at its 8 inputs.
__device__ __forceinline__ f32x4_t down_step(const uint16_t* A, const uint16_t* X, int64_t k,
                                             int64_t K, f32x4_t acc) {
  bf16x8_t wa[kDeep], xa[kDeep];
#pragma unroll
  for (int i = 0; i < kDeep; ++i) {
    // past K: the first inputs again, not multiplied
    const int64_t at = k + i * kStep < K ? k + i * kStep : 0;
    wa[i] = *reinterpret_cast<const bf16x8_t*>(A + at);
    xa[i] = *reinterpret_cast<const bf16x8_t*>(X + at);
  }
#pragma unroll
  for (int i = 0; i < kDeep; ++i)
    if (k + i * kStep < K)
      acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wa[i], xa[i], acc, 0, 0, 0);
  return acc;
}

__global__ __launch_bounds__(kThreads) void k_lora_down(const LoraArgs a, const LoraShape sh) {
  __shared__ int list[16];
  __shared__ float part[4][16][17];
  const int m = row_of_block();
  if (m >= (int)a.M) return;
  const Rows rows = rows_of(a, m, list);
  if (rows.count == 0 || rows.id < 0) return;
  int u = blockIdx.x;
  const int chunk = u % sh.chunks;
  u /= sh.chunks;
  const int tile = u % sh.tiles, seg = u / sh.tiles;
  const int rank = (int)a.rank, r0 = tile * 16;
  // (every adapter reads its first 16 ranks: no wait for how many it has)
  if (r0 > 0 && a.ranks && r0 >= a.ranks[rows.id]) return;
  const int lane = threadIdx.x & 63, n = lane & 15, g = lane >> 4;
  const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t K = a.K;
  // ranks and rows past the last repeat it: what they give is not stored
  const int r = r0 + n < rank ? r0 + n : rank - 1;
  const int row = list[n < rows.count ? n : 0];
  const uint16_t* A = a.segs[seg].a + ((int64_t)rows.id * rank + r) * K + g * 8;
  const uint16_t* X = a.x + (int64_t)row * K + g * 8;
  f32x4_t acc = {0.0f, 0.0f, 0.0f, 0.0f};
  int64_t k = (int64_t)chunk * sh.turns * kTurn + wv * (kDeep * kStep);
  for (int turn = 0; turn < sh.turns; ++turn, k += kTurn) acc = down_step(A, X, k, K, acc);
  // acc[i]: rank r0 + g * 4 + i, row n
#pragma unroll
  for (int i = 0; i < 4; ++i) part[wv][n][g * 4 + i] = acc[i];
  __syncthreads();
  const int tr = threadIdx.x & 15, tn = threadIdx.x >> 4;
  if (tn < rows.count && r0 + tr < rank)
    sh.t[(((int64_t)chunk * a.n_segments + seg) * a.M + list[tn]) * rank + r0 + tr] =
        (part[0][tn][tr] + part[1][tn][tr]) + (part[2][tn][tr] + part[3][tn][tr]);
}

// t in LDS as three bf16: [part][row][rank, padded to 32], rows 16 bytes apart
// from a multiple of the banks.
__device__ __forceinline__ int lds_row(int rank) { return (rank + 31) / 32 * 32 + 8; }
__device__ __forceinline__ void put_t(uint16_t* lds_t, int ld, int row, int r, float v) {
#pragma unroll
  for (int p = 0; p < 3; ++p) {
    const uint32_t u = __float_as_uint(v) & 0xFFFF0000u;
    lds_t[(p * 16 + row) * ld + r] = (uint16_t)(u >> 16);
    v -= __uint_as_float(u);   // exact
  }
}

// A wavefront's 64 outputs from n0 on (the lane's 4: n0 + c * 4 ..) of up to 16
// rows. G: groups of 8 ranks that a matrix instruction takes of one output (4, or
// 1 and 2 for ranks of 8 and 16: then it holds 4 / G outputs' groups, and one
// output's at a time enter it, the others as zeros).
template <int G>
struct Up {
  static constexpr int kPer = 4 / G;   // outputs of a load
  const LoraSegment& s;
  const uint16_t* const B;
  const int rank, c, g;
  const int64_t n0;
  u32x4_t w[2][G];                     // two steps of 8 G ranks
  f32x4_t y[4];                        // base of the lane's rows g * 4 + i

  __device__ __forceinline__ Up(const LoraSegment& s_, int id, int rank_, int64_t first)
      : s(s_), B(s_.b + (int64_t)id * s_.N * rank_), rank(rank_), c(threadIdx.x & 15),
        g((threadIdx.x & 63) >> 4), n0(first + c * 4) {}
  __device__ __forceinline__ void load(int step, u32x4_t (&to)[G]) const {
    const int r = step * 8 * G + g % G * 8;
#pragma unroll
    for (int q = 0; q < G; ++q) {
      int64_t n = n0 + q * kPer + g / G;
      n = n < s.N ? n : s.N - 1;       // not stored
      to[q] = *reinterpret_cast<const u32x4_t*>(B + n * rank + (r < rank ? r : 0));
    }
  }
  __device__ __forceinline__ void load_base(const int* list, int count) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      y[i] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
      if (!s.base || g * 4 + i >= count || n0 >= s.N) continue;
      const float* p = s.base + (int64_t)list[g * 4 + i] * s.N + n0;
      if (s.wide) {
        y[i] = *reinterpret_cast<const f32x4_t*>(p);
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) y[i][j] = n0 + j < s.N ? p[j] : 0.0f;
      }
    }
  }
  __device__ __forceinline__ void multiply(u32x4_t (&v)[G], int step, int own,
                                           const uint16_t* lds_t, int ld, f32x4_t (&acc)[4]) const {
    const int r = step * 8 * G + g % G * 8;
    if ((step + 1) * 8 * G > own) {    // ranks past the adapter's own
#pragma unroll
      for (int q = 0; q < G; ++q)
#pragma unroll
        for (int d = 0; d < 4; ++d) {
          const int left = own - (r + 2 * d);
          v[q][d] &= left >= 2 ? 0xFFFFFFFFu : left == 1 ? 0xFFFFu : 0u;
        }
    }
    bf16x8_t tf[3];
#pragma unroll
    for (int p = 0; p < 3; ++p)
      tf[p] = *reinterpret_cast<const bf16x8_t*>(&lds_t[(p * 16 + c) * ld + r]);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      u32x4_t b = v[j / kPer];
      if (G < 4) {
        const bool mine = g / G == j % kPer;
#pragma unroll
        for (int d = 0; d < 4; ++d) b[d] = mine ? b[d] : 0u;
      }
#pragma unroll
      for (int p = 2; p >= 0; --p)     // the smallest parts first
        acc[j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(tf[p], __builtin_bit_cast(bf16x8_t, b),
                                                         acc[j], 0, 0, 0);
    }
  }
  // After load() of steps 0 and 1 (where there is one) and load_base().
  __device__ __forceinline__ void finish(int own, float alpha, const uint16_t* lds_t,
                                         const int* list, int count) {
    const int ld = lds_row(rank), steps = (own + 8 * G - 1) / (8 * G);
    f32x4_t acc[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[j] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
    if (G < 4) {                       // one step
      if (steps) multiply(w[0], 0, own, lds_t, ld, acc);
    } else {
      for (int i = 0; i < steps; i += 2) {
        multiply(w[0], i, own, lds_t, ld, acc);
        if (i + 2 < steps) load(i + 2, w[0]);
        if (i + 1 < steps) multiply(w[1], i + 1, own, lds_t, ld, acc);
        if (i + 3 < steps) load(i + 3, w[1]);
      }
    }
    // acc[j][i]: row g * 4 + i, output n0 + j
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (g * 4 + i >= count || n0 >= s.N) continue;
      float* p = s.y + (int64_t)list[g * 4 + i] * s.N + n0;
      f32x4_t v;
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] = fmaf(alpha, acc[j][i], y[i][j]);
      if (s.wide) {
        *reinterpret_cast<f32x4_t*>(p) = v;
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (n0 + j < s.N) p[j] = v[j];
      }
    }
  }
};

// Rows without an adapter: the base, where y is another array.
__device__ __forceinline__ void copy_base(const LoraSegment& s, const int* list, int count,
                                          int64_t first, int64_t end) {
  if (s.base == s.y) return;
  for (int i = 0; i < count; ++i) {
    const int64_t at = (int64_t)list[i] * s.N;
    for (int64_t n = first + threadIdx.x; n < end; n += blockDim.x)
      s.y[at + n] = s.base ? s.base[at + n] : 0.0f;
  }
}

__device__ __forceinline__ int own_ranks(const LoraArgs& a, int id) {
  const int rank = (int)a.rank, own = a.ranks ? a.ranks[id] : rank;
  return own < 0 ? 0 : own > rank ? rank : own;
}

template <int G>
__global__ __launch_bounds__(kThreads) void k_lora_up(const LoraArgs a, const LoraShape sh) {
  __shared__ int list[16];
  extern __shared__ __align__(16) uint16_t lds_t[];
  const int m = row_of_block();
  if (m >= (int)a.M) return;
  const Rows rows = rows_of(a, m, list);
  if (rows.count == 0) return;
  int block = blockIdx.x, seg = 0;
  while (block >= a.segs[seg].blocks) block -= a.segs[seg++].blocks;
  const LoraSegment& s = a.segs[seg];
  const int64_t first = (int64_t)block * kOuts, end = first + kOuts < s.N ? first + kOuts : s.N;
  if (rows.id < 0) return copy_base(s, list, rows.count, first, end);
  const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), rank = (int)a.rank;
  Up<G> up(s, rows.id, rank, first + wv * 64);
  up.load(0, up.w[0]);
  up.load_base(list, rows.count);
  const float alpha = a.alpha ? a.alpha[rows.id] : 1.0f;
  const int own = own_ranks(a, rows.id), ld = lds_row(rank), pad = ld - 8;
  if (G == 4 && own > 32) up.load(1, up.w[1]);
  const int64_t step = a.n_segments * a.M * rank;
  for (int i = threadIdx.x; i < 16 * pad; i += kThreads) {
    const int tn = i / pad, tr = i - tn * pad;
    float v = 0.0f;
    if (tn < rows.count && tr < own) {
      const float* t = sh.t + ((int64_t)seg * a.M + list[tn]) * rank + tr;
      float x[kMaxChunks];             // all on their way at once
#pragma unroll
      for (int q = 0; q < kMaxChunks; ++q) x[q] = q < sh.chunks ? t[q * step] : 0.0f;
#pragma unroll
      for (int q = 0; q < kMaxChunks; ++q) v += x[q];
    }
    put_t(lds_t, ld, tn, tr, v);
  }
  __syncthreads();
  up.finish(own, alpha, lds_t, list, rows.count);
}

// All in one: 16 wavefronts, each 64 outputs; of t they take 256 inputs each in
// turn, four of them a piece of k_lora_down's, summed in its order.
template <int G>
__global__ __launch_bounds__(1024) void k_lora_all(const LoraArgs a, const LoraShape sh) {
  __shared__ int list[16];
  __shared__ float part[16][16][17];
  extern __shared__ __align__(16) uint16_t lds_t[];
  const int m = blockIdx.y;
  const Rows rows = rows_of(a, m, list);
  if (rows.count == 0) return;
  int block = blockIdx.x, seg = 0;
  while (block >= a.segs[seg].blocks) block -= a.segs[seg++].blocks;
  const LoraSegment& s = a.segs[seg];
  const int64_t first = (int64_t)block * kAllOuts;
  const int64_t end = first + kAllOuts < s.N ? first + kAllOuts : s.N;
  if (rows.id < 0) return copy_base(s, list, rows.count, first, end);
  const int lane = threadIdx.x & 63, n = lane & 15, g = lane >> 4;
  const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), rank = (int)a.rank;
  const int64_t K = a.K;
  Up<G> up(s, rows.id, rank, first + wv * 64);
  up.load(0, up.w[0]);
  const float alpha = a.alpha ? a.alpha[rows.id] : 1.0f;
  const int own = own_ranks(a, rows.id), ld = lds_row(rank), pad = ld - 8;
  const uint16_t* X = a.x + (int64_t)list[n < rows.count ? n : 0] * K + g * 8;
  const int tr = threadIdx.x & 15, tn = (threadIdx.x >> 4) & 15;
  for (int r0 = 0; r0 < pad; r0 += 16) {
    float v = 0.0f;
    if (r0 < own) {
      const int r = r0 + n < rank ? r0 + n : rank - 1;
      const uint16_t* A = s.a + ((int64_t)rows.id * rank + r) * K + g * 8;
      for (int64_t k0 = 0; k0 < K; k0 += 4 * kTurn) {
        const f32x4_t acc = down_step(A, X, k0 + wv * (kDeep * kStep), K, f32x4_t{0, 0, 0, 0});
        __syncthreads();               // the last turn's parts are read
#pragma unroll
        for (int i = 0; i < 4; ++i) part[wv][n][g * 4 + i] = acc[i];
        __syncthreads();
        if (threadIdx.x < 256 && tn < rows.count && r0 + tr < own)
          for (int q = 0; q < 4 && k0 + q * kTurn < K; ++q)
            v += (part[4 * q][tn][tr] + part[4 * q + 1][tn][tr]) +
                 (part[4 * q + 2][tn][tr] + part[4 * q + 3][tn][tr]);
      }
    }
    if (threadIdx.x < 256) put_t(lds_t, ld, tn, r0 + tr, v);
  }
  up.load_base(list, rows.count);
  if (G == 4 && own > 32) up.load(1, up.w[1]);
  __syncthreads();
  up.finish(own, alpha, lds_t, list, rows.count);
}

// K in chunks of whole turns, kMaxChunks at most.
void split(int64_t K, int& chunks, int& turns) {
  const int64_t all = (K + kTurn - 1) / kTurn;
  turns = (int)((all + kMaxChunks - 1) / kMaxChunks);
  chunks = turns ? (int)((all + turns - 1) / turns) : 0;
}

// One launch where a workgroup makes t quickly enough by itself (one CU reads some
// 30 GB/s of A) and few make it. One against two (and a launch more), other inputs
// each time, us: K 4096, 6144 outputs in three projections, rank 16: 1 row 9.9 / 9.9,
// 32 rows 10.9 / 12.4, 64 19.6 / 15.1; rank 64: 1 row 26 / 10.8; K 12288, rank 32:
// 34 / 10.3; 24576 outputs in two, rank 16: 4 rows 10.3 / 10.3, 16 18.4 / 12.0.
bool all_in_one(const LoraArgs& a, const LoraShape& sh) {
  if (sh.turns > 1) return false;   // its order is that of one turn a piece
  int64_t blocks = 0;
  for (int s = 0; s < a.n_segments; ++s) blocks += (a.segs[s].N + kAllOuts - 1) / kAllOuts;
  return a.rank * a.K <= 1 << 16 && a.M * blocks <= 192;
}

}  // namespace

size_t lora_workspace_bytes(int64_t M, int64_t K, int64_t rank, int64_t n_segments) {
  int chunks, turns;
  split(K, chunks, turns);
  return ((size_t)chunks * n_segments * M * rank * sizeof(float) + 255) & ~(size_t)255;
}

hipError_t launch_lora(LoraArgs& a, hipStream_t stream) {
  LoraShape sh;
  split(a.K, sh.chunks, sh.turns);
  sh.tiles = (int)((a.rank + 15) / 16);
  sh.t = (float*)a.workspace;
  const bool one = all_in_one(a, sh);
  const int outs = one ? kAllOuts : kOuts;   // of a workgroup
  sh.blocks = 0;
  for (int s = 0; s < a.n_segments; ++s) {
    LoraSegment& g = a.segs[s];
    g.blocks = (int)((g.N + outs - 1) / outs);
    g.wide = g.N % 4 == 0 && (((uintptr_t)g.y | (uintptr_t)g.base) & 15) == 0;
    sh.blocks += g.blocks;
  }
  if (sh.blocks == 0) return hipSuccess;
  // (row_of_block's)
  const uint32_t eighths = a.M >= 16 ? 8 : 1, rows = ((uint32_t)a.M + eighths - 1) / eighths;
  if (!one && sh.chunks && a.n_adapters) {   // without inputs, or adapters, the sums are empty
    hipLaunchKernelGGL(k_lora_down,
                       dim3((uint32_t)(a.n_segments * sh.tiles * sh.chunks), rows, eighths),
                       dim3(kThreads), 0, stream, a, sh);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  const size_t lds = (size_t)3 * 16 * ((a.rank + 31) / 32 * 32 + 8) * sizeof(uint16_t);
  const dim3 grid((uint32_t)sh.blocks, one ? (uint32_t)a.M : rows, one ? 1 : eighths), block(one ? 1024 : kThreads);
  const auto kernel = a.rank == 8    ? (one ? k_lora_all<1> : k_lora_up<1>)
                      : a.rank == 16 ? (one ? k_lora_all<2> : k_lora_up<2>)
                                     : (one ? k_lora_all<4> : k_lora_up<4>);
  hipLaunchKernelGGL(kernel, grid, block, lds, stream, a, sh);
  return hipGetLastError();
}

}  // namespace nvfp4
