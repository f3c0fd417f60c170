// lora.hip -- low-rank adapters of many requests beside shared projections:
// row m of x has adapter e = ids[m], and for every projection s of x
//   y_s[m] = base_s[m] + alpha[e] B_s[e] (A_s[e] x[m])
// with A_s[e] [rank, K] and B_s[e] [N_s, rank] in bf16.
//
// Bound: the bytes of the adapters that occur, each read once for up to 16 rows
// that share it, and of y; for a few tokens the latency of two launches, each
// three loads that wait for each other (ids, then weights or sums, then y).
//
// Rows are grouped on the device: a workgroup is launched for every row and
// finds the rows of the same adapter among the ids (two ballots); it works if
// its row is the first, 17th, .. of them and takes that one and the next 15,
// which fill the 16 rows (columns) of the matrix instructions.
//   k_lora_down  t[m, r] = A x[m]: a workgroup per (row, projection, 16 ranks,
//                chunk of K); its wavefronts split the chunk and meet in LDS;
//                chunks leave partial sums (fp32) in the workspace.
//   k_lora_up    a workgroup per (row, 256 outputs): the chunks' sums, in a
//                fixed order, as three bf16 each (all 24 bits), times B.
// A's and x's products are exact in the matrix cores' fp32 sums. No atomics.
#include "elems.h"
#include "internal.h"

namespace nvfp4 {

namespace {

constexpr int kThreads = 256;
constexpr int kStep = 32;          // inputs per matrix instruction
constexpr int kDeep = 8;           // of them per wavefront and turn
constexpr int kTurn = 4 * kDeep * kStep;   // inputs of a workgroup's turn: 1024
constexpr int kMaxChunks = 16;
constexpr int kOuts = 256;         // outputs per workgroup

struct LoraShape {
  int chunks, turns;               // chunks of K, turns of a chunk
  int tiles;                       // tiles of 16 ranks
  int blocks;                      // workgroups per row of k_lora_up
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

__global__ __launch_bounds__(kThreads) void k_lora_down(const LoraArgs a, const LoraShape sh) {
  __shared__ int list[16];
  __shared__ float part[4][16][17];
  const int m = blockIdx.y;
  const Rows rows = rows_of(a, m, list);
  if (rows.count == 0 || rows.id < 0) return;
  int u = blockIdx.x;
  const int chunk = u % sh.chunks;
  u /= sh.chunks;
  const int tile = u % sh.tiles, seg = u / sh.tiles;
  const int rank = (int)a.rank;
  const int own = a.ranks ? a.ranks[rows.id] : rank;
  const int r0 = tile * 16;
  if (r0 >= own) return;
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
  for (int turn = 0; turn < sh.turns; ++turn, k += kTurn) {
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
  }
  // acc[i]: rank r0 + g * 4 + i, row n
#pragma unroll
  for (int i = 0; i < 4; ++i) part[wv][n][g * 4 + i] = acc[i];
  __syncthreads();
  const int tr = threadIdx.x & 15, tn = threadIdx.x >> 4;
  if (tn < rows.count && r0 + tr < rank)
    sh.t[(((int64_t)chunk * a.n_segments + seg) * a.M + list[tn]) * rank + r0 + tr] =
        (part[0][tn][tr] + part[1][tn][tr]) + (part[2][tn][tr] + part[3][tn][tr]);
}

// G: groups of 8 ranks that a matrix instruction takes of one output (4, or 1
// and 2 for ranks of 8 and 16: then it holds 4 / G outputs' groups, and one
// output's at a time enter it, the others as zeros).
template <int G>
__global__ __launch_bounds__(kThreads) void k_lora_up(const LoraArgs a, const LoraShape sh) {
  __shared__ int list[16];
  // t as three bf16: [part][row][rank], rows 16 bytes apart from a bank's multiple
  extern __shared__ __align__(16) uint16_t lds_t[];
  const int m = blockIdx.y;
  const Rows rows = rows_of(a, m, list);
  if (rows.count == 0) return;
  int block = blockIdx.x, seg = 0;
  while (block >= a.segs[seg].blocks) block -= a.segs[seg++].blocks;
  const LoraSegment& s = a.segs[seg];
  const int64_t N = s.N;
  const int lane = threadIdx.x & 63, c = lane & 15, g = lane >> 4;
  const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t n0 = (int64_t)block * kOuts + wv * 64 + c * 4;   // the lane's 4 outputs
  const int rank = (int)a.rank;
  if (rows.id < 0) {
    if (s.base == s.y) return;
    for (int i = g; i < rows.count; i += 4) {
      const int64_t at = (int64_t)list[i] * N + n0;
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (n0 + j < N) s.y[at + j] = s.base ? s.base[at + j] : 0.0f;
    }
    return;
  }
  int own = a.ranks ? a.ranks[rows.id] : rank;
  own = own < 0 ? 0 : own > rank ? rank : own;
  const float alpha = a.alpha ? a.alpha[rows.id] : 1.0f;
  const int pad = (rank + 31) / 32 * 32, ld = pad + 8;
  for (int i = threadIdx.x; i < 16 * pad; i += kThreads) {
    const int tn = i / pad, tr = i - tn * pad;
    float v = 0.0f;
    if (tn < rows.count && tr < own) {
      const float* t = sh.t + ((int64_t)seg * a.M + list[tn]) * rank + tr;
      const int64_t step = a.n_segments * a.M * rank;
      for (int q = 0; q < sh.chunks; ++q) v += t[q * step];
    }
#pragma unroll
    for (int p = 0; p < 3; ++p) {
      const uint32_t u = __float_as_uint(v) & 0xFFFF0000u;
      lds_t[(p * 16 + tn) * ld + tr] = (uint16_t)(u >> 16);
      v -= __uint_as_float(u);   // exact
    }
  }
  __syncthreads();
  const uint16_t* B = s.b + (int64_t)rows.id * N * rank;
  f32x4_t acc[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) acc[j] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
  constexpr int kLoads = G;          // per 32 / (4 / G) ranks
  constexpr int kPer = 4 / G;        // outputs of a load
  const int r_lane = (g % G) * 8;
  for (int r0 = 0; r0 < own; r0 += 8 * G) {
    u32x4_t w[kLoads];
    const int r = r0 + r_lane;
#pragma unroll
    for (int q = 0; q < kLoads; ++q) {
      int64_t n = n0 + q * kPer + g / G;
      n = n < N ? n : N - 1;         // not stored
      w[q] = *reinterpret_cast<const u32x4_t*>(B + n * rank + (r < rank ? r : 0));
    }
    if (r0 + 8 * G > own) {
      // ranks past the adapter's own
#pragma unroll
      for (int q = 0; q < kLoads; ++q)
#pragma unroll
        for (int d = 0; d < 4; ++d) {
          const int left = own - (r + 2 * d);
          w[q][d] &= left >= 2 ? 0xFFFFFFFFu : left == 1 ? 0xFFFFu : 0u;
        }
    }
    bf16x8_t tf[3];
#pragma unroll
    for (int p = 0; p < 3; ++p)
      tf[p] = *reinterpret_cast<const bf16x8_t*>(&lds_t[(p * 16 + c) * ld + r]);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      u32x4_t b = w[j / kPer];
      if (G < 4) {
        const bool mine = g / G == j % kPer;
#pragma unroll
        for (int d = 0; d < 4; ++d) b[d] = mine ? b[d] : 0u;
      }
#pragma unroll
      for (int p = 2; p >= 0; --p)
        acc[j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(tf[p], __builtin_bit_cast(bf16x8_t, b),
                                                         acc[j], 0, 0, 0);
    }
  }
  // acc[j][i]: row g * 4 + i, output n0 + j
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (g * 4 + i >= rows.count || n0 >= N) continue;
    const int64_t at = (int64_t)list[g * 4 + i] * N + n0;
    if (s.wide) {
      f32x4_t v = {0.0f, 0.0f, 0.0f, 0.0f};
      if (s.base) v = *reinterpret_cast<const f32x4_t*>(s.base + at);
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] = fmaf(alpha, acc[j][i], v[j]);
      *reinterpret_cast<f32x4_t*>(s.y + at) = v;
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (n0 + j < N) s.y[at + j] = fmaf(alpha, acc[j][i], s.base ? s.base[at + j] : 0.0f);
    }
  }
}

// K in chunks of whole turns, kMaxChunks at most.
void split(int64_t K, int& chunks, int& turns) {
  const int64_t all = (K + kTurn - 1) / kTurn;
  turns = (int)((all + kMaxChunks - 1) / kMaxChunks);
  chunks = turns ? (int)((all + turns - 1) / turns) : 0;
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
  sh.blocks = 0;
  for (int s = 0; s < a.n_segments; ++s) {
    LoraSegment& g = a.segs[s];
    g.blocks = (int)((g.N + kOuts - 1) / kOuts);
    g.wide = g.N % 4 == 0 && (((uintptr_t)g.y | (uintptr_t)g.base) & 15) == 0;
    sh.blocks += g.blocks;
  }
  if (sh.blocks == 0) return hipSuccess;
  if (sh.chunks && a.n_adapters) {   // without inputs, or adapters, the sums are empty
    hipLaunchKernelGGL(k_lora_down,
                       dim3((uint32_t)(a.n_segments * sh.tiles * sh.chunks), (uint32_t)a.M),
                       dim3(kThreads), 0, stream, a, sh);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  const size_t lds = (size_t)3 * 16 * ((a.rank + 31) / 32 * 32 + 8) * sizeof(uint16_t);
  const dim3 grid((uint32_t)sh.blocks, (uint32_t)a.M);
  if (a.rank == 8)
    hipLaunchKernelGGL(k_lora_up<1>, grid, dim3(kThreads), lds, stream, a, sh);
  else if (a.rank == 16)
    hipLaunchKernelGGL(k_lora_up<2>, grid, dim3(kThreads), lds, stream, a, sh);
  else
    hipLaunchKernelGGL(k_lora_up<4>, grid, dim3(kThreads), lds, stream, a, sh);
  return hipGetLastError();
}

}  // namespace nvfp4
