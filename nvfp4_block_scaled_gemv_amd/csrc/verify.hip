// verify.hip -- verification of drafted tokens against the target's
// probabilities, from given random numbers (speculative sampling).
//
// Draft j of a sequence is kept while u_j q_j[d_j] < p_j[d_j] (without draft
// probabilities the draft is certain: q_j[d_j] = 1). At the first one that is
// not, the next token is drawn from max(p_j - q_j, 0) (from p_j where that is
// zero everywhere); if all are kept, from the target's row after them:
//   token = the lowest v with  sum_{i <= v} r_i > u * sum_i r_i.
// All sums are in 64 bits: neighbouring borders of the cumulated sum lie 1e-6
// apart at these vocabularies, so 32-bit sums would pick another token every
// few dozen calls.
//
// Bound: the one row of p and one of q that the draw reads; the other rows
// give one number each. Two launches: k_verify_sums, a workgroup per 1024
// values of the row, finds the row (every workgroup for itself: a gather of Q
// numbers) and sums its piece; k_verify_draw, a workgroup per sequence, finds
// the piece that holds the border, then the token in it (the workspace may hold
// anything, so the sums' workgroups cannot count their arrivals in it). Measured:
// one sequence of 4 drafts, 151936 entries: 3.6 + 3.6 us, each the latency of two
// dependent loads; 16 of them with draft probabilities, 19.4 MB: 7.6 + 5.1 us.
#include "elems.h"
#include "internal.h"

namespace nvfp4 {

namespace {

// Values per workgroup of the sums: 16 sequences 6.4 us, more with 2048 or 4096.
constexpr int kPiece = 1024;
constexpr int kPer = kPiece / 256;

// The drafts of a sequence that are real.
__device__ __forceinline__ int drafts_of(const VerifyArgs& a, int b) {
  const int Q = (int)a.Q;
  if (!a.n_draft) return Q;
  const int n = a.n_draft[b];
  return n < 0 ? 0 : n < Q ? n : Q;
}
// The number of kept drafts; every thread of the wavefront gets it. Q < 64.
__device__ __forceinline__ int kept(const VerifyArgs& a, int b, int& nd) {
  const int lane = threadIdx.x & 63, Q = (int)a.Q;
  nd = drafts_of(a, b);
  bool ok = false;
  if (lane < nd) {
    const int d = a.draft[(int64_t)b * Q + lane];
    if (d >= 0 && d < a.V) {
      const double pt = a.p[((int64_t)b * (Q + 1) + lane) * a.V + d];
      const double qt = a.q ? (double)a.q[((int64_t)b * Q + lane) * a.V + d] : 1.0;
      ok = (double)a.u_accept[(int64_t)b * Q + lane] * qt < pt;   // exact product
    }
  }
  const uint64_t no = ~__ballot(ok);
  const int n = no ? __builtin_ctzll(no) : 64;
  return n < nd ? n : nd;
}

// The weights of the draw: r = max(p - q, 0) at a refused draft, else p.
struct Row {
  const float* p;
  const float* q;   // NULL: none to take off
  int cut;          // without draft probabilities: the refused token, else -1
};
__device__ __forceinline__ Row row_of(const VerifyArgs& a, int b, int n, int nd) {
  Row r;
  r.p = a.p + ((int64_t)b * (a.Q + 1) + n) * a.V;
  r.q = n < nd && a.q ? a.q + ((int64_t)b * a.Q + n) * a.V : nullptr;
  r.cut = n < nd && !a.q ? a.draft[(int64_t)b * a.Q + n] : -1;
  return r;
}
__device__ __forceinline__ double weight(const Row& r, int64_t v, float p, float q) {
  const double d = (double)p - (double)q;
  return r.q ? (d > 0.0 ? d : 0.0) : v == r.cut ? 0.0 : (double)p;
}
// kPer values of p and q at first, first + step, ..; past the row its last one
// (their weight is left out): no branch between the loads.
__device__ __forceinline__ void load_row(const Row& r, int64_t first, int step, int64_t V,
                                         float (&p)[kPer], float (&q)[kPer]) {
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int64_t v = first + i * step;
    p[i] = r.p[v < V ? v : V - 1];
  }
#pragma unroll
  for (int i = 0; i < kPer; ++i) q[i] = 0.0f;
  if (r.q) {
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int64_t v = first + i * step;
      q[i] = r.q[v < V ? v : V - 1];
    }
  }
}

__device__ __forceinline__ double wave_sum_f64(double v) {
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) v += __shfl_xor(v, off, 64);
  return v;
}

__global__ __launch_bounds__(256) void k_verify_sums(const VerifyArgs a, int pieces) {
  __shared__ double lds[4][2];
  const int b = blockIdx.y, piece = blockIdx.x;
  int nd;
  const int n = kept(a, b, nd);
  const Row r = row_of(a, b, n, nd);
  if (piece == 0 && threadIdx.x <= (unsigned)a.Q) {
    const int j = threadIdx.x;
    if (j != n) a.tokens[(int64_t)b * (a.Q + 1) + j] = j < n ? a.draft[(int64_t)b * a.Q + j] : -1;
    if (j == 0) a.accepted[b] = n;
  }
  const int64_t v0 = (int64_t)piece * kPiece;
  float p[kPer], q[kPer];
  load_row(r, v0 + threadIdx.x, 256, a.V, p, q);
  double sr = 0.0, sp = 0.0;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int64_t v = v0 + i * 256 + threadIdx.x;
    sr += v < a.V ? weight(r, v, p[i], q[i]) : 0.0;
    sp += v < a.V ? (double)p[i] : 0.0;
  }
  sr = wave_sum_f64(sr);
  sp = wave_sum_f64(sp);
  if ((threadIdx.x & 63) == 0) {
    lds[threadIdx.x >> 6][0] = sr;
    lds[threadIdx.x >> 6][1] = sp;
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    double* o = (double*)a.workspace + ((int64_t)b * pieces + piece) * 2;
    o[0] = (lds[0][0] + lds[1][0]) + (lds[2][0] + lds[3][0]);
    o[1] = (lds[0][1] + lds[1][1]) + (lds[2][1] + lds[3][1]);
  }
}

// Inclusive sums over the 64 lanes of a wavefront.
__device__ __forceinline__ double wave_scan(double v) {
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) {
    const double o = __shfl_up(v, off, 64);
    if (lane >= off) v += o;
  }
  return v;
}
__device__ __forceinline__ double lane_f64(double v, int lane) {
  const int64_t u = __builtin_bit_cast(int64_t, v);
  const uint32_t lo = __builtin_amdgcn_readlane((int)u, lane);
  const uint32_t hi = __builtin_amdgcn_readlane((int)(u >> 32), lane);
  return __builtin_bit_cast(double, ((uint64_t)hi << 32) | lo);
}

// The first index i below n with sum_{j <= i} x(j) > target, and the sum
// before it; n if there is none. By one wavefront: a run of `per` numbers per
// lane. The lanes' sums and a lane's own add up in different orders, so a
// border may move by a rounding between them: only an i with x(i) > 0 is
// taken. total: of all (target_of(total) is the target).
template <typename X, typename T>
__device__ __forceinline__ int first_past(int n, X x, T target_of, double& before, double& total) {
  const int lane = threadIdx.x & 63;
  const int per = (n + 63) / 64, i0 = lane * per;
  const int i1 = i0 + per < n ? i0 + per : n;
  double mine = 0.0;
  for (int i = i0; i < i1; ++i) mine += x(i);
  const double incl = wave_scan(mine);
  total = lane_f64(incl, 63);
  const double target = target_of(total);
  const uint64_t past = __ballot(incl > target), some = __ballot(mine > 0.0);
  before = 0.0;
  if (!past || !some) return n;
  const int l = past & some ? __builtin_ctzll(past & some) : 63 - __builtin_clzll(some);
  double run = incl - mine, at = run;
  int found = i0;
  for (int i = i0; i < i1; ++i) {
    const double xi = x(i);
    if (xi > 0.0) {
      found = i;
      at = run;
    }
    run += xi;
    if (run > target) break;
  }
  before = lane_f64(at, l);
  return __builtin_amdgcn_readlane(found, l);
}

// Every wavefront finds the piece for itself (no barrier); the four of them
// then share its values.
__global__ __launch_bounds__(256) void k_verify_draw(const VerifyArgs a, int pieces) {
  __shared__ double lds[4];
  __shared__ int ldsi[2][4];
  const int b = blockIdx.x, lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
  const int n = a.accepted[b];   // by k_verify_sums
  const int nd = drafts_of(a, b);
  Row r = row_of(a, b, n, nd);
  const double u = a.u_sample[b];
  const double* sums = (const double*)a.workspace + (int64_t)b * pieces * 2;
  double target = 0.0, before, total;
  auto target_of = [&](double sum) { return target = u * sum; };
  int piece = first_past(pieces, [&](int i) { return sums[2 * i]; }, target_of, before, total);
  if (!(total > 0.0)) {   // p <= q everywhere: draw from p
    r.q = nullptr;
    r.cut = -1;
    piece = first_past(pieces, [&](int i) { return sums[2 * i + 1]; }, target_of, before, total);
  }
  int32_t* const out = a.tokens + (int64_t)b * (a.Q + 1) + n;
  if (piece >= pieces) {   // nothing passes: u >= 1, or no probability at all
    if (threadIdx.x == 0) *out = (int)a.V - 1;
    return;
  }
  // kPer consecutive values per thread
  const int64_t v0 = (int64_t)piece * kPiece + threadIdx.x * kPer;
  float p[kPer], q[kPer];
  load_row(r, v0, 1, a.V, p, q);
  double w[kPer], sum = 0.0;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    w[i] = v0 + i < a.V ? weight(r, v0 + i, p[i], q[i]) : 0.0;
    sum += w[i];
  }
  const double incl = wave_scan(sum);
  if (lane == 63) lds[wv] = incl;
  __syncthreads();
  double run = before + (incl - sum);
  for (int k = 0; k < wv; ++k) run += lds[k];
  int token = 0x7FFFFFFF, last = -1;   // the first past the target, the last with a weight
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    run += w[i];
    if (w[i] > 0.0) last = (int)(v0 + i);
    if (token == 0x7FFFFFFF && run > target && w[i] > 0.0) token = (int)(v0 + i);
  }
  // values rise with the lane: the first lane that has one, the last that does
  const uint64_t hit = __ballot(token != 0x7FFFFFFF), any = __ballot(last >= 0);
  if (lane == 0) {
    ldsi[0][wv] = -1;
    ldsi[1][wv] = -1;
  }
  if (hit && lane == __builtin_ctzll(hit)) ldsi[0][wv] = token;
  if (any && lane == 63 - __builtin_clzll(any)) ldsi[1][wv] = last;
  __syncthreads();
  if (threadIdx.x) return;
  int pick = -1, end = (int)a.V - 1;
  for (int k = 0; k < 4; ++k) {
    if (pick < 0) pick = ldsi[0][k];
    if (ldsi[1][k] >= 0) end = ldsi[1][k];
  }
  *out = pick >= 0 ? pick : end;
}

int64_t pieces_of(int64_t V) { return (V + kPiece - 1) / kPiece; }

}  // namespace

size_t verify_workspace_bytes(int64_t B, int64_t V) {
  return ((size_t)B * (size_t)pieces_of(V) * 2 * sizeof(double) + 255) & ~(size_t)255;
}

hipError_t launch_verify_draft(const VerifyArgs& a, hipStream_t stream) {
  const int pieces = (int)pieces_of(a.V);
  hipLaunchKernelGGL(k_verify_sums, dim3((uint32_t)pieces, (uint32_t)a.B), dim3(256), 0, stream, a,
                     pieces);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(k_verify_draw, dim3((uint32_t)a.B), dim3(256), 0, stream, a, pieces);
  return hipGetLastError();
}

}  // namespace nvfp4
