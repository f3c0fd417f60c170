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
// give one number each. Two launches: k_verify_sums, a workgroup per 2048
// values of the row, finds the row (every workgroup for itself: a gather of Q
// numbers) and sums its piece; k_verify_draw, a workgroup per sequence, finds
// the piece that holds the border, then the token in it.
#include "elems.h"
#include "internal.h"

namespace nvfp4 {

namespace {

constexpr int kPiece = 2048;     // values per workgroup of the sums
constexpr int kPer = kPiece / 256;

// The number of kept drafts; every thread of the wavefront gets it. Q <= 64.
__device__ __forceinline__ int kept(const VerifyArgs& a, int b, int& nd) {
  const int lane = threadIdx.x & 63, Q = (int)a.Q;
  nd = Q;
  if (a.n_draft) {
    const int n = a.n_draft[b];
    nd = n < 0 ? 0 : n < Q ? n : Q;
  }
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
__device__ __forceinline__ double weight(const Row& r, int64_t v, double p) {
  if (r.q) {
    const double d = p - (double)r.q[v];
    return d > 0.0 ? d : 0.0;
  }
  return v == r.cut ? 0.0 : p;
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
  double sr = 0.0, sp = 0.0;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int64_t v = v0 + i * 256 + threadIdx.x;
    if (v < a.V) {
      const double p = r.p[v];
      sr += weight(r, v, p);
      sp += p;
    }
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

// Inclusive sums over the 256 threads; total: of all.
__device__ __forceinline__ double block_scan(double v, double* lds, double& total) {
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) {
    const double o = __shfl_up(v, off, 64);
    if (lane >= off) v += o;
  }
  __syncthreads();   // the last use of lds is over
  if (lane == 63) lds[wv] = v;
  __syncthreads();
  double base = 0.0;
  for (int w = 0; w < wv; ++w) base += lds[w];
  total = ((lds[0] + lds[1]) + lds[2]) + lds[3];
  return v + base;
}
// The lowest index that any thread offers (INT_MAX: none).
__device__ __forceinline__ int block_min(int v, int* lds) {
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) {
    const int o = __shfl_xor(v, off, 64);
    v = o < v ? o : v;
  }
  __syncthreads();
  if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
  __syncthreads();
  int m = lds[0];
  for (int w = 1; w < 4; ++w) m = lds[w] < m ? lds[w] : m;
  return m;
}

__global__ __launch_bounds__(256) void k_verify_draw(const VerifyArgs a, int pieces) {
  __shared__ double lds[4];
  __shared__ int ldsi[4];
  __shared__ double lds_before;
  const int b = blockIdx.x;
  int nd;
  const int n = kept(a, b, nd);
  Row r = row_of(a, b, n, nd);
  const double* sums = (const double*)a.workspace + (int64_t)b * pieces * 2;
  // totals of the weights and of p: every thread a run of pieces
  const int per = (pieces + 255) / 256;
  const int i0 = threadIdx.x * per;
  double mine = 0.0, mine_p = 0.0;
  for (int i = i0; i < i0 + per && i < pieces; ++i) {
    mine += sums[2 * i];
    mine_p += sums[2 * i + 1];
  }
  double total, total_p;
  double incl = block_scan(mine, lds, total);
  const double incl_p = block_scan(mine_p, lds, total_p);
  int which = 0;
  if (!(total > 0.0)) {   // p <= q everywhere: draw from p
    which = 1;
    r.q = nullptr;
    r.cut = -1;
    incl = incl_p;
    mine = mine_p;
    total = total_p;
  }
  const double target = (double)a.u_sample[b] * total;
  // the piece: the first whose inclusive sum passes the target
  int found = 0x7FFFFFFF;
  double before = incl - mine;
  if (incl > target) {
    double run = before;
    for (int i = i0; i < i0 + per && i < pieces; ++i) {
      const double next = run + sums[2 * i + which];
      if (next > target) {
        found = i;
        before = run;
        break;
      }
      run = next;
    }
    if (found == 0x7FFFFFFF) {   // a rounding apart from the scan's own sum
      const int last = i0 + per < pieces ? i0 + per : pieces;
      found = last - 1;
      before = run - sums[2 * found + which];
    }
  }
  const int piece = block_min(found, ldsi);
  if (piece == 0x7FFFFFFF) {   // nothing passes: u >= 1, or no probability at all
    if (threadIdx.x == 0) a.tokens[(int64_t)b * (a.Q + 1) + n] = (int)a.V - 1;
    return;
  }
  if (found == piece) lds_before = before;
  __syncthreads();
  before = lds_before;
  // the token: 8 consecutive values per thread
  const int64_t v0 = (int64_t)piece * kPiece + threadIdx.x * kPer;
  double w[kPer], sum = 0.0;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    w[i] = v0 + i < a.V ? weight(r, v0 + i, r.p[v0 + i]) : 0.0;
    sum += w[i];
  }
  double all;
  const double upto = block_scan(sum, lds, all) + before;
  int token = 0x7FFFFFFF, last = -1;
  double run = upto - sum;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    run += w[i];
    if (w[i] > 0.0) last = (int)(v0 + i);
    if (token == 0x7FFFFFFF && run > target && w[i] > 0.0) token = (int)(v0 + i);
  }
  const int pick = block_min(token, ldsi);
  const int end = -block_min(-last, ldsi);   // the piece's last value with a weight
  if (threadIdx.x == 0)
    a.tokens[(int64_t)b * (a.Q + 1) + n] = pick != 0x7FFFFFFF ? pick : end >= 0 ? end : (int)a.V - 1;
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
