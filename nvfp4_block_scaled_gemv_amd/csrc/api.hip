// api.hip -- the extern "C" boundary: host-side argument checks, then the
// launches on the caller's stream. No allocation, no synchronisation.
#include <stdarg.h>
#include <stdio.h>
#include <string.h>

#include <mutex>

#include "nvfp4_gemv.h"
#include "internal.h"

static_assert(NVFP4_MAX_M == NVFP4_MAX_M_INTERNAL, "M limit mismatch");
static_assert(NVFP4_MOE_MAX_M == NVFP4_MOE_MAX_M_INTERNAL, "MoE M limit mismatch");
static_assert(NVFP4_MAX_TOPK == NVFP4_MAX_TOPK_INTERNAL, "topk limit mismatch");

namespace {

thread_local char g_last_error[512] = "";

nvfp4_status fail(nvfp4_status st, const char* fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(g_last_error, sizeof(g_last_error), fmt, ap);
  va_end(ap);
  return st;
}

void clear_error() { g_last_error[0] = '\0'; }

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// [a, a + na) and [b, b + nb) share a byte.
bool overlap(const void* a, size_t na, const void* b, size_t nb) {
  if (!a || !b || na == 0 || nb == 0) return false;
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x < y + nb && y < x + na;
}

nvfp4_status hip_result(hipError_t e, const char* what) {
  if (e != hipSuccess)
    return fail(NVFP4_ERR_HIP, "%s: %s (%s)", what, hipGetErrorName(e), hipGetErrorString(e));
  return NVFP4_OK;
}

}  // namespace

static_assert(NVFP4_MAX_SEGMENTS == nvfp4::kMaxSegments, "segment limit mismatch");

extern "C" {

int nvfp4_abi_version(void) { return NVFP4_ABI_VERSION; }

const char* nvfp4_status_string(int status) {
  switch (status) {
    case NVFP4_OK: return "ok";
    case NVFP4_ERR_NULL: return "null pointer";
    case NVFP4_ERR_SHAPE: return "invalid shape";
    case NVFP4_ERR_ALIGN: return "misaligned pointer";
    case NVFP4_ERR_UNSUPPORTED: return "unsupported size";
    case NVFP4_ERR_WORKSPACE: return "workspace too small";
    case NVFP4_ERR_HIP: return "HIP error";
    case NVFP4_ERR_ALIAS: return "output overlaps an input";
    default: return "unknown status";
  }
}

const char* nvfp4_last_error(void) { return g_last_error; }

nvfp4_status nvfp4_pack(const float* W, int64_t N, int64_t K, uint8_t* codes,
                        uint8_t* scales, float* gscale, const float* gscale_override,
                        hipStream_t stream) {
  clear_error();
  if (N < 0 || K < 0 || (K % 16) != 0)
    return fail(NVFP4_ERR_SHAPE, "nvfp4_pack: need N >= 0, K >= 0, K %% 16 == 0 (N=%lld K=%lld)",
                (long long)N, (long long)K);
  const size_t numel = (size_t)N * (size_t)K;
  if (!gscale || (numel && (!W || !codes || !scales)))
    return fail(NVFP4_ERR_NULL, "nvfp4_pack: W, codes, scales and gscale must be non-NULL");
  if (!aligned(W, 16) || !aligned(codes, 8) || !aligned(gscale, 4) ||
      (gscale_override && !aligned(gscale_override, 4)))
    return fail(NVFP4_ERR_ALIGN, "nvfp4_pack: W must be 16-byte, codes 8-byte, gscale 4-byte aligned");
  const size_t wb = numel * 4, cb = numel / 2, sb = numel / 16;
  if (overlap(codes, cb, W, wb) || overlap(scales, sb, W, wb) || overlap(gscale, 4, W, wb) ||
      overlap(codes, cb, scales, sb) || overlap(codes, cb, gscale, 4) ||
      overlap(scales, sb, gscale, 4) || overlap(gscale, 4, gscale_override, 4))
    return fail(NVFP4_ERR_ALIAS, "nvfp4_pack: outputs overlap each other or an input");
  return hip_result(nvfp4::launch_pack(W, N, K, codes, scales, gscale, gscale_override, stream),
                    "nvfp4_pack launch");
}

nvfp4_status nvfp4_dequant(const uint8_t* codes, const uint8_t* scales, const float* gscale,
                           int64_t N, int64_t K, float* W_out, hipStream_t stream) {
  clear_error();
  if (N < 0 || K < 0 || (K % 32) != 0)
    return fail(NVFP4_ERR_SHAPE, "nvfp4_dequant: need N >= 0, K >= 0, K %% 32 == 0 (N=%lld K=%lld)",
                (long long)N, (long long)K);
  const size_t numel = (size_t)N * (size_t)K;
  if (numel == 0) return NVFP4_OK;
  if (!codes || !scales || !gscale || !W_out)
    return fail(NVFP4_ERR_NULL, "nvfp4_dequant: NULL pointer");
  if (!aligned(codes, 16) || !aligned(W_out, 16) || !aligned(gscale, 4))
    return fail(NVFP4_ERR_ALIGN, "nvfp4_dequant: codes and W_out must be 16-byte aligned");
  if (overlap(W_out, numel * 4, codes, numel / 2) || overlap(W_out, numel * 4, scales, numel / 16) ||
      overlap(W_out, numel * 4, gscale, 4))
    return fail(NVFP4_ERR_ALIAS, "nvfp4_dequant: W_out overlaps an input");
  return hip_result(nvfp4::launch_dequant(codes, scales, gscale, N, K, W_out, stream),
                    "nvfp4_dequant launch");
}

nvfp4_status nvfp4_gemv(const uint8_t* codes, const uint8_t* scales, const float* gscale,
                        const uint16_t* x, int64_t M, int64_t N, int64_t K, float* y,
                        hipStream_t stream) {
  clear_error();
  if (M < 0 || N < 0 || K < 0 || (K % 32) != 0)
    return fail(NVFP4_ERR_SHAPE, "nvfp4_gemv: need M, N, K >= 0 and K %% 32 == 0 (M=%lld N=%lld K=%lld)",
                (long long)M, (long long)N, (long long)K);
  if (M > NVFP4_MAX_M || N > NVFP4_MAX_N || K > NVFP4_MAX_K)
    return fail(NVFP4_ERR_UNSUPPORTED,
                "nvfp4_gemv: M=%lld (max %d), N=%lld (max %lld), K=%lld (max %lld)",
                (long long)M, NVFP4_MAX_M, (long long)N, (long long)NVFP4_MAX_N, (long long)K,
                (long long)NVFP4_MAX_K);
  if (M == 0 || N == 0) return NVFP4_OK;
  if (!y) return fail(NVFP4_ERR_NULL, "nvfp4_gemv: y is NULL");
  if (!aligned(y, 4)) return fail(NVFP4_ERR_ALIGN, "nvfp4_gemv: y must be 4-byte aligned");
  const size_t yb = (size_t)M * (size_t)N * 4;
  if (K == 0) return hip_result(nvfp4::launch_fill_zero(y, (size_t)M * (size_t)N, stream),
                                "nvfp4_gemv zero fill");
  if (!codes || !scales || !gscale || !x) return fail(NVFP4_ERR_NULL, "nvfp4_gemv: NULL input");
  if (!aligned(codes, 16) || !aligned(scales, 2) || !aligned(x, 16) || !aligned(gscale, 4))
    return fail(NVFP4_ERR_ALIGN,
                "nvfp4_gemv: codes and x must be 16-byte, scales 2-byte, gscale 4-byte aligned");
  const size_t nk = (size_t)N * (size_t)K;
  if (overlap(y, yb, codes, nk / 2) || overlap(y, yb, scales, nk / 16) ||
      overlap(y, yb, gscale, 4) || overlap(y, yb, x, (size_t)M * (size_t)K * 2))
    return fail(NVFP4_ERR_ALIAS, "nvfp4_gemv: y overlaps an input");
  return hip_result(nvfp4::launch_gemv(codes, scales, gscale, x, (int)M, N, K, y, stream),
                    "nvfp4_gemv launch");
}

nvfp4_status nvfp4_gemv_segments(const nvfp4_gemv_segment* segs, int64_t n_segments,
                                 const uint16_t* x, int64_t M, int64_t K, hipStream_t stream) {
  clear_error();
  if (n_segments < 0 || M < 0 || K < 0 || (K % 32) != 0)
    return fail(NVFP4_ERR_SHAPE,
                "nvfp4_gemv_segments: need n_segments, M, K >= 0 and K %% 32 == 0 "
                "(n=%lld M=%lld K=%lld)",
                (long long)n_segments, (long long)M, (long long)K);
  if (n_segments > NVFP4_MAX_SEGMENTS || M > NVFP4_MAX_M || K > NVFP4_MAX_K)
    return fail(NVFP4_ERR_UNSUPPORTED,
                "nvfp4_gemv_segments: n_segments=%lld (max %d), M=%lld (max %d), K=%lld (max %lld)",
                (long long)n_segments, NVFP4_MAX_SEGMENTS, (long long)M, NVFP4_MAX_M,
                (long long)K, (long long)NVFP4_MAX_K);
  if (n_segments == 0 || M == 0) return NVFP4_OK;
  if (!segs) return fail(NVFP4_ERR_NULL, "nvfp4_gemv_segments: segs is NULL");
  nvfp4::SegDesc d[NVFP4_MAX_SEGMENTS];
  int n = 0;
  int64_t total_n = 0;
  for (int64_t s = 0; s < n_segments; ++s) {
    const nvfp4_gemv_segment& g = segs[s];
    if (g.N < 0)
      return fail(NVFP4_ERR_SHAPE, "nvfp4_gemv_segments: segment %lld has N=%lld < 0",
                  (long long)s, (long long)g.N);
    if (g.N > NVFP4_MAX_N - total_n)
      return fail(NVFP4_ERR_UNSUPPORTED, "nvfp4_gemv_segments: the segments' N exceed %lld",
                  (long long)NVFP4_MAX_N);
    total_n += g.N;
    if (g.N == 0) continue;
    if (!g.y) return fail(NVFP4_ERR_NULL, "nvfp4_gemv_segments: segment %lld y is NULL", (long long)s);
    if (!aligned(g.y, 4))
      return fail(NVFP4_ERR_ALIGN, "nvfp4_gemv_segments: segment %lld y must be 4-byte aligned",
                  (long long)s);
    if (K > 0) {
      if (!g.codes || !g.scales || !g.gscale || !x)
        return fail(NVFP4_ERR_NULL, "nvfp4_gemv_segments: segment %lld has a NULL input",
                    (long long)s);
      if (!aligned(g.codes, 16) || !aligned(g.scales, 2) || !aligned(g.gscale, 4) ||
          !aligned(x, 16))
        return fail(NVFP4_ERR_ALIGN,
                    "nvfp4_gemv_segments: segment %lld: codes and x must be 16-byte, scales "
                    "2-byte, gscale 4-byte aligned", (long long)s);
    }
    d[n++] = {g.codes, g.scales, g.gscale, g.y, g.N};
  }
  if (n == 0) return NVFP4_OK;
  // no output may overlap any input or another output
  for (int a = 0; a < n; ++a) {
    const size_t ya = (size_t)M * (size_t)d[a].N * 4;
    if (K > 0 && overlap(d[a].y, ya, x, (size_t)M * (size_t)K * 2))
      return fail(NVFP4_ERR_ALIAS, "nvfp4_gemv_segments: an output overlaps x");
    for (int b = 0; b < n; ++b) {
      const size_t nk = (size_t)d[b].N * (size_t)K;
      if (K > 0 && (overlap(d[a].y, ya, d[b].codes, nk / 2) ||
                    overlap(d[a].y, ya, d[b].scales, nk / 16) ||
                    overlap(d[a].y, ya, d[b].gscale, 4)))
        return fail(NVFP4_ERR_ALIAS, "nvfp4_gemv_segments: an output overlaps an input");
      if (b != a && overlap(d[a].y, ya, d[b].y, (size_t)M * (size_t)d[b].N * 4))
        return fail(NVFP4_ERR_ALIAS, "nvfp4_gemv_segments: two outputs overlap");
    }
  }
  if (K == 0) {
    for (int a = 0; a < n; ++a) {
      const nvfp4_status st =
          hip_result(nvfp4::launch_fill_zero(d[a].y, (size_t)M * (size_t)d[a].N, stream),
                     "nvfp4_gemv_segments zero fill");
      if (st != NVFP4_OK) return st;
    }
    return NVFP4_OK;
  }
  return hip_result(nvfp4::launch_gemv_segments(d, n, x, (int)M, K, stream),
                    "nvfp4_gemv_segments launch");
}

nvfp4_status nvfp4_quantize_act(const uint16_t* x, int64_t M, int64_t K, const float* gscale_x,
                                uint8_t* codes_x, uint8_t* scales_x, hipStream_t stream) {
  clear_error();
  if (M < 0 || K < 0 || (K % 32) != 0)
    return fail(NVFP4_ERR_SHAPE,
                "nvfp4_quantize_act: need M, K >= 0 and K %% 32 == 0 (M=%lld K=%lld)",
                (long long)M, (long long)K);
  const size_t numel = (size_t)M * (size_t)K;
  if (numel == 0) return NVFP4_OK;
  if (!x || !gscale_x || !codes_x || !scales_x)
    return fail(NVFP4_ERR_NULL, "nvfp4_quantize_act: NULL pointer");
  if (!aligned(x, 16) || !aligned(codes_x, 8) || !aligned(gscale_x, 4))
    return fail(NVFP4_ERR_ALIGN,
                "nvfp4_quantize_act: x must be 16-byte, codes 8-byte, gscale_x 4-byte aligned");
  const size_t xb = numel * 2, cb = numel / 2, sb = numel / 16;
  if (overlap(codes_x, cb, x, xb) || overlap(scales_x, sb, x, xb) ||
      overlap(codes_x, cb, gscale_x, 4) || overlap(scales_x, sb, gscale_x, 4) ||
      overlap(codes_x, cb, scales_x, sb))
    return fail(NVFP4_ERR_ALIAS, "nvfp4_quantize_act: outputs overlap each other or an input");
  return hip_result(nvfp4::launch_quantize_act(x, M, K, gscale_x, codes_x, scales_x, stream),
                    "nvfp4_quantize_act launch");
}

size_t nvfp4_gemv_w4a4_workspace_bytes(int64_t M, int64_t K) {
  if (M < 0 || K < 0) return 0;
  return nvfp4::w4a4_layout(M, K).total;
}

nvfp4_status nvfp4_gemv_w4a4(const uint8_t* codes_w, const uint8_t* scales_w,
                             const float* gscale_w, const uint8_t* codes_x,
                             const uint8_t* scales_x, const float* gscale_x, int64_t M,
                             int64_t N, int64_t K, float* y, void* workspace,
                             size_t workspace_bytes, hipStream_t stream) {
  clear_error();
  if (M < 0 || N < 0 || K < 0 || (K % 32) != 0)
    return fail(NVFP4_ERR_SHAPE,
                "nvfp4_gemv_w4a4: need M, N, K >= 0 and K %% 32 == 0 (M=%lld N=%lld K=%lld)",
                (long long)M, (long long)N, (long long)K);
  if (M > NVFP4_MAX_M || N > NVFP4_MAX_N || K > NVFP4_MAX_K)
    return fail(NVFP4_ERR_UNSUPPORTED,
                "nvfp4_gemv_w4a4: M=%lld (max %d), N=%lld (max %lld), K=%lld (max %lld)",
                (long long)M, NVFP4_MAX_M, (long long)N, (long long)NVFP4_MAX_N, (long long)K,
                (long long)NVFP4_MAX_K);
  if (M == 0 || N == 0) return NVFP4_OK;
  if (!y) return fail(NVFP4_ERR_NULL, "nvfp4_gemv_w4a4: y is NULL");
  if (!aligned(y, 4)) return fail(NVFP4_ERR_ALIGN, "nvfp4_gemv_w4a4: y must be 4-byte aligned");
  const size_t yb = (size_t)M * (size_t)N * 4;
  if (K == 0) return hip_result(nvfp4::launch_fill_zero(y, (size_t)M * (size_t)N, stream),
                                "nvfp4_gemv_w4a4 zero fill");
  if (!codes_w || !scales_w || !gscale_w || !codes_x || !scales_x || !gscale_x)
    return fail(NVFP4_ERR_NULL, "nvfp4_gemv_w4a4: NULL input");
  const size_t need = nvfp4::w4a4_layout(M, K).total;
  if (!workspace || workspace_bytes < need)
    return fail(NVFP4_ERR_WORKSPACE, "nvfp4_gemv_w4a4: workspace of %zu bytes needed, %zu given",
                need, workspace ? workspace_bytes : (size_t)0);
  if (!aligned(codes_w, 16) || !aligned(scales_w, 2) || !aligned(gscale_w, 4) ||
      !aligned(codes_x, 16) || !aligned(scales_x, 2) || !aligned(gscale_x, 4) ||
      !aligned(workspace, 256))
    return fail(NVFP4_ERR_ALIGN,
                "nvfp4_gemv_w4a4: codes 16-byte, scales 2-byte, scales of the tensors 4-byte, "
                "workspace 256-byte aligned");
  const size_t nk = (size_t)N * (size_t)K, mk = (size_t)M * (size_t)K;
  const void* ins[] = {codes_w, scales_w, gscale_w, codes_x, scales_x, gscale_x};
  const size_t insz[] = {nk / 2, nk / 16, 4, mk / 2, mk / 16, 4};
  for (int i = 0; i < 6; ++i)
    if (overlap(y, yb, ins[i], insz[i]) || overlap(workspace, need, ins[i], insz[i]))
      return fail(NVFP4_ERR_ALIAS, "nvfp4_gemv_w4a4: y or workspace overlaps input %d", i);
  if (overlap(y, yb, workspace, need))
    return fail(NVFP4_ERR_ALIAS, "nvfp4_gemv_w4a4: y overlaps the workspace");
  return hip_result(nvfp4::launch_gemv_w4a4(codes_w, scales_w, gscale_w, codes_x, scales_x,
                                            gscale_x, (int)M, N, K, y, workspace, stream),
                    "nvfp4_gemv_w4a4 launch");
}

nvfp4_status nvfp4_gemv_w4a4_segments(const nvfp4_gemv_segment* segs, int64_t n_segments,
                                      const uint8_t* codes_x, const uint8_t* scales_x,
                                      const float* gscale_x, int64_t M, int64_t K,
                                      void* workspace, size_t workspace_bytes,
                                      hipStream_t stream) {
  clear_error();
  const char* fn = "nvfp4_gemv_w4a4_segments";
  if (n_segments < 0 || M < 0 || K < 0 || (K % 32) != 0)
    return fail(NVFP4_ERR_SHAPE, "%s: need n_segments, M, K >= 0 and K %% 32 == 0 "
                "(n=%lld M=%lld K=%lld)", fn, (long long)n_segments, (long long)M, (long long)K);
  if (n_segments > NVFP4_MAX_SEGMENTS || M > NVFP4_MAX_M || K > NVFP4_MAX_K)
    return fail(NVFP4_ERR_UNSUPPORTED, "%s: n_segments=%lld (max %d), M=%lld (max %d), K=%lld (max %lld)",
                fn, (long long)n_segments, NVFP4_MAX_SEGMENTS, (long long)M, NVFP4_MAX_M,
                (long long)K, (long long)NVFP4_MAX_K);
  if (n_segments == 0 || M == 0) return NVFP4_OK;
  if (!segs) return fail(NVFP4_ERR_NULL, "%s: segs is NULL", fn);
  nvfp4::SegDesc d[NVFP4_MAX_SEGMENTS];
  int n = 0;
  int64_t total_n = 0;
  for (int64_t s = 0; s < n_segments; ++s) {
    const nvfp4_gemv_segment& g = segs[s];
    if (g.N < 0)
      return fail(NVFP4_ERR_SHAPE, "%s: segment %lld has N=%lld < 0", fn, (long long)s,
                  (long long)g.N);
    if (g.N > NVFP4_MAX_N - total_n)
      return fail(NVFP4_ERR_UNSUPPORTED, "%s: the segments' N exceed %lld", fn,
                  (long long)NVFP4_MAX_N);
    total_n += g.N;
    if (g.N == 0) continue;
    if (!g.y) return fail(NVFP4_ERR_NULL, "%s: segment %lld y is NULL", fn, (long long)s);
    if (!aligned(g.y, 4))
      return fail(NVFP4_ERR_ALIGN, "%s: segment %lld y must be 4-byte aligned", fn,
                  (long long)s);
    if (K > 0) {
      if (!g.codes || !g.scales || !g.gscale)
        return fail(NVFP4_ERR_NULL, "%s: segment %lld has a NULL input", fn, (long long)s);
      if (!aligned(g.codes, 16) || !aligned(g.scales, 2) || !aligned(g.gscale, 4))
        return fail(NVFP4_ERR_ALIGN, "%s: segment %lld: codes must be 16-byte, scales 2-byte, "
                    "gscale 4-byte aligned", fn, (long long)s);
    }
    d[n++] = {g.codes, g.scales, g.gscale, g.y, g.N};
  }
  if (n == 0) return NVFP4_OK;
  if (K > 0) {
    if (!codes_x || !scales_x || !gscale_x)
      return fail(NVFP4_ERR_NULL, "%s: NULL activation input", fn);
    if (!aligned(codes_x, 16) || !aligned(scales_x, 2) || !aligned(gscale_x, 4))
      return fail(NVFP4_ERR_ALIGN, "%s: codes_x 16-byte, scales_x 2-byte, gscale_x 4-byte "
                  "aligned", fn);
  }
  const size_t need = nvfp4::w4a4_layout(M, K).total;
  if (K > 0) {
    if (!workspace || workspace_bytes < need)
      return fail(NVFP4_ERR_WORKSPACE, "%s: workspace of %zu bytes needed, %zu given", fn, need,
                  workspace ? workspace_bytes : (size_t)0);
    if (!aligned(workspace, 256))
      return fail(NVFP4_ERR_ALIGN, "%s: workspace must be 256-byte aligned", fn);
  }
  // no output (or the workspace) may overlap any input, another output or the workspace
  const size_t mk = (size_t)M * (size_t)K;
  for (int a = 0; a < n; ++a) {
    const size_t ya = (size_t)M * (size_t)d[a].N * 4;
    if (K > 0 && (overlap(d[a].y, ya, codes_x, mk / 2) || overlap(d[a].y, ya, scales_x, mk / 16) ||
                  overlap(d[a].y, ya, gscale_x, 4) || overlap(d[a].y, ya, workspace, need)))
      return fail(NVFP4_ERR_ALIAS, "%s: an output overlaps the activations or the workspace", fn);
    for (int b = 0; b < n; ++b) {
      const size_t nk = (size_t)d[b].N * (size_t)K;
      if (K > 0 && (overlap(d[a].y, ya, d[b].codes, nk / 2) ||
                    overlap(d[a].y, ya, d[b].scales, nk / 16) ||
                    overlap(d[a].y, ya, d[b].gscale, 4)))
        return fail(NVFP4_ERR_ALIAS, "%s: an output overlaps an input", fn);
      if (K > 0 && (overlap(workspace, need, d[b].codes, nk / 2) ||
                    overlap(workspace, need, d[b].scales, nk / 16) ||
                    overlap(workspace, need, d[b].gscale, 4)))
        return fail(NVFP4_ERR_ALIAS, "%s: the workspace overlaps an input", fn);
      if (b != a && overlap(d[a].y, ya, d[b].y, (size_t)M * (size_t)d[b].N * 4))
        return fail(NVFP4_ERR_ALIAS, "%s: two outputs overlap", fn);
    }
  }
  if (K > 0 && (overlap(workspace, need, codes_x, mk / 2) ||
                overlap(workspace, need, scales_x, mk / 16) || overlap(workspace, need, gscale_x, 4)))
    return fail(NVFP4_ERR_ALIAS, "%s: the workspace overlaps the activations", fn);
  if (K == 0) {
    for (int a = 0; a < n; ++a) {
      const nvfp4_status st =
          hip_result(nvfp4::launch_fill_zero(d[a].y, (size_t)M * (size_t)d[a].N, stream),
                     "nvfp4_gemv_w4a4_segments zero fill");
      if (st != NVFP4_OK) return st;
    }
    return NVFP4_OK;
  }
  return hip_result(nvfp4::launch_gemv_w4a4_segments(d, n, codes_x, scales_x, gscale_x, (int)M,
                                                     K, workspace, stream),
                    "nvfp4_gemv_w4a4_segments launch");
}

namespace {

// The checks that the three norm entry points share. `y` (yb bytes, aligned to
// ya) and `extra` (eb bytes, an output, 4-byte aligned) are theirs; extra_in:
// a float[1] input.
nvfp4_status norm_checks(const char* fn, const void* x, int x_type, const void* residual,
                         void* residual_out, int residual_type, const uint16_t* weight,
                         float eps, int64_t M, int64_t H, int64_t unit, const void* y, size_t yb,
                         size_t ya, const void* extra, size_t eb, size_t ea,
                         const float* extra_in, nvfp4::NormArgs* a, bool* nothing) {
  *nothing = false;
  if (M < 0 || H < 0 || H % unit != 0)
    return fail(NVFP4_ERR_SHAPE, "%s: need M, H >= 0 and H %% %lld == 0 (M=%lld H=%lld)", fn,
                (long long)unit, (long long)M, (long long)H);
  if ((x_type != NVFP4_BF16 && x_type != NVFP4_F32) ||
      (residual && residual_type != NVFP4_BF16 && residual_type != NVFP4_F32))
    return fail(NVFP4_ERR_SHAPE, "%s: x and residual are bf16 or fp32 (types %d, %d)", fn, x_type,
                residual_type);
  if (!(eps >= 0.0f) || eps > 3.0e38f)
    return fail(NVFP4_ERR_SHAPE, "%s: eps must be finite and >= 0", fn);
  if (M > NVFP4_MAX_ROWS || H > NVFP4_NORM_MAX_H)
    return fail(NVFP4_ERR_UNSUPPORTED, "%s: M=%lld (max %d), H=%lld (max %d)", fn, (long long)M,
                NVFP4_MAX_ROWS, (long long)H, NVFP4_NORM_MAX_H);
  if (M == 0 || H == 0) {
    *nothing = true;
    return NVFP4_OK;
  }
  if (!x || !weight || !y || (ea && !extra) || (!residual) != (!residual_out))
    return fail(NVFP4_ERR_NULL, "%s: NULL pointer (residual and residual_out go together)", fn);
  if (!aligned(x, 16) || !aligned(residual, 16) || !aligned(residual_out, 16) ||
      !aligned(weight, 16) || !aligned(y, ya) || (ea && !aligned(extra, ea)) ||
      !aligned(extra_in, 4))
    return fail(NVFP4_ERR_ALIGN,
                "%s: x, residual, residual_out and weight must be 16-byte aligned, the output "
                "%d-byte", fn, (int)ya);
  const size_t numel = (size_t)M * (size_t)H;
  const size_t xb = numel * (x_type == NVFP4_F32 ? 4 : 2);
  const size_t rb = residual ? numel * (residual_type == NVFP4_F32 ? 4 : 2) : 0;
  const size_t wb = (size_t)H * 2;
  const void* outs[3] = {y, extra, residual_out};
  const size_t ob[3] = {yb, eb, rb};
  for (int i = 0; i < 3; ++i) {
    if (overlap(outs[i], ob[i], x, xb) || overlap(outs[i], ob[i], weight, wb) ||
        overlap(outs[i], ob[i], extra_in, 4) ||
        (outs[i] != residual && overlap(outs[i], ob[i], residual, rb)) ||
        (i < 2 && outs[i] == residual && overlap(outs[i], ob[i], residual, rb)))
      return fail(NVFP4_ERR_ALIAS, "%s: an output overlaps an input", fn);
    for (int j = 0; j < i; ++j)
      if (overlap(outs[i], ob[i], outs[j], ob[j]))
        return fail(NVFP4_ERR_ALIAS, "%s: two outputs overlap", fn);
  }
  *a = {};
  a->x = x;
  a->residual = residual;
  a->residual_out = residual_out;
  a->weight = weight;
  a->M = M;
  a->H = H;
  a->eps = eps;
  a->x_f32 = x_type == NVFP4_F32;
  a->residual_f32 = residual_type == NVFP4_F32;
  a->out = const_cast<void*>(y);
  a->out_scales = const_cast<void*>(extra);
  return NVFP4_OK;
}

}  // namespace

nvfp4_status nvfp4_add_rmsnorm(const void* x, int x_type, const void* residual,
                               void* residual_out, int residual_type, const uint16_t* weight,
                               float eps, int64_t M, int64_t H, uint16_t* y, hipStream_t stream) {
  clear_error();
  nvfp4::NormArgs a;
  bool nothing;
  const size_t numel = M > 0 && H > 0 ? (size_t)M * (size_t)H : 0;
  const nvfp4_status st =
      norm_checks("nvfp4_add_rmsnorm", x, x_type, residual, residual_out, residual_type, weight,
                  eps, M, H, 8, y, numel * 2, 16, nullptr, 0, 0, nullptr, &a, &nothing);
  if (st != NVFP4_OK || nothing) return st;
  a.form = nvfp4::NormForm::bf16;
  return hip_result(nvfp4::launch_add_rmsnorm(a, stream), "nvfp4_add_rmsnorm launch");
}

nvfp4_status nvfp4_add_rmsnorm_e4m3(const void* x, int x_type, const void* residual,
                                    void* residual_out, int residual_type,
                                    const uint16_t* weight, float eps, int64_t M, int64_t H,
                                    int64_t group, uint8_t* y8, float* scales,
                                    hipStream_t stream) {
  clear_error();
  if ((group != 0 && group != 32 && group != 64 && group != 128) ||
      (group != 0 && H % group != 0))
    return fail(NVFP4_ERR_SHAPE,
                "nvfp4_add_rmsnorm_e4m3: group must be 0, 32, 64 or 128 and divide H "
                "(group=%lld H=%lld)", (long long)group, (long long)H);
  nvfp4::NormArgs a;
  bool nothing;
  const size_t numel = M > 0 && H > 0 ? (size_t)M * (size_t)H : 0;
  const nvfp4_status st =
      norm_checks("nvfp4_add_rmsnorm_e4m3", x, x_type, residual, residual_out, residual_type,
                  weight, eps, M, H, 8, y8, numel, 8, scales,
                  group ? numel / (size_t)group * 4 : M > 0 ? (size_t)M * 4 : 0, 4, nullptr, &a,
                  &nothing);
  if (st != NVFP4_OK || nothing) return st;
  a.form = nvfp4::NormForm::e4m3;
  a.group = (int)group;
  return hip_result(nvfp4::launch_add_rmsnorm(a, stream), "nvfp4_add_rmsnorm_e4m3 launch");
}

nvfp4_status nvfp4_add_rmsnorm_nvfp4(const void* x, int x_type, const void* residual,
                                     void* residual_out, int residual_type,
                                     const uint16_t* weight, float eps, int64_t M, int64_t H,
                                     const float* gscale, uint8_t* codes, uint8_t* scales,
                                     hipStream_t stream) {
  clear_error();
  nvfp4::NormArgs a;
  bool nothing;
  const size_t numel = M > 0 && H > 0 ? (size_t)M * (size_t)H : 0;
  const nvfp4_status st =
      norm_checks("nvfp4_add_rmsnorm_nvfp4", x, x_type, residual, residual_out, residual_type,
                  weight, eps, M, H, 32, codes, numel / 2, 8, scales, numel / 16, 1, gscale, &a,
                  &nothing);
  if (st != NVFP4_OK || nothing) return st;
  if (!gscale) return fail(NVFP4_ERR_NULL, "nvfp4_add_rmsnorm_nvfp4: gscale is NULL");
  a.form = nvfp4::NormForm::nvfp4;
  a.gscale = gscale;
  return hip_result(nvfp4::launch_add_rmsnorm(a, stream), "nvfp4_add_rmsnorm_nvfp4 launch");
}

}  // extern "C"

namespace {

// Bytes from a cache's first to past its last element (0: none).
size_t cache_bytes(const nvfp4_kv_cache& c) {
  if (c.num_blocks == 0) return 0;
  const int64_t last = (c.num_blocks - 1) * c.stride_block + (c.page - 1) * c.stride_token +
                       (c.n_kv_heads - 1) * c.stride_head + c.D;
  return (size_t)last * (c.type == NVFP4_E4M3 ? 1 : 2);
}

nvfp4_status cache_checks(const char* fn, const nvfp4_kv_cache& c) {
  if (c.type != NVFP4_BF16 && c.type != NVFP4_E4M3)
    return fail(NVFP4_ERR_SHAPE, "%s: the cache is bf16 or E4M3 (type %d)", fn, c.type);
  const int64_t unit = c.type == NVFP4_E4M3 ? 16 : 8;
  if (c.num_blocks < 0 || c.page < 1 || c.n_kv_heads < 1 || c.D < 1 || c.stride_block < c.D ||
      c.stride_token < c.D || c.stride_head < c.D || c.stride_block % unit ||
      c.stride_token % unit || c.stride_head % unit)
    return fail(NVFP4_ERR_SHAPE,
                "%s: cache num_blocks=%lld page=%lld heads=%lld D=%lld: need num_blocks >= 0, the "
                "others >= 1, and strides (%lld, %lld, %lld) >= D, multiples of %lld", fn,
                (long long)c.num_blocks, (long long)c.page, (long long)c.n_kv_heads,
                (long long)c.D, (long long)c.stride_block, (long long)c.stride_token,
                (long long)c.stride_head, (long long)unit);
  if (c.num_blocks > 0x7FFFFFFF || c.page > (1 << 20) || c.n_kv_heads > NVFP4_MAX_HEADS ||
      c.D > NVFP4_ROPE_MAX_D || c.stride_token >= (1 << 26) || c.stride_head >= (1LL << 40) ||
      c.stride_block >= (1LL << 40) || (__int128)c.num_blocks * c.stride_block >= (1LL << 58))
    return fail(NVFP4_ERR_UNSUPPORTED,
                "%s: cache num_blocks=%lld page=%lld heads=%lld D=%lld stride_token=%lld is past a "
                "limit", fn, (long long)c.num_blocks, (long long)c.page, (long long)c.n_kv_heads,
                (long long)c.D, (long long)c.stride_token);
  // the scales are read also where there is no page
  if (c.type == NVFP4_E4M3 && (!c.k_scale || !c.v_scale))
    return fail(NVFP4_ERR_NULL, "%s: an E4M3 cache needs k_scale and v_scale", fn);
  if (c.type == NVFP4_E4M3 && (!aligned(c.k_scale, 4) || !aligned(c.v_scale, 4)))
    return fail(NVFP4_ERR_ALIGN, "%s: k_scale and v_scale must be 4-byte aligned", fn);
  if (c.num_blocks == 0) return NVFP4_OK;
  if (!c.k || !c.v || c.k == c.v)
    return fail(NVFP4_ERR_NULL, "%s: the cache's k and v must be non-NULL and differ", fn);
  if (!aligned(c.k, 16) || !aligned(c.v, 16))
    return fail(NVFP4_ERR_ALIGN, "%s: the cache must be 16-byte aligned", fn);
  return NVFP4_OK;
}

nvfp4_status cache4_checks(const char* fn, const nvfp4_kv_cache4& c) {
  const int64_t cb = c.D / 2, sb = c.D / 16;   // bytes of a head
  if (c.num_blocks < 0 || c.page < 1 || c.n_kv_heads < 1 || c.D < 1 || c.D % 64 ||
      c.stride_block < cb || c.stride_token < cb || c.stride_head < cb || c.stride_block % 16 ||
      c.stride_token % 16 || c.stride_head % 16 || c.scale_stride_block < sb ||
      c.scale_stride_token < sb || c.scale_stride_head < sb || c.scale_stride_block % 4 ||
      c.scale_stride_token % 4 || c.scale_stride_head % 4)
    return fail(NVFP4_ERR_SHAPE,
                "%s: cache num_blocks=%lld page=%lld heads=%lld D=%lld: need num_blocks >= 0, the "
                "others >= 1, D %% 64 == 0, strides of the codes (%lld, %lld, %lld) >= D / 2, "
                "multiples of 16, and of the scales (%lld, %lld, %lld) >= D / 16, multiples of 4",
                fn, (long long)c.num_blocks, (long long)c.page, (long long)c.n_kv_heads,
                (long long)c.D, (long long)c.stride_block, (long long)c.stride_token,
                (long long)c.stride_head, (long long)c.scale_stride_block,
                (long long)c.scale_stride_token, (long long)c.scale_stride_head);
  const int64_t far = 1LL << 40;
  if (c.num_blocks > 0x7FFFFFFF || c.page > (1 << 20) || c.n_kv_heads > NVFP4_MAX_HEADS ||
      c.D > NVFP4_ROPE_MAX_D || c.stride_token >= (1 << 26) ||
      c.scale_stride_token >= (1 << 26) || c.stride_head >= far || c.stride_block >= 1LL << 35 ||
      c.scale_stride_head >= far || c.scale_stride_block >= 1LL << 33 ||
      (__int128)c.num_blocks * c.stride_block >= (1LL << 58) ||
      (__int128)c.num_blocks * c.scale_stride_block >= (1LL << 58))
    return fail(NVFP4_ERR_UNSUPPORTED,
                "%s: cache num_blocks=%lld page=%lld heads=%lld D=%lld or a stride is past a limit",
                fn, (long long)c.num_blocks, (long long)c.page, (long long)c.n_kv_heads,
                (long long)c.D);
  // the tensor scales are read also where there is no page
  if (!c.k_gscale || !c.v_gscale)
    return fail(NVFP4_ERR_NULL, "%s: the cache's k_gscale or v_gscale is NULL", fn);
  if (!aligned(c.k_gscale, 4) || !aligned(c.v_gscale, 4))
    return fail(NVFP4_ERR_ALIGN, "%s: k_gscale and v_gscale must be 4-byte aligned", fn);
  if (c.num_blocks == 0) return NVFP4_OK;
  if (!c.k || !c.v || !c.k_scales || !c.v_scales || c.k == c.v || c.k_scales == c.v_scales)
    return fail(NVFP4_ERR_NULL,
                "%s: the cache's codes and scales must be non-NULL, and differ for k and v", fn);
  if (!aligned(c.k, 16) || !aligned(c.v, 16) || !aligned(c.k_scales, 4) ||
      !aligned(c.v_scales, 4))
    return fail(NVFP4_ERR_ALIGN,
                "%s: the cache's codes must be 16-byte, its scales 4-byte aligned", fn);
  return NVFP4_OK;
}

// A cache's arrays, whatever it is held in: what a call writes or reads of it,
// and its one or two fp32 scales.
struct CacheArrays {
  const void* p[4];
  size_t n[4];
  const float* scale[2];
};
CacheArrays arrays_of(const nvfp4_kv_cache& c) {
  const size_t n = cache_bytes(c);
  const bool scaled = c.type == NVFP4_E4M3;
  return {{c.k, c.v, nullptr, nullptr},
          {n, n, 0, 0},
          {scaled ? c.k_scale : nullptr, scaled ? c.v_scale : nullptr}};
}
CacheArrays arrays_of(const nvfp4_kv_cache4& c) {
  size_t nc = 0, ns = 0;
  if (c.num_blocks) {
    nc = (size_t)((c.num_blocks - 1) * c.stride_block + (c.page - 1) * c.stride_token +
                  (c.n_kv_heads - 1) * c.stride_head + c.D / 2);
    ns = (size_t)((c.num_blocks - 1) * c.scale_stride_block + (c.page - 1) * c.scale_stride_token +
                  (c.n_kv_heads - 1) * c.scale_stride_head + c.D / 16);
  }
  return {{c.k, c.v, c.k_scales, c.v_scales}, {nc, nc, ns, ns}, {c.k_gscale, c.v_gscale}};
}
// [p, p + n) meets one of the arrays or scales.
bool overlap(const void* p, size_t n, const CacheArrays& c) {
  for (int i = 0; i < 4; ++i)
    if (overlap(p, n, c.p[i], c.n[i])) return true;
  return overlap(p, n, c.scale[0], 4) || overlap(p, n, c.scale[1], 4);
}

// What RopeArgs and AttnArgs (Attn4Args) hold of a cache.
template <class Args>
void put_cache(Args& a, const nvfp4_kv_cache& c) {
  a.cache_e4m3 = c.type == NVFP4_E4M3;
  a.k_cache = c.k;
  a.v_cache = c.v;
  a.num_blocks = c.num_blocks;
  a.page = c.page;
  a.Hkv = c.n_kv_heads;
  a.sb = c.stride_block;
  a.st = c.stride_token;
  a.sh = c.stride_head;
  a.k_scale = a.cache_e4m3 ? c.k_scale : nullptr;
  a.v_scale = a.cache_e4m3 ? c.v_scale : nullptr;
}
template <class Args>
void put_cache(Args& a, const nvfp4_kv_cache4& c) {
  a.cache_nvfp4 = true;
  a.k_cache = c.k;
  a.v_cache = c.v;
  a.k_blocks = c.k_scales;
  a.v_blocks = c.v_scales;
  a.num_blocks = c.num_blocks;
  a.page = c.page;
  a.Hkv = c.n_kv_heads;
  a.sb = c.stride_block;
  a.st = c.stride_token;
  a.sh = c.stride_head;
  a.block_sb = c.scale_stride_block;
  a.block_st = c.scale_stride_token;
  a.block_sh = c.scale_stride_head;
  a.k_scale = c.k_gscale;
  a.v_scale = c.v_gscale;
}
// A cache's attention: its arguments, workspace and launcher.
nvfp4::AttnArgs attn_args(const nvfp4_kv_cache& c) {
  nvfp4::AttnArgs a = {};
  put_cache(a, c);
  return a;
}
nvfp4::Attn4Args attn_args(const nvfp4_kv_cache4& c) {
  nvfp4::Attn4Args a = {};
  put_cache(a, c);
  return a;
}
size_t attn_need(const nvfp4::AttnArgs& a) { return nvfp4::attn_workspace_need(a); }
size_t attn_need(const nvfp4::Attn4Args& a) {
  return nvfp4::attn4_workspace_bytes(a.Hq / a.Hkv * a.Q, a.Hkv, a.D);
}
hipError_t launch_attn(const nvfp4::AttnArgs& a, hipStream_t stream) {
  return nvfp4::launch_paged_attention(a, stream);
}
hipError_t launch_attn(const nvfp4::Attn4Args& a, hipStream_t stream) {
  return nvfp4::launch_paged_attention4(a, stream);
}
nvfp4_status checks_of(const char* fn, const nvfp4_kv_cache& c) { return cache_checks(fn, c); }
nvfp4_status checks_of(const char* fn, const nvfp4_kv_cache4& c) { return cache4_checks(fn, c); }

template <class Cache>
nvfp4_status rope_checked(const char* fn, const void* q, int64_t q_stride, const void* k,
                          int64_t k_stride, const void* v, int64_t v_stride, int x_type,
                          const int64_t* positions, const int64_t* slots, const float* inv_freq,
                          int64_t T, int64_t Hq, int64_t D, int64_t R, int interleaved,
                          float rope_scale, uint16_t* q_out, const Cache* cache,
                          hipStream_t stream) {
  clear_error();
  if (T < 0 || Hq < 0 || D < 16 || D % 16 || R < 0 || R > D || R % 16)
    return fail(NVFP4_ERR_SHAPE,
                "%s: need T, Hq >= 0, D >= 16, 0 <= R <= D, D and R multiples of 16 (T=%lld "
                "Hq=%lld D=%lld R=%lld)", fn, (long long)T, (long long)Hq, (long long)D,
                (long long)R);
  if (x_type != NVFP4_BF16 && x_type != NVFP4_F32)
    return fail(NVFP4_ERR_SHAPE, "%s: q, k and v are bf16 or fp32 (type %d)", fn, x_type);
  if (interleaved != 0 && interleaved != 1)
    return fail(NVFP4_ERR_SHAPE, "%s: interleaved is 0 or 1", fn);
  if (!(rope_scale > -3.0e38f && rope_scale < 3.0e38f))
    return fail(NVFP4_ERR_SHAPE, "%s: rope_scale must be finite", fn);
  if (T > NVFP4_MAX_ROWS || Hq > NVFP4_MAX_HEADS || D > NVFP4_ROPE_MAX_D)
    return fail(NVFP4_ERR_UNSUPPORTED, "%s: T=%lld (max %d), Hq=%lld (max %d), D=%lld (max %d)",
                fn, (long long)T, NVFP4_MAX_ROWS, (long long)Hq, NVFP4_MAX_HEADS, (long long)D,
                NVFP4_ROPE_MAX_D);
  int64_t Hkv = 0;
  if (cache) {
    const nvfp4_status st = checks_of(fn, *cache);
    if (st != NVFP4_OK) return st;
    Hkv = cache->n_kv_heads;
    if (cache->D != D)
      return fail(NVFP4_ERR_SHAPE, "%s: D=%lld, the cache has %lld", fn, (long long)D,
                  (long long)cache->D);
  }
  const int64_t unit = x_type == NVFP4_F32 ? 4 : 8;
  if ((Hq && (q_stride < Hq * D || q_stride % unit)) ||
      (Hkv && (k_stride < Hkv * D || v_stride < Hkv * D || k_stride % unit || v_stride % unit)))
    return fail(NVFP4_ERR_SHAPE,
                "%s: token strides (%lld, %lld, %lld) must hold the heads and be multiples of "
                "%lld", fn, (long long)q_stride, (long long)k_stride, (long long)v_stride,
                (long long)unit);
  const int64_t most = 1LL << 36;
  if (q_stride > most || k_stride > most || v_stride > most)
    return fail(NVFP4_ERR_UNSUPPORTED, "%s: a token stride is past %lld", fn, (long long)most);
  if (T == 0 || (Hq == 0 && Hkv == 0)) return NVFP4_OK;
  if ((Hq && (!q || !q_out)) || (Hkv && (!k || !v || !slots)) || !positions ||
      (R > 0 && !inv_freq))
    return fail(NVFP4_ERR_NULL, "%s: NULL pointer", fn);
  if ((Hq && (!aligned(q, 16) || !aligned(q_out, 16))) ||
      (Hkv && (!aligned(k, 16) || !aligned(v, 16) || !aligned(slots, 8))) ||
      !aligned(positions, 8) || !aligned(inv_freq, 4))
    return fail(NVFP4_ERR_ALIGN,
                "%s: q, k, v and q_out must be 16-byte, positions and slots 8-byte aligned", fn);
  const size_t es = x_type == NVFP4_F32 ? 4 : 2;
  const size_t qb = Hq ? ((size_t)(T - 1) * q_stride + Hq * D) * es : 0;
  const size_t kb = Hkv ? ((size_t)(T - 1) * k_stride + Hkv * D) * es : 0;
  const size_t vb = Hkv ? ((size_t)(T - 1) * v_stride + Hkv * D) * es : 0;
  const size_t ob = (size_t)T * Hq * D * 2, tb = (size_t)T * 8, fb = (size_t)R * 2;
  const CacheArrays none = {};
  const CacheArrays ca = cache ? arrays_of(*cache) : none;
  const void* outs[5] = {Hq ? q_out : nullptr, ca.p[0], ca.p[1], ca.p[2], ca.p[3]};
  const size_t obytes[5] = {ob, ca.n[0], ca.n[1], ca.n[2], ca.n[3]};
  for (int i = 0; i < 5; ++i) {
    const void* o = outs[i];
    const size_t n = obytes[i];
    if ((Hq && overlap(o, n, q, qb)) || (Hkv && overlap(o, n, k, kb)) ||
        (Hkv && overlap(o, n, v, vb)) || overlap(o, n, positions, tb) ||
        (Hkv && overlap(o, n, slots, tb)) || overlap(o, n, inv_freq, fb) ||
        overlap(o, n, ca.scale[0], 4) || overlap(o, n, ca.scale[1], 4))
      return fail(NVFP4_ERR_ALIAS, "%s: an output overlaps an input", fn);
    // the cache's arrays may lie in each other's gaps; q_out may not lie in theirs
    if (i > 0 && overlap(o, n, outs[0], ob))
      return fail(NVFP4_ERR_ALIAS, "%s: q_out overlaps the cache", fn);
  }
  nvfp4::RopeArgs a = {};
  a.q = q;
  a.k = k;
  a.v = v;
  a.q_stride = q_stride;
  a.k_stride = k_stride;
  a.v_stride = v_stride;
  a.positions = positions;
  a.slots = slots;
  a.inv_freq = inv_freq;
  a.T = T;
  a.Hq = Hq;
  a.D = D;
  a.R = R;
  a.rope_scale = rope_scale;
  a.x_f32 = x_type == NVFP4_F32;
  a.interleaved = interleaved != 0;
  a.q_out = q_out;
  if (cache) {
    put_cache(a, *cache);
  } else {
    a.page = 1;
  }
  return hip_result(nvfp4::launch_rope_append(a, stream), fn);
}

}  // namespace

extern "C" {

nvfp4_status nvfp4_rope_append(const void* q, int64_t q_stride, const void* k, int64_t k_stride,
                               const void* v, int64_t v_stride, int x_type,
                               const int64_t* positions, const int64_t* slots,
                               const float* inv_freq, int64_t T, int64_t Hq, int64_t D,
                               int64_t R, int interleaved, float rope_scale, uint16_t* q_out,
                               const nvfp4_kv_cache* cache, hipStream_t stream) {
  return rope_checked("nvfp4_rope_append", q, q_stride, k, k_stride, v, v_stride, x_type,
                      positions, slots, inv_freq, T, Hq, D, R, interleaved, rope_scale, q_out,
                      cache, stream);
}

nvfp4_status nvfp4_rope_append_nvfp4(const void* q, int64_t q_stride, const void* k,
                                     int64_t k_stride, const void* v, int64_t v_stride,
                                     int x_type, const int64_t* positions, const int64_t* slots,
                                     const float* inv_freq, int64_t T, int64_t Hq, int64_t D,
                                     int64_t R, int interleaved, float rope_scale,
                                     uint16_t* q_out, const nvfp4_kv_cache4* cache,
                                     hipStream_t stream) {
  const char* fn = "nvfp4_rope_append_nvfp4";
  if (!cache) {
    clear_error();
    return fail(NVFP4_ERR_NULL, "%s: cache is NULL", fn);
  }
  return rope_checked(fn, q, q_stride, k, k_stride, v, v_stride, x_type, positions, slots,
                      inv_freq, T, Hq, D, R, interleaved, rope_scale, q_out, cache, stream);
}

}  // extern "C"

namespace {

bool attn_sizes(int64_t B, int64_t Q, int64_t Hq, int64_t Hkv, int64_t D) {
  return B >= 0 && Q >= 0 && Hkv >= 1 && Hq >= 0 && Hq % Hkv == 0 && B <= NVFP4_ATTN_MAX_B &&
         Q <= NVFP4_ATTN_MAX_Q && Hq <= NVFP4_MAX_HEADS && (D == 64 || D == 128 || D == 256);
}

template <class Cache>
nvfp4_status attn_checked(const char* fn, const uint16_t* q, const Cache* cache,
                          const int32_t* block_table, const int32_t* seq_lens, int64_t B,
                          int64_t Q, int64_t Hq, int64_t max_blocks, float scale, int64_t window,
                          const nvfp4_attn_scores* scores, uint16_t* out, void* workspace,
                          size_t workspace_bytes, hipStream_t stream) {
  clear_error();
  if (!cache) return fail(NVFP4_ERR_NULL, "%s: cache is NULL", fn);
  const nvfp4_status st = checks_of(fn, *cache);
  if (st != NVFP4_OK) return st;
  const int64_t Hkv = cache->n_kv_heads, D = cache->D;
  if (B < 0 || Q < 0 || Hq < 0 || Hq % Hkv || max_blocks < 0 || window < 0)
    return fail(NVFP4_ERR_SHAPE,
                "%s: need B, Q, max_blocks, window >= 0 and Hq a multiple of the cache's heads "
                "(B=%lld Q=%lld Hq=%lld Hkv=%lld)", fn, (long long)B, (long long)Q,
                (long long)Hq, (long long)Hkv);
  if (!(scale > -3.0e38f && scale < 3.0e38f))
    return fail(NVFP4_ERR_SHAPE, "%s: scale must be finite", fn);
  const float softcap = scores ? scores->softcap : 0.0f;
  const float* slopes = scores ? scores->slopes : nullptr;
  if (!(softcap == 0.0f || (softcap >= 1e-6f && softcap <= 1e30f)))
    return fail(NVFP4_ERR_SHAPE, "%s: softcap must be 0 (none) or 1e-6 .. 1e30", fn);
  if (!attn_sizes(B, Q, Hq, Hkv, D))
    return fail(NVFP4_ERR_UNSUPPORTED,
                "%s: B=%lld (max %d), Q=%lld (max %d), Hq=%lld (max %d), D=%lld (64, 128 or 256)",
                fn, (long long)B, NVFP4_ATTN_MAX_B, (long long)Q, NVFP4_ATTN_MAX_Q,
                (long long)Hq, NVFP4_MAX_HEADS, (long long)D);
  if (max_blocks > 0x7FFFFFFF || window > 0x7FFFFFFF)
    return fail(NVFP4_ERR_UNSUPPORTED, "%s: max_blocks=%lld or window=%lld is past 2^31 - 1", fn,
                (long long)max_blocks, (long long)window);
  if (B == 0 || Q == 0 || Hq == 0) return NVFP4_OK;
  auto a = attn_args(*cache);
  a.B = B;
  a.Q = Q;
  a.Hq = Hq;
  a.D = D;
  a.max_blocks = max_blocks;
  a.window = window;
  if (!nvfp4::attn_fits(a))
    return fail(NVFP4_ERR_UNSUPPORTED,
                "%s: more than 2^31 tiles of 32 keys (B * max_blocks * page), or than 2^22 "
                "sequences times row tiles of all heads", fn);
  if (!q || !seq_lens || !out || (max_blocks && !block_table))
    return fail(NVFP4_ERR_NULL, "%s: NULL pointer", fn);
  if (!aligned(q, 16) || !aligned(out, 16) || !aligned(block_table, 4) || !aligned(seq_lens, 4) ||
      !aligned(slopes, 4))
    return fail(NVFP4_ERR_ALIGN,
                "%s: q and out must be 16-byte, block_table, seq_lens and slopes 4-byte aligned",
                fn);
  a.cap = softcap * 1.4426950408889634f;
  a.cap_inv = softcap > 0.0f ? 1.0f / a.cap : 0.0f;
  a.slopes = slopes;
  const size_t need = attn_need(a);
  if (!workspace || workspace_bytes < need)
    return fail(NVFP4_ERR_WORKSPACE, "%s: the workspace needs %zu bytes, %zu given", fn, need,
                workspace ? workspace_bytes : (size_t)0);
  if (!aligned(workspace, 256))
    return fail(NVFP4_ERR_ALIGN, "%s: the workspace must be 256-byte aligned", fn);
  const size_t qb = (size_t)B * Q * Hq * D * 2;
  const size_t tb = (size_t)B * max_blocks * 4, lb = (size_t)B * 4;
  const CacheArrays ca = arrays_of(*cache);
  const void* outs[2] = {out, workspace};
  const size_t ob[2] = {qb, need};
  for (int i = 0; i < 2; ++i)
    if (overlap(outs[i], ob[i], q, qb) || overlap(outs[i], ob[i], ca) ||
        overlap(outs[i], ob[i], block_table, tb) || overlap(outs[i], ob[i], seq_lens, lb) ||
        overlap(outs[i], ob[i], slopes, (size_t)Hq * 4))
      return fail(NVFP4_ERR_ALIAS, "%s: the output or the workspace overlaps an input", fn);
  if (overlap(out, qb, workspace, need))
    return fail(NVFP4_ERR_ALIAS, "%s: the output and the workspace overlap", fn);
  a.q = q;
  a.table = block_table;
  a.lens = seq_lens;
  a.scale = scale;
  a.out = out;
  a.workspace = workspace;
  return hip_result(launch_attn(a, stream), fn);
}

}  // namespace

extern "C" {

size_t nvfp4_paged_attention_workspace_bytes(int64_t B, int64_t Q, int64_t Hq, int64_t Hkv,
                                             int64_t D) {
  if (!attn_sizes(B, Q, Hq, Hkv, D) || Hq == 0) return 0;
  return nvfp4::attn_workspace_bytes(B, Q, Hq, Hkv, D);
}

nvfp4_status nvfp4_paged_attention(const uint16_t* q, const nvfp4_kv_cache* cache,
                                   const int32_t* block_table, const int32_t* seq_lens,
                                   int64_t B, int64_t Q, int64_t Hq, int64_t max_blocks,
                                   float scale, int64_t window, uint16_t* out, void* workspace,
                                   size_t workspace_bytes, hipStream_t stream) {
  return attn_checked("nvfp4_paged_attention", q, cache, block_table, seq_lens, B, Q, Hq,
                      max_blocks, scale, window, nullptr, out, workspace, workspace_bytes, stream);
}

nvfp4_status nvfp4_paged_attention_scored(const uint16_t* q, const nvfp4_kv_cache* cache,
                                          const int32_t* block_table, const int32_t* seq_lens,
                                          int64_t B, int64_t Q, int64_t Hq, int64_t max_blocks,
                                          float scale, int64_t window,
                                          const nvfp4_attn_scores* scores, uint16_t* out,
                                          void* workspace, size_t workspace_bytes,
                                          hipStream_t stream) {
  return attn_checked("nvfp4_paged_attention_scored", q, cache, block_table, seq_lens, B, Q, Hq,
                      max_blocks, scale, window, scores, out, workspace, workspace_bytes, stream);
}

nvfp4_status nvfp4_paged_attention_nvfp4(const uint16_t* q, const nvfp4_kv_cache4* cache,
                                         const int32_t* block_table, const int32_t* seq_lens,
                                         int64_t B, int64_t Q, int64_t Hq, int64_t max_blocks,
                                         float scale, int64_t window,
                                         const nvfp4_attn_scores* scores, uint16_t* out,
                                         void* workspace, size_t workspace_bytes,
                                         hipStream_t stream) {
  return attn_checked("nvfp4_paged_attention_nvfp4", q, cache, block_table, seq_lens, B, Q, Hq,
                      max_blocks, scale, window, scores, out, workspace, workspace_bytes, stream);
}

namespace {

bool lora_sizes(int64_t M, int64_t K, int64_t rank, int64_t n_segments) {
  return M >= 0 && K >= 0 && K % 32 == 0 && rank >= 8 && rank % 8 == 0 && n_segments >= 0;
}
bool lora_limits(int64_t M, int64_t K, int64_t rank, int64_t n_segments) {
  return M <= NVFP4_MAX_M && K <= NVFP4_MAX_K && rank <= NVFP4_LORA_MAX_RANK &&
         n_segments <= NVFP4_MAX_SEGMENTS;
}

}  // namespace

size_t nvfp4_lora_workspace_bytes(int64_t M, int64_t K, int64_t rank, int64_t n_segments) {
  if (!lora_sizes(M, K, rank, n_segments) || !lora_limits(M, K, rank, n_segments)) return 0;
  return nvfp4::lora_workspace_bytes(M, K, rank, n_segments);
}

nvfp4_status nvfp4_lora_segments(const nvfp4_lora_segment* segs, int64_t n_segments,
                                 int64_t n_adapters, int64_t rank, const int32_t* ids,
                                 const int32_t* ranks, const float* alpha, const uint16_t* x,
                                 int64_t M, int64_t K, void* workspace, size_t workspace_bytes,
                                 hipStream_t stream) {
  clear_error();
  const char* fn = "nvfp4_lora_segments";
  if (!lora_sizes(M, K, rank, n_segments) || n_adapters < 0)
    return fail(NVFP4_ERR_SHAPE,
                "%s: need n_segments, n_adapters, M, K >= 0, K %% 32 == 0, rank >= 8 and rank %% 8 "
                "== 0 (n=%lld adapters=%lld rank=%lld M=%lld K=%lld)", fn, (long long)n_segments,
                (long long)n_adapters, (long long)rank, (long long)M, (long long)K);
  if (!lora_limits(M, K, rank, n_segments) || n_adapters > NVFP4_LORA_MAX_ADAPTERS)
    return fail(NVFP4_ERR_UNSUPPORTED,
                "%s: n_segments=%lld (max %d), n_adapters=%lld (max %d), rank=%lld (max %d), "
                "M=%lld (max %d), K=%lld (max %lld)", fn, (long long)n_segments,
                NVFP4_MAX_SEGMENTS, (long long)n_adapters, NVFP4_LORA_MAX_ADAPTERS,
                (long long)rank, NVFP4_LORA_MAX_RANK, (long long)M, NVFP4_MAX_M, (long long)K,
                (long long)NVFP4_MAX_K);
  if (n_segments == 0 || M == 0) return NVFP4_OK;
  if (!segs) return fail(NVFP4_ERR_NULL, "%s: segs is NULL", fn);
  nvfp4::LoraArgs a = {};
  int64_t total_n = 0;
  for (int64_t i = 0; i < n_segments; ++i) {
    const nvfp4_lora_segment& g = segs[i];
    if (g.N < 0)
      return fail(NVFP4_ERR_SHAPE, "%s: segment %lld has N=%lld < 0", fn, (long long)i,
                  (long long)g.N);
    if (g.N > NVFP4_MAX_N - total_n)
      return fail(NVFP4_ERR_UNSUPPORTED, "%s: the segments' N exceed %lld", fn,
                  (long long)NVFP4_MAX_N);
    total_n += g.N;
    if (g.N == 0) continue;
    if (!g.y || (n_adapters && (!g.b || (K && !g.a))))
      return fail(NVFP4_ERR_NULL, "%s: segment %lld has a NULL pointer", fn, (long long)i);
    if (!aligned(g.a, 16) || !aligned(g.b, 16) || !aligned(g.y, 4) || !aligned(g.base, 4))
      return fail(NVFP4_ERR_ALIGN,
                  "%s: segment %lld: a and b must be 16-byte, base and y 4-byte aligned", fn,
                  (long long)i);
    nvfp4::LoraSegment& d = a.segs[a.n_segments++];
    d.a = g.a;
    d.b = g.b;
    d.base = g.base;
    d.y = g.y;
    d.N = g.N;
  }
  if (a.n_segments == 0) return NVFP4_OK;
  if (!ids || (K && !x)) return fail(NVFP4_ERR_NULL, "%s: ids or x is NULL", fn);
  if (!aligned(ids, 4) || !aligned(ranks, 4) || !aligned(alpha, 4) || !aligned(x, 16))
    return fail(NVFP4_ERR_ALIGN, "%s: x must be 16-byte, ids, ranks and alpha 4-byte aligned", fn);
  const size_t need = nvfp4::lora_workspace_bytes(M, K, rank, n_segments);
  if (need && (!workspace || workspace_bytes < need))
    return fail(NVFP4_ERR_WORKSPACE, "%s: the workspace needs %zu bytes, %zu given", fn, need,
                workspace ? workspace_bytes : (size_t)0);
  if (need && !aligned(workspace, 256))
    return fail(NVFP4_ERR_ALIGN, "%s: the workspace must be 256-byte aligned", fn);
  const size_t xb = (size_t)M * K * 2, eb = (size_t)n_adapters * 4;
  for (int i = 0; i <= a.n_segments; ++i) {
    const bool ws = i == a.n_segments;   // the workspace, after the outputs
    const void* o = ws ? workspace : a.segs[i].y;
    const size_t n = ws ? need : (size_t)M * a.segs[i].N * 4;
    if (overlap(o, n, ids, (size_t)M * 4) || overlap(o, n, ranks, eb) ||
        overlap(o, n, alpha, eb) || overlap(o, n, x, xb))
      return fail(NVFP4_ERR_ALIAS, "%s: an output or the workspace overlaps an input", fn);
    for (int j = 0; j < a.n_segments; ++j) {
      const nvfp4::LoraSegment& g = a.segs[j];
      const size_t yb = (size_t)M * g.N * 4;
      const bool in_place = i == j && g.base == g.y;
      if (overlap(o, n, g.a, (size_t)n_adapters * rank * K * 2) ||
          overlap(o, n, g.b, (size_t)n_adapters * rank * g.N * 2) ||
          (!in_place && overlap(o, n, g.base, yb)))
        return fail(NVFP4_ERR_ALIAS, "%s: an output or the workspace overlaps an input", fn);
      if (i != j && overlap(o, n, g.y, yb))
        return fail(NVFP4_ERR_ALIAS, "%s: two outputs, or one and the workspace, overlap", fn);
    }
  }
  a.x = x;
  a.ids = ids;
  a.ranks = ranks;
  a.alpha = alpha;
  a.n_adapters = n_adapters;
  a.rank = rank;
  a.M = M;
  a.K = K;
  a.workspace = workspace;
  return hip_result(nvfp4::launch_lora(a, stream), "nvfp4_lora_segments launch");
}

namespace {

bool verify_sizes(int64_t B, int64_t V) {
  return B >= 0 && V >= 1 && B <= NVFP4_VERIFY_MAX_B && V <= NVFP4_VERIFY_MAX_V;
}

}  // namespace

size_t nvfp4_verify_draft_workspace_bytes(int64_t B, int64_t V) {
  return verify_sizes(B, V) ? nvfp4::verify_workspace_bytes(B, V) : 0;
}

nvfp4_status nvfp4_verify_draft(const float* target_p, const float* draft_p, const int32_t* draft,
                                const int32_t* n_draft, const float* u_accept,
                                const float* u_sample, int64_t B, int64_t Q, int64_t V,
                                int32_t* tokens, int32_t* n_accepted, void* workspace,
                                size_t workspace_bytes, hipStream_t stream) {
  clear_error();
  const char* fn = "nvfp4_verify_draft";
  if (B < 0 || Q < 0 || V < 1)
    return fail(NVFP4_ERR_SHAPE, "%s: need B, Q >= 0 and V >= 1 (B=%lld Q=%lld V=%lld)", fn,
                (long long)B, (long long)Q, (long long)V);
  if (!verify_sizes(B, V) || Q > NVFP4_VERIFY_MAX_Q)
    return fail(NVFP4_ERR_UNSUPPORTED, "%s: B=%lld (max %d), Q=%lld (max %d), V=%lld (max %d)",
                fn, (long long)B, NVFP4_VERIFY_MAX_B, (long long)Q, NVFP4_VERIFY_MAX_Q,
                (long long)V, NVFP4_VERIFY_MAX_V);
  if (B == 0) return NVFP4_OK;
  if (!target_p || !u_sample || !tokens || !n_accepted || (Q && (!draft || !u_accept)))
    return fail(NVFP4_ERR_NULL, "%s: NULL pointer", fn);
  if (!aligned(target_p, 4) || !aligned(draft_p, 4) || !aligned(draft, 4) ||
      !aligned(n_draft, 4) || !aligned(u_accept, 4) || !aligned(u_sample, 4) ||
      !aligned(tokens, 4) || !aligned(n_accepted, 4))
    return fail(NVFP4_ERR_ALIGN, "%s: every pointer must be 4-byte aligned", fn);
  const size_t need = nvfp4::verify_workspace_bytes(B, V);
  if (!workspace || workspace_bytes < need)
    return fail(NVFP4_ERR_WORKSPACE, "%s: the workspace needs %zu bytes, %zu given", fn, need,
                workspace ? workspace_bytes : (size_t)0);
  if (!aligned(workspace, 256))
    return fail(NVFP4_ERR_ALIGN, "%s: the workspace must be 256-byte aligned", fn);
  const size_t pb = (size_t)B * (Q + 1) * V * 4, qb = (size_t)B * Q * V * 4;
  const size_t db = (size_t)B * Q * 4, bb = (size_t)B * 4;
  const void* outs[3] = {tokens, n_accepted, workspace};
  const size_t ob[3] = {(size_t)B * (Q + 1) * 4, bb, need};
  for (int i = 0; i < 3; ++i) {
    if (overlap(outs[i], ob[i], target_p, pb) || overlap(outs[i], ob[i], draft_p, qb) ||
        overlap(outs[i], ob[i], draft, db) || overlap(outs[i], ob[i], n_draft, bb) ||
        overlap(outs[i], ob[i], u_accept, db) || overlap(outs[i], ob[i], u_sample, bb))
      return fail(NVFP4_ERR_ALIAS, "%s: an output or the workspace overlaps an input", fn);
    for (int j = 0; j < i; ++j)
      if (overlap(outs[i], ob[i], outs[j], ob[j]))
        return fail(NVFP4_ERR_ALIAS, "%s: two outputs overlap", fn);
  }
  nvfp4::VerifyArgs a = {};
  a.p = target_p;
  a.q = Q ? draft_p : nullptr;
  a.draft = draft;
  a.n_draft = n_draft;
  a.u_accept = u_accept;
  a.u_sample = u_sample;
  a.B = B;
  a.Q = Q;
  a.V = V;
  a.tokens = tokens;
  a.accepted = n_accepted;
  a.workspace = workspace;
  return hip_result(nvfp4::launch_verify_draft(a, stream), "nvfp4_verify_draft launch");
}

nvfp4_status nvfp4_stream_read(const void* buf, size_t bytes, uint32_t* sink,
                               hipStream_t stream) {
  clear_error();
  if (bytes % 16 != 0)
    return fail(NVFP4_ERR_SHAPE, "nvfp4_stream_read: bytes=%zu is not a multiple of 16", bytes);
  if (bytes == 0) return NVFP4_OK;
  if (!buf || !sink) return fail(NVFP4_ERR_NULL, "nvfp4_stream_read: NULL pointer");
  if (!aligned(buf, 16) || !aligned(sink, 4))
    return fail(NVFP4_ERR_ALIGN, "nvfp4_stream_read: buf must be 16-byte, sink 4-byte aligned");
  if (overlap(sink, 4, buf, bytes))
    return fail(NVFP4_ERR_ALIAS, "nvfp4_stream_read: sink overlaps buf");
  return hip_result(nvfp4::launch_stream_read(buf, bytes, sink, stream),
                    "nvfp4_stream_read launch");
}

nvfp4_status nvfp4_check_device_faults(hipStream_t stream) {
  clear_error();
  uint32_t fault = 0u;
  const hipError_t e = nvfp4::splitk_take_fault(stream, &fault);
  if (e != hipSuccess)
    return fail(NVFP4_ERR_HIP, "nvfp4_check_device_faults: %s (%s)", hipGetErrorName(e),
                hipGetErrorString(e));
  if (fault != 0u)
    return fail(NVFP4_ERR_HIP,
                "nvfp4_check_device_faults: a split-K GEMV slot wait gave up (fault word %#x); "
                "the tiles concerned hold NaN",
                fault);
  return NVFP4_OK;
}

void nvfp4_debug_set_wait_limit(int polls) { nvfp4::splitk_set_spin_limit(polls); }

size_t nvfp4_moe_workspace_bytes(int64_t M, int64_t H, int64_t I, int64_t topk) {
  if (M < 0 || H < 0 || I < 0 || topk < 0) return 0;
  return nvfp4::moe_layout(M, H, I, topk, 0, false).total;
}

size_t nvfp4_moe_shared_workspace_bytes(int64_t M, int64_t H, int64_t I, int64_t topk,
                                        int64_t I_shared) {
  if (M < 0 || H < 0 || I < 0 || topk < 0 || I_shared < 0) return 0;
  return nvfp4::moe_layout(M, H, I, topk, I_shared, false).total;
}

size_t nvfp4_moe_w4a4_workspace_bytes(int64_t M, int64_t H, int64_t I, int64_t topk,
                                      int64_t I_shared) {
  if (M < 0 || H < 0 || I < 0 || topk < 0 || I_shared < 0) return 0;
  return nvfp4::moe_layout(M, H, I, topk, I_shared, true).total;
}

}  // extern "C"

namespace {

// The current device's scratch array of nvfp4_moe_gemv_noalloc (defined at
// the end of this file), or NULL with the error text set.
void* device_scratch(const char* fn);

// Checks and launch shared by nvfp4_moe_gemv, nvfp4_moe_shared_gemv,
// nvfp4_moe_w4a4_gemv and nvfp4_moe_gemv_noalloc (shared == NULL: no shared
// expert; w4a4: the routed experts take NVFP4 activations with the static
// scales ga13 and ga2; own_ws: the workspace is the library's scratch array,
// looked up after every host-side check, just before the launch).
nvfp4_status moe_checked(const char* fn, const uint8_t* w13_codes, const uint8_t* w13_scales,
                         const float* w13_gscale, const uint8_t* w2_codes,
                         const uint8_t* w2_scales, const float* w2_gscale, const uint16_t* x,
                         const int32_t* expert_ids, const float* gate_w, int64_t M, int64_t E,
                         int64_t H, int64_t I, int64_t topk, const nvfp4_moe_shared* shared,
                         bool w4a4, const float* ga13, const float* ga2, float* y,
                         void* workspace, size_t workspace_bytes, hipStream_t stream,
                         bool own_ws = false) {
  clear_error();
  if (M < 0 || E < 1 || H <= 0 || I <= 0 || topk < 1 || (H % 32) != 0 || (I % 32) != 0)
    return fail(NVFP4_ERR_SHAPE,
                "%s: need M >= 0, E >= 1, topk >= 1, H, I > 0 and multiples of 32 "
                "(M=%lld E=%lld H=%lld I=%lld topk=%lld)",
                fn, (long long)M, (long long)E, (long long)H, (long long)I, (long long)topk);
  const int64_t Is = shared ? shared->I : 0;
  if (shared && (Is <= 0 || (Is % 32) != 0))
    return fail(NVFP4_ERR_SHAPE, "%s: shared expert width I=%lld must be > 0 and a multiple of 32",
                fn, (long long)Is);
  if (M > NVFP4_MOE_MAX_M || topk > NVFP4_MAX_TOPK || I > NVFP4_MOE_MAX_I || Is > NVFP4_MOE_MAX_I ||
      H > NVFP4_MOE_MAX_H)
    return fail(NVFP4_ERR_UNSUPPORTED,
                "%s: M=%lld (max %d), topk=%lld (max %d), I=%lld, shared I=%lld (max %d), "
                "H=%lld (max %d)", fn,
                (long long)M, NVFP4_MOE_MAX_M, (long long)topk, NVFP4_MAX_TOPK, (long long)I,
                (long long)Is, NVFP4_MOE_MAX_I, (long long)H, NVFP4_MOE_MAX_H);
  if (M == 0) return NVFP4_OK;
  if (!w13_codes || !w13_scales || !w13_gscale || !w2_codes || !w2_scales || !w2_gscale || !x ||
      !expert_ids || !gate_w || !y)
    return fail(NVFP4_ERR_NULL, "%s: NULL pointer", fn);
  if (shared && (!shared->w13_codes || !shared->w13_scales || !shared->w13_gscale ||
                 !shared->w2_codes || !shared->w2_scales || !shared->w2_gscale))
    return fail(NVFP4_ERR_NULL, "%s: NULL pointer in the shared expert", fn);
  if (w4a4 && (!ga13 || !ga2)) return fail(NVFP4_ERR_NULL, "%s: NULL static input scale", fn);
  const size_t need = nvfp4::moe_layout(M, H, I, topk, Is, w4a4).total;
  if (own_ws && need > (size_t)NVFP4_NOALLOC_SCRATCH_BYTES)
    return fail(NVFP4_ERR_UNSUPPORTED,
                "%s: M * topk * I * 2 = %zu bytes of activations exceed the %d-byte scratch "
                "array (use nvfp4_moe_gemv with a workspace)",
                fn, need, NVFP4_NOALLOC_SCRATCH_BYTES);
  if (!own_ws && (!workspace || workspace_bytes < need))
    return fail(NVFP4_ERR_WORKSPACE, "%s: workspace of %zu bytes needed, %zu given", fn, need,
                workspace ? workspace_bytes : (size_t)0);
  if (!aligned(w13_codes, 16) || !aligned(w2_codes, 16) || !aligned(w13_scales, 2) ||
      !aligned(w2_scales, 2) || !aligned(x, 16) || !aligned(y, 16) ||
      (!own_ws && !aligned(workspace, 256)) ||
      !aligned(expert_ids, 4) || !aligned(gate_w, 4) || !aligned(w13_gscale, 4) ||
      !aligned(w2_gscale, 4))
    return fail(NVFP4_ERR_ALIGN, "%s: alignment rule broken (see nvfp4_gemv.h)", fn);
  if (shared && (!aligned(shared->w13_codes, 16) || !aligned(shared->w2_codes, 16) ||
                 !aligned(shared->w13_scales, 2) || !aligned(shared->w2_scales, 2) ||
                 !aligned(shared->w13_gscale, 4) || !aligned(shared->w2_gscale, 4)))
    return fail(NVFP4_ERR_ALIGN, "%s: alignment rule broken in the shared expert", fn);
  if (w4a4 && (!aligned(ga13, 4) || !aligned(ga2, 4)))
    return fail(NVFP4_ERR_ALIGN, "%s: static input scales must be 4-byte aligned", fn);
  const size_t e13 = (size_t)E * 2 * (size_t)I * (size_t)H, e2 = (size_t)E * (size_t)H * (size_t)I;
  const size_t s13 = 2 * (size_t)Is * (size_t)H, s2 = (size_t)H * (size_t)Is;
  const size_t yb = (size_t)M * (size_t)H * 4, S = (size_t)(M * topk);
  const void* ins[] = {w13_codes, w13_scales, w13_gscale, w2_codes, w2_scales, w2_gscale, x,
                       expert_ids, gate_w,
                       shared ? shared->w13_codes : nullptr, shared ? shared->w13_scales : nullptr,
                       shared ? shared->w13_gscale : nullptr, shared ? shared->w2_codes : nullptr,
                       shared ? shared->w2_scales : nullptr, shared ? shared->w2_gscale : nullptr,
                       w4a4 ? ga13 : nullptr, w4a4 ? ga2 : nullptr};
  const size_t insz[] = {e13 / 2, e13 / 16, (size_t)E * 4, e2 / 2, e2 / 16, (size_t)E * 4,
                         (size_t)M * (size_t)H * 2, S * 4, S * 4,
                         s13 / 2, s13 / 16, 4, s2 / 2, s2 / 16, 4, 4, 4};
  // (the library's own scratch array cannot overlap a caller buffer)
  for (int i = 0; i < 17; ++i) {
    if (overlap(y, yb, ins[i], insz[i]) ||
        (!own_ws && overlap(workspace, need, ins[i], insz[i])))
      return fail(NVFP4_ERR_ALIAS, "%s: y or workspace overlaps input %d", fn, i);
  }
  if (!own_ws && overlap(y, yb, workspace, need))
    return fail(NVFP4_ERR_ALIAS, "%s: y overlaps the workspace", fn);
  if (own_ws) {
    workspace = device_scratch(fn);
    if (!workspace) return NVFP4_ERR_HIP;
  }
  nvfp4::MoeShared sh = {};
  if (shared) {
    sh.c13 = shared->w13_codes;
    sh.s13 = shared->w13_scales;
    sh.g13 = shared->w13_gscale;
    sh.c2 = shared->w2_codes;
    sh.s2 = shared->w2_scales;
    sh.g2 = shared->w2_gscale;
    sh.I = Is;
  }
  const nvfp4::MoeW4a4 q = {ga13, ga2};
  return hip_result(nvfp4::launch_moe(w13_codes, w13_scales, w13_gscale, w2_codes, w2_scales,
                                      w2_gscale, x, expert_ids, gate_w, (int)M, E, H, I,
                                      (int)topk, shared ? &sh : nullptr, w4a4 ? &q : nullptr, y,
                                      workspace, stream),
                    fn);
}

}  // namespace

extern "C" {

nvfp4_status nvfp4_moe_gemv(const uint8_t* w13_codes, const uint8_t* w13_scales,
                            const float* w13_gscale, const uint8_t* w2_codes,
                            const uint8_t* w2_scales, const float* w2_gscale, const uint16_t* x,
                            const int32_t* expert_ids, const float* gate_w, int64_t M, int64_t E,
                            int64_t H, int64_t I, int64_t topk, float* y, void* workspace,
                            size_t workspace_bytes, hipStream_t stream) {
  return moe_checked("nvfp4_moe_gemv", w13_codes, w13_scales, w13_gscale, w2_codes, w2_scales,
                     w2_gscale, x, expert_ids, gate_w, M, E, H, I, topk, nullptr, false, nullptr,
                     nullptr, y, workspace, workspace_bytes, stream);
}

nvfp4_status nvfp4_moe_shared_gemv(const uint8_t* w13_codes, const uint8_t* w13_scales,
                                   const float* w13_gscale, const uint8_t* w2_codes,
                                   const uint8_t* w2_scales, const float* w2_gscale,
                                   const uint16_t* x, const int32_t* expert_ids,
                                   const float* gate_w, int64_t M, int64_t E, int64_t H,
                                   int64_t I, int64_t topk, const nvfp4_moe_shared* shared,
                                   float* y, void* workspace, size_t workspace_bytes,
                                   hipStream_t stream) {
  if (!shared) {
    clear_error();
    return fail(NVFP4_ERR_NULL, "nvfp4_moe_shared_gemv: NULL shared expert");
  }
  return moe_checked("nvfp4_moe_shared_gemv", w13_codes, w13_scales, w13_gscale, w2_codes,
                     w2_scales, w2_gscale, x, expert_ids, gate_w, M, E, H, I, topk, shared, false,
                     nullptr, nullptr, y, workspace, workspace_bytes, stream);
}

nvfp4_status nvfp4_moe_w4a4_gemv(const uint8_t* w13_codes, const uint8_t* w13_scales,
                                 const float* w13_gscale, const uint8_t* w2_codes,
                                 const uint8_t* w2_scales, const float* w2_gscale,
                                 const uint16_t* x, const float* gscale_x, const float* gscale_h,
                                 const int32_t* expert_ids, const float* gate_w, int64_t M,
                                 int64_t E, int64_t H, int64_t I, int64_t topk,
                                 const nvfp4_moe_shared* shared, float* y, void* workspace,
                                 size_t workspace_bytes, hipStream_t stream) {
  return moe_checked("nvfp4_moe_w4a4_gemv", w13_codes, w13_scales, w13_gscale, w2_codes,
                     w2_scales, w2_gscale, x, expert_ids, gate_w, M, E, H, I, topk, shared, true,
                     gscale_x, gscale_h, y, workspace, workspace_bytes, stream);
}

}  // extern "C"

// ---------------------------------------------------------------------------
// nvfp4_moe_gemv_noalloc: nvfp4_moe_gemv with its workspace (the bf16 SwiGLU
// activations h) in a file-scope device array instead of caller memory, for
// callers that cannot allocate. Each device the library runs on holds its own
// copy of the array until the process ends. In host code `scratch` only names
// the symbol: its device address is looked up once per device with
// hipGetSymbolAddress (with that device current) and that address is what
// the kernels receive.

namespace {

static __device__ __align__(256) unsigned char scratch[NVFP4_NOALLOC_SCRATCH_BYTES];

constexpr int kMaxDevices = 64;
std::mutex g_scratch_mu;
void* g_scratch_ptr[kMaxDevices] = {};

// The current device's address of `scratch` (looked up on the first call on
// that device), or NULL with the error text set.
void* device_scratch(const char* fn) {
  int dev = -1;
  const hipError_t e = hipGetDevice(&dev);
  if (e != hipSuccess) {
    fail(NVFP4_ERR_HIP, "%s: hipGetDevice: %s", fn, hipGetErrorString(e));
    return nullptr;
  }
  if (dev < 0 || dev >= kMaxDevices) {
    fail(NVFP4_ERR_UNSUPPORTED, "%s: device %d is past the %d devices this entry point serves",
         fn, dev, kMaxDevices);
    return nullptr;
  }
  std::lock_guard<std::mutex> lock(g_scratch_mu);
  if (!g_scratch_ptr[dev]) {
    void* ptr = nullptr;
    const hipError_t r = hipGetSymbolAddress((void**)&ptr, HIP_SYMBOL(scratch));
    if (r != hipSuccess || !ptr) {
      fail(NVFP4_ERR_HIP, "%s: hipGetSymbolAddress(scratch) on device %d: %s", fn, dev,
           hipGetErrorString(r));
      return nullptr;
    }
    g_scratch_ptr[dev] = ptr;
  }
  return g_scratch_ptr[dev];
}

}  // namespace

extern "C" {

nvfp4_status nvfp4_moe_gemv_noalloc(const uint8_t* w13_codes, const uint8_t* w13_scales,
                                    const float* w13_gscale, const uint8_t* w2_codes,
                                    const uint8_t* w2_scales, const float* w2_gscale,
                                    const uint16_t* x, const int32_t* expert_ids,
                                    const float* gate_w, int64_t M, int64_t E, int64_t H,
                                    int64_t I, int64_t topk, float* y, hipStream_t stream) {
  return moe_checked("nvfp4_moe_gemv_noalloc", w13_codes, w13_scales, w13_gscale, w2_codes,
                     w2_scales, w2_gscale, x, expert_ids, gate_w, M, E, H, I, topk, nullptr,
                     false, nullptr, nullptr, y, nullptr, 0, stream, /*own_ws=*/true);
}

}  // extern "C"
