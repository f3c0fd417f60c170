"""NVFP4 g16 W4A16 small-M GEMV for MI355X (gfx950): a thin Python binding.

Every function here marshals torch tensors into the C ABI declared in
``include/nvfp4_gemv.h`` and calls ``libnvfp4_gemv.so``; all computation runs
in the library's HIP kernels on the tensors' device, on the current torch
stream. PyTorch only provides device memory and streams. There is no CPU
fallback: if the library is not built, every call raises.

Functions (same names as the C entry points, without the prefix):
  pack(W[, gscale_override])             -> codes, scales, gscale
  dequant(codes, scales, gscale)         -> W_hat (fp32)
  gemv(codes, scales, gscale, x)         -> y (fp32 [M, N])
  gemv_segments([(codes, scales, gscale), ...], x) -> [y_s] (one launch)
  quantize_act(x, gscale_x)              -> codes_x, scales_x (static input scale)
  gemv_w4a4(codes, scales, gscale, codes_x, scales_x, gscale_x) -> y (fp32)
  moe_workspace_bytes(M, H, I, topk)     -> int
  moe_gemv(w13..., w2..., x, ids, gate_w[, workspace]) -> y (fp32 [M, H])
  moe_shared_workspace_bytes(M, H, I, topk, I_shared) -> int
  moe_shared_gemv(w13..., w2..., x, ids, gate_w, shared[, workspace]) -> y
  moe_gemv_noalloc_into(w13..., w2..., x, ids, gate_w, y)  (no workspace)
  add_rmsnorm(x, weight, eps[, residual])         -> y (bf16), residual_out
  add_rmsnorm_e4m3(x, weight, eps[, residual, group]) -> y8, scales, residual_out
  add_rmsnorm_nvfp4(x, weight, eps, gscale[, residual]) -> codes, scales, residual_out
  rope_append(q, k, v, positions, slots, inv_freq, k_cache, v_cache, ...) -> q_out (bf16)
  rope_append_nvfp4(q, k, v, positions, slots, inv_freq, k_cache, v_cache, ...) -> q_out (bf16)
  paged_attention(q, k_cache, v_cache, block_table, seq_lens, ...) -> out (bf16)
  paged_attention_scored(q, k_cache, v_cache, block_table, seq_lens, softcap, slopes, ...) -> out
  paged_attention_nvfp4(q, k_cache, v_cache, block_table, seq_lens, ...) -> out (bf16)
  lora_segments([(a, b), ...], x, ids[, bases, alpha, ranks]) -> [y_s] (fp32 [M, N_s])
  verify_draft(target_p, draft_p, draft, u_accept, u_sample, ...) -> tokens, n_accepted
  paged_attention_workspace_bytes(B, Q, Hq, Hkv, D), verify_draft_workspace_bytes(B, V),
  lora_workspace_bytes(M, K, rank, n_segments)
  stream_read(buf, sink)                 (measurement aid: one pure read of buf)
The ``*_into`` variants write into caller-provided outputs.
"""
from __future__ import annotations

import ctypes
import os

import torch

from . import traffic  # noqa: F401  (algorithmic byte model, pure Python)

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libnvfp4_gemv.so")
HEADER_PATH = os.path.join(os.path.dirname(_HERE), "include", "nvfp4_gemv.h")

# The size limits of include/nvfp4_gemv.h (NVFP4_MAX_M, NVFP4_MOE_MAX_M,
# NVFP4_MAX_TOPK, NVFP4_MAX_N, NVFP4_MAX_K, NVFP4_MOE_MAX_I, NVFP4_MOE_MAX_H).
MAX_M = 128
MOE_MAX_M = 8
MAX_TOPK = 16
MAX_N = 1 << 30
MAX_K = 1 << 20
MOE_MAX_I = 1 << 24
MOE_MAX_H = 1 << 24
# NVFP4_MAX_ROWS, NVFP4_NORM_MAX_H, NVFP4_MAX_HEADS, NVFP4_ROPE_MAX_D,
# NVFP4_ATTN_MAX_B, NVFP4_ATTN_MAX_Q, NVFP4_VERIFY_MAX_Q / _B / _V.
MAX_ROWS = 1 << 21
NORM_MAX_H = 1 << 15
MAX_HEADS = 1024
ROPE_MAX_D = 512
ATTN_MAX_B = 4096
ATTN_MAX_Q = 64
VERIFY_MAX_Q = 63
VERIFY_MAX_B = 4096
VERIFY_MAX_V = 1 << 24
# NVFP4_LORA_MAX_RANK, NVFP4_LORA_MAX_ADAPTERS.
LORA_MAX_RANK = 256
LORA_MAX_ADAPTERS = 1 << 20
# NVFP4_NOALLOC_SCRATCH_BYTES: the device array of nvfp4_moe_gemv_noalloc.
NOALLOC_SCRATCH_BYTES = 4 << 20

_VP = ctypes.c_void_p
_I64 = ctypes.c_int64
_lib = None


class Nvfp4Error(RuntimeError):
    def __init__(self, fn: str, status: int, detail: str):
        super().__init__(f"{fn} failed: status {status} ({detail})")
        self.status = status


class GemvSegment(ctypes.Structure):
    """nvfp4_gemv_segment: one matrix of a fused multi-projection GEMV."""
    _fields_ = [("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p),
                ("gscale", ctypes.c_void_p), ("y", ctypes.c_void_p), ("N", ctypes.c_int64)]


MAX_SEGMENTS = 8


class MoeShared(ctypes.Structure):
    """nvfp4_moe_shared: the shared expert of a MoE call."""
    _fields_ = [("w13_codes", ctypes.c_void_p), ("w13_scales", ctypes.c_void_p),
                ("w13_gscale", ctypes.c_void_p), ("w2_codes", ctypes.c_void_p),
                ("w2_scales", ctypes.c_void_p), ("w2_gscale", ctypes.c_void_p),
                ("I", ctypes.c_int64)]


class KvCache(ctypes.Structure):
    """nvfp4_kv_cache: a paged key-value cache."""
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_scale", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p), ("num_blocks", ctypes.c_int64),
                ("page", ctypes.c_int64), ("n_kv_heads", ctypes.c_int64), ("D", ctypes.c_int64),
                ("stride_block", ctypes.c_int64), ("stride_token", ctypes.c_int64),
                ("stride_head", ctypes.c_int64), ("type", ctypes.c_int)]


class KvCache4(ctypes.Structure):
    """nvfp4_kv_cache4: a paged key-value cache in NVFP4."""
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_scales", ctypes.c_void_p),
                ("v_scales", ctypes.c_void_p), ("k_gscale", ctypes.c_void_p),
                ("v_gscale", ctypes.c_void_p), ("num_blocks", ctypes.c_int64),
                ("page", ctypes.c_int64), ("n_kv_heads", ctypes.c_int64), ("D", ctypes.c_int64),
                ("stride_block", ctypes.c_int64), ("stride_token", ctypes.c_int64),
                ("stride_head", ctypes.c_int64), ("scale_stride_block", ctypes.c_int64),
                ("scale_stride_token", ctypes.c_int64), ("scale_stride_head", ctypes.c_int64)]


class AttnScores(ctypes.Structure):
    """nvfp4_attn_scores: the cap and the bias of attention's scores."""
    _fields_ = [("softcap", ctypes.c_float), ("slopes", ctypes.c_void_p)]


class LoraSegment(ctypes.Structure):
    """nvfp4_lora_segment: one projection's adapters."""
    _fields_ = [("a", ctypes.c_void_p), ("b", ctypes.c_void_p), ("base", ctypes.c_void_p),
                ("y", ctypes.c_void_p), ("N", ctypes.c_int64)]


# nvfp4_dtype
_BF16, _F32, _E4M3 = 0, 1, 2
_ACT_TYPES = {torch.bfloat16: _BF16, torch.float32: _F32}
_CACHE_TYPES = {torch.bfloat16: _BF16, torch.float8_e4m3fn: _E4M3}


def lib() -> ctypes.CDLL:
    """The loaded C library (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(
                f"{LIB_PATH} is not built; run "
                "`python -m nvfp4_block_scaled_gemv_amd.build` (no CPU fallback exists)")
        L = ctypes.CDLL(LIB_PATH)
        L.nvfp4_abi_version.restype = ctypes.c_int
        L.nvfp4_abi_version.argtypes = []
        L.nvfp4_status_string.restype = ctypes.c_char_p
        L.nvfp4_status_string.argtypes = [ctypes.c_int]
        L.nvfp4_last_error.restype = ctypes.c_char_p
        L.nvfp4_last_error.argtypes = []
        L.nvfp4_pack.restype = ctypes.c_int
        L.nvfp4_pack.argtypes = [_VP, _I64, _I64, _VP, _VP, _VP, _VP, _VP]
        L.nvfp4_dequant.restype = ctypes.c_int
        L.nvfp4_dequant.argtypes = [_VP, _VP, _VP, _I64, _I64, _VP, _VP]
        L.nvfp4_gemv.restype = ctypes.c_int
        L.nvfp4_gemv.argtypes = [_VP, _VP, _VP, _VP, _I64, _I64, _I64, _VP, _VP]
        L.nvfp4_gemv_segments.restype = ctypes.c_int
        L.nvfp4_gemv_segments.argtypes = [ctypes.POINTER(GemvSegment), _I64, _VP, _I64, _I64,
                                          _VP]
        L.nvfp4_quantize_act.restype = ctypes.c_int
        L.nvfp4_quantize_act.argtypes = [_VP, _I64, _I64, _VP, _VP, _VP, _VP]
        L.nvfp4_gemv_w4a4_workspace_bytes.restype = ctypes.c_size_t
        L.nvfp4_gemv_w4a4_workspace_bytes.argtypes = [_I64, _I64]
        L.nvfp4_gemv_w4a4.restype = ctypes.c_int
        L.nvfp4_gemv_w4a4.argtypes = [_VP] * 6 + [_I64] * 3 + [_VP, _VP, ctypes.c_size_t, _VP]
        L.nvfp4_gemv_w4a4_segments.restype = ctypes.c_int
        L.nvfp4_gemv_w4a4_segments.argtypes = [ctypes.POINTER(GemvSegment), _I64, _VP, _VP, _VP,
                                               _I64, _I64, _VP, ctypes.c_size_t, _VP]
        L.nvfp4_moe_workspace_bytes.restype = ctypes.c_size_t
        L.nvfp4_moe_workspace_bytes.argtypes = [_I64, _I64, _I64, _I64]
        L.nvfp4_moe_gemv.restype = ctypes.c_int
        L.nvfp4_moe_gemv.argtypes = [_VP] * 9 + [_I64] * 5 + [_VP, _VP, ctypes.c_size_t, _VP]
        L.nvfp4_moe_shared_workspace_bytes.restype = ctypes.c_size_t
        L.nvfp4_moe_shared_workspace_bytes.argtypes = [_I64] * 5
        L.nvfp4_moe_shared_gemv.restype = ctypes.c_int
        L.nvfp4_moe_shared_gemv.argtypes = ([_VP] * 9 + [_I64] * 5 +
                                            [ctypes.POINTER(MoeShared), _VP, _VP,
                                             ctypes.c_size_t, _VP])
        L.nvfp4_moe_w4a4_workspace_bytes.restype = ctypes.c_size_t
        L.nvfp4_moe_w4a4_workspace_bytes.argtypes = [_I64] * 5
        L.nvfp4_moe_w4a4_gemv.restype = ctypes.c_int
        L.nvfp4_moe_w4a4_gemv.argtypes = ([_VP] * 11 + [_I64] * 5 +
                                          [ctypes.POINTER(MoeShared), _VP, _VP,
                                           ctypes.c_size_t, _VP])
        L.nvfp4_moe_gemv_noalloc.restype = ctypes.c_int
        L.nvfp4_moe_gemv_noalloc.argtypes = [_VP] * 9 + [_I64] * 5 + [_VP, _VP]
        norm = [_VP, ctypes.c_int, _VP, _VP, ctypes.c_int, _VP, ctypes.c_float, _I64, _I64]
        L.nvfp4_add_rmsnorm.restype = ctypes.c_int
        L.nvfp4_add_rmsnorm.argtypes = norm + [_VP, _VP]
        L.nvfp4_add_rmsnorm_e4m3.restype = ctypes.c_int
        L.nvfp4_add_rmsnorm_e4m3.argtypes = norm + [_I64, _VP, _VP, _VP]
        L.nvfp4_add_rmsnorm_nvfp4.restype = ctypes.c_int
        L.nvfp4_add_rmsnorm_nvfp4.argtypes = norm + [_VP] * 4
        L.nvfp4_rope_append.restype = ctypes.c_int
        L.nvfp4_rope_append.argtypes = ([_VP, _I64] * 3 + [ctypes.c_int] + [_VP] * 3 +
                                        [_I64] * 4 + [ctypes.c_int, ctypes.c_float, _VP,
                                                      ctypes.POINTER(KvCache), _VP])
        L.nvfp4_paged_attention_workspace_bytes.restype = ctypes.c_size_t
        L.nvfp4_paged_attention_workspace_bytes.argtypes = [_I64] * 5
        L.nvfp4_paged_attention.restype = ctypes.c_int
        L.nvfp4_paged_attention.argtypes = [_VP, ctypes.POINTER(KvCache), _VP, _VP, _I64, _I64,
                                            _I64, _I64, ctypes.c_float, _I64, _VP, _VP,
                                            ctypes.c_size_t, _VP]
        L.nvfp4_rope_append_nvfp4.restype = ctypes.c_int
        L.nvfp4_rope_append_nvfp4.argtypes = ([_VP, _I64] * 3 + [ctypes.c_int] + [_VP] * 3 +
                                              [_I64] * 4 + [ctypes.c_int, ctypes.c_float, _VP,
                                                            ctypes.POINTER(KvCache4), _VP])
        for name, cache in (("scored", KvCache), ("nvfp4", KvCache4)):
            f = getattr(L, "nvfp4_paged_attention_" + name)
            f.restype = ctypes.c_int
            f.argtypes = [_VP, ctypes.POINTER(cache), _VP, _VP, _I64, _I64, _I64, _I64,
                          ctypes.c_float, _I64, ctypes.POINTER(AttnScores), _VP, _VP,
                          ctypes.c_size_t, _VP]
        L.nvfp4_lora_workspace_bytes.restype = ctypes.c_size_t
        L.nvfp4_lora_workspace_bytes.argtypes = [_I64] * 4
        L.nvfp4_lora_segments.restype = ctypes.c_int
        L.nvfp4_lora_segments.argtypes = [ctypes.POINTER(LoraSegment), _I64, _I64, _I64, _VP, _VP,
                                          _VP, _VP, _I64, _I64, _VP, ctypes.c_size_t, _VP]
        L.nvfp4_verify_draft_workspace_bytes.restype = ctypes.c_size_t
        L.nvfp4_verify_draft_workspace_bytes.argtypes = [_I64, _I64]
        L.nvfp4_verify_draft.restype = ctypes.c_int
        L.nvfp4_verify_draft.argtypes = [_VP] * 6 + [_I64] * 3 + [_VP] * 3 + [ctypes.c_size_t,
                                                                             _VP]
        L.nvfp4_stream_read.restype = ctypes.c_int
        L.nvfp4_stream_read.argtypes = [_VP, ctypes.c_size_t, _VP, _VP]
        L.nvfp4_check_device_faults.restype = ctypes.c_int
        L.nvfp4_check_device_faults.argtypes = [_VP]
        L.nvfp4_debug_set_wait_limit.restype = None
        L.nvfp4_debug_set_wait_limit.argtypes = [ctypes.c_int]
        _lib = L
    return _lib


def _check(fn: str, status: int) -> None:
    if status != 0:
        L = lib()
        detail = (L.nvfp4_last_error() or b"").decode() or \
            L.nvfp4_status_string(status).decode()
        raise Nvfp4Error(fn, status, detail)


# The current stream's raw handle for a device index: torch's own accessor
# when it has one (about 0.06 us a call, against about 1.8 us for building a
# Stream object through torch.cuda.current_stream).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(t: torch.Tensor) -> int:
    if _raw_stream is not None:
        return _raw_stream(t.get_device())
    return torch.cuda.current_stream(t.device).cuda_stream


def _p(t) -> int | None:
    return None if t is None else t.data_ptr()


def _dev(*ts):
    d = None
    for t in ts:
        if t is None:
            continue
        if not t.is_cuda:
            raise ValueError("tensors must be on a HIP device")
        if not t.is_contiguous():
            raise ValueError("tensors must be contiguous")
        if d is None:
            d = t.device
        elif t.device != d:
            raise ValueError("tensors must be on one device")
    return d


def _dtype(t, *dts, name="tensor"):
    if t.dtype not in dts:
        raise TypeError(f"{name} must be one of {dts}, got {t.dtype}")


# ------------------------------------------------------------------ pack

def pack_into(W, codes, scales, gscale, gscale_override=None) -> None:
    _dev(W, codes, scales, gscale, gscale_override)
    _dtype(W, torch.float32, name="W")
    N, K = W.shape
    _check("nvfp4_pack", lib().nvfp4_pack(_p(W), N, K, _p(codes), _p(scales), _p(gscale),
                                          _p(gscale_override), _stream(W)))


def pack(W: torch.Tensor, gscale_override: torch.Tensor | None = None):
    """fp32 W[N, K] -> (codes u8[N, K/2], scales u8[N, K/16], gscale f32[1])."""
    N, K = W.shape
    codes = torch.empty((N, K // 2), dtype=torch.uint8, device=W.device)
    scales = torch.empty((N, K // 16), dtype=torch.uint8, device=W.device)
    gscale = torch.empty((1,), dtype=torch.float32, device=W.device)
    pack_into(W, codes, scales, gscale, gscale_override)
    return codes, scales, gscale


# --------------------------------------------------------------- dequant

def dequant_into(codes, scales, gscale, out) -> None:
    _dev(codes, scales, gscale, out)
    N, K = codes.shape[0], codes.shape[1] * 2
    _check("nvfp4_dequant", lib().nvfp4_dequant(_p(codes), _p(scales), _p(gscale), N, K,
                                                _p(out), _stream(codes)))


def dequant(codes, scales, gscale) -> torch.Tensor:
    N, K = codes.shape[0], codes.shape[1] * 2
    out = torch.empty((N, K), dtype=torch.float32, device=codes.device)
    dequant_into(codes, scales, gscale, out)
    return out


# ----------------------------------------------------------- measurement

def stream_read(buf: torch.Tensor, sink: torch.Tensor, nbytes: int | None = None) -> None:
    """Read the first `nbytes` (default: all) bytes of `buf` once on the
    device (the read-bandwidth ceiling of the benchmark); `sink` is a
    uint32/int32 [1] device tensor that keeps the loads alive."""
    _dev(buf, sink)
    n = buf.numel() * buf.element_size() if nbytes is None else int(nbytes)
    _check("nvfp4_stream_read", lib().nvfp4_stream_read(_p(buf), n, _p(sink), _stream(buf)))


# ------------------------------------------------------------ diagnostics

def check_device_faults(stream=None) -> None:
    """Wait for `stream` (default: torch's current stream) and raise if a
    kernel gave up a bounded internal wait since the last check (the fault
    word is cleared by the read)."""
    s = torch.cuda.current_stream() if stream is None else stream
    _check("nvfp4_check_device_faults", lib().nvfp4_check_device_faults(s.cuda_stream))


def debug_set_wait_limit(polls: int) -> None:
    """Test hook: polls before the split-K slot wait gives up (0: default,
    negative: give up at once)."""
    lib().nvfp4_debug_set_wait_limit(int(polls))


# ------------------------------------------------------------------ gemv

def gemv_into(codes, scales, gscale, x, y) -> None:
    """y[M, N] (fp32) = g * decode(W) . x^T for bf16 x[M, K]."""
    _dev(codes, scales, gscale, x, y)
    _dtype(x, torch.bfloat16, torch.int16, torch.uint16, name="x")
    _dtype(y, torch.float32, name="y")
    N, K = codes.shape[0], codes.shape[1] * 2
    M = x.shape[0]
    if x.shape[1] != K or tuple(y.shape) != (M, N):
        raise ValueError(f"shape mismatch: codes {tuple(codes.shape)}, x {tuple(x.shape)}, "
                         f"y {tuple(y.shape)}")
    _check("nvfp4_gemv", lib().nvfp4_gemv(_p(codes), _p(scales), _p(gscale), _p(x), M, N, K,
                                          _p(y), _stream(codes)))


def gemv(codes, scales, gscale, x) -> torch.Tensor:
    y = torch.empty((x.shape[0], codes.shape[0]), dtype=torch.float32, device=codes.device)
    gemv_into(codes, scales, gscale, x, y)
    return y


def gemv_segments_into(mats, x, ys) -> None:
    """One launch for several matrices reading the same x[M, K]:
    ys[s] = g_s * decode(W_s) . x^T, mats[s] = (codes, scales, gscale)."""
    if len(mats) != len(ys):
        raise ValueError("one output per matrix")
    if len(mats) > MAX_SEGMENTS:
        raise ValueError(f"at most {MAX_SEGMENTS} matrices per launch")
    _dev(x, *ys, *[t for m in mats for t in m])
    _dtype(x, torch.bfloat16, torch.int16, torch.uint16, name="x")
    M, K = x.shape
    segs = (GemvSegment * max(1, len(mats)))()
    for i, ((c, sc, g), y) in enumerate(zip(mats, ys)):
        _dtype(y, torch.float32, name="y")
        N = c.shape[0]
        if c.shape[1] * 2 != K or tuple(y.shape) != (M, N):
            raise ValueError(f"segment {i}: codes {tuple(c.shape)}, x {tuple(x.shape)}, "
                             f"y {tuple(y.shape)}")
        segs[i] = GemvSegment(_p(c), _p(sc), _p(g), _p(y), N)
    _check("nvfp4_gemv_segments",
           lib().nvfp4_gemv_segments(segs, len(mats), _p(x), M, K, _stream(x)))


def gemv_segments(mats, x):
    """[y_s] for mats = [(codes, scales, gscale), ...] sharing x (one launch)."""
    ys = [torch.empty((x.shape[0], c.shape[0]), dtype=torch.float32, device=x.device)
          for c, _, _ in mats]
    gemv_segments_into(mats, x, ys)
    return ys


# ------------------------------------------------------------------ w4a4

def quantize_act_into(x, gscale_x, codes_x, scales_x) -> None:
    """bf16 x[M, K] -> NVFP4 codes_x u8[M, K/2], scales_x u8[M, K/16] with the
    static input scale gscale_x (fp32 [1])."""
    _dev(x, gscale_x, codes_x, scales_x)
    _dtype(x, torch.bfloat16, torch.int16, torch.uint16, name="x")
    M, K = x.shape
    if tuple(codes_x.shape) != (M, K // 2) or tuple(scales_x.shape) != (M, K // 16):
        raise ValueError("codes_x / scales_x have the wrong shape")
    _check("nvfp4_quantize_act", lib().nvfp4_quantize_act(
        _p(x), M, K, _p(gscale_x), _p(codes_x), _p(scales_x), _stream(x)))


def quantize_act(x, gscale_x):
    M, K = x.shape
    codes_x = torch.empty((M, K // 2), dtype=torch.uint8, device=x.device)
    scales_x = torch.empty((M, K // 16), dtype=torch.uint8, device=x.device)
    quantize_act_into(x, gscale_x, codes_x, scales_x)
    return codes_x, scales_x


def gemv_w4a4_workspace_bytes(M: int, K: int) -> int:
    return int(lib().nvfp4_gemv_w4a4_workspace_bytes(M, K))


def gemv_w4a4_into(codes, scales, gscale, codes_x, scales_x, gscale_x, y, workspace) -> None:
    """y[M, N] (fp32) = g_w g_x decode(W) . decode(x)^T, both NVFP4 g16."""
    _dev(codes, scales, gscale, codes_x, scales_x, gscale_x, y, workspace)
    _dtype(y, torch.float32, name="y")
    N, K = codes.shape[0], codes.shape[1] * 2
    M = codes_x.shape[0]
    if codes_x.shape[1] * 2 != K or tuple(scales_x.shape) != (M, K // 16) \
            or tuple(y.shape) != (M, N):
        raise ValueError(f"shape mismatch: codes {tuple(codes.shape)}, codes_x "
                         f"{tuple(codes_x.shape)}, y {tuple(y.shape)}")
    _check("nvfp4_gemv_w4a4", lib().nvfp4_gemv_w4a4(
        _p(codes), _p(scales), _p(gscale), _p(codes_x), _p(scales_x), _p(gscale_x), M, N, K,
        _p(y), _p(workspace), workspace.numel() * workspace.element_size(), _stream(codes)))


def gemv_w4a4(codes, scales, gscale, codes_x, scales_x, gscale_x,
              workspace: torch.Tensor | None = None) -> torch.Tensor:
    M, K = codes_x.shape[0], codes_x.shape[1] * 2
    if workspace is None:
        workspace = torch.empty(max(gemv_w4a4_workspace_bytes(M, K), 256), dtype=torch.uint8,
                                device=codes.device)
    y = torch.empty((M, codes.shape[0]), dtype=torch.float32, device=codes.device)
    gemv_w4a4_into(codes, scales, gscale, codes_x, scales_x, gscale_x, y, workspace)
    return y


def gemv_w4a4_segments_into(mats, codes_x, scales_x, gscale_x, ys, workspace) -> None:
    """One launch (two at M >= 3) for several weight matrices on the same
    NVFP4 activations: ys[s] = g_s g_x decode(W_s) . decode(x)^T,
    mats[s] = (codes, scales, gscale)."""
    if len(mats) != len(ys):
        raise ValueError("one output per matrix")
    if len(mats) > MAX_SEGMENTS:
        raise ValueError(f"at most {MAX_SEGMENTS} matrices per launch")
    _dev(codes_x, scales_x, gscale_x, workspace, *ys, *[t for m in mats for t in m])
    M, K = codes_x.shape[0], codes_x.shape[1] * 2
    segs = (GemvSegment * max(1, len(mats)))()
    for i, ((c, sc, g), y) in enumerate(zip(mats, ys)):
        _dtype(y, torch.float32, name="y")
        N = c.shape[0]
        if c.shape[1] * 2 != K or tuple(y.shape) != (M, N):
            raise ValueError(f"segment {i}: codes {tuple(c.shape)}, codes_x "
                             f"{tuple(codes_x.shape)}, y {tuple(y.shape)}")
        segs[i] = GemvSegment(_p(c), _p(sc), _p(g), _p(y), N)
    _check("nvfp4_gemv_w4a4_segments", lib().nvfp4_gemv_w4a4_segments(
        segs, len(mats), _p(codes_x), _p(scales_x), _p(gscale_x), M, K, _p(workspace),
        workspace.numel() * workspace.element_size(), _stream(codes_x)))


def gemv_w4a4_segments(mats, codes_x, scales_x, gscale_x, workspace=None):
    """[y_s] for mats = [(codes, scales, gscale), ...] on the same NVFP4 x."""
    M, K = codes_x.shape[0], codes_x.shape[1] * 2
    if workspace is None:
        workspace = torch.empty(max(gemv_w4a4_workspace_bytes(M, K), 256), dtype=torch.uint8,
                                device=codes_x.device)
    ys = [torch.empty((M, c.shape[0]), dtype=torch.float32, device=codes_x.device)
          for c, _, _ in mats]
    gemv_w4a4_segments_into(mats, codes_x, scales_x, gscale_x, ys, workspace)
    return ys


# ------------------------------------------------------------------- moe

def moe_workspace_bytes(M: int, H: int, I: int, topk: int) -> int:
    return int(lib().nvfp4_moe_workspace_bytes(M, H, I, topk))


def moe_gemv_into(w13_codes, w13_scales, w13_gscale, w2_codes, w2_scales, w2_gscale,
                  x, expert_ids, gate_w, y, workspace) -> None:
    _dev(w13_codes, w13_scales, w13_gscale, w2_codes, w2_scales, w2_gscale, x,
         expert_ids, gate_w, y, workspace)
    _dtype(x, torch.bfloat16, torch.int16, torch.uint16, name="x")
    _dtype(expert_ids, torch.int32, name="expert_ids")
    _dtype(gate_w, torch.float32, name="gate_w")
    E, twoI, Hh = w13_codes.shape
    H, I = Hh * 2, twoI // 2
    M, topk = expert_ids.shape
    if tuple(w2_codes.shape) != (E, H, I // 2) or tuple(x.shape) != (M, H) \
            or tuple(gate_w.shape) != (M, topk) or tuple(y.shape) != (M, H):
        raise ValueError("inconsistent MoE shapes")
    _check("nvfp4_moe_gemv", lib().nvfp4_moe_gemv(
        _p(w13_codes), _p(w13_scales), _p(w13_gscale), _p(w2_codes), _p(w2_scales),
        _p(w2_gscale), _p(x), _p(expert_ids), _p(gate_w), M, E, H, I, topk, _p(y),
        _p(workspace), workspace.numel() * workspace.element_size(), _stream(x)))


def moe_gemv(w13_codes, w13_scales, w13_gscale, w2_codes, w2_scales, w2_gscale, x,
             expert_ids, gate_w, workspace: torch.Tensor | None = None) -> torch.Tensor:
    E, twoI, Hh = w13_codes.shape
    H, I = Hh * 2, twoI // 2
    M, topk = expert_ids.shape
    if workspace is None:
        workspace = torch.empty(max(moe_workspace_bytes(M, H, I, topk), 256),
                                dtype=torch.uint8, device=x.device)
    y = torch.empty((M, H), dtype=torch.float32, device=x.device)
    moe_gemv_into(w13_codes, w13_scales, w13_gscale, w2_codes, w2_scales, w2_gscale, x,
                  expert_ids, gate_w, y, workspace)
    return y


def moe_gemv_noalloc_into(w13_codes, w13_scales, w13_gscale, w2_codes, w2_scales, w2_gscale,
                          x, expert_ids, gate_w, y) -> None:
    """moe_gemv_into without a workspace: the library's own device array
    holds the SwiGLU activations (calls on one device must not overlap)."""
    _dev(w13_codes, w13_scales, w13_gscale, w2_codes, w2_scales, w2_gscale, x,
         expert_ids, gate_w, y)
    _dtype(x, torch.bfloat16, torch.int16, torch.uint16, name="x")
    _dtype(expert_ids, torch.int32, name="expert_ids")
    _dtype(gate_w, torch.float32, name="gate_w")
    E, twoI, Hh = w13_codes.shape
    H, I = Hh * 2, twoI // 2
    M, topk = expert_ids.shape
    if tuple(w2_codes.shape) != (E, H, I // 2) or tuple(x.shape) != (M, H) \
            or tuple(gate_w.shape) != (M, topk) or tuple(y.shape) != (M, H):
        raise ValueError("inconsistent MoE shapes")
    _check("nvfp4_moe_gemv_noalloc", lib().nvfp4_moe_gemv_noalloc(
        _p(w13_codes), _p(w13_scales), _p(w13_gscale), _p(w2_codes), _p(w2_scales),
        _p(w2_gscale), _p(x), _p(expert_ids), _p(gate_w), M, E, H, I, topk, _p(y),
        _stream(x)))


def moe_workspace_layout(M: int, H: int, I: int, topk: int) -> dict:
    """Byte offsets inside the MoE workspace (for inspecting the bf16 SwiGLU
    activations h[M*topk, I] after a call)."""
    S = M * topk
    return {"h": 0, "total": (S * I * 2 + 255) & ~255}


def moe_shared_workspace_bytes(M: int, H: int, I: int, topk: int, I_shared: int) -> int:
    return int(lib().nvfp4_moe_shared_workspace_bytes(M, H, I, topk, I_shared))


def moe_shared_gemv_into(w13_codes, w13_scales, w13_gscale, w2_codes, w2_scales, w2_gscale,
                         x, expert_ids, gate_w, shared, y, workspace) -> None:
    """`shared` = (codes13 [2Is, H/2], scales13 [2Is, H/16], gscale13 [1],
    codes2 [H, Is/2], scales2 [H, Is/16], gscale2 [1]) device tensors."""
    sc13, ss13, sg13, sc2, ss2, sg2 = shared
    _dev(w13_codes, w13_scales, w13_gscale, w2_codes, w2_scales, w2_gscale, x,
         expert_ids, gate_w, y, workspace, sc13, ss13, sg13, sc2, ss2, sg2)
    _dtype(x, torch.bfloat16, torch.int16, torch.uint16, name="x")
    _dtype(expert_ids, torch.int32, name="expert_ids")
    _dtype(gate_w, torch.float32, name="gate_w")
    E, twoI, Hh = w13_codes.shape
    H, I = Hh * 2, twoI // 2
    M, topk = expert_ids.shape
    Is = sc13.shape[0] // 2
    if tuple(w2_codes.shape) != (E, H, I // 2) or tuple(x.shape) != (M, H) \
            or tuple(gate_w.shape) != (M, topk) or tuple(y.shape) != (M, H) \
            or tuple(sc13.shape) != (2 * Is, H // 2) or tuple(sc2.shape) != (H, Is // 2):
        raise ValueError("inconsistent MoE shapes")
    sh = MoeShared(_p(sc13), _p(ss13), _p(sg13), _p(sc2), _p(ss2), _p(sg2), Is)
    _check("nvfp4_moe_shared_gemv", lib().nvfp4_moe_shared_gemv(
        _p(w13_codes), _p(w13_scales), _p(w13_gscale), _p(w2_codes), _p(w2_scales),
        _p(w2_gscale), _p(x), _p(expert_ids), _p(gate_w), M, E, H, I, topk, ctypes.byref(sh),
        _p(y), _p(workspace), workspace.numel() * workspace.element_size(), _stream(x)))


def moe_shared_gemv(w13_codes, w13_scales, w13_gscale, w2_codes, w2_scales, w2_gscale, x,
                    expert_ids, gate_w, shared,
                    workspace: torch.Tensor | None = None) -> torch.Tensor:
    E, twoI, Hh = w13_codes.shape
    H, I = Hh * 2, twoI // 2
    M, topk = expert_ids.shape
    Is = shared[0].shape[0] // 2
    if workspace is None:
        workspace = torch.empty(max(moe_shared_workspace_bytes(M, H, I, topk, Is), 256),
                                dtype=torch.uint8, device=x.device)
    y = torch.empty((M, H), dtype=torch.float32, device=x.device)
    moe_shared_gemv_into(w13_codes, w13_scales, w13_gscale, w2_codes, w2_scales, w2_gscale, x,
                         expert_ids, gate_w, shared, y, workspace)
    return y


def moe_shared_workspace_layout(M: int, H: int, I: int, topk: int, I_shared: int) -> dict:
    """Byte offsets inside the workspace of nvfp4_moe_shared_gemv: the routed
    h[M*topk, I] and the shared hs[M, I_shared] bf16 activations."""
    hs = (M * topk * I * 2 + 255) & ~255
    return {"h": 0, "hs": hs, "total": (hs + M * I_shared * 2 + 255) & ~255}


def moe_w4a4_workspace_bytes(M: int, H: int, I: int, topk: int, I_shared: int = 0) -> int:
    return int(lib().nvfp4_moe_w4a4_workspace_bytes(M, H, I, topk, I_shared))


def moe_w4a4_gemv_into(w13_codes, w13_scales, w13_gscale, w2_codes, w2_scales, w2_gscale,
                       x, gscale_x, gscale_h, expert_ids, gate_w, y, workspace,
                       shared=None) -> None:
    """W4A4 routed experts (static input scales gscale_x for x and gscale_h
    for h, fp32 [1] device tensors) and an optional W4A16 shared expert
    (the tuple of moe_shared_gemv_into)."""
    extra = list(shared) if shared is not None else []
    _dev(w13_codes, w13_scales, w13_gscale, w2_codes, w2_scales, w2_gscale, x, gscale_x,
         gscale_h, expert_ids, gate_w, y, workspace, *extra)
    _dtype(x, torch.bfloat16, torch.int16, torch.uint16, name="x")
    _dtype(expert_ids, torch.int32, name="expert_ids")
    _dtype(gate_w, torch.float32, name="gate_w")
    _dtype(gscale_x, torch.float32, name="gscale_x")
    _dtype(gscale_h, torch.float32, name="gscale_h")
    E, twoI, Hh = w13_codes.shape
    H, I = Hh * 2, twoI // 2
    M, topk = expert_ids.shape
    if tuple(w2_codes.shape) != (E, H, I // 2) or tuple(x.shape) != (M, H) \
            or tuple(gate_w.shape) != (M, topk) or tuple(y.shape) != (M, H):
        raise ValueError("inconsistent MoE shapes")
    sh = None
    if shared is not None:
        sc13, ss13, sg13, sc2, ss2, sg2 = shared
        Is = sc13.shape[0] // 2
        if tuple(sc13.shape) != (2 * Is, H // 2) or tuple(sc2.shape) != (H, Is // 2):
            raise ValueError("inconsistent shared expert shapes")
        sh = MoeShared(_p(sc13), _p(ss13), _p(sg13), _p(sc2), _p(ss2), _p(sg2), Is)
    _check("nvfp4_moe_w4a4_gemv", lib().nvfp4_moe_w4a4_gemv(
        _p(w13_codes), _p(w13_scales), _p(w13_gscale), _p(w2_codes), _p(w2_scales),
        _p(w2_gscale), _p(x), _p(gscale_x), _p(gscale_h), _p(expert_ids), _p(gate_w),
        M, E, H, I, topk, ctypes.byref(sh) if sh is not None else None,
        _p(y), _p(workspace), workspace.numel() * workspace.element_size(), _stream(x)))


def moe_w4a4_gemv(w13_codes, w13_scales, w13_gscale, w2_codes, w2_scales, w2_gscale, x,
                  gscale_x, gscale_h, expert_ids, gate_w, shared=None,
                  workspace: torch.Tensor | None = None) -> torch.Tensor:
    E, twoI, Hh = w13_codes.shape
    H, I = Hh * 2, twoI // 2
    M, topk = expert_ids.shape
    Is = shared[0].shape[0] // 2 if shared is not None else 0
    if workspace is None:
        workspace = torch.empty(max(moe_w4a4_workspace_bytes(M, H, I, topk, Is), 256),
                                dtype=torch.uint8, device=x.device)
    y = torch.empty((M, H), dtype=torch.float32, device=x.device)
    moe_w4a4_gemv_into(w13_codes, w13_scales, w13_gscale, w2_codes, w2_scales, w2_gscale, x,
                       gscale_x, gscale_h, expert_ids, gate_w, y, workspace, shared=shared)
    return y


def moe_w4a4_workspace_layout(M: int, H: int, I: int, topk: int, I_shared: int = 0) -> dict:
    """Byte offsets inside the workspace of nvfp4_moe_w4a4_gemv: h[M*topk, I]
    (bf16 SwiGLU output), hs[M, I_shared], and h and x on the NVFP4 grid
    (bf16 e2m1 * s): hq[M*topk, I], xq[M, H]."""
    def a(v):
        return (v + 255) & ~255
    hs = a(M * topk * I * 2)
    hq = a(hs + M * I_shared * 2)
    xq = a(hq + M * topk * I * 2)
    return {"h": 0, "hs": hs, "hq": hq, "xq": xq, "total": a(xq + M * H * 2)}


# ------------------------------------------------- between the GEMVs: norms
# These calls take a few microseconds on the device, so their checks are kept
# to what the C side cannot see, one attribute at a time.

# The current device's index without the initialisation check of
# torch.cuda.current_device (a device tensor is at hand wherever it is asked).
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _same_device(d, *ts) -> None:
    """Tensors (None is skipped) on the HIP device of index d (-1: none), which
    must be the current one: the library launches there."""
    if d < 0:
        raise ValueError("tensors must be on a HIP device")
    if d != _current_device():
        raise ValueError(f"tensors are on device {d}, the current one is {_current_device()}")
    for t in ts:
        if t is not None and t.get_device() != d:
            raise ValueError("tensors must be on one HIP device")


def _contiguous(*ts) -> None:
    for t in ts:
        if t is not None and not t.is_contiguous():
            raise ValueError("tensors must be contiguous")


def _norm_args(x, weight, residual, residual_out, *outs):
    """The arguments that the three norms share, checked."""
    _same_device(x.get_device(), weight, residual, residual_out, *outs)
    _contiguous(x, weight, residual, residual_out, *outs)
    xt = _ACT_TYPES.get(x.dtype)
    if xt is None or weight.dtype is not torch.bfloat16:
        raise TypeError(f"x must be bf16 or fp32 and weight bf16, got {x.dtype}, {weight.dtype}")
    M, H = shape = x.shape
    if weight.shape != (H,):
        raise ValueError(f"weight must have shape ({H},), got {tuple(weight.shape)}")
    if residual is None:
        if residual_out is not None:
            raise ValueError("residual and residual_out go together")
        return x.data_ptr(), xt, None, None, 0, weight.data_ptr(), M, H
    if residual_out is None:
        raise ValueError("residual and residual_out go together")
    rt = _ACT_TYPES.get(residual.dtype)
    if rt is None or residual_out.dtype is not residual.dtype:
        raise TypeError("residual must be bf16 or fp32, residual_out the same")
    if residual.shape != shape or residual_out.shape != shape:
        raise ValueError("residual and residual_out must have x's shape")
    return (x.data_ptr(), xt, residual.data_ptr(), residual_out.data_ptr(), rt,
            weight.data_ptr(), M, H)


def add_rmsnorm_into(x, weight, eps, y, residual=None, residual_out=None) -> None:
    """y[M, H] (bf16) = s rsqrt(mean s^2 + eps) weight with s = x + residual,
    which goes to residual_out (may be residual itself). x is bf16 or fp32
    (a GEMV's output), so is the residual."""
    *a, M, H = _norm_args(x, weight, residual, residual_out, y)
    if y.dtype is not torch.bfloat16 or y.shape != x.shape:
        raise ValueError("y must be bf16 and have x's shape")
    _check("nvfp4_add_rmsnorm", lib().nvfp4_add_rmsnorm(*a, eps, M, H, y.data_ptr(), _stream(x)))


def add_rmsnorm(x, weight, eps, residual=None):
    """(y, residual_out); residual_out is None without a residual."""
    y = torch.empty(x.shape, dtype=torch.bfloat16, device=x.device)
    r = None if residual is None else torch.empty_like(residual)
    add_rmsnorm_into(x, weight, eps, y, residual, r)
    return y, r


def add_rmsnorm_e4m3_into(x, weight, eps, y8, scales, residual=None, residual_out=None) -> None:
    """add_rmsnorm_into with y8 (float8_e4m3fn [M, H]) and scales fp32
    [M, H / group]: groups of 32, 64 or 128, or a whole row ([M, 1])."""
    *a, M, H = _norm_args(x, weight, residual, residual_out, y8, scales)
    if y8.dtype is not torch.float8_e4m3fn or scales.dtype is not torch.float32 \
            or y8.shape != x.shape or scales.dim() != 2 or scales.shape[0] != M:
        raise ValueError("y8 must be float8_e4m3fn with x's shape, scales fp32 [M, H / group]")
    n = scales.shape[1]
    if n < 1 or H % n:
        raise ValueError(f"scales has {n} columns, which do not divide H = {H}")
    group = 0 if n == 1 else H // n
    _check("nvfp4_add_rmsnorm_e4m3", lib().nvfp4_add_rmsnorm_e4m3(
        *a, eps, M, H, group, y8.data_ptr(), scales.data_ptr(), _stream(x)))


def add_rmsnorm_e4m3(x, weight, eps, residual=None, group: int = 0):
    """(y8, scales, residual_out); group 0 (a scale for each row), 32, 64 or
    128, dividing H."""
    M, H = x.shape
    if group not in (0, 32, 64, 128) or (group and H % group):
        raise ValueError(f"group must be 0, 32, 64 or 128 and divide H = {H}, got {group}")
    y8 = torch.empty((M, H), dtype=torch.float8_e4m3fn, device=x.device)
    scales = torch.empty((M, H // group if group else 1), dtype=torch.float32, device=x.device)
    r = None if residual is None else torch.empty_like(residual)
    add_rmsnorm_e4m3_into(x, weight, eps, y8, scales, residual, r)
    return y8, scales, r


def add_rmsnorm_nvfp4_into(x, weight, eps, gscale, codes, scales, residual=None,
                           residual_out=None) -> None:
    """add_rmsnorm_into with the NVFP4 activations of gemv_w4a4 (static input
    scale gscale, fp32 [1]): codes u8[M, H/2], scales u8[M, H/16]."""
    *a, M, H = _norm_args(x, weight, residual, residual_out, gscale, codes, scales)
    if gscale.dtype is not torch.float32 or codes.dtype is not torch.uint8 \
            or scales.dtype is not torch.uint8 or codes.shape != (M, H // 2) \
            or scales.shape != (M, H // 16) or gscale.numel() != 1:
        raise ValueError("gscale must be fp32 [1], codes u8 [M, H/2], scales u8 [M, H/16]")
    _check("nvfp4_add_rmsnorm_nvfp4", lib().nvfp4_add_rmsnorm_nvfp4(
        *a, eps, M, H, gscale.data_ptr(), codes.data_ptr(), scales.data_ptr(), _stream(x)))


def add_rmsnorm_nvfp4(x, weight, eps, gscale, residual=None):
    """(codes, scales, residual_out)."""
    M, H = x.shape
    codes = torch.empty((M, H // 2), dtype=torch.uint8, device=x.device)
    scales = torch.empty((M, H // 16), dtype=torch.uint8, device=x.device)
    r = None if residual is None else torch.empty_like(residual)
    add_rmsnorm_nvfp4_into(x, weight, eps, gscale, codes, scales, residual, r)
    return codes, scales, r


# -------------------------------------------- between the GEMVs: attention

def _kv_cache(k_cache, v_cache, k_scale, v_scale) -> KvCache:
    """The descriptor of caches [blocks, page, heads, D] (any strides with
    contiguous elements, the same for both)."""
    ct = _CACHE_TYPES.get(k_cache.dtype)
    if ct is None or v_cache.dtype is not k_cache.dtype:
        raise TypeError("the caches must both be bf16 or float8_e4m3fn")
    st, sv = k_cache.stride(), v_cache.stride()
    # the stride of a dimension of one says nothing
    if k_cache.dim() != 4 or v_cache.shape != k_cache.shape or st[3] != 1 \
            or (sv != st and any(n > 1 and a != b for n, a, b in zip(k_cache.shape, st, sv))):
        raise ValueError("the caches must have one shape [blocks, page, heads, D] and the same "
                         "strides, the last one 1")
    nb, page, heads, D = k_cache.shape
    if ct == _E4M3:
        if k_scale is None or v_scale is None:
            raise ValueError("an e4m3 cache needs k_scale and v_scale")
        if k_scale.dtype is not torch.float32 or v_scale.dtype is not torch.float32 \
                or k_scale.numel() != 1 or v_scale.numel() != 1:
            raise TypeError("k_scale and v_scale must be fp32 [1]")
        ks, vs = k_scale.data_ptr(), v_scale.data_ptr()
    else:
        ks = vs = None
    return KvCache(k_cache.data_ptr(), v_cache.data_ptr(), ks, vs, nb, page, heads, D,
                   st[0] if nb > 1 else D, st[1] if page > 1 else D, st[2] if heads > 1 else D,
                   ct)


def rope_append_into(q, k, v, positions, slots, inv_freq, q_out, k_cache, v_cache, k_scale=None,
                     v_scale=None, interleaved: bool = False, rope_scale: float = 1.0) -> None:
    """Rotary positions of q[T, Hq, D] and k[T, Hkv, D] (bf16 or fp32; a
    token's heads contiguous, tokens at any stride, so views of one fused
    projection), q to q_out (bf16 [T, Hq, D]), k and v into the pages
    k_cache, v_cache[blocks, page, Hkv, D] at slots (int64 [T], page number *
    page size + place; outside the cache: not written). positions int64 [T];
    inv_freq fp32 [R / 2] turns the first R elements of each head. q and q_out
    may be None (only append); k, v, slots and the caches may be (only
    rotate)."""
    x = k if q is None else q
    if x is None:
        raise ValueError("neither q nor k is given")
    if (k is None) != (v is None) or (k is not None and (k_cache is None or v_cache is None)):
        raise ValueError("k, v and the caches go together")
    _same_device(x.get_device(), q, k, v, positions, slots, inv_freq, q_out, k_cache, v_cache,
                 k_scale, v_scale)
    c = None if k is None else _kv_cache(k_cache, v_cache, k_scale, v_scale)
    _rope_append("nvfp4_rope_append", lib().nvfp4_rope_append, x, q, k, v, positions, slots,
                 inv_freq, q_out, c, interleaved, rope_scale)


def _rope_append(name, fn, x, q, k, v, positions, slots, inv_freq, q_out, c, interleaved,
                 rope_scale) -> None:
    """The call of either append; x: q or k, c: the cache's descriptor (with k)."""
    xt = _ACT_TYPES.get(x.dtype)
    if xt is None:
        raise TypeError(f"q, k and v must be bf16 or fp32, got {x.dtype}")
    T, _, D = x.shape
    if positions.dtype is not torch.int64 or positions.shape != (T,) \
            or not positions.is_contiguous():
        raise ValueError("positions must be contiguous int64 [T]")
    if inv_freq.dtype is not torch.float32 or inv_freq.dim() != 1 or not inv_freq.is_contiguous():
        raise ValueError("inv_freq must be contiguous fp32 [R / 2]")
    qp = qs = op = kp = ks = vp = vs = sp = cache = None
    Hq = 0
    if q is not None:
        Hq, st = q.shape[1], q.stride()
        if st[2] != 1 or (st[1] != D and Hq > 1):
            raise ValueError("the heads of a token of q must be contiguous")
        if q_out is None or q_out.dtype is not torch.bfloat16 or q_out.shape != q.shape \
                or not q_out.is_contiguous():
            raise ValueError("q_out must be contiguous bf16 with q's shape")
        qp, qs, op = q.data_ptr(), st[0], q_out.data_ptr()
        if T == 1:   # one token's stride says nothing
            qs = Hq * D
    if k is not None:
        Hkv, st, sv = c.n_kv_heads, k.stride(), v.stride()
        if k.dtype is not x.dtype or v.dtype is not x.dtype or k.shape != (T, Hkv, D) \
                or v.shape != k.shape or c.D != D:
            raise ValueError(f"k and v must be {x.dtype} [{T}, {Hkv}, {c.D}], got "
                             f"{tuple(k.shape)}, {tuple(v.shape)}")
        if st[2] != 1 or sv[2] != 1 or ((st[1] != D or sv[1] != D) and Hkv > 1):
            raise ValueError("the heads of a token of k and v must be contiguous")
        if slots is None or slots.dtype is not torch.int64 or slots.shape != (T,) \
                or not slots.is_contiguous():
            raise ValueError("slots must be contiguous int64 [T]")
        kp, ks, vp, vs, sp = k.data_ptr(), st[0], v.data_ptr(), sv[0], slots.data_ptr()
        if T == 1:
            ks = vs = Hkv * D
        cache = ctypes.byref(c)
    _check(name, fn(
        qp, qs or 0, kp, ks or 0, vp, vs or 0, xt, positions.data_ptr(), sp,
        inv_freq.data_ptr(), T, Hq, D, 2 * inv_freq.shape[0], 1 if interleaved else 0,
        rope_scale, op, cache, _stream(x)))


def rope_append(q, k, v, positions, slots, inv_freq, k_cache, v_cache, k_scale=None, v_scale=None,
                interleaved: bool = False, rope_scale: float = 1.0):
    """q_out (bf16 [T, Hq, D]; None without q)."""
    q_out = None if q is None else torch.empty(q.shape, dtype=torch.bfloat16, device=q.device)
    rope_append_into(q, k, v, positions, slots, inv_freq, q_out, k_cache, v_cache, k_scale,
                     v_scale, interleaved, rope_scale)
    return q_out


def _kv_cache4(k_cache, v_cache) -> KvCache4:
    """The descriptor of an NVFP4 cache: two triples (codes u8 [blocks, page,
    heads, D / 2], scales u8 [blocks, page, heads, D / 16], gscale fp32 [1]), any
    strides with contiguous bytes, the same for both."""
    (kc, ks, kg), (vc, vs, vg) = k_cache, v_cache
    if kc.dtype is not torch.uint8 or vc.dtype is not torch.uint8 \
            or ks.dtype is not torch.uint8 or vs.dtype is not torch.uint8 \
            or kg.dtype is not torch.float32 or vg.dtype is not torch.float32 \
            or kg.numel() != 1 or vg.numel() != 1:
        raise TypeError("codes and scales must be uint8, gscale fp32 [1]")
    if kc.dim() != 4 or vc.shape != kc.shape or vs.shape != ks.shape \
            or ks.shape != (*kc.shape[:3], kc.shape[3] // 8) or kc.shape[3] % 32:
        raise ValueError("codes must be [blocks, page, heads, D / 2], D a multiple of 64, and "
                         "scales [blocks, page, heads, D / 16]")
    for a, b in ((kc, vc), (ks, vs)):
        st, sv = a.stride(), b.stride()
        # the stride of a dimension of one says nothing
        if st[3] != 1 or sv[3] != 1 or \
                (sv != st and any(n > 1 and x != y for n, x, y in zip(a.shape, st, sv))):
            raise ValueError("codes (scales) of k and v must have the same strides, the last one 1")
    nb, page, heads, half = kc.shape
    st, ss = kc.stride(), ks.stride()

    def strides(s, n):   # (of a dimension of one: any that is allowed)
        any_ = (n + 15) // 16 * 16
        return (s[0] if nb > 1 else any_, s[1] if page > 1 else any_, s[2] if heads > 1 else any_)
    return KvCache4(kc.data_ptr(), vc.data_ptr(), ks.data_ptr(), vs.data_ptr(), kg.data_ptr(),
                    vg.data_ptr(), nb, page, heads, 2 * half, *strides(st, half),
                    *strides(ss, half // 8))


def rope_append_nvfp4_into(q, k, v, positions, slots, inv_freq, q_out, k_cache, v_cache,
                           interleaved: bool = False, rope_scale: float = 1.0) -> None:
    """rope_append_into with an NVFP4 cache: k_cache and v_cache are triples
    (codes u8 [blocks, page, Hkv, D / 2], scales u8 [blocks, page, Hkv, D / 16],
    gscale fp32 [1])."""
    x = k if q is None else q
    if x is None:
        raise ValueError("neither q nor k is given")
    if (k is None) != (v is None):
        raise ValueError("k and v go together")
    _same_device(x.get_device(), q, k, v, positions, slots, inv_freq, q_out, *k_cache, *v_cache)
    c = _kv_cache4(k_cache, v_cache)
    _rope_append("nvfp4_rope_append_nvfp4", lib().nvfp4_rope_append_nvfp4, x, q, k, v, positions,
                 slots, inv_freq, q_out, c, interleaved, rope_scale)


def rope_append_nvfp4(q, k, v, positions, slots, inv_freq, k_cache, v_cache,
                      interleaved: bool = False, rope_scale: float = 1.0):
    """q_out (bf16 [T, Hq, D]; None without q)."""
    q_out = None if q is None else torch.empty(q.shape, dtype=torch.bfloat16, device=q.device)
    rope_append_nvfp4_into(q, k, v, positions, slots, inv_freq, q_out, k_cache, v_cache,
                           interleaved, rope_scale)
    return q_out


def paged_attention_workspace_bytes(B: int, Q: int, Hq: int, Hkv: int, D: int) -> int:
    return int(lib().nvfp4_paged_attention_workspace_bytes(B, Q, Hq, Hkv, D))


def paged_attention_into(q, k_cache, v_cache, block_table, seq_lens, out, workspace,
                         scale: float | None = None, window: int = 0, k_scale=None,
                         v_scale=None) -> None:
    """Attention of the T / B newest tokens of each of B sequences over pages
    k_cache, v_cache[blocks, page, Hkv, D] (bf16, or e4m3 with k_scale,
    v_scale fp32 [1]). q and out bf16 [T, Hq, D], sequence by sequence;
    block_table int32 [B, max_blocks]; seq_lens int32 [B], the new tokens
    included; scale defaults to D ** -0.5; window > 0: each token sees the
    last `window` keys up to itself."""
    _same_device(q.get_device(), k_cache, v_cache, block_table, seq_lens, out, workspace, k_scale,
                 v_scale)
    _paged_attention("nvfp4_paged_attention", lib().nvfp4_paged_attention, q,
                     _kv_cache(k_cache, v_cache, k_scale, v_scale), block_table, seq_lens, out,
                     workspace, scale, window)


def _paged_attention(name, fn, q, c, block_table, seq_lens, out, workspace, scale, window,
                     *scores) -> None:
    """The call of any attention; c: the cache's descriptor."""
    if q.dtype is not torch.bfloat16 or out.dtype is not torch.bfloat16 \
            or block_table.dtype is not torch.int32 or seq_lens.dtype is not torch.int32:
        raise TypeError("q and out must be bf16, block_table and seq_lens int32")
    _contiguous(q, out, block_table, seq_lens, workspace)
    T, Hq, D = q.shape
    B, width = block_table.shape
    if seq_lens.shape != (B,) or out.shape != q.shape or D != c.D or (T % B if B else T):
        raise ValueError(f"shape mismatch: q {tuple(q.shape)}, out {tuple(out.shape)}, "
                         f"block_table {tuple(block_table.shape)}, seq_lens "
                         f"{tuple(seq_lens.shape)}, D {c.D}")
    _check(name, fn(
        q.data_ptr(), ctypes.byref(c), block_table.data_ptr(), seq_lens.data_ptr(), B,
        T // B if B else 0, Hq, width, D ** -0.5 if scale is None else scale, window, *scores,
        out.data_ptr(), workspace.data_ptr(), workspace.nbytes, _stream(q)))


def paged_attention(q, k_cache, v_cache, block_table, seq_lens, scale: float | None = None,
                    window: int = 0, k_scale=None, v_scale=None,
                    workspace: torch.Tensor | None = None) -> torch.Tensor:
    workspace, out = _attn_outputs(q, block_table, k_cache.shape[2], workspace)
    paged_attention_into(q, k_cache, v_cache, block_table, seq_lens, out, workspace, scale,
                         window, k_scale, v_scale)
    return out


def _attn_outputs(q, block_table, Hkv, workspace):
    """The workspace of an attention call (a new one where None is given) and its
    output."""
    T, Hq, D = q.shape
    B = block_table.shape[0]
    if workspace is None:
        n = paged_attention_workspace_bytes(B, T // B if B else 0, Hq, Hkv, D)
        workspace = torch.empty(max(n, 256), dtype=torch.uint8, device=q.device)
    return workspace, torch.empty_like(q)


def _scores(softcap, slopes, Hq):
    """nvfp4_attn_scores (None: neither cap nor bias)."""
    if slopes is not None:
        if slopes.dtype is not torch.float32 or slopes.shape != (Hq,) \
                or not slopes.is_contiguous():
            raise ValueError(f"slopes must be contiguous fp32 [{Hq}]")
    elif not softcap:
        return None
    return ctypes.byref(AttnScores(softcap, _p(slopes)))


def paged_attention_scored_into(q, k_cache, v_cache, block_table, seq_lens, out, workspace,
                                softcap: float = 0.0, slopes=None, scale: float | None = None,
                                window: int = 0, k_scale=None, v_scale=None) -> None:
    """paged_attention_into with scores z capped (softcap > 0: softcap * tanh(z /
    softcap)), then biased by distance (slopes fp32 [Hq]: + slopes[h] * (key -
    token's position))."""
    _same_device(q.get_device(), k_cache, v_cache, block_table, seq_lens, out, workspace, k_scale,
                 v_scale, slopes)
    _paged_attention("nvfp4_paged_attention_scored", lib().nvfp4_paged_attention_scored, q,
                     _kv_cache(k_cache, v_cache, k_scale, v_scale), block_table, seq_lens, out,
                     workspace, scale, window, _scores(softcap, slopes, q.shape[1]))


def paged_attention_scored(q, k_cache, v_cache, block_table, seq_lens, softcap: float = 0.0,
                           slopes=None, scale: float | None = None, window: int = 0, k_scale=None,
                           v_scale=None, workspace: torch.Tensor | None = None) -> torch.Tensor:
    workspace, out = _attn_outputs(q, block_table, k_cache.shape[2], workspace)
    paged_attention_scored_into(q, k_cache, v_cache, block_table, seq_lens, out, workspace,
                                softcap, slopes, scale, window, k_scale, v_scale)
    return out


def paged_attention_nvfp4_into(q, k_cache, v_cache, block_table, seq_lens, out, workspace,
                               scale: float | None = None, window: int = 0, softcap: float = 0.0,
                               slopes=None) -> None:
    """paged_attention_into over an NVFP4 cache (the triples of
    rope_append_nvfp4_into), with the cap and bias of
    paged_attention_scored_into."""
    _same_device(q.get_device(), block_table, seq_lens, out, workspace, slopes, *k_cache, *v_cache)
    _paged_attention("nvfp4_paged_attention_nvfp4", lib().nvfp4_paged_attention_nvfp4, q,
                     _kv_cache4(k_cache, v_cache), block_table, seq_lens, out, workspace, scale,
                     window, _scores(softcap, slopes, q.shape[1]))


def paged_attention_nvfp4(q, k_cache, v_cache, block_table, seq_lens, scale: float | None = None,
                          window: int = 0, softcap: float = 0.0, slopes=None,
                          workspace: torch.Tensor | None = None) -> torch.Tensor:
    workspace, out = _attn_outputs(q, block_table, k_cache[0].shape[2], workspace)
    paged_attention_nvfp4_into(q, k_cache, v_cache, block_table, seq_lens, out, workspace, scale,
                               window, softcap, slopes)
    return out


# ------------------------------------------- beside the GEMVs: low-rank adapters

def lora_workspace_bytes(M: int, K: int, rank: int, n_segments: int) -> int:
    return int(lib().nvfp4_lora_workspace_bytes(M, K, rank, n_segments))


def lora_segments_into(mats, x, ids, ys, workspace, bases=None, alpha=None, ranks=None) -> None:
    """ys[s][m] = bases[s][m] + alpha[e] B_s[e] (A_s[e] x[m]) with e = ids[m], for
    all rows m (an id outside the adapters: the base alone). mats: per projection
    of x (bf16 [M, K]) its adapters (a bf16 [E, rank, K], b bf16 [E, N, rank]); ids
    int32 [M]; ys fp32 [M, N]; bases: what the projections gave (fp32, ys itself
    for in place; None: zeros); alpha fp32 [E] (None: 1); ranks int32 [E]: how
    many of its ranks an adapter uses (None: all)."""
    if not mats or len(ys) != len(mats) or (bases is not None and len(bases) != len(mats)):
        raise ValueError("mats, ys and bases must have the same length, at least one")
    bases = [None] * len(mats) if bases is None else bases
    flat = [t for m in mats for t in m]
    _same_device(x.get_device(), ids, workspace, alpha, ranks, *flat, *ys, *bases)
    _contiguous(x, ids, workspace, alpha, ranks, *flat, *ys, *bases)
    M, K = x.shape
    E, rank, _ = mats[0][0].shape
    if x.dtype is not torch.bfloat16 or ids.dtype is not torch.int32 \
            or (alpha is not None and alpha.dtype is not torch.float32) \
            or (ranks is not None and ranks.dtype is not torch.int32):
        raise TypeError("x must be bf16, ids and ranks int32, alpha fp32")
    if ids.shape != (M,) or (alpha is not None and alpha.shape != (E,)) \
            or (ranks is not None and ranks.shape != (E,)):
        raise ValueError(f"ids must be [{M}], alpha and ranks [{E}]")
    segs = (LoraSegment * len(mats))()
    for i, ((a, b), base, y) in enumerate(zip(mats, bases, ys)):
        if a.dtype is not torch.bfloat16 or b.dtype is not torch.bfloat16 \
                or y.dtype is not torch.float32 \
                or (base is not None and base.dtype is not torch.float32):
            raise TypeError("a and b must be bf16, bases and ys fp32")
        N = b.shape[1]
        if a.shape != (E, rank, K) or b.shape != (E, N, rank) or y.shape != (M, N) \
                or (base is not None and base.shape != (M, N)):
            raise ValueError(f"projection {i}: a must be [{E}, {rank}, {K}], b [{E}, N, {rank}], "
                             f"base and y [{M}, N]; got {tuple(a.shape)}, {tuple(b.shape)}, "
                             f"{None if base is None else tuple(base.shape)}, {tuple(y.shape)}")
        segs[i] = LoraSegment(a.data_ptr(), b.data_ptr(), _p(base), y.data_ptr(), N)
    _check("nvfp4_lora_segments", lib().nvfp4_lora_segments(
        segs, len(mats), E, rank, ids.data_ptr(), _p(ranks), _p(alpha), x.data_ptr(), M, K,
        workspace.data_ptr(), workspace.nbytes, _stream(x)))


def lora_segments(mats, x, ids, bases=None, alpha=None, ranks=None,
                  workspace: torch.Tensor | None = None):
    """[y_s]."""
    if workspace is None:
        n = lora_workspace_bytes(x.shape[0], x.shape[1], mats[0][0].shape[1], len(mats))
        workspace = torch.empty(max(n, 256), dtype=torch.uint8, device=x.device)
    ys = [torch.empty((x.shape[0], b.shape[1]), dtype=torch.float32, device=x.device)
          for _, b in mats]
    lora_segments_into(mats, x, ids, ys, workspace, bases, alpha, ranks)
    return ys


# ------------------------------------------------- after the LM head: drafts

def verify_draft_workspace_bytes(B: int, V: int) -> int:
    return int(lib().nvfp4_verify_draft_workspace_bytes(B, V))


def verify_draft_into(target_p, draft_p, draft, u_accept, u_sample, tokens, n_accepted, workspace,
                      n_draft=None) -> None:
    """Speculative verification: target_p fp32 [B, Q + 1, V], draft_p fp32
    [B, Q, V] (None: the drafts are certain), draft int32 [B, Q], u_accept
    fp32 [B, Q] and u_sample fp32 [B] in [0, 1); n_draft int32 [B]: how many
    of the drafts are real (None: all). tokens int32 [B, Q + 1]: the kept
    drafts, the token drawn after them, then -1; n_accepted int32 [B]."""
    _same_device(target_p.get_device(), draft_p, draft, u_accept, u_sample, tokens, n_accepted,
                 workspace, n_draft)
    _contiguous(target_p, draft_p, draft, u_accept, u_sample, tokens, n_accepted, workspace,
                n_draft)
    f, i = torch.float32, torch.int32
    if target_p.dtype is not f or (draft_p is not None and draft_p.dtype is not f) \
            or u_accept.dtype is not f or u_sample.dtype is not f or draft.dtype is not i \
            or tokens.dtype is not i or n_accepted.dtype is not i \
            or (n_draft is not None and n_draft.dtype is not i):
        raise TypeError("probabilities and u must be fp32, draft, tokens, n_accepted and n_draft "
                        "int32")
    B, Q1, V = target_p.shape
    Q = Q1 - 1
    if draft.shape != (B, Q) or u_accept.shape != (B, Q) or u_sample.shape != (B,) \
            or tokens.shape != (B, Q1) or n_accepted.shape != (B,) \
            or (draft_p is not None and draft_p.shape != (B, Q, V)) \
            or (n_draft is not None and n_draft.shape != (B,)):
        raise ValueError(f"shapes do not fit target_p {tuple(target_p.shape)}")
    _check("nvfp4_verify_draft", lib().nvfp4_verify_draft(
        target_p.data_ptr(), _p(draft_p), draft.data_ptr(), _p(n_draft), u_accept.data_ptr(),
        u_sample.data_ptr(), B, Q, V, tokens.data_ptr(), n_accepted.data_ptr(),
        workspace.data_ptr(), workspace.nbytes, _stream(target_p)))


def verify_draft(target_p, draft_p, draft, u_accept, u_sample, n_draft=None,
                 workspace: torch.Tensor | None = None):
    """(tokens, n_accepted)."""
    B, Q1, V = target_p.shape
    if workspace is None:
        workspace = torch.empty(max(verify_draft_workspace_bytes(B, V), 256), dtype=torch.uint8,
                                device=target_p.device)
    tokens = torch.empty((B, Q1), dtype=torch.int32, device=target_p.device)
    n_accepted = torch.empty((B,), dtype=torch.int32, device=target_p.device)
    verify_draft_into(target_p, draft_p, draft, u_accept, u_sample, tokens, n_accepted, workspace,
                      n_draft)
    return tokens, n_accepted
