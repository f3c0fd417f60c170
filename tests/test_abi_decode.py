"""Host checks of the entry points of a decode step between the GEMVs (norm,
rotation and append, paged attention, verification of drafts): every call here
is refused, or has nothing to do, before any HIP call. Nothing is launched."""
import ctypes
import re

import pytest
import torch

import nvfp4_block_scaled_gemv_amd as nv

OK, ERR_NULL, ERR_SHAPE, ERR_ALIGN, ERR_UNSUPPORTED, ERR_WORKSPACE, ERR_HIP, ERR_ALIAS = range(8)
BF16, F32, E4M3 = 0, 1, 2

# Fake, never-dereferenced device addresses, far apart.
A = [0x7F0000000000 + i * 0x100000000 for i in range(16)]


@pytest.fixture(scope="module")
def L():
    return nv.lib()


def test_limits_match_the_header():
    text = open(nv.HEADER_PATH).read()
    defs = dict(re.findall(r"#define NVFP4_([A-Z_0-9]+) \(?([0-9]+(?: << [0-9]+)?)\)?", text))
    for name in ("MAX_ROWS", "NORM_MAX_H", "MAX_HEADS", "ROPE_MAX_D", "ATTN_MAX_B", "ATTN_MAX_Q",
                 "VERIFY_MAX_Q", "VERIFY_MAX_B", "VERIFY_MAX_V"):
        assert eval(defs[name]) == getattr(nv, name), name


# ------------------------------------------------------------------- norms

def norm(L, form="bf16", x=A[0], xt=F32, r=A[1], ro=A[2], rt=BF16, w=A[3], eps=1e-6, M=2, H=128,
         y=A[4], extra=A[5], group=0, g=A[6]):
    if form == "bf16":
        return L.nvfp4_add_rmsnorm(x, xt, r, ro, rt, w, eps, M, H, y, None)
    if form == "e4m3":
        return L.nvfp4_add_rmsnorm_e4m3(x, xt, r, ro, rt, w, eps, M, H, group, y, extra, None)
    return L.nvfp4_add_rmsnorm_nvfp4(x, xt, r, ro, rt, w, eps, M, H, g, y, extra, None)


@pytest.mark.parametrize("form", ["bf16", "e4m3", "nvfp4"])
def test_norm_checks(L, form):
    unit = 32 if form == "nvfp4" else 8
    assert norm(L, form, H=128 + unit // 2) == ERR_SHAPE
    assert norm(L, form, M=-1) == ERR_SHAPE
    assert norm(L, form, H=-unit) == ERR_SHAPE
    assert norm(L, form, xt=E4M3) == ERR_SHAPE
    assert norm(L, form, rt=E4M3) == ERR_SHAPE
    assert norm(L, form, eps=-1.0) == ERR_SHAPE
    assert norm(L, form, eps=float("nan")) == ERR_SHAPE
    assert norm(L, form, eps=float("inf")) == ERR_SHAPE
    assert norm(L, form, M=nv.MAX_ROWS + 1) == ERR_UNSUPPORTED
    assert norm(L, form, H=nv.NORM_MAX_H + 128) == ERR_UNSUPPORTED
    assert norm(L, form, M=0) == OK
    assert norm(L, form, H=0) == OK
    assert norm(L, form, x=None) == ERR_NULL
    assert norm(L, form, w=None) == ERR_NULL
    assert norm(L, form, y=None) == ERR_NULL
    assert norm(L, form, ro=None) == ERR_NULL          # residual without residual_out
    assert norm(L, form, r=None) == ERR_NULL           # and the reverse
    assert norm(L, form, x=A[0] + 8) == ERR_ALIGN
    assert norm(L, form, r=A[1] + 8) == ERR_ALIGN
    assert norm(L, form, ro=A[2] + 8) == ERR_ALIGN
    assert norm(L, form, w=A[3] + 8) == ERR_ALIGN
    assert norm(L, form, y=A[4] + 4) == ERR_ALIGN
    assert norm(L, form, y=A[0] + 512) == ERR_ALIAS    # on x
    assert norm(L, form, y=A[1]) == ERR_ALIAS          # on the residual
    assert norm(L, form, y=A[2]) == ERR_ALIAS          # on residual_out
    assert norm(L, form, y=A[3] + 16) == ERR_ALIAS     # on the weight
    assert norm(L, form, ro=A[1] + 16) == ERR_ALIAS    # residual_out shifted over the residual
    assert norm(L, form, ro=A[0]) == ERR_ALIAS         # residual_out on x
    if form != "bf16":
        assert norm(L, form, extra=None) == ERR_NULL
        assert norm(L, form, extra=A[4] + 32) == ERR_ALIAS
    if form == "e4m3":
        assert norm(L, form, extra=A[5] + 2) == ERR_ALIGN
        assert norm(L, form, group=16) == ERR_SHAPE
        assert norm(L, form, group=128, H=192) == ERR_SHAPE
        assert norm(L, form, group=-32) == ERR_SHAPE
    if form == "nvfp4":
        assert norm(L, form, g=None) == ERR_NULL
        assert norm(L, form, g=A[6] + 2) == ERR_ALIGN
        assert norm(L, form, g=A[4]) == ERR_ALIAS      # codes over gscale


# ---------------------------------------------------------- rotation, append

def cache(k=A[8], v=A[9], ks=None, vs=None, nb=4, page=16, heads=2, D=64, sb=None, st=None,
          sh=None, t=BF16):
    st = heads * D if st is None else st
    return nv.KvCache(k, v, ks, vs, nb, page, heads, D, page * st if sb is None else sb, st,
                      D if sh is None else sh, t)


def rope(L, q=A[0], qs=256, k=A[1], ks=128, v=A[2], vs=128, xt=F32, pos=A[3], slots=A[4],
         f=A[5], T=3, Hq=4, D=64, R=64, inter=0, scale=1.0, out=A[6], c="default"):
    c = cache() if c == "default" else c
    return L.nvfp4_rope_append(q, qs, k, ks, v, vs, xt, pos, slots, f, T, Hq, D, R, inter, scale,
                               out, None if c is None else ctypes.byref(c), None)


def test_rope_append_checks(L):
    assert rope(L, T=-1) == ERR_SHAPE
    assert rope(L, D=72, R=64, c=None) == ERR_SHAPE
    assert rope(L, D=0, R=0, c=None) == ERR_SHAPE
    assert rope(L, R=8) == ERR_SHAPE
    assert rope(L, R=80) == ERR_SHAPE                    # past D
    assert rope(L, xt=E4M3) == ERR_SHAPE
    assert rope(L, inter=2) == ERR_SHAPE
    assert rope(L, scale=float("inf")) == ERR_SHAPE
    assert rope(L, scale=float("nan")) == ERR_SHAPE
    assert rope(L, D=128, R=64) == ERR_SHAPE             # not the cache's D
    assert rope(L, qs=255) == ERR_SHAPE                  # shorter than the heads
    assert rope(L, qs=258) == ERR_SHAPE                  # not 16 bytes
    assert rope(L, xt=BF16, ks=132) == ERR_SHAPE
    assert rope(L, vs=64) == ERR_SHAPE
    assert rope(L, qs=(1 << 36) + 4) == ERR_UNSUPPORTED
    assert rope(L, T=nv.MAX_ROWS + 1) == ERR_UNSUPPORTED
    assert rope(L, Hq=nv.MAX_HEADS + 1, qs=1 << 20) == ERR_UNSUPPORTED
    assert rope(L, D=528, R=16, qs=4 * 528, c=None) == ERR_UNSUPPORTED
    assert rope(L, T=0) == OK
    assert rope(L, q=None, k=None, v=None, Hq=0, c=None) == OK
    for name in ("q", "k", "v", "pos", "slots", "f", "out"):
        assert rope(L, **{name: None}) == ERR_NULL, name
    for name, i in (("q", 0), ("k", 1), ("v", 2), ("out", 6)):
        assert rope(L, **{name: A[i] + 8}) == ERR_ALIGN, name
    assert rope(L, pos=A[3] + 4) == ERR_ALIGN
    assert rope(L, slots=A[4] + 4) == ERR_ALIGN
    for name in ("q", "k", "v", "pos", "slots", "f"):     # q_out on every input
        assert rope(L, **{name: A[6]}) == ERR_ALIAS, name
    assert rope(L, out=A[8] + 64) == ERR_ALIAS            # on the cache
    assert rope(L, k=A[9]) == ERR_ALIAS                   # an input inside the cache


def test_cache_checks(L):
    def both(c):
        n = nv.paged_attention_workspace_bytes(1, 1, 4, 2, 64)
        r = L.nvfp4_paged_attention(A[0], ctypes.byref(c), A[1], A[2], 1, 1, 4, 2, 0.125, 0, A[3],
                                    A[4], n, None)
        assert rope(L, c=c) == r
        return r

    assert both(cache(t=F32)) == ERR_SHAPE
    assert both(cache(nb=-1)) == ERR_SHAPE
    assert both(cache(page=0)) == ERR_SHAPE
    assert both(cache(st=56)) == ERR_SHAPE                # a token inside another
    assert both(cache(st=132)) == ERR_SHAPE               # not 16 bytes
    assert both(cache(sh=68)) == ERR_SHAPE
    assert both(cache(sb=1028)) == ERR_SHAPE
    assert both(cache(t=E4M3, ks=A[10], vs=A[11], sh=72)) == ERR_SHAPE   # not 16 bytes
    assert both(cache(page=(1 << 20) + 1, sb=1 << 30)) == ERR_UNSUPPORTED
    assert both(cache(st=1 << 26)) == ERR_UNSUPPORTED
    assert both(cache(sb=1 << 40)) == ERR_UNSUPPORTED
    assert both(cache(nb=1 << 31)) == ERR_UNSUPPORTED
    assert both(cache(k=None)) == ERR_NULL
    assert both(cache(v=None)) == ERR_NULL
    assert both(cache(v=A[8])) == ERR_NULL                # k and v the same array
    assert both(cache(t=E4M3, ks=A[10])) == ERR_NULL
    assert both(cache(t=E4M3, ks=A[10], nb=0)) == ERR_NULL   # read also without a page
    assert both(cache(k=A[8] + 8)) == ERR_ALIGN
    assert both(cache(t=E4M3, ks=A[10] + 2, vs=A[11])) == ERR_ALIGN


# ------------------------------------------------------------ paged attention

def attn(L, q=A[0], c=None, table=A[1], lens=A[2], B=2, Q=3, Hq=4, width=2, scale=0.125, window=0,
         out=A[3], ws=A[4], wb=None):
    c = cache() if c is None else c
    n = nv.paged_attention_workspace_bytes(B, Q, Hq, c.n_kv_heads, c.D) if wb is None else wb
    return L.nvfp4_paged_attention(q, ctypes.byref(c), table, lens, B, Q, Hq, width, scale, window,
                                   out, ws, n, None)


def test_paged_attention_checks(L):
    assert L.nvfp4_paged_attention(A[0], None, A[1], A[2], 1, 1, 4, 2, 0.1, 0, A[3], A[4], 1 << 30,
                                   None) == ERR_NULL
    assert attn(L, B=-1) == ERR_SHAPE
    assert attn(L, Q=-1) == ERR_SHAPE
    assert attn(L, Hq=3) == ERR_SHAPE                     # not a multiple of the heads
    assert attn(L, width=-1) == ERR_SHAPE
    assert attn(L, window=-1) == ERR_SHAPE
    assert attn(L, scale=float("inf")) == ERR_SHAPE
    assert attn(L, scale=float("nan")) == ERR_SHAPE
    assert attn(L, B=nv.ATTN_MAX_B + 1, wb=1 << 30) == ERR_UNSUPPORTED
    assert attn(L, Q=nv.ATTN_MAX_Q + 1, wb=1 << 30) == ERR_UNSUPPORTED
    assert attn(L, Hq=nv.MAX_HEADS + 2, wb=1 << 30) == ERR_UNSUPPORTED
    assert attn(L, c=cache(D=96), wb=1 << 30) == ERR_UNSUPPORTED
    assert attn(L, width=1 << 31) == ERR_UNSUPPORTED
    assert attn(L, window=1 << 31) == ERR_UNSUPPORTED
    # more steps of 128 keys than 31 bits: 4096 sequences of 2^31 keys
    assert attn(L, B=4096, width=0x7FFFFFFF) == ERR_UNSUPPORTED
    # more workgroups than a launch holds: 4096 sequences x 4096 row tiles
    assert attn(L, B=4096, Q=64, Hq=1024, c=cache(heads=1, D=256)) == ERR_UNSUPPORTED
    assert attn(L, B=0, wb=0) == OK
    assert attn(L, Q=0, wb=0) == OK
    assert attn(L, Hq=0, wb=0) == OK
    for name in ("q", "table", "lens", "out"):
        assert attn(L, **{name: None}) == ERR_NULL, name
    assert attn(L, q=A[0] + 8) == ERR_ALIGN
    assert attn(L, out=A[3] + 8) == ERR_ALIGN
    assert attn(L, table=A[1] + 2) == ERR_ALIGN
    assert attn(L, lens=A[2] + 2) == ERR_ALIGN
    need = nv.paged_attention_workspace_bytes(2, 3, 4, 2, 64)
    assert need > 0
    assert attn(L, wb=need - 1) == ERR_WORKSPACE
    assert attn(L, ws=None) == ERR_WORKSPACE
    assert attn(L, ws=A[4] + 64) == ERR_ALIGN
    assert attn(L, out=A[0]) == ERR_ALIAS
    assert attn(L, out=A[8]) == ERR_ALIAS                 # on K
    assert attn(L, out=A[9] + 64) == ERR_ALIAS            # on V
    assert attn(L, out=A[1]) == ERR_ALIAS
    assert attn(L, ws=A[2]) == ERR_ALIAS                  # the workspace on seq_lens
    assert attn(L, ws=A[3]) == ERR_ALIAS                  # and on out
    eight = cache(t=E4M3, ks=A[10], vs=A[11])
    assert attn(L, c=eight, ws=A[11]) == ERR_ALIAS        # and on v_scale


def test_paged_attention_workspace_bytes():
    f = nv.paged_attention_workspace_bytes
    assert f(1, 1, 4, 3, 64) == 0 and f(1, 1, 4, 2, 96) == 0 and f(-1, 1, 4, 2, 64) == 0
    assert f(0, 1, 4, 2, 64) == 0 and f(1, 0, 4, 2, 64) == 0 and f(1, 1, 0, 2, 64) == 0
    assert f(1, 65, 4, 2, 64) == 0 and f(4097, 1, 4, 2, 64) == 0
    # it goes by the rows of a head, not by the sequences
    assert f(1, 1, 32, 8, 128) == f(64, 1, 32, 8, 128) < f(1, 2, 32, 8, 128)


# ----------------------------------------------------------------- verification

def verify(L, p=A[0], q=A[1], d=A[2], n=A[3], ua=A[4], us=A[5], B=2, Q=3, V=1000, tok=A[6],
           acc=A[7], ws=A[8], wb=None):
    wb = nv.verify_draft_workspace_bytes(B, V) if wb is None else wb
    return L.nvfp4_verify_draft(p, q, d, n, ua, us, B, Q, V, tok, acc, ws, wb, None)


def test_verify_draft_checks(L):
    assert verify(L, B=-1) == ERR_SHAPE
    assert verify(L, Q=-1) == ERR_SHAPE
    assert verify(L, V=0) == ERR_SHAPE
    assert verify(L, B=nv.VERIFY_MAX_B + 1, wb=1 << 30) == ERR_UNSUPPORTED
    assert verify(L, Q=nv.VERIFY_MAX_Q + 1) == ERR_UNSUPPORTED
    assert verify(L, V=nv.VERIFY_MAX_V + 1, wb=1 << 30) == ERR_UNSUPPORTED
    assert verify(L, B=0) == OK
    for name in ("p", "d", "ua", "us", "tok", "acc"):
        assert verify(L, **{name: None}) == ERR_NULL, name
    for i, name in enumerate(("p", "q", "d", "n", "ua", "us", "tok", "acc")):
        assert verify(L, **{name: A[i] + 2}) == ERR_ALIGN, name
    need = nv.verify_draft_workspace_bytes(2, 1000)
    assert need >= 2 * 2 * 8
    assert verify(L, wb=need - 1) == ERR_WORKSPACE
    assert verify(L, ws=None) == ERR_WORKSPACE
    assert verify(L, ws=A[8] + 128) == ERR_ALIGN
    for i in range(6):
        assert verify(L, tok=A[i]) == ERR_ALIAS
        assert verify(L, acc=A[i]) == ERR_ALIAS
        assert verify(L, ws=A[i]) == ERR_ALIAS
    assert verify(L, acc=A[6]) == ERR_ALIAS
    assert verify(L, ws=A[7]) == ERR_ALIAS
    assert nv.verify_draft_workspace_bytes(1, 0) == 0
    assert nv.verify_draft_workspace_bytes(-1, 10) == 0


def test_bindings_raise_without_device_tensors():
    bf, f = torch.bfloat16, torch.float32
    x, w = torch.zeros(2, 64), torch.ones(64, dtype=bf)
    with pytest.raises(ValueError):
        nv.add_rmsnorm(x, w, 1e-6)
    c = torch.zeros(2, 16, 1, 64, dtype=bf)
    one = torch.zeros(2, dtype=torch.int64)
    with pytest.raises(ValueError):
        nv.rope_append(torch.zeros(2, 1, 64), torch.zeros(2, 1, 64), torch.zeros(2, 1, 64), one,
                       one, torch.ones(32), c, c.clone())
    with pytest.raises(ValueError):
        nv.paged_attention(torch.zeros(1, 1, 64, dtype=bf), c, c.clone(),
                           torch.zeros(1, 2, dtype=torch.int32), torch.ones(1, dtype=torch.int32))
    with pytest.raises(ValueError):
        nv.verify_draft(torch.zeros(1, 2, 8), None, torch.zeros(1, 1, dtype=torch.int32),
                        torch.zeros(1, 1, dtype=f), torch.zeros(1, dtype=f))
    with pytest.raises(ValueError, match="go together"):      # k without v, or without pages
        nv.rope_append(None, torch.zeros(2, 1, 64), None, one, one, torch.ones(32), c, c.clone())
    with pytest.raises(ValueError, match="go together"):
        nv.rope_append(torch.zeros(2, 1, 64), None, torch.zeros(2, 1, 64), one, one,
                       torch.ones(32), c, c.clone())
    with pytest.raises(ValueError, match="go together"):
        nv.rope_append(None, torch.zeros(2, 1, 64), torch.zeros(2, 1, 64), one, one,
                       torch.ones(32), None, None)
