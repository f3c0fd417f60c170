"""Host checks of the NVFP4 cache's entry points, of scored attention and of the
adapters: every call here is refused, or has nothing to do, before any HIP call.
Nothing is launched."""
import ctypes
import re

import pytest

import nvfp4_block_scaled_gemv_amd as nv

OK, ERR_NULL, ERR_SHAPE, ERR_ALIGN, ERR_UNSUPPORTED, ERR_WORKSPACE, ERR_HIP, ERR_ALIAS = range(8)
BF16, F32, E4M3 = 0, 1, 2

# Fake, never-dereferenced device addresses, far apart.
A = [0x7F0000000000 + i * 0x100000000 for i in range(20)]


@pytest.fixture(scope="module")
def L():
    return nv.lib()


def test_limits_match_the_header():
    text = open(nv.HEADER_PATH).read()
    defs = dict(re.findall(r"#define NVFP4_([A-Z_0-9]+) \(?([0-9]+(?: << [0-9]+)?)\)?", text))
    for name in ("LORA_MAX_RANK", "LORA_MAX_ADAPTERS"):
        assert eval(defs[name]) == getattr(nv, name), name


def cache4(k=A[8], v=A[9], ks=A[10], vs=A[11], kg=A[12], vg=A[13], nb=4, page=16, heads=2, D=64,
           **strides):
    d = dict(stride_block=page * heads * D // 2, stride_token=heads * D // 2, stride_head=D // 2,
             scale_stride_block=page * heads * D // 16, scale_stride_token=heads * D // 16,
             scale_stride_head=D // 16)
    d.update(strides)
    return nv.KvCache4(k, v, ks, vs, kg, vg, nb, page, heads, D, *d.values())


BAD_CACHES = [
    (dict(nb=-1), ERR_SHAPE), (dict(page=0), ERR_SHAPE), (dict(heads=0), ERR_SHAPE),
    (dict(stride_head=16), ERR_SHAPE), (dict(stride_token=72), ERR_SHAPE),
    (dict(stride_block=8), ERR_SHAPE), (dict(scale_stride_head=2), ERR_SHAPE),
    (dict(scale_stride_token=10), ERR_SHAPE), (dict(scale_stride_block=0), ERR_SHAPE),
    (dict(stride_head=-32), ERR_SHAPE), (dict(nb=1 << 31), ERR_UNSUPPORTED),
    (dict(page=(1 << 20) + 1), ERR_UNSUPPORTED), (dict(heads=1025), ERR_UNSUPPORTED),
    (dict(stride_token=1 << 26), ERR_UNSUPPORTED), (dict(scale_stride_token=1 << 26), ERR_UNSUPPORTED),
    (dict(stride_block=1 << 35), ERR_UNSUPPORTED), (dict(stride_head=1 << 40), ERR_UNSUPPORTED),
    (dict(scale_stride_head=1 << 40), ERR_UNSUPPORTED),
    (dict(scale_stride_block=1 << 33), ERR_UNSUPPORTED),
    (dict(nb=1 << 30, stride_block=1 << 29), ERR_UNSUPPORTED),
    (dict(k=None), ERR_NULL), (dict(vs=None), ERR_NULL), (dict(kg=None), ERR_NULL),
    (dict(vg=None, nb=0), ERR_NULL), (dict(v=A[8]), ERR_NULL), (dict(vs=A[10]), ERR_NULL),
    (dict(k=A[8] + 8), ERR_ALIGN), (dict(vs=A[11] + 2), ERR_ALIGN), (dict(kg=A[12] + 2), ERR_ALIGN),
]


def rope(L, q=A[0], qs=256, k=A[1], ks=128, v=A[2], vs=128, xt=F32, pos=A[3], slots=A[4],
         f=A[5], T=3, Hq=4, D=64, R=64, inter=0, scale=1.0, out=A[6], c="default"):
    c = cache4() if c == "default" else c
    return L.nvfp4_rope_append_nvfp4(q, qs, k, ks, v, vs, xt, pos, slots, f, T, Hq, D, R, inter,
                                     scale, out, None if c is None else ctypes.byref(c), None)


def test_append_checks(L):
    assert rope(L, c=None) == ERR_NULL
    assert rope(L, T=-1) == ERR_SHAPE
    assert rope(L, R=8) == ERR_SHAPE
    assert rope(L, xt=E4M3) == ERR_SHAPE
    assert rope(L, inter=2) == ERR_SHAPE
    assert rope(L, D=128) == ERR_SHAPE                   # not the cache's D
    assert rope(L, D=96, c=cache4(D=96, stride_head=48, stride_token=96, stride_block=1536,
                                  scale_stride_head=8, scale_stride_token=16,
                                  scale_stride_block=256)) == ERR_SHAPE
    assert rope(L, D=576, c=cache4(D=576)) == ERR_UNSUPPORTED
    assert rope(L, vs=64) == ERR_SHAPE
    for bad, want in BAD_CACHES:
        assert rope(L, c=cache4(**bad)) == want, bad
    assert rope(L, T=0) == OK
    for name in ("q", "k", "v", "pos", "slots", "f", "out"):
        assert rope(L, **{name: None}) == ERR_NULL, name
    assert rope(L, k=A[1] + 8) == ERR_ALIGN
    # q_out, codes and scales on inputs, q_out on the cache, scales on the gscale
    assert rope(L, out=A[0]) == ERR_ALIAS
    assert rope(L, out=A[8] + 4032) == ERR_ALIAS
    assert rope(L, out=A[11] + 496) == ERR_ALIAS
    for name in ("k", "v", "ks", "vs"):
        for over in (A[1], A[2], A[3], A[4], A[5], A[12], A[13]):
            assert rope(L, c=cache4(**{name: over})) == ERR_ALIAS, (name, hex(over))


def attn(L, q=A[0], c="default", table=A[1], lens=A[2], B=2, Q=1, Hq=4, width=4, scale=0.125,
         window=0, scores=None, out=A[3], ws=A[4], wsb=None, which="nvfp4"):
    c = (cache4() if which == "nvfp4" else
         nv.KvCache(A[8], A[9], None, None, 4, 16, 2, 64, 2048, 128, 64, BF16)) \
        if c == "default" else c
    wsb = (1 << 32) - 256 if wsb is None else wsb
    f = getattr(L, "nvfp4_paged_attention_" + which)
    return f(q, None if c is None else ctypes.byref(c), table, lens, B, Q, Hq, width, scale,
             window, None if scores is None else ctypes.byref(scores), out, ws, wsb, None)


@pytest.mark.parametrize("which", ["nvfp4", "scored"])
def test_attention_checks(L, which):
    def a(**kw):
        return attn(L, which=which, **kw)
    assert a(c=None) == ERR_NULL
    assert a(B=-1) == ERR_SHAPE
    assert a(Hq=5) == ERR_SHAPE                          # not a multiple of the cache's heads
    assert a(width=-1) == ERR_SHAPE
    assert a(window=-1) == ERR_SHAPE
    assert a(scale=float("nan")) == ERR_SHAPE
    for cap in (-1.0, float("nan"), float("inf"), 1e-7, 2e30):
        assert a(scores=nv.AttnScores(cap, None)) == ERR_SHAPE, cap
    assert a(scores=nv.AttnScores(30.0, A[5] + 2)) == ERR_ALIGN
    assert a(B=nv.ATTN_MAX_B + 1) == ERR_UNSUPPORTED
    assert a(Q=nv.ATTN_MAX_Q + 1) == ERR_UNSUPPORTED
    assert a(Hq=1026) == ERR_UNSUPPORTED
    assert a(width=1 << 31) == ERR_UNSUPPORTED
    assert a(B=4096, Q=64, Hq=1024) == ERR_UNSUPPORTED   # sequences times row tiles
    assert a(B=0) == OK and a(Q=0) == OK and a(Hq=0) == OK
    for name in ("q", "table", "lens", "out"):
        assert a(**{name: None}) == ERR_NULL, name
    assert a(q=A[0] + 8) == ERR_ALIGN
    assert a(ws=A[4] + 16) == ERR_ALIGN
    need = L.nvfp4_paged_attention_workspace_bytes(2, 1, 4, 2, 64)
    assert a(wsb=need - 1) == ERR_WORKSPACE and a(ws=None) == ERR_WORKSPACE
    slopes = nv.AttnScores(0.0, A[5])
    for over in (A[0], A[1], A[2], A[8], A[9]):
        assert a(out=over) == ERR_ALIAS, hex(over)
        assert a(ws=over) == ERR_ALIAS, hex(over)
    assert a(out=A[5], scores=slopes) == ERR_ALIAS
    assert a(ws=A[5], scores=slopes) == ERR_ALIAS
    assert a(out=A[4]) == ERR_ALIAS
    if which == "nvfp4":
        for over in (A[10], A[11], A[12], A[13]):
            assert a(out=over) == ERR_ALIAS, hex(over)
            assert a(ws=over) == ERR_ALIAS, hex(over)
        for bad, want in BAD_CACHES:
            assert a(c=cache4(**bad)) == want, bad
        for D in (192, 320, 512):
            assert a(c=cache4(D=D)) == ERR_UNSUPPORTED


def test_workspace_of_any_attention(L):
    """One query serves every cache; it grows neither with B nor with lengths, and
    is 0 for what is refused."""
    w = L.nvfp4_paged_attention_workspace_bytes
    assert w(1, 1, 32, 8, 128) == w(64, 1, 32, 8, 128) > 0
    assert w(1, 1, 32, 8, 96) == 0 and w(0, 1, 32, 8, 128) == 0


def lora(L, segs="default", n=None, E=3, rank=16, ids=A[2], ranks=None, alpha=None, x=A[3], M=2,
         K=64, ws=A[4], wsb=1 << 24):
    if segs == "default":
        segs = [(A[0], A[1], None, A[5], 32)]
    arr = None if segs is None else (nv.LoraSegment * max(len(segs), 1))(
        *[nv.LoraSegment(*s) for s in segs])
    return L.nvfp4_lora_segments(arr, len(segs) if n is None else n, E, rank, ids, ranks, alpha, x,
                                 M, K, ws, wsb, None)


def seg(a=A[0], b=A[1], base=None, y=A[5], N=32):
    return [(a, b, base, y, N)]


def test_lora_checks(L):
    for bad in (dict(n=-1), dict(E=-1), dict(M=-1), dict(K=-32), dict(K=48), dict(rank=0),
                dict(rank=12), dict(rank=-8), dict(segs=seg(N=-1))):
        assert lora(L, **bad) == ERR_SHAPE, bad
    for bad in (dict(n=9), dict(E=nv.LORA_MAX_ADAPTERS + 1), dict(M=nv.MAX_M + 1),
                dict(K=nv.MAX_K + 32), dict(rank=nv.LORA_MAX_RANK + 8),
                dict(segs=seg(N=nv.MAX_N + 1))):
        assert lora(L, **bad) == ERR_UNSUPPORTED, bad
    assert lora(L, segs=[(A[0], A[1], None, A[5], nv.MAX_N // 2 + 1)] * 2) == ERR_UNSUPPORTED
    assert lora(L, n=0) == OK and lora(L, M=0) == OK and lora(L, segs=seg(N=0, y=None)) == OK
    for bad in (dict(segs=None, n=1), dict(segs=seg(a=None)), dict(segs=seg(b=None)),
                dict(segs=seg(y=None)), dict(ids=None), dict(x=None)):
        assert lora(L, **bad) == ERR_NULL, bad
    for bad in (dict(segs=seg(a=A[0] + 8)), dict(segs=seg(b=A[1] + 8)), dict(segs=seg(y=A[5] + 2)),
                dict(segs=seg(base=A[6] + 2)), dict(ids=A[2] + 2), dict(ranks=A[6] + 1),
                dict(alpha=A[6] + 1), dict(x=A[3] + 8), dict(ws=A[4] + 128)):
        assert lora(L, **bad) == ERR_ALIGN, bad
    need = nv.lora_workspace_bytes(2, 64, 16, 1)
    assert need >= 2 * 16 * 4
    assert lora(L, wsb=need - 1) == ERR_WORKSPACE and lora(L, ws=None) == ERR_WORKSPACE
    for over in (A[0], A[1], A[2], A[3], A[6], A[7]):
        kw = dict(ranks=A[6], alpha=A[7])
        assert lora(L, segs=seg(y=over), **kw) == ERR_ALIAS, hex(over)
        assert lora(L, ws=over, **kw) == ERR_ALIAS, hex(over)
    assert lora(L, segs=seg(base=A[5] + 16)) == ERR_ALIAS            # over y, shifted
    assert lora(L, ws=A[5]) == ERR_ALIAS                             # workspace on y
    assert lora(L, segs=seg(base=A[4])) == ERR_ALIAS                 # base in the workspace
    two = seg() + seg(a=A[6], b=A[7], y=A[5] + 128)
    assert lora(L, segs=two) == ERR_ALIAS                            # two outputs
    two = seg() + seg(a=A[6], b=A[7], y=A[8], base=A[5])
    assert lora(L, segs=two) == ERR_ALIAS                            # another's y as a base


def test_lora_workspace(L):
    w = nv.lora_workspace_bytes
    assert w(1, 0, 16, 1) == 0 and w(0, 64, 16, 1) == 0
    for bad in ((129, 64, 16, 1), (1, 48, 16, 1), (1, 64, 12, 1), (1, 64, 264, 1), (1, 64, 16, 9),
                (-1, 64, 16, 1), (1, 64, 0, 1)):
        assert w(*bad) == 0
    assert w(128, nv.MAX_K, 256, 8) <= 32 << 20
