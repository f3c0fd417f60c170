"""Rotary positions and the append to a paged cache on the GPU against a plain
64-bit form: both layouts, part of the head, far positions, bf16 and E4M3
caches in several orders, padded tokens, views of one projection's output."""
import pytest
import torch

import nvfp4_block_scaled_gemv_amd as nv
from decode_ref import gen, inv_freq, normal, rotate
from gpu_util import DEV, say

pytestmark = pytest.mark.gpu

BF16, F32, E4M3 = torch.bfloat16, torch.float32, torch.float8_e4m3fn


def make_cache(order, nb, page, Hkv, D, dtype, fill=0):
    """Two caches [nb, page, Hkv, D] in the given memory order, bytes `fill`."""
    n = 1 if dtype is E4M3 else 2
    shape = {"nhd": (2, nb, page, Hkv, D), "hnd": (2, nb, Hkv, page, D),
             "beside": (nb, 2, page, Hkv, D), "wide": (2, nb, page, Hkv, D + 32)}[order]
    raw = torch.full(shape[:-1] + (shape[-1] * n,), fill, dtype=torch.uint8, device=DEV).view(dtype)
    if order == "hnd":
        raw = raw.transpose(2, 3)
    if order == "beside":
        return raw[:, 0], raw[:, 1]
    return raw[0][..., :D], raw[1][..., :D]


def bytes_of(t):
    return t.contiguous().view(torch.uint8).cpu()


# half a step of bf16 around a value that fp32 arithmetic leaves within 8 steps
# of 2^-24 of |x0| + |x1| (angle 2^-24, sine and cosine 2 of them, products
# and sum one each), times the scale
def tol_of(exact, x0x1):
    return exact.abs() * 2.0 ** -8 + x0x1 * 8 * 2.0 ** -24 + 1e-37


def pair_size(x, R, interleaved, scale):
    """|x0| + |x1| for every element of x (0 beyond R), in 64 bits."""
    a = x.double().abs()
    out = torch.zeros_like(a)
    if R:
        r = a[..., :R]
        if interleaved:
            s = r[..., 0::2] + r[..., 1::2]
            out[..., 0:R:2] = s
            out[..., 1:R:2] = s
        else:
            s = r[..., :R // 2] + r[..., R // 2:]
            out[..., :R] = torch.cat([s, s], -1)
    return out * abs(scale)


CASES = [
    # T, Hq, Hkv, D, R, page, xt, cache type, interleaved, order, first position
    (1, 32, 8, 128, 128, 16, F32, BF16, False, "nhd", 0),
    (5, 32, 8, 128, 128, 16, F32, BF16, False, "hnd", 32768),
    (5, 32, 8, 128, 64, 64, BF16, E4M3, True, "nhd", 1 << 20),
    (3, 4, 1, 64, 64, 1, BF16, BF16, True, "beside", 7),
    (64, 2, 2, 64, 32, 20, F32, E4M3, False, "wide", 100000),
    (65, 8, 8, 256, 256, 256, BF16, BF16, False, "nhd", 5),
    (130, 1, 1, 16, 16, 3, F32, BF16, True, "nhd", 0),
    (257, 2, 1, 96, 48, 7, F32, E4M3, False, "hnd", 999983),
    (71, 7, 1, 80, 32, 16, BF16, E4M3, True, "beside", 1 << 26),
    (9, 3, 3, 512, 512, 5, BF16, BF16, False, "wide", 12),
    (100, 28, 4, 128, 0, 32, F32, BF16, False, "nhd", 3),
    (600, 5, 5, 48, 48, 16, BF16, BF16, True, "hnd", 123),
]


@pytest.mark.parametrize("T,Hq,Hkv,D,R,page,xt,ct,inter,order,first", CASES)
def test_rope_append(T, Hq, Hkv, D, R, page, xt, ct, inter, order, first):
    say(f"[rope] T={T} Hq={Hq} Hkv={Hkv} D={D} R={R} page={page} {xt} {ct} {inter} {order}")
    g = gen(T + D + R)
    scale = 1.0 if T % 2 else 1.25
    qkv = normal(g, T, Hq + 2 * Hkv, D, dtype=xt)
    x = qkv.to(DEV)
    q, k, v = x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]
    pos = first + torch.randperm(3 * T, generator=g)[:T]
    nb = T // page + 4
    slots = torch.randperm(nb * page, generator=g)[:T]
    if T > 2:                       # padding, and a slot behind the cache
        slots[1], slots[T - 1] = -1, nb * page
    freq = inv_freq(R) if R else torch.empty(0)
    ks, vs = torch.tensor([0.02]), torch.tensor([0.003])
    kc, vc = make_cache(order, nb, page, Hkv, D, ct, 0x35)
    kb, vb = bytes_of(kc), bytes_of(vc)
    out = nv.rope_append(q, k, v, pos.to(DEV), slots.to(DEV), freq.to(DEV), kc, vc,
                         ks.to(DEV) if ct is E4M3 else None, vs.to(DEV) if ct is E4M3 else None,
                         interleaved=inter, rope_scale=scale)
    torch.cuda.synchronize()
    hq, hk, hv = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
    want = rotate(hq, pos, freq, inter, scale)
    tol = tol_of(want, pair_size(hq, R, inter, scale))
    assert torch.all((out.cpu().double() - want).abs() <= tol)
    live = [t for t in range(T) if 0 <= int(slots[t]) < nb * page]
    at = slots[live]
    for cache, before, rows, s, turned in ((kc, kb, hk, ks, True), (vc, vb, hv, vs, False)):
        want = rotate(rows, pos, freq, inter, scale) if turned else rows.double()
        size = pair_size(rows, R if turned else 0, inter, scale)
        got = cache.contiguous().cpu().view(torch.uint8).view(nb * page, -1)
        vals = got[at].contiguous().view(ct).float().double().view(len(live), Hkv, D)
        if ct is E4M3:
            w = (want / s.double())[live].clamp(-448, 448)
            z = (size / s.double())[live]
            half = torch.maximum(w.abs() * 2.0 ** -4, torch.tensor(2.0 ** -10).double())
            assert torch.all((vals - w).abs() <= half + (z + w.abs()) * 8 * 2.0 ** -24)
        else:
            assert torch.all((vals - want[live]).abs() <= tol_of(want, size)[live])
        # every other slot as it was
        rest = torch.ones(nb * page, dtype=torch.bool)
        rest[at] = False
        assert torch.equal(got[rest], before.view(nb * page, -1)[rest])


def test_far_positions_stay_exact():
    """At position 2^20 + 5 a product of position and frequency in 32 bits would
    be 0.06 rad off; the bound here is that of one bf16 rounding."""
    x = torch.zeros(1, 1, 128)
    x[..., :64] = 1.0
    pos = torch.tensor([(1 << 20) + 5])
    f = inv_freq(128, 10000.0)
    out = nv.rope_append(x.to(DEV), None, None, pos.to(DEV), None, f.to(DEV), None, None)
    want = rotate(x, pos, f, False)
    assert torch.all((out.cpu().double() - want).abs() <= tol_of(want, torch.ones(1, 1, 128)))


def test_only_append_and_only_rotate():
    g = gen(3)
    T, Hkv, D = 4, 2, 64
    k, v = normal(g, T, Hkv, D), normal(g, T, Hkv, D)
    pos, slots, f = torch.arange(T), torch.tensor([3, 0, 7, 5]), inv_freq(D)
    kc, vc = make_cache("nhd", 2, 4, Hkv, D, BF16)
    r = nv.rope_append(None, k.to(DEV), v.to(DEV), pos.to(DEV), slots.to(DEV), f.to(DEV), kc, vc)
    assert r is None
    assert torch.equal(vc.reshape(8, Hkv, D)[slots].cpu(), v.to(BF16))
    q = nv.rope_append(k.to(DEV), None, None, pos.to(DEV), None, f.to(DEV), None, None)
    assert torch.equal(q, kc.reshape(8, Hkv, D)[slots.to(DEV)])   # the same rotation


def test_infinities_and_nan_are_kept():
    """bf16 keeps them; an E4M3 cache saturates infinities and keeps NaN; other
    elements are as without them."""
    T, D = 1, 64
    x = torch.ones(T, 1, D)
    x[0, 0, 3], x[0, 0, 9], x[0, 0, 11] = float("inf"), float("nan"), -float("inf")
    one = torch.zeros(T, dtype=torch.int64)
    for ct in (BF16, E4M3):
        kc, vc = make_cache("nhd", 1, 1, 1, D, ct)
        s = torch.ones(1, device=DEV) if ct is E4M3 else None
        nv.rope_append(None, x.to(DEV), x.to(DEV), one.to(DEV), one.to(DEV),
                       torch.empty(0, device=DEV), kc, vc, s, s)
        got = vc.float().cpu().view(D)
        top = 448.0 if ct is E4M3 else float("inf")
        assert got[3] == top and got[11] == -top and torch.isnan(got[9])
        assert torch.all(got[[i for i in range(D) if i not in (3, 9, 11)]] == 1)


def test_slots_past_32_bits_are_refused_quietly():
    """Slots whose page number does not fit 32 bits lie outside the cache."""
    kc, vc = make_cache("nhd", 2, 2, 1, 16, BF16, 0x11)
    before = bytes_of(kc)
    x = torch.ones(3, 1, 16, device=DEV)
    slots = torch.tensor([1 << 33, -(1 << 40), (1 << 62)], device=DEV)
    pos = torch.zeros(3, dtype=torch.int64, device=DEV)
    nv.rope_append(None, x, x, pos, slots, inv_freq(16).to(DEV), kc, vc)
    torch.cuda.synchronize()
    assert torch.equal(bytes_of(kc), before) and torch.equal(bytes_of(vc), before)
