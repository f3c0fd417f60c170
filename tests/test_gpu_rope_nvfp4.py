"""Rotation and append to an NVFP4 cache on the GPU: v, and k where nothing
turns, bit for bit as the oracle packs them; turned k within the encoding's
steps of the 64-bit rotation; q as the other append gives it; every other byte
of the cache as it was."""
import pytest
import torch

import nvfp4_block_scaled_gemv_amd as nv
from decode_ref import gen, inv_freq, normal, rotate
from gpu_util import DEV, say
from serving_ref import decode4, encode4, place4
from test_gpu_rope import pair_size

pytestmark = pytest.mark.gpu

BF16, F32, E4M3 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
GK, GV = 4.5 / 2688, 0.7 / 2688

CASES = [
    # T, Hq, Hkv, D, R, page, xt, interleaved, order, first position
    (1, 32, 8, 128, 128, 16, F32, False, "nhd", 0),
    (5, 32, 8, 128, 128, 16, F32, False, "hnd", 32768),
    (5, 32, 8, 128, 64, 64, BF16, True, "nhd", 1 << 20),
    (3, 4, 1, 64, 64, 1, BF16, True, "beside", 7),
    (64, 2, 2, 64, 32, 20, F32, False, "wide", 100000),
    (65, 8, 8, 256, 256, 256, BF16, False, "nhd", 5),
    (130, 1, 1, 64, 16, 3, F32, False, "nhd", 0),          # pairs 8 apart: inside a block
    (257, 2, 1, 192, 48, 7, F32, False, "hnd", 999983),    # 24 apart: across blocks
    (71, 7, 1, 128, 112, 16, BF16, False, "beside", 1 << 26),
    (9, 3, 3, 512, 512, 5, BF16, False, "wide", 12),
    (100, 28, 4, 128, 0, 32, F32, False, "nhd", 3),
    (600, 5, 5, 64, 48, 16, BF16, True, "hnd", 123),
    (300, 0, 1, 64, 64, 16, F32, False, "nhd", 50),        # only append, several tokens a workgroup
]


def fresh(order, nb, page, Hkv, D, byte=0x35):
    z = [(torch.full((nb, page, Hkv, D // 2), byte, dtype=torch.uint8),
          torch.full((nb, page, Hkv, D // 16), byte, dtype=torch.uint8), g) for g in (GK, GV)]
    return place4(z, order, DEV)


def within(got_codes, got_scales, want, size, g):
    """The stored values against the exact ones: the block scale is E4M3(amax / (6
    g)) (half a step: 2^-4 of it, 2^-10 below its normal numbers), a value then off
    by at most half its own step of E2M1, 0.25, 0.5 or 1 for magnitudes t to 2, 4 and
    6 of the scale. Past 6 the largest code remains, off by t - 6: t <= 6 r / s is
    at most 6 (1 + 2^-4) at the normal scales, but where a scale of 2^-9 stands for an
    r of up to 1.5 2^-9 it comes to 9. The rotation's fp32 moves both by 8 of 2^-24
    of the pair's size."""
    D = want.shape[-1]
    s = got_scales.view(E4M3).double()
    amax = want.abs().unflatten(-1, (D // 16, 16)).amax(-1)
    err = size.unflatten(-1, (D // 16, 16)).amax(-1) * 8 * 2.0 ** -24
    r = (amax / (6 * g)).clamp(max=448)
    off = torch.maximum(r * 2.0 ** -4, torch.tensor(2.0 ** -10).double())
    assert torch.all((s - r).abs() <= off * (1 + 2.0 ** -20) + err / (6 * g))
    step = (s * g).repeat_interleave(16, -1)
    t = want.abs() / step.clamp(min=1e-300)
    half = torch.where(t <= 2, 0.25, torch.where(t <= 4, 0.5, (t - 6).clamp(min=1.0)))
    vals = decode4(got_codes, got_scales, g)
    # a value next to a border may take either side's step
    slack = size * 8 * 2.0 ** -24 * (1 + 1e-6) + want.abs() * 2.0 ** -22
    full = amax.repeat_interleave(16, -1) > 6 * 448 * g * (1 - 2.0 ** -20)
    ok = ((vals - want).abs() <= half * step + slack) | full
    # a block whose scale is zero holds zeros
    ok |= (step == 0) & (vals == 0) & (want.abs() <= 6 * g * 2.0 ** -10 * (1 + 1e-6) + slack)
    assert ok.all(), torch.nonzero(~ok)[0].tolist()


@pytest.mark.parametrize("T,Hq,Hkv,D,R,page,xt,inter,order,first", CASES)
def test_append(T, Hq, Hkv, D, R, page, xt, inter, order, first):
    say(f"[rope4] T={T} Hq={Hq} Hkv={Hkv} D={D} R={R} page={page} {xt} {inter} {order}")
    g = gen(T + D + R)
    scale = 1.0 if T % 2 else 1.25
    qkv = normal(g, T, Hq + 2 * Hkv, D, dtype=xt)
    qkv[T // 2, Hq:, :16] = 0                              # a block of zeros
    qkv[T // 2, Hq:, 16:32] *= 1e-5                        # one below every scale, or nearly
    x = qkv.to(DEV)
    q, k, v = x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]
    pos = first + torch.randperm(3 * T, generator=g)[:T]
    nb = T // page + 4
    slots = torch.randperm(nb * page, generator=g)[:T]
    if T > 2:                       # padding, a slot behind the cache
        slots[1], slots[T - 1] = -1, nb * page
    freq = inv_freq(R) if R else torch.empty(0)
    cache = fresh(order, nb, page, Hkv, D)
    out = nv.rope_append_nvfp4(q if Hq else None, k, v, pos.to(DEV), slots.to(DEV), freq.to(DEV),
                               *cache, interleaved=inter, rope_scale=scale)
    torch.cuda.synchronize()
    if Hq:
        kb = torch.zeros(nb, page, Hkv, D, dtype=BF16, device=DEV)
        same = nv.rope_append(q, k, v, pos.to(DEV), slots.to(DEV), freq.to(DEV), kb,
                              torch.zeros_like(kb), interleaved=inter, rope_scale=scale)
        assert torch.equal(out, same)
    hk, hv = qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
    live = [t for t in range(T) if 0 <= int(slots[t]) < nb * page]
    at = slots[live]
    rest = torch.ones(nb * page, dtype=torch.bool)
    rest[at] = False
    for (c, s, _), rows, gs, turned in ((cache[0], hk, GK, R > 0), (cache[1], hv, GV, False)):
        c, s = c.cpu().reshape(nb * page, Hkv, -1), s.cpu().reshape(nb * page, Hkv, -1)
        assert torch.all(c[rest] == 0x35) and torch.all(s[rest] == 0x35)
        if not turned:
            wc, ws = encode4(rows[live].float(), gs)
            assert torch.equal(c[at], wc) and torch.equal(s[at], ws)
        else:
            want = rotate(rows, pos, freq, inter, scale)[live]
            within(c[at].contiguous(), s[at].contiguous(), want,
                   pair_size(rows, R, inter, scale)[live], float(torch.tensor(gs)))
            # blocks that do not turn: bit for bit
            wc, ws = encode4(rows[live][..., R:].float(), gs) if R < D else (None, None)
            if R < D:
                assert torch.equal(c[at][..., R // 2:], wc) and torch.equal(s[at][..., R // 16:], ws)


def test_no_byte_outside_the_heads():
    """Caches in wider rows: what lies between the heads stays."""
    T, Hkv, D, page = 6, 2, 64, 4
    g = gen(2)
    k = normal(g, T, Hkv, D).to(DEV)
    raw = torch.full((2, 2, page, Hkv, 48), 0x5A, dtype=torch.uint8, device=DEV)
    rs = torch.full((2, 2, page, Hkv, 8), 0x5A, dtype=torch.uint8, device=DEV)
    one = torch.full((1,), GK, device=DEV)
    pos, slots = torch.arange(T, device=DEV), torch.tensor([0, 7, 2, 5, 1, 4], device=DEV)
    nv.rope_append_nvfp4(None, k, k, pos, slots, inv_freq(D).to(DEV),
                         (raw[0][..., :32], rs[0][..., :4], one),
                         (raw[1][..., :32], rs[1][..., :4], one))
    torch.cuda.synchronize()
    assert torch.all(raw[..., 32:] == 0x5A) and torch.all(rs[..., 4:] == 0x5A)
    assert not torch.all(raw[..., :32] == 0x5A)


def test_infinities_and_nan():
    """An infinite element saturates its block; a NaN makes its block NaN, codes
    0; the blocks beside them are as without."""
    D = 64
    x = normal(gen(4), 1, 1, D)
    clean = fresh("nhd", 1, 1, 1, D)
    z = torch.zeros(1, dtype=torch.int64, device=DEV)
    nv.rope_append_nvfp4(None, x.to(DEV), x.to(DEV), z, z, torch.empty(0, device=DEV), *clean)
    y = x.clone()
    y[0, 0, 3], y[0, 0, 20], y[0, 0, 37] = float("inf"), float("nan"), -float("inf")
    got = fresh("nhd", 1, 1, 1, D)
    nv.rope_append_nvfp4(None, y.to(DEV), y.to(DEV), z, z, torch.empty(0, device=DEV), *got)
    for (c, s, _), (c0, s0, _), g in zip(got, clean, (GK, GV)):
        c, s, c0, s0 = (t.cpu().flatten() for t in (c, s, c0, s0))
        assert s.tolist()[:3] == [0x7E, 0x7F, 0x7E] and s[3] == s0[3]
        assert torch.all(c[8:16] == 0) and torch.equal(c[24:], c0[24:])
        v = decode4(c[None], s[None], 1.0)[0]
        assert v[3] == 6 * 448 and v[37] == -6 * 448
        want, _ = encode4(y[0, 0, :16].clamp(max=6 * 448 * g)[None], g)
        assert torch.equal(c[:8], want[0]) or g == GV


def test_slots_past_32_bits_are_not_written():
    cache = fresh("nhd", 2, 2, 1, 64, 0x11)
    x = torch.ones(3, 1, 64, device=DEV)
    slots = torch.tensor([1 << 33, -(1 << 40), (1 << 62)], device=DEV)
    pos = torch.zeros(3, dtype=torch.int64, device=DEV)
    nv.rope_append_nvfp4(None, x, x, pos, slots, inv_freq(64).to(DEV), *cache)
    torch.cuda.synchronize()
    assert all(torch.all(t == 0x11) for c in cache for t in c[:2])


@pytest.mark.parametrize("g", [1e-30, 2.0 ** -100, 1.0, 1e30])
def test_any_tensor_scale(g):
    """Tensor scales at which every block saturates, or is zero."""
    x = normal(gen(5), 4, 2, 64)
    x[1] *= 1e-20
    x[2] *= 1e20
    c = [(torch.zeros(4, 1, 2, 32, dtype=torch.uint8, device=DEV),
          torch.zeros(4, 1, 2, 4, dtype=torch.uint8, device=DEV),
          torch.full((1,), g, device=DEV)) for _ in range(2)]
    s = torch.arange(4, device=DEV)
    nv.rope_append_nvfp4(None, x.to(DEV), x.to(DEV), s, s, torch.empty(0, device=DEV), *c)
    wc, ws = encode4(x, g)
    for codes, scales, _ in c:
        assert torch.equal(codes[:, 0].cpu(), wc) and torch.equal(scales[:, 0].cpu(), ws)
