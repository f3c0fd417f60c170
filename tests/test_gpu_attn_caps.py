"""Caps from one end of their range to the other over every cache: queries and
tensor scales small enough that a score's share of the cap leaves fp32's normal
numbers, tables of either form, and scores whose difference shows the tanh."""
import math

import pytest
import torch

import nvfp4_block_scaled_gemv_amd as nv
import test_gpu_attn_nvfp4 as four
import test_gpu_attn_scored as scored
from gpu_util import DEV, say
from serving_ref import attention, build4, decode4, place4
from test_gpu_paged_attn import BF16, E4M3, build

pytestmark = pytest.mark.gpu

CACHES = ["bf16", "e4m3", "nvfp4"]


def widened(table, Hkv, page):
    """A table of 2^19 keys of all heads: two heads side by side where they fit."""
    width = (1 << 19) // (Hkv * table.shape[0] * page) + 1
    return torch.cat([table, torch.full((table.shape[0], width), -1, dtype=torch.int32)], 1)


def capped(cache, lens, Q, Hq, Hkv, D, page, cap, std, wide, seed, scale=None, gk=4.5 / 2688):
    """The call on queries of deviation `std`, within the bound of its cache's
    tests."""
    scale = D ** -0.5 if scale is None else scale
    if cache == "nvfp4":
        q, table, ln, parts = build4(lens, Q, Hq, Hkv, D, page, seed=seed, gk=gk, q_std=std)
        table = widened(table, Hkv, page) if wide else table
        got = four.run(q, place4(parts, "nhd", DEV), table, ln, softcap=cap, scale=scale)
        return four.check(got, q, parts, table, ln, scale, 0, cap)
    ct = BF16 if cache == "bf16" else E4M3
    q, k, v, table, ln, kc, vc, ks, vs = build(lens, Q, Hq, Hkv, D, page, ct, seed=seed)
    q = (q.double() * std).to(BF16)
    table = widened(table, Hkv, page) if wide else table
    got = scored.run(q, table, ln, kc, vc, ks, vs, ct, softcap=cap, scale=scale)
    return scored.check(got, q, k, v, table, ln, scale, 0, ks, vs, cap, None)


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("std", [0.1, 0.5, 2.0])
@pytest.mark.parametrize("cap", [1e-6, 1.0, 1e28, 3e29, 1e30])
@pytest.mark.parametrize("cache", CACHES)
def test_caps_and_small_queries(cache, cap, std, wide):
    say(f"[caps] {cache} cap={cap} std={std} wide={wide}")
    r = capped(cache, [400, 33, 0], 1, 16, 4, 128, 16, cap, std, wide, seed=41)
    say(f"  max err / tol = {r:.3f}")


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("cache,D,Q,page", [("nvfp4", 64, 5, 20), ("nvfp4", 256, 2, 64),
                                            ("nvfp4", 128, 5, 16), ("e4m3", 64, 2, 20),
                                            ("bf16", 256, 5, 16)])
def test_large_caps_in_other_forms(cache, D, Q, page, wide):
    say(f"[caps] {cache} D={D} Q={Q} page={page} wide={wide}")
    r = capped(cache, [300, 77], Q, 8, 2, D, page, 1e30, 0.1, wide, seed=42)
    say(f"  max err / tol = {r:.3f}")


@pytest.mark.parametrize("cache", CACHES)
def test_a_small_factor_and_large_queries(cache):
    """Scores of order one from queries of 2^20 and a factor (or tensor scale) of 2^-20
    beside: the factor over the cap is below fp32's normal numbers, the scores are not."""
    q, gk, scale = 2.0 ** 20, 4.5 / 2688, 2.0 ** -20 / 8
    if cache == "nvfp4":
        gk, scale = gk * 2.0 ** -10, 2.0 ** -10 / 8
    r = capped(cache, [200], 2, 8, 2, 64, 16, 1e30, q, False, 43, scale, gk)
    say(f"  max err / tol = {r:.3f}")


@pytest.mark.parametrize("cap,z1,z2", [
    (500.0, 149.5, 151.0),              # both in tanh's near part
    (500.0, 624.0, 628.0),              # on either side of 1.25
    (500.0, 1000.0, 1008.0),            # both beyond
    (2000.0, 2492.0, 2504.0), (40.0, 49.0, 51.0), (1e30, 100.0, 101.5), (3.0, 3.0, 4.5)])
@pytest.mark.parametrize("cache", CACHES)
def test_the_difference_of_two_capped_scores(cache, cap, z1, z2):
    """Keys with one of two scores, exact in every cache, and values 1 and -1 in such
    numbers that the sum nearly cancels: it moves by the scores' errors, (1 + |o|) of
    the larger. A capped score is off by 2^-21 of it and six roundings of 2^-24 of the
    score (the factor's product, its log2, the score's product, the cap's log2, the
    bias of none, the difference to the largest). Sums over the keys add 2^-16 at
    most (2^7 additions of 2^-24 in a chain, twice), the output its 2^-8."""
    D, keys, page = 64, 600, 16
    c1, c2 = (cap * math.tanh(z / cap) for z in (z1, z2))
    n1 = round(keys / (1 + math.exp(c1 - c2)))            # n1 e^c1 = (keys - n1) e^c2
    first = torch.arange(keys) < n1
    # q = (q0, q1), keys (1, 0.5) and (1, 1), a factor of 1 / 8
    q1 = 16.0 * (z2 - z1)
    q0 = 8.0 * z1 - q1 / 2
    assert torch.tensor([q0, q1], dtype=BF16).tolist() == [q0, q1]
    table = torch.arange((keys + page - 1) // page, dtype=torch.int32)[None]
    nb = table.shape[1]
    q = torch.zeros(1, 1, D, dtype=BF16)
    q[..., 0], q[..., 1] = q0, q1
    k = torch.zeros(nb * page, 1, D)
    v = torch.zeros(nb * page, 1, D)
    k[:, :, 0] = 1.0
    k[:keys, 0, 1] = torch.where(first, 0.5, 1.0)
    v[:keys, 0] = torch.where(first, 1.0, -1.0)[:, None]
    # in turn, so that no chain of additions meets one sign only
    turn = torch.randperm(keys, generator=torch.Generator().manual_seed(3))
    k[:keys], v[:keys] = k[:keys][turn], v[:keys][turn]
    k, v = k.view(nb, page, 1, D), v.view(nb, page, 1, D)
    ln = torch.tensor([keys], dtype=torch.int32)
    ref = attention(q, k, v, table, ln, 0.125, 0, cap)
    assert float(ref.abs().max()) < 2.0 ** -7, float(ref.abs().max())
    if cache == "nvfp4":
        code = {0.0: 0, 0.5: 1, 1.0: 2, -1.0: 10}
        parts = []
        for x in (k, v):
            c = x.clone()
            for val, i in code.items():
                c[x == val] = i
            c = c.to(torch.uint8)
            s = torch.full((*x.shape[:3], D // 16), 0x38, dtype=torch.uint8)   # 1.0
            parts.append((c[..., 0::2] | (c[..., 1::2] << 4), s, 1.0))
            assert torch.equal(decode4(*parts[-1]).float(), x)
        got = four.run(q, place4(parts, "nhd", DEV), table, ln, softcap=cap, scale=0.125)
    else:
        ct = BF16 if cache == "bf16" else E4M3
        got = scored.run(q, table, ln, k.to(ct).to(DEV), v.to(ct).to(DEV), 1.0, 1.0, ct,
                         softcap=cap, scale=0.125)
    off = 2.0 ** -21 * max(abs(c1), abs(c2)) + 6 * 2.0 ** -24 * max(z1, z2)
    tol = 2 * (1 + ref.abs()) * off + 2.0 ** -16 + ref.abs() * 2.0 ** -8
    say(f"[caps] {cache} cap={cap}: max err / tol = {float(((got - ref).abs() / tol).max()):.3f}")
    assert torch.all((got - ref).abs() <= tol)
