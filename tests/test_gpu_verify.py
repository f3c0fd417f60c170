"""Verification of drafted tokens on the GPU against a plain 64-bit form. The
outputs are whole numbers and have to be equal; every case says how near its
comparisons came to their borders (the reference's own sums are exact to far
less than that)."""
import numpy as np
import pytest
import torch

import nvfp4_block_scaled_gemv_amd as nv
from decode_ref import gen, verify
from gpu_util import DEV, say

pytestmark = pytest.mark.gpu


def case(B, Q, V, seed, spread=2.5, near=0.7):
    g = gen(seed)
    z = torch.randn(B, Q + 1, V, generator=g) * spread
    p = torch.softmax(z, -1)
    q = torch.softmax(z[:, :Q] + torch.randn(B, Q, V, generator=g) * near, -1)
    draft = torch.multinomial(q.view(B * Q, V), 1, generator=g).view(B, Q).int() if Q \
        else torch.zeros(B, 0, dtype=torch.int32)
    return p, q, draft, torch.rand(B, Q, generator=g), torch.rand(B, generator=g)


def check(p, q, draft, ua, us, n_draft=None, what=""):
    tokens, acc = nv.verify_draft(p.to(DEV), None if q is None else q.to(DEV), draft.to(DEV),
                                  ua.to(DEV), us.to(DEV),
                                  None if n_draft is None else n_draft.to(DEV))
    rt, ra, margin = verify(p, q, draft, ua, us, n_draft)
    say(f"[verify] {what} kept {ra.tolist()[:8]} margin {margin:.1e}")
    assert margin > 1e-13      # far from a border that 64-bit sums could miss
    assert np.array_equal(acc.cpu().numpy(), ra)
    assert np.array_equal(tokens.cpu().numpy(), rt)
    return ra


@pytest.mark.parametrize("B,Q,V", [(1, 1, 5), (3, 4, 1000), (2, 7, 2048), (2, 3, 2049), (1, 4, 151936),
                                   (5, 2, 33333), (16, 1, 4097), (1, 63, 300), (2, 0, 5000),
                                   (70, 3, 257), (1, 2, 1), (1, 1, 600000)])
@pytest.mark.parametrize("with_q", [True, False])
def test_verify(B, Q, V, with_q):
    p, q, draft, ua, us = case(B, Q, V, B * 31 + Q + V)
    check(p, q if with_q else None, draft, ua, us, what=f"B={B} Q={Q} V={V} q={with_q}")


@pytest.mark.parametrize("with_q", [True, False])
def test_all_kept_none_kept(with_q):
    p, q, draft, ua, us = case(4, 5, 3001, 3)
    qq = q if with_q else None
    assert check(p, qq, draft, torch.zeros_like(ua), us, what="u = 0").tolist() == [5] * 4
    # q = 1 at the draft and nothing of it in p: never kept
    q2, p2 = q.clone(), p.clone()
    for b in range(4):
        for j in range(5):
            p2[b, j, draft[b, j]] = 0.0
    assert check(p2, q2 if with_q else None, draft, ua, us, what="p = 0").tolist() == [0] * 4


def test_padded_and_bad_drafts():
    p, q, draft, ua, us = case(6, 4, 999, 4)
    ua = ua * 0
    n = torch.tensor([4, 0, 2, 3, -1, 9], dtype=torch.int32)
    draft[2, 2:] = -1
    ra = check(p, q, draft, ua, us, n, what="n_draft")
    assert ra.tolist() == [4, 0, 2, 3, 0, 4]
    draft[0, 1], draft[3, 0] = -1, 999          # not a token: refused there
    for qq in (q, None):
        ra = check(p, qq, draft, ua, us, n, what="bad drafts")
        assert ra.tolist() == [1, 0, 2, 0, 0, 4]


def test_the_same_distribution():
    """p = q bit for bit: u < 1 keeps every draft; a forced refusal (a draft
    that is not a token) finds nothing left and draws from p."""
    p, q, draft, ua, us = case(3, 2, 5000, 5)
    q = p[:, :2].clone()
    assert check(p, q, draft, ua, us, what="p = q").tolist() == [2, 2, 2]
    draft[:, 1] = -1
    assert check(p, q, draft, ua, us, what="p = q, refused").tolist() == [1, 1, 1]


def test_sparse_rows():
    """Rows with few nonzero entries: the border lies on them, at both ends of
    the pieces, and u = 0 takes the first of them."""
    V = 3 * 2048 + 5
    for at in ([0], [V - 1], [2047, 2048], [0, 2048, V - 1], [4095, 4096, 6144]):
        p = torch.zeros(1, 1, V)
        p[0, 0, at] = torch.tensor([0.5 + i for i in range(len(at))])
        for u in (0.0, 0.3, 0.77, 0.999999):
            us = torch.tensor([u])
            tokens, acc = nv.verify_draft(p.to(DEV), None, torch.zeros(1, 0, dtype=torch.int32,
                                                                       device=DEV),
                                          torch.zeros(1, 0, device=DEV), us.to(DEV))
            rt, _, _ = verify(p, None, torch.zeros(1, 0), torch.zeros(1, 0), us)
            assert int(tokens[0, 0]) == int(rt[0, 0]) and int(rt[0, 0]) in at


@pytest.mark.parametrize("V,count", [(300, 64), (5000, 512), (151936, 4096)])
def test_exact_borders(V, count):
    """`count` equal weights of a power of two at random places: every sum is
    exact, and u = i / count is the border itself, which belongs to the entry
    after it."""
    g = gen(V)
    at = torch.randperm(V, generator=g)[:count].sort().values
    p = torch.zeros(1, 1, V)
    p[0, 0, at] = 1.0 / count
    B = 128
    i = torch.randint(0, count, (B,), generator=g)
    below = torch.nextafter((i + 1).float() / count, torch.zeros(()))
    none = torch.zeros(B, 0, dtype=torch.int32, device=DEV)
    pg = p.to(DEV).expand(B, 1, V).contiguous()
    for u in (i.float() / count, below):
        tokens, acc = nv.verify_draft(pg, None, none, torch.zeros(B, 0, device=DEV), u.to(DEV))
        assert torch.equal(tokens[:, 0].cpu().long(), at[i])


def test_every_token_has_weight():
    """u at the fp32 neighbours of the borders of rows that are mostly zeros:
    whatever the rounding of a sum, an entry without weight is never drawn."""
    V, B = 60000, 512
    g = gen(12)
    row = torch.zeros(V)
    at = torch.randperm(V, generator=g)[:300].sort().values
    row[at] = torch.rand(300, generator=g) ** 4
    c = torch.cumsum(row.double(), 0)
    u = (c[at] / c[-1]).float()[torch.randint(0, 299, (B,), generator=g)]
    u[::3] = torch.nextafter(u[::3], torch.zeros(()))
    none = torch.zeros(B, 0, dtype=torch.int32, device=DEV)
    tokens, _ = nv.verify_draft(row.to(DEV).expand(B, 1, V).contiguous(), None, none,
                                torch.zeros(B, 0, device=DEV), u.to(DEV))
    t = tokens[:, 0].cpu().long()
    assert torch.all(row[t] > 0)
    # and it is the border's: the sums around it enclose the target
    target = u.double() * c[-1]
    assert torch.all((c[t] > target - 1e-9) & (c[t] - row[t].double() <= target + 1e-9))


def test_nothing_to_draw_from():
    """Zeros, NaN and u = 1 give a token inside the vocabulary."""
    V = 2500
    zero = torch.zeros(0, device=DEV)
    none = torch.zeros(1, 0, dtype=torch.int32, device=DEV)
    for p, u in ((torch.zeros(1, 1, V), 0.5), (torch.full((1, 1, V), float("nan")), 0.5),
                 (torch.full((1, 1, V), 1.0 / V), 1.0), (torch.full((1, 1, V), float("inf")), 0.5)):
        tokens, acc = nv.verify_draft(p.to(DEV), None, none, zero.view(1, 0),
                                      torch.tensor([u], device=DEV))
        assert int(acc[0]) == 0 and 0 <= int(tokens[0, 0]) < V
    assert int(tokens[0, 0]) >= 0


def test_follows_the_distribution():
    """Speculative sampling leaves the target's distribution: over 4096
    sequences with one draft each, the first token's counts against p (5
    standard deviations of a binomial count; seeded, so it is the same run
    every time)."""
    g = gen(7)
    B, V = 4096, 8
    z = torch.randn(V, generator=g)
    p1 = torch.softmax(z, -1)
    q1 = torch.softmax(z + torch.randn(V, generator=g), -1)
    p = p1.expand(B, 2, V).contiguous()
    q = q1.expand(B, 1, V).contiguous()
    draft = torch.multinomial(q1, B, replacement=True, generator=g).int().view(B, 1)
    tokens, acc = nv.verify_draft(p.to(DEV), q.to(DEV), draft.to(DEV),
                                  torch.rand(B, 1, generator=g).to(DEV),
                                  torch.rand(B, generator=g).to(DEV))
    first = tokens[:, 0].cpu().long()
    count = torch.bincount(first, minlength=V).double()
    want = p1.double() * B
    assert torch.all((count - want).abs() <= 5 * (want * (1 - p1.double())).sqrt() + 1)
