"""The decode operators at the largest sizes that the header allows, against
64-bit forms (of some rows, where the whole would take long)."""
import numpy as np
import pytest
import torch

import nvfp4_block_scaled_gemv_amd as nv
from decode_ref import attention, gen, rmsnorm, verify
from gpu_util import DEV

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


def rand(seed, *shape, dtype=torch.float32):
    g = torch.Generator(DEV).manual_seed(seed)
    return torch.randn(*shape, device=DEV, generator=g).to(dtype)


@pytest.mark.parametrize("M,H", [(nv.MAX_ROWS, 8), (nv.MAX_ROWS - 1, 32), (3, nv.NORM_MAX_H)])
def test_norm(M, H):
    x, w = rand(1, M, H, dtype=BF16), (1 + 0.1 * rand(2, H)).to(BF16)
    r = rand(3, M, H, dtype=BF16)
    y, s = nv.add_rmsnorm(x, w, 1e-6, r)
    yr, sr = rmsnorm(x, w, 1e-6, r)
    # half a bf16 step, and the fp32 sum of at most 2^15 squares in a tree of
    # VPT * 8 terms per lane and 10 levels, taken as 64 steps of 2^-24
    assert torch.all((y.double() - yr).abs() <= yr.abs() * (2.0 ** -8 + 64 * 2.0 ** -24) + 1e-37)
    assert torch.equal(s, (x.float() + r.float()).to(BF16))


def test_append():
    """2^21 tokens of one head of 16, every slot of the cache taken once."""
    T, D = nv.MAX_ROWS, 16
    q, k, v = (rand(i, T, 1, D, dtype=BF16) for i in (4, 5, 6))
    pos = torch.arange(T, device=DEV)
    slots = torch.randperm(T, device=DEV, generator=torch.Generator(DEV).manual_seed(7))
    kc = torch.zeros(T // 64, 64, 1, D, dtype=BF16, device=DEV)
    vc = torch.zeros_like(kc)
    f = torch.tensor([1.0, 0.5, 0.1, 0.01, 1e-3, 1e-4, 1e-5, 1e-6], device=DEV)
    qo = nv.rope_append(q, k, v, pos, slots, f, kc, vc)
    assert torch.equal(vc.view(T, D)[slots], v.view(T, D))
    a = pos.double()[:, None] * f.double()
    for x, got in ((q, qo.view(T, D)), (k, kc.view(T, D)[slots])):
        x0, x1 = x.view(T, D).double()[:, :8], x.view(T, D).double()[:, 8:]
        want = torch.cat((x0 * a.cos() - x1 * a.sin(), x1 * a.cos() + x0 * a.sin()), -1)
        # half a bf16 step, and sine and cosine within 2^-22
        size = (x0.abs() + x1.abs()).repeat(1, 2)
        assert torch.all((got.double() - want).abs() <= want.abs() * 2.0 ** -8 + size * 2.0 ** -21)


def test_append_many_heads():
    """1024 query and 1024 key-value heads of 512."""
    T, Hd, D = 3, nv.MAX_HEADS, nv.ROPE_MAX_D
    q, k, v = (rand(i, T, Hd, D, dtype=BF16) for i in (8, 9, 10))
    kc = torch.zeros(2, 4, Hd, D, dtype=BF16, device=DEV)
    vc = torch.zeros_like(kc)
    slots = torch.tensor([6, 0, 3], device=DEV)
    qo = nv.rope_append(q, k, v, torch.zeros(T, dtype=torch.int64, device=DEV), slots,
                        torch.ones(D // 2, device=DEV), kc, vc)
    assert torch.equal(qo, q)                     # position 0 turns nothing
    assert torch.equal(kc.view(8, Hd, D)[slots], k) and torch.equal(vc.view(8, Hd, D)[slots], v)
    assert int((kc.view(8, Hd, D).abs().amax((1, 2)) > 0).sum()) == T


def attn_check(q, kc, vc, table, lens, rows, got):
    """Some of the sequences' outputs against the 64-bit form: half a bf16 step
    of the output, and 2^-11 of the values, of which none is above 6 (their
    probabilities lose 2^-16, the scores 64 products' sums of |q k| / 8 about
    12 twice 2 * 64 * 2^-24 * 12, sums over the keys 2^-14)."""
    B = table.shape[0]
    Q = q.shape[0] // B
    for b in rows:
        ref = attention(q.view(B, Q, *q.shape[1:])[b].cpu(), kc.cpu(), vc.cpu(), table[b:b + 1].cpu(),
                        lens[b:b + 1].cpu(), q.shape[-1] ** -0.5)
        err = (got.view(B, Q, *q.shape[1:])[b].cpu().double() - ref).abs()
        assert torch.all(err <= ref.abs() * 2.0 ** -8 + 6 * 2.0 ** -11), b


def test_attention_many_sequences():
    B, D, page = nv.ATTN_MAX_B, 64, 16
    lens = torch.arange(B, device=DEV).int() % 150
    kc, vc = rand(11, 500, page, 1, D, dtype=BF16), rand(12, 500, page, 1, D, dtype=BF16)
    table = torch.randint(0, 500, (B, 10), device=DEV, dtype=torch.int32,
                          generator=torch.Generator(DEV).manual_seed(13))
    q = rand(14, B, 4, D, dtype=BF16)
    got = nv.paged_attention(q, kc, vc, table, lens)
    attn_check(q, kc, vc, table, lens, (0, 1, 33, 149, 2000, B - 1), got)
    # long rows of the table: the split form
    wide = torch.cat((table, torch.full((B, 90), -1, dtype=torch.int32, device=DEV)), 1)
    got = nv.paged_attention(q, kc, vc, wide.contiguous(), lens)
    attn_check(q, kc, vc, wide, lens, (0, 1, 33, 149, 2000, B - 1), got)
    assert torch.all(got[lens == 0] == 0)


@pytest.mark.parametrize("Hq,Hkv,Q,L", [(1024, 1, 64, 200), (1024, 1, 64, 1500), (1024, 1024, 1, 70),
                                        (1024, 1024, 1, 1100)])
def test_attention_many_heads(Hq, Hkv, Q, L):
    D, page, B = 64, 32, 2
    n = (L + page - 1) // page
    kc, vc = rand(15, n + 1, page, Hkv, D, dtype=BF16), rand(16, n + 1, page, Hkv, D, dtype=BF16)
    table = torch.stack((torch.arange(n), torch.arange(n).flip(0) + 1)).int().to(DEV)
    lens = torch.tensor([L, L - 7], dtype=torch.int32, device=DEV)
    q = rand(17, B * Q, Hq, D, dtype=BF16)
    got = nv.paged_attention(q, kc, vc, table, lens)
    attn_check(q, kc, vc, table, lens, (0, 1), got)


def test_attention_all_heads_and_sequences():
    """4096 sequences of 1024 heads: the largest launch."""
    B, Hd, D, page = nv.ATTN_MAX_B, nv.MAX_HEADS, 64, 4
    kc, vc = rand(18, 3, page, Hd, D, dtype=BF16), rand(19, 3, page, Hd, D, dtype=BF16)
    table = torch.randint(0, 3, (B, 2), device=DEV, dtype=torch.int32,
                          generator=torch.Generator(DEV).manual_seed(20))
    lens = torch.arange(B, device=DEV).int() % 9
    q = rand(21, B, Hd, D, dtype=BF16)
    got = nv.paged_attention(q, kc, vc, table, lens)
    attn_check(q, kc, vc, table, lens, (0, 1, 8, B - 1), got)


@pytest.mark.parametrize("B,Q,V", [(1, 1, nv.VERIFY_MAX_V), (1, 0, nv.VERIFY_MAX_V - 1),
                                   (nv.VERIFY_MAX_B, 1, 70), (2, nv.VERIFY_MAX_Q, 1025)])
def test_verify(B, Q, V):
    g = gen(B + Q + V)
    p = torch.rand(B, Q + 1, V, generator=g) ** 4
    p /= p.sum(-1, keepdim=True)
    q = torch.rand(B, Q, V, generator=g) ** 4
    q /= q.sum(-1, keepdim=True)
    draft = torch.randint(0, V, (B, Q), generator=g, dtype=torch.int32)
    ua, us = torch.rand(B, Q, generator=g), torch.rand(B, generator=g)
    tokens, acc = nv.verify_draft(p.to(DEV), q.to(DEV), draft.to(DEV), ua.to(DEV), us.to(DEV))
    rt, ra, margin = verify(p, q, draft, ua, us)
    assert margin > 1e-13      # far from a border that 64-bit sums could miss
    assert np.array_equal(acc.cpu().numpy(), ra) and np.array_equal(tokens.cpu().numpy(), rt)
