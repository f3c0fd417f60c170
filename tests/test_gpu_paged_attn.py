"""Attention over a paged cache on the GPU against a plain 64-bit form: head
layouts, head sizes, page sizes that fit tiles and that do not, one and several
new tokens, windows, lengths from zero to many workgroups per sequence, pages
that do not exist, values that no token may see."""
import pytest
import torch

import nvfp4_block_scaled_gemv_amd as nv
from decode_ref import attention, gen, normal
from gpu_util import DEV, say
from test_gpu_rope import make_cache

pytestmark = pytest.mark.gpu

BF16, E4M3 = torch.bfloat16, torch.float8_e4m3fn


def build(lens, Q, Hq, Hkv, D, page, ct, order="nhd", seed=1, spare=3):
    """Inputs on the CPU (q, k, v, table, lens) and the caches on the GPU, with
    every sequence's pages scattered and unused table entries out of range."""
    g = gen(seed)
    B = len(lens)
    used = [(max(n, 0) + page - 1) // page for n in lens]
    width = max(max(used), 1)
    nb = sum(used) + spare
    perm = torch.randperm(nb, generator=g)
    table = torch.full((B, width), -7, dtype=torch.int32)
    at = 0
    for b, n in enumerate(used):
        table[b, :n] = perm[at:at + n]
        at += n
    q = normal(g, B * Q, Hq, D, dtype=BF16)
    ks, vs = (0.02, 0.015) if ct is E4M3 else (1.0, 1.0)
    k = (normal(g, nb, page, Hkv, D) / ks).clamp(-448, 448).to(ct)
    v = (normal(g, nb, page, Hkv, D) / vs).clamp(-448, 448).to(ct)
    kc, vc = make_cache(order, nb, page, Hkv, D, ct)
    kc.copy_(k)
    vc.copy_(v)
    return q, k, v, table, torch.tensor(lens, dtype=torch.int32), kc, vc, ks, vs


def scales(ct, ks, vs):
    if ct is not E4M3:
        return None, None
    return torch.full((1,), ks, device=DEV), torch.full((1,), vs, device=DEV)


def run(q, table, lens, kc, vc, ks, vs, ct, scale=None, window=0):
    a, b = scales(ct, ks, vs)
    out = nv.paged_attention(q.to(DEV), kc, vc, table.to(DEV), lens.to(DEV), scale=scale,
                             window=window, k_scale=a, v_scale=b)
    torch.cuda.synchronize()
    return out.cpu().double()


def check(got, q, k, v, table, lens, scale, window, ks, vs):
    """The bound. A probability enters the product with V as two bf16 (2^-16 of
    it at most is lost, and not in the sum), the scores are off by the products'
    fp32 sums (D terms of at most |q||k|, 2^-24 each for D / 32 + 8 additions,
    taken as 2 D 2^-24 sum |q k|) and the output by half a bf16 step; sums over
    the keys in fp32 add 2^-24 per addition of the longest chain, taken as
    2^-14 in all. With a = sum_j p_j |v_j| the error is at most
    a * (2^-16 + 2 * dscore + 2^-14) + |o| 2^-8."""
    ref = attention(q, k, v, table, lens, scale, window, ks, vs)
    a = attention(q, k, v.double().abs(), table, lens, scale, window, ks, vs)
    D = q.shape[-1]
    size = q.double().norm(dim=-1).max() * (k.double() * ks).norm(dim=-1).max() * scale
    dscore = 2 * D * 2.0 ** -24 * float(size)
    tol = a * (2.0 ** -16 + 2 * dscore + 2.0 ** -14) + ref.abs() * 2.0 ** -8 + 1e-30
    err = (got - ref).abs()
    bad = ~(err <= tol)
    assert not bad.any(), (int(bad.sum()), float((err / tol).max()), torch.nonzero(bad)[0].tolist())
    return float((err / tol).max())


CASES = [
    # lens, Q, Hq, Hkv, D, page, type, window, order
    ([1], 1, 4, 1, 64, 16, BF16, 0, "nhd"),
    ([33], 1, 32, 8, 128, 16, BF16, 0, "nhd"),
    ([700], 1, 32, 8, 128, 16, BF16, 0, "nhd"),
    ([700], 1, 32, 8, 128, 16, E4M3, 0, "hnd"),
    ([5000], 1, 8, 2, 128, 256, BF16, 0, "beside"),
    ([129, 0, 1, 64, 128, 500, 31], 1, 8, 2, 64, 32, BF16, 0, "nhd"),
    ([1000, 3, 777], 5, 32, 8, 128, 64, BF16, 0, "nhd"),
    ([1000, 3, 777], 5, 32, 8, 128, 64, E4M3, 0, "wide"),
    ([300, 2], 3, 16, 16, 64, 20, BF16, 100, "nhd"),
    ([300, 2], 3, 16, 16, 64, 20, E4M3, 7, "hnd"),
    ([260, 515], 2, 4, 4, 256, 16, BF16, 0, "nhd"),
    ([260, 515], 2, 4, 4, 256, 1, E4M3, 0, "nhd"),
    ([97, 200], 1, 6, 2, 128, 1, BF16, 0, "hnd"),
    ([97, 200], 8, 8, 1, 128, 7, BF16, 0, "nhd"),        # 64 rows: two tiles of 32
    ([150], 5, 16, 1, 256, 48, BF16, 0, "nhd"),          # 80 rows of a 256 head
    ([400, 90, 1], 1, 64, 1, 64, 16, E4M3, 33, "nhd"),   # 64 heads on one
    ([150, 1300], 5, 16, 2, 256, 20, BF16, 0, "nhd"),    # 40 rows of a 256 head, odd pages
    ([150, 1300], 5, 16, 2, 256, 16, E4M3, 90, "hnd"),
    ([700, 20], 3, 32, 2, 128, 3, E4M3, 0, "nhd"),       # 48 rows, one key of three to a page
    ([1025, 513, 512], 1, 8, 8, 128, 16, BF16, 0, "hnd"),
    ([63] * 70, 1, 2, 1, 64, 16, BF16, 0, "nhd"),        # more sequences than lanes
    ([1, 2, 3, 4, 5, 6, 7, 8] * 17, 2, 4, 2, 64, 16, BF16, 0, "nhd"),
    ([2049], 64, 1, 1, 64, 128, BF16, 500, "nhd"),
    ([40000], 1, 5, 1, 64, 16, BF16, 0, "nhd"),          # one head over many workgroups
]


@pytest.mark.parametrize("lens,Q,Hq,Hkv,D,page,ct,window,order", CASES)
def test_paged_attention(lens, Q, Hq, Hkv, D, page, ct, window, order):
    say(f"[attn] lens={lens[:8]} x{len(lens)} Q={Q} Hq={Hq} Hkv={Hkv} D={D} page={page} {ct} "
        f"window={window} {order}")
    q, k, v, table, ln, kc, vc, ks, vs = build(lens, Q, Hq, Hkv, D, page, ct, order, seed=D + page)
    scale = D ** -0.5
    got = run(q, table, ln, kc, vc, ks, vs, ct, window=window)
    r = check(got, q, k, v, table, ln, scale, window, ks, vs)
    say(f"  max err / tol = {r:.3f}")


def test_large_scores():
    """Scores of hundreds: the running maximum moves by far more than the slack,
    up and down; near one-hot rows."""
    q, k, v, table, ln, kc, vc, ks, vs = build([900, 130], 1, 8, 2, 128, 16, BF16, seed=5)
    got = run(q, table, ln, kc, vc, ks, vs, BF16, scale=4.0)
    check(got, q, k, v, table, ln, 4.0, 0, ks, vs)
    # keys in ascending order of score: every turn moves the maximum
    k2 = k.clone()
    base = torch.linspace(-3, 3, 900)
    for i in range(900):
        k2[table[0, i // 16], i % 16] = base[i].to(BF16)
    kc.copy_(k2)
    q2 = torch.ones_like(q)
    got = run(q2, table, ln, kc, vc, ks, vs, BF16, scale=1.0)
    check(got, q2, k2, v, table, ln, 1.0, 0, ks, vs)


@pytest.mark.parametrize("page", [16, 5])
def test_what_no_token_sees_does_not_reach_it(page):
    """NaN and infinities in the places behind each sequence, in pages that
    nobody has, before the window, and at the later new tokens: the rows that
    do not see them are bit for bit as without."""
    lens, Q, window = [70, 37, 2], 3, 20
    args = build(lens, Q, 4, 2, 64, page, BF16, seed=9)
    q, k, v, table, ln, kc, vc, ks, vs = args
    clean = run(q, table, ln, kc, vc, ks, vs, BF16, window=window)
    nb = k.shape[0]
    seen = torch.zeros(nb, page, dtype=torch.bool)
    for b, n in enumerate(lens):
        for j in range(max(0, n - Q - window + 1), n):
            seen[table[b, j // page], j % page] = True
    for bad in (float("nan"), float("inf"), -float("inf")):
        k2, v2 = k.clone(), v.clone()
        k2[~seen], v2[~seen] = bad, bad
        kc.copy_(k2)
        vc.copy_(v2)
        got = run(q, table, ln, kc, vc, ks, vs, BF16, window=window)
        assert torch.equal(got, clean)
        # the newest token's key and value: only its own row sees them
        n = lens[0]
        k2[table[0, (n - 1) // page], (n - 1) % page] = bad
        v2[table[0, (n - 1) // page], (n - 1) % page] = bad
        kc.copy_(k2)
        vc.copy_(v2)
        got = run(q, table, ln, kc, vc, ks, vs, BF16, window=window)
        assert torch.equal(got[:Q - 1], clean[:Q - 1]) and torch.equal(got[Q:], clean[Q:])
        assert torch.isnan(got[Q - 1]).all() or bad == -float("inf")


@pytest.mark.parametrize("D,Q,ct", [(64, 1, BF16), (128, 3, E4M3), (256, 2, BF16)])
def test_values_that_are_not_finite_stay_in_their_sequence(D, Q, ct):
    """A NaN value that every token of its sequence sees gives NaN in its
    dimension, an infinite one infinity or NaN (its probability is the sum of
    two bf16, the second of either sign or zero: inf + inf, inf - inf or
    inf + 0 inf); other sequences and heads stay as they were."""
    q, k, v, table, ln, kc, vc, ks, vs = build([1500, 700, 90], Q, 4, 2, D, 16, ct, seed=11)
    clean = run(q, table, ln, kc, vc, ks, vs, ct)
    for bad in (float("nan"),) if ct is E4M3 else (float("nan"), float("inf")):
        v2 = v.clone()
        v2.view(torch.uint8 if ct is E4M3 else torch.int16)[table[1, 20], 3, 1, 5] = \
            torch.tensor([bad]).to(ct).view(torch.uint8 if ct is E4M3 else torch.int16)[0]
        vc.copy_(v2)
        got = run(q, table, ln, kc, vc, ks, vs, ct)
        assert torch.equal(got[:Q], clean[:Q]) and torch.equal(got[2 * Q:], clean[2 * Q:])
        assert torch.equal(got[Q:2 * Q, :2], clean[Q:2 * Q, :2])
        hit = got[Q:2 * Q, 2:, 5]
        assert torch.all(torch.isnan(hit) | ((hit == bad) if bad == bad else False))


def test_pages_that_do_not_exist_hide_their_keys():
    for page in (16, 6):
        q, k, v, table, ln, kc, vc, ks, vs = build([200, 90, 40], 2, 8, 2, 128, page, BF16, seed=3)
        table[0, 2] = -1
        table[0, 5] = k.shape[0]
        table[1, 0] = 0x7FFFFFFF
        table[2, :] = -0x80000000        # a sequence with no page at all
        got = run(q, table, ln, kc, vc, ks, vs, BF16)
        check(got, q, k, v, table, ln, 128 ** -0.5, 0, ks, vs)
        assert torch.all(got[4:] == 0)


def test_lengths_outside_the_table():
    """Longer than the table's row counts as the row; negative as empty."""
    q, k, v, table, ln, kc, vc, ks, vs = build([64, 64, 64], 1, 4, 2, 64, 16, BF16, seed=4)
    ln = torch.tensor([1000000, -5, 0x7FFFFFFF], dtype=torch.int32)
    got = run(q, table, ln, kc, vc, ks, vs, BF16)
    check(got, q, k, v, table, ln, 0.125, 0, ks, vs)
    assert torch.all(got[1] == 0)


def test_no_pages_at_all():
    q = torch.ones(2, 4, 64, dtype=BF16, device=DEV)
    empty = torch.empty(0, 16, 2, 64, dtype=BF16, device=DEV)
    out = nv.paged_attention(q, empty, empty.clone(), torch.zeros(2, 3, dtype=torch.int32,
                                                                  device=DEV),
                             torch.tensor([5, 9], dtype=torch.int32, device=DEV))
    assert torch.all(out == 0)
    k = torch.ones(1, 16, 2, 64, dtype=BF16, device=DEV)
    out = nv.paged_attention(q, k, k.clone(), torch.zeros(2, 0, dtype=torch.int32, device=DEV),
                             torch.tensor([5, 9], dtype=torch.int32, device=DEV))
    assert torch.all(out == 0)


def test_rows_repeat_and_the_split_is_fixed():
    """The same call gives the same bits, whatever the workspace held."""
    q, k, v, table, ln, kc, vc, ks, vs = build([9000, 100, 4000], 1, 32, 8, 128, 16, BF16, seed=6)
    n = nv.paged_attention_workspace_bytes(3, 1, 32, 8, 128)
    dq, dt, dl = q.to(DEV), table.to(DEV), ln.to(DEV)
    outs = []
    for fill in (0, 0x7F, 0xFF):
        ws = torch.full((n,), fill, dtype=torch.uint8, device=DEV)
        outs.append(nv.paged_attention(dq, kc, vc, dt, dl, workspace=ws))
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])
    check(outs[0].cpu().double(), q, k, v, table, ln, 128 ** -0.5, 0, ks, vs)


def test_cache_past_4_gib():
    """Pages whose element offset passes 2^32: 40000 pages of 256 KiB, the
    sequence's first and last page at both ends (10 GiB each for K and V; only
    the used pages are written)."""
    nb, page, Hkv, D = 40000, 128, 8, 128
    kc = torch.empty(nb, page, Hkv, D, dtype=BF16, device=DEV)
    vc = torch.empty(nb, page, Hkv, D, dtype=BF16, device=DEV)
    g = gen(8)
    ids = torch.tensor([[nb - 1, 0, nb // 2, 33333]], dtype=torch.int32)
    k, v = normal(g, 4, page, Hkv, D, dtype=BF16), normal(g, 4, page, Hkv, D, dtype=BF16)
    pos = torch.arange(4 * page)
    slots = ids[0].long()[pos // page] * page + pos % page
    nv.rope_append(None, k.view(-1, Hkv, D).to(DEV), v.view(-1, Hkv, D).to(DEV), pos.to(DEV),
                   slots.to(DEV), torch.empty(0, device=DEV), kc, vc)
    q = normal(g, 1, 8, D, dtype=BF16)
    ln = torch.tensor([500], dtype=torch.int32)
    got = run(q, ids, ln, kc, vc, 1.0, 1.0, BF16)
    check(got, q, k, v, torch.arange(4, dtype=torch.int32)[None], ln, D ** -0.5, 0, 1.0, 1.0)


def test_one_scale_for_a_cache():
    """A scale for each head is refused (the first would count for all)."""
    q, k, v, table, ln, kc, vc, ks, vs = build([40], 1, 4, 2, 64, 16, E4M3)
    two, one = torch.ones(2, device=DEV), torch.ones(1, device=DEV)
    for a, b in ((two, one), (one, two), (one.double(), one)):
        with pytest.raises(TypeError):
            nv.paged_attention(q.to(DEV), kc, vc, table.to(DEV), ln.to(DEV), k_scale=a, v_scale=b)
    x = torch.ones(1, 64, device=DEV)
    with pytest.raises(ValueError):
        nv.add_rmsnorm_nvfp4(x, torch.ones(64, dtype=BF16, device=DEV), 1e-6, two)
