"""Low-rank adapters on the GPU against a plain 64-bit form: ranks, numbers of
rows and of rows that share an adapter, ragged sizes, several projections, rows
without an adapter, adapters' own ranks, in place and beside the GEMV."""
import pytest
import torch

import nvfp4_block_scaled_gemv_amd as nv
from decode_ref import gen, normal
from gpu_util import DEV, say
from serving_ref import adapters

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


def make(M, K, Ns, E, rank, seed=1):
    g = gen(seed)
    mats = [(normal(g, E, rank, K, std=K ** -0.5 if K else 1.0, dtype=BF16),
             normal(g, E, n, rank, std=0.1, dtype=BF16)) for n in Ns]
    return g, mats, normal(g, M, K, dtype=BF16)


def dev(x):
    return None if x is None else [t.to(DEV) for t in x] if isinstance(x, list) else x.to(DEV)


def run(mats, x, ids, bases=None, alpha=None, ranks=None):
    ys = nv.lora_segments([(a.to(DEV), b.to(DEV)) for a, b in mats], dev(x), dev(ids), dev(bases),
                          dev(alpha), dev(ranks))
    torch.cuda.synchronize()
    return [y.cpu().double() for y in ys]


def check(got, mats, x, ids, bases=None, alpha=None, ranks=None):
    worst = 0.0
    for y, (ref, tol) in zip(got, adapters(mats, x, ids, bases, alpha, ranks)):
        err = (y - ref).abs()
        bad = ~(err <= tol)
        assert not bad.any(), (int(bad.sum()), float((err / tol).max()),
                               torch.nonzero(bad)[0].tolist())
        worst = max(worst, float((err / tol).max())) if err.numel() else worst
        # as a whole: roundings of 2^-24, some tens of them in a row, of either sign
        if ref.numel() and float(ref.norm()):
            assert float(err.norm() / ref.norm()) < 2.0 ** -20
    return worst


CASES = [
    # M, K, Ns, E, rank, ids' range
    (1, 32, [1], 1, 8, 1),
    (1, 4096, [4096, 1024, 1024], 3, 16, 3),
    (2, 256, [333, 5], 4, 8, 4),
    (3, 1024, [64], 2, 24, 2),
    (8, 1056, [257, 256, 255], 5, 32, 5),
    (16, 2048, [1000], 3, 64, 1),
    (17, 2048, [1000], 3, 16, 1),                 # two workgroups of one adapter
    (33, 512, [100, 4], 40, 40, 40),
    (64, 320, [130], 7, 128, 7),
    (65, 96, [513], 2, 8, 2),
    (128, 4096, [300], 1, 16, 1),                 # all rows on one adapter
    (128, 1120, [70, 512], 128, 16, 128),
    (128, 64, [31], 3, 256, 3),
    (5, 12288, [512], 2, 16, 2),
    (2, 20000 // 32 * 32, [64], 2, 104, 2),       # chunks of two turns
    (127, 512, [1, 2, 3, 4, 5, 6, 7, 8], 9, 16, 9),
]


@pytest.mark.parametrize("M,K,Ns,E,rank,upto", CASES)
def test_adapters(M, K, Ns, E, rank, upto):
    say(f"[lora] M={M} K={K} Ns={Ns} E={E} rank={rank}")
    g, mats, x = make(M, K, Ns, E, rank, seed=M + K)
    ids = torch.randint(0, upto, (M,), generator=g, dtype=torch.int32)
    got = run(mats, x, ids)
    say(f"  plain {check(got, mats, x, ids):.3f}")
    # a base, factors, ranks of their own, rows without an adapter
    bases = [normal(g, M, n) for n in Ns]
    alpha = normal(g, E)
    ranks = torch.randint(-1, rank + 3, (E,), generator=g, dtype=torch.int32)
    if M > 1:
        for i, bad in enumerate((-1, E, 0x7FFFFFFF, -0x80000000)):
            if i * 5 + 1 < M:
                ids[i * 5 + 1] = bad
    got = run(mats, x, ids, bases, alpha, ranks)
    say(f"  all {check(got, mats, x, ids, bases, alpha, ranks):.3f}")
    none = [m for m, e in enumerate(ids.tolist()) if not 0 <= e < E]
    for y, b in zip(got, bases):
        assert torch.equal(y[none], b[none].double())


@pytest.mark.parametrize("N", [1024, 1023])
def test_in_place_and_into_unaligned_rows(N):
    """base and y one array; arrays that start 4 bytes off 16; what lies beside
    them stays."""
    M, K, E, rank = 6, 512, 3, 16
    g, mats, x = make(M, K, [N], E, rank, seed=3)
    ids = torch.tensor([0, -1, 2, 0, 1, 7], dtype=torch.int32)
    base = normal(g, M, N)
    want = run(mats, x, ids, [base])[0]
    a = [(mats[0][0].to(DEV), mats[0][1].to(DEV))]
    ws = torch.empty(nv.lora_workspace_bytes(M, K, rank, 1), dtype=torch.uint8, device=DEV)
    for off in (0, 1):
        buf = torch.full((M * N + 8,), 7.0, device=DEV)
        y = buf[off:off + M * N].view(M, N)
        y.copy_(base)
        nv.lora_segments_into(a, x.to(DEV), ids.to(DEV), [y], ws, bases=[y])
        torch.cuda.synchronize()
        assert torch.equal(y.cpu().double(), want)
        assert torch.all(buf[:off] == 7) and torch.all(buf[off + M * N:] == 7)


def test_the_same_bits_whoever_shares_the_call():
    """A row's result does not depend on the other rows, nor on the workspace."""
    M, K, E, rank = 40, 4096, 4, 16
    g, mats, x = make(M, K, [384], E, rank, seed=4)
    ids = torch.randint(0, E, (M,), generator=g, dtype=torch.int32)
    a = [(mats[0][0].to(DEV), mats[0][1].to(DEV))]
    n = nv.lora_workspace_bytes(M, K, rank, 1)
    outs = []
    for fill in (0, 0x7F, 0xFF):
        ws = torch.full((n,), fill, dtype=torch.uint8, device=DEV)
        outs.append(nv.lora_segments(a, x.to(DEV), ids.to(DEV), workspace=ws)[0])
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])
    for m in (0, 7, 39):
        alone = nv.lora_segments(a, x[m:m + 1].to(DEV), ids[m:m + 1].to(DEV))[0]
        assert torch.equal(alone[0], outs[0][m])


def test_what_is_not_an_adapters_own_may_be_anything():
    """NaN in the ranks past an adapter's own, in adapters that no row has and in
    outputs of other rows of B reach nobody."""
    M, K, E, rank, N = 9, 256, 4, 16, 70
    g, mats, x = make(M, K, [N], E, rank, seed=5)
    ids = torch.tensor([0, 1, 0, 2, 1, 0, 2, 2, -1], dtype=torch.int32)
    for rank_of in ([16, 8, 5, 16], [1, 0, 9, 0], [15, 16, 7, 3]):
        ranks = torch.tensor(rank_of, dtype=torch.int32)
        want = run(mats, x, ids, None, None, ranks)
        check(want, mats, x, ids, None, None, ranks)
        a, b = (t.clone() for t in mats[0])
        for e, r in enumerate(rank_of):
            a[e, r:], b[e, :, r:] = float("nan"), float("inf")
        a[3], b[3] = float("nan"), float("nan")
        got = run([(a, b)], x, ids, None, None, ranks)
        assert torch.equal(got[0], want[0])
    for rank in (8, 16, 32):
        g, mats, x = make(M, K, [N], E, rank, seed=rank)
        want = run(mats, x, ids)[0]
        a, b = (t.clone() for t in mats[0])
        b[:, 33] = float("inf")
        b[:, 66] = float("nan")
        got = run([(a, b)], x, ids)[0]
        keep = [n for n in range(N) if n not in (33, 66)]
        assert torch.equal(got[:, keep], want[:, keep])
        assert not torch.isfinite(got[:8, [33, 66]]).any()
        # a row of x that is not finite
        x2 = x.clone()
        x2[4, 5] = float("nan")
        got = run(mats, x2, ids)[0]
        rest = [m for m in range(M) if m != 4]
        assert torch.equal(got[rest], want[rest]) and torch.isnan(got[4]).all()


def test_sizes_of_nothing():
    g, mats, x = make(3, 0, [5], 2, 8, seed=6)
    base = [normal(g, 3, 5)]
    ids = torch.tensor([0, 1, -1], dtype=torch.int32)
    assert torch.equal(run(mats, x, ids, base)[0], base[0].double())
    assert torch.all(run(mats, x, ids)[0] == 0)
    g, mats, x = make(3, 64, [5], 0, 8, seed=7)           # no adapter at all
    assert torch.equal(run(mats, x, ids, base)[0], base[0].double())
    g, mats, x = make(0, 64, [5], 2, 8, seed=8)
    assert run(mats, x, ids[:0])[0].shape == (0, 5)
    g, mats, x = make(3, 64, [0, 7], 2, 8, seed=9)        # an empty projection
    got = run(mats, x, ids)
    assert got[0].shape == (3, 0)
    check(got[1:], mats[1:], x, ids)


def test_adapters_past_4_gib():
    """An adapter whose elements lie past 2^32 bytes, and past 2^31 elements."""
    E, rank, K, N = 70000, 64, 512, 64                    # A: 4.6 GB
    a = torch.empty(E, rank, K, dtype=BF16, device=DEV)
    b = torch.empty(E, N, rank, dtype=BF16, device=DEV)
    g, mats, x = make(3, K, [N], 3, rank, seed=10)
    at = torch.tensor([0, E - 1, 66000], device=DEV)
    a[at], b[at] = mats[0][0].to(DEV), mats[0][1].to(DEV)
    got = nv.lora_segments([(a, b)], x.to(DEV), at.to(torch.int32))[0].cpu().double()
    check([got], mats, x, torch.arange(3, dtype=torch.int32))


def test_one_launch_and_two_give_the_same_bits():
    """Few rows of a small rank take one launch, many two; the order of every sum
    is the same: a row alone gives the bits that it has among 128."""
    for K, rank, Ns in ((4096, 16, [300, 8]), (1056, 8, [1025]), (5152, 8, [64])):
        g, mats, x = make(128, K, Ns * 2, 8, rank, seed=K)
        mats = mats[:len(Ns)]
        ids = torch.randint(0, 8, (128,), generator=g, dtype=torch.int32)
        wide = [(a, b.repeat(1, 12, 1)) for a, b in mats]    # more outputs: two launches
        many = run(wide, x, ids)
        for m in (0, 77, 127):
            alone = run(mats, x[m:m + 1], ids[m:m + 1])
            for y, z, n in zip(alone, many, Ns):
                assert torch.equal(y[0], z[m, :n])
