"""Attention over bf16 and E4M3 caches with capped scores and biases by
distance against a plain 64-bit form; without either it is paged_attention."""
import pytest
import torch

import nvfp4_block_scaled_gemv_amd as nv
from gpu_util import DEV, say
from serving_ref import attention, slopes_of
from test_gpu_paged_attn import BF16, E4M3, build, run as run_plain, scales

pytestmark = pytest.mark.gpu


def run(q, table, lens, kc, vc, ks, vs, ct, slopes=None, **kw):
    a, b = scales(ct, ks, vs)
    out = nv.paged_attention_scored(q.to(DEV), kc, vc, table.to(DEV), lens.to(DEV), k_scale=a,
                                    v_scale=b, slopes=None if slopes is None else slopes.to(DEV),
                                    **kw)
    torch.cuda.synchronize()
    return out.cpu().double()


def check(got, q, k, v, table, lens, scale, window, ks, vs, softcap, slopes):
    """The bound of plain attention over these caches, with scores off by 2^-20 of
    their largest more: the cap (2^-21 of it), and six roundings of 2^-24 for the
    scale's products, the bias's product and addition and the factors of log2."""
    top = [0.0]

    def weigh(z, w, vh):
        top[0] = max(top[0], float(z.abs().max()))
    kd, vd = k.double() * ks, v.double() * vs
    ref = attention(q, kd, vd, table, lens, scale, window, softcap, slopes, weigh)
    a = attention(q, kd, vd.abs(), table, lens, scale, window, softcap, slopes)
    D = q.shape[-1]
    size = float(q.double().norm(dim=-1).max() * kd.norm(dim=-1).max()) * abs(scale)
    dz = 2 * D * 2.0 ** -24 * size + 2.0 ** -20 * top[0]
    tol = a * (2.0 ** -23 + 2 * dz + 2.0 ** -14) + ref.abs() * 2.0 ** -8 + 1e-30
    err = (got - ref).abs()
    bad = ~(err <= tol)
    assert not bad.any(), (int(bad.sum()), float((err / tol).max()), torch.nonzero(bad)[0].tolist())
    return float((err / tol).max())


CASES = [
    # lens, Q, Hq, Hkv, D, page, type, window, order, softcap, bias
    ([1], 1, 4, 1, 64, 16, BF16, 0, "nhd", 30.0, False),
    ([700], 1, 32, 8, 128, 16, BF16, 0, "nhd", 50.0, False),
    ([700], 1, 32, 8, 128, 16, E4M3, 0, "hnd", 0.0, True),
    ([129, 0, 1, 64, 128, 500, 31], 1, 8, 2, 64, 32, BF16, 0, "nhd", 1.0, True),
    ([1000, 3, 777], 5, 32, 8, 128, 64, BF16, 0, "nhd", 0.0, True),
    ([1000, 3, 777], 5, 32, 8, 128, 64, E4M3, 300, "wide", 20.0, True),
    ([300, 2], 3, 16, 16, 64, 20, BF16, 100, "nhd", 5.0, False),
    ([260, 515], 2, 4, 4, 256, 16, BF16, 0, "nhd", 8.0, True),
    ([260, 515], 2, 4, 4, 256, 1, E4M3, 0, "nhd", 0.0, True),
    ([97, 200], 8, 8, 1, 128, 7, BF16, 0, "nhd", 0.01, False),
    ([150, 1300], 5, 16, 2, 256, 16, E4M3, 90, "hnd", 12.0, False),
    ([5000], 1, 8, 2, 128, 256, BF16, 0, "beside", 0.0, True),
    ([2049], 64, 1, 1, 64, 128, BF16, 500, "nhd", 3.0, True),
]


@pytest.mark.parametrize("lens,Q,Hq,Hkv,D,page,ct,window,order,cap,bias", CASES)
def test_scored(lens, Q, Hq, Hkv, D, page, ct, window, order, cap, bias):
    say(f"[scored] lens={lens[:8]} x{len(lens)} Q={Q} Hq={Hq} Hkv={Hkv} D={D} page={page} {ct} "
        f"window={window} {order} cap={cap} bias={bias}")
    q, k, v, table, ln, kc, vc, ks, vs = build(lens, Q, Hq, Hkv, D, page, ct, order, seed=D + page)
    q = q * 4
    slopes = slopes_of(Hq) if bias else None
    got = run(q, table, ln, kc, vc, ks, vs, ct, slopes, softcap=cap, window=window)
    r = check(got, q, k, v, table, ln, D ** -0.5, window, ks, vs, cap, slopes)
    say(f"  max err / tol = {r:.3f}")


@pytest.mark.parametrize("ct", [BF16, E4M3])
def test_without_either_it_is_paged_attention(ct):
    args = build([1000, 33, 0], 2, 8, 2, 128, 16, ct, seed=2)
    q, k, v, table, ln, kc, vc, ks, vs = args
    want = run_plain(q, table, ln, kc, vc, ks, vs, ct, window=200)
    assert torch.equal(run(q, table, ln, kc, vc, ks, vs, ct, window=200), want)
    # slopes of zero: the same up to the bits that the addition of zero keeps
    got = run(q, table, ln, kc, vc, ks, vs, ct, torch.zeros(8), window=200)
    assert torch.equal(got, want)


def test_slopes_of_either_sign_over_far_keys():
    """Keys that are weighed more the farther they are, and less, 20000 of them."""
    q, k, v, table, ln, kc, vc, ks, vs = build([20000], 1, 4, 2, 64, 64, BF16, seed=12)
    slopes = torch.tensor([-2.0 ** -8, 2.0 ** -8, -1.0, 1.0])
    got = run(q, table, ln, kc, vc, ks, vs, BF16, slopes)
    check(got, q, k, v, table, ln, 0.125, 0, ks, vs, 0.0, slopes)


@pytest.mark.parametrize("cap", [1e-6, 0.5, 1e30])
def test_caps_at_the_ends(cap):
    """A cap below every score leaves a plain mean, one above all changes nothing
    that shows."""
    q, k, v, table, ln, kc, vc, ks, vs = build([400], 2, 8, 2, 128, 16, BF16, seed=13)
    got = run(q, table, ln, kc, vc, ks, vs, BF16, softcap=cap)
    check(got, q, k, v, table, ln, 128 ** -0.5, 0, ks, vs, cap, None)


def test_a_cap_makes_infinite_scores_finite():
    """An infinite key's score is +-cap, a NaN one's NaN."""
    q, k, v, table, ln, kc, vc, ks, vs = build([40], 1, 2, 1, 64, 16, BF16, seed=14)
    q = torch.ones_like(q)
    k[table[0, 0], 3, 0, 0] = float("inf")
    kc.copy_(k)
    got = run(q, table, ln, kc, vc, ks, vs, BF16, softcap=10.0)
    k2 = k.clone()
    k2[table[0, 0], 3, 0] = 1e30
    check(got, q, k2.clamp(max=1e3), v, table, ln, 0.125, 0, ks, vs, 10.0, None)
    k[table[0, 0], 3, 0, 0] = float("nan")
    kc.copy_(k)
    assert torch.isnan(run(q, table, ln, kc, vc, ks, vs, BF16, softcap=10.0)).all()


@pytest.mark.parametrize("cap,spread", [(50.0, 1.0), (50.0, 9.0), (2.0, 9.0), (500.0, 60.0)])
def test_tanh_near_and_far(cap, spread):
    """Tiles whose scores all lie in tanh's near part, in both, and far out, against
    a weighted mean that shows the scores' errors: 2^-21 of the cap at most."""
    q, k, v, table, ln, kc, vc, ks, vs = build([300], 1, 4, 1, 64, 16, BF16, seed=15)
    q = q * spread
    got = run(q, table, ln, kc, vc, ks, vs, BF16, softcap=cap)
    check(got, q, k, v, table, ln, 0.125, 0, ks, vs, cap, None)


def paired(lens, Q, G, Hkv, page, seed, order="nhd"):
    """An E4M3 cache with heads of 64 and a table wide enough for the form that takes
    two heads side by side."""
    q, k, v, table, ln, kc, vc, ks, vs = build(lens, Q, G * Hkv, Hkv, 64, page, E4M3, order,
                                               seed=seed)
    width = (1 << 19) // (Hkv * len(lens) * page) + 1
    table = torch.cat([table, torch.full((len(lens), width), -1, dtype=torch.int32)], 1)
    return q, k, v, table, ln, kc, vc, ks, vs


PAIRS = [
    # lens, Q, G, Hkv, page, window, order, softcap, bias
    ([1], 1, 1, 2, 16, 0, "nhd", 30.0, False),
    ([700], 1, 1, 16, 20, 0, "nhd", 0.0, True),
    ([5000, 0, 1, 17, 333], 1, 4, 8, 16, 0, "nhd", 20.0, True),
    ([5000, 0, 1, 17, 333], 2, 4, 8, 20, 0, "hnd", 0.0, True),
    ([1000, 3, 777], 4, 2, 4, 4, 0, "wide", 5.0, False),
    ([1000, 3, 777], 8, 1, 2, 64, 0, "beside", 0.0, True),
    ([15, 16, 2049], 3, 1, 6, 48, 0, "nhd", 50.0, True),
]


@pytest.mark.parametrize("lens,Q,G,Hkv,page,window,order,cap,bias", PAIRS)
def test_two_heads_side_by_side(lens, Q, G, Hkv, page, window, order, cap, bias):
    say(f"[scored pairs] lens={lens} Q={Q} G={G} Hkv={Hkv} page={page} {order} cap={cap} "
        f"bias={bias}")
    q, k, v, table, ln, kc, vc, ks, vs = paired(lens, Q, G, Hkv, page, 16, order)
    q = q * 4
    slopes = slopes_of(G * Hkv) if bias else None
    got = run(q, table, ln, kc, vc, ks, vs, E4M3, slopes, softcap=cap, window=window)
    check(got, q, k, v, table, ln, 0.125, window, ks, vs, cap, slopes)
    assert torch.equal(got, run(q, table, ln, kc, vc, ks, vs, E4M3, slopes, softcap=cap,
                                window=window))


@pytest.mark.parametrize("page", [16, 20])
def test_side_by_side_with_a_window(page):
    """A window of 2^16 keys, of 90000 and of 300."""
    q, k, v, table, ln, kc, vc, ks, vs = build([90000, 300], 2, 8, 8, 64, page, E4M3, seed=17)
    slopes = slopes_of(8) / 64
    got = run(q, table, ln, kc, vc, ks, vs, E4M3, slopes, window=1 << 16)
    check(got, q, k, v, table, ln, 0.125, 1 << 16, ks, vs, 0.0, slopes)


@pytest.mark.parametrize("page", [16, 20])
def test_side_by_side_unseen_and_nan_values(page):
    """NaN behind each sequence and in pages that nobody has leave every row as it
    was, bit for bit; a NaN value stays with the rows of its head that see it."""
    lens, Q = [70, 700, 2], 2
    q, k, v, table, ln, kc, vc, ks, vs = paired(lens, Q, 2, 4, page, 18)
    slopes = slopes_of(8)
    clean = run(q, table, ln, kc, vc, ks, vs, E4M3, slopes, softcap=9.0)
    check(clean, q, k, v, table, ln, 0.125, 0, ks, vs, 9.0, slopes)
    seen = torch.zeros(kc.shape[0], page, dtype=torch.bool)
    for b, n in enumerate(lens):
        for j in range(n):
            seen[table[b, j // page], j % page] = True
    for c in (kc, vc):
        c.view(torch.uint8)[(~seen).to(DEV)] = 0x7F
    got = run(q, table, ln, kc, vc, ks, vs, E4M3, slopes, softcap=9.0)
    assert torch.equal(got, clean)
    vc.view(torch.uint8)[table[1, 699 // page], 699 % page, 1, 5] = 0xFF
    got = run(q, table, ln, kc, vc, ks, vs, E4M3, slopes, softcap=9.0).view(3, 2, 4, 2, 64)
    was = clean.view(3, 2, 4, 2, 64)
    assert torch.isnan(got[1, 1, 1, :, 5]).all()
    got[1, 1, 1] = was[1, 1, 1]
    assert torch.equal(got, was)
