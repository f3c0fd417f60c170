"""How many bits of a probability attention over a paged cache uses: values
that cancel under their weights leave an output far below them, in which a
rounding of the probabilities to fewer bits than fp32's 24 would stand out."""
import math

import pytest
import torch

import nvfp4_block_scaled_gemv_amd as nv
from decode_ref import attention, gen
from gpu_util import DEV, say
from test_gpu_rope import make_cache

pytestmark = pytest.mark.gpu

BF16, E4M3 = torch.bfloat16, torch.float8_e4m3fn

# The fp32 number whose fp32 product with fp32(log2 e) is exactly 1: the kernel's
# scores, in powers of two, are then q . k itself, without a rounding. (In 64
# bits the product is 1 + 2.7e-9, 2^-28.4.)
SCALE = 0.6931471824645996


def cancelling(lens, Hkv, D, page, ct, seed):
    """Caches in which every sequence and head has a few keys of weight whose
    values cancel, dimension by dimension, to the last bits of ct; all others
    have a weight of 2^-60 and the value zero. Key 0 of the few has the score 0,
    so it is the maximum."""
    g = gen(seed)
    n = 3 if ct is BF16 else 5
    B = len(lens)
    used = [(x + page - 1) // page for x in lens]
    nb = sum(used) + 1
    table = torch.full((B, max(used)), -1, dtype=torch.int32)
    perm = torch.randperm(nb, generator=g)
    k = torch.zeros(nb, page, Hkv, D)
    v = torch.zeros(nb, page, Hkv, D)
    k[..., 0] = -60.0
    at = 0
    for b, u in enumerate(used):
        table[b, :u] = perm[at:at + u]
        at += u
        first = int(torch.randint(0, max(1, lens[b] - 32), (1,), generator=g)) // 32 * 32
        keys = first + torch.randperm(min(32, lens[b] - first - 4), generator=g)[:n]
        pages, place = table[b, keys // page].long(), keys % page
        # scores in [-1, -0.25]: one number of bf16, or two of E4M3, the second
        # of which counts a 64th
        s = -(0.25 + 0.75 * torch.rand(n, Hkv, generator=g))
        s[0] = 0
        hi = s.to(ct).float()
        lo = ((s - hi) * 64).to(ct).float() if ct is E4M3 else torch.zeros_like(s)
        k[pages, place, :, 0] = hi
        k[pages, place, :, 1] = lo
        p = torch.exp2(hi.double() + lo.double() / 64)[..., None]
        rest = torch.zeros(Hkv, D, dtype=torch.float64)
        for j in list(range(1, n)) + [0]:
            x = (1 + torch.rand(Hkv, D, generator=g).double()) * (128 if ct is E4M3 else 1) \
                if j == 1 else -rest / p[j]
            x = x.float().to(ct).double()
            v[pages[j], place[j]] = x.float()
            rest += p[j] * x
    kc, vc = make_cache("nhd", nb, page, Hkv, D, ct)
    kc.copy_(k.to(ct))
    vc.copy_(v.to(ct))
    return k.to(ct), v.to(ct), kc, vc, table, torch.tensor(lens, dtype=torch.int32)


CASES = [
    # lens, Q, G, Hkv, D, page, type: the whole form (tables of few keys), the
    # split one (heads of 256, wide tables); one row tile and two
    ([40, 64, 200], 1, 1, 8, 64, 16, BF16),
    ([40, 64, 200], 1, 4, 8, 128, 16, BF16),
    ([40, 64, 200], 1, 4, 8, 128, 16, E4M3),
    ([300, 41], 5, 5, 2, 128, 20, BF16),
    ([300, 41], 5, 5, 2, 128, 16, E4M3),
    ([1500, 40, 700], 1, 2, 8, 64, 16, E4M3),
    ([1500, 40, 700], 1, 4, 8, 128, 16, BF16),
    ([1500, 40, 700], 4, 5, 4, 128, 16, BF16),
    ([1500, 40, 700], 4, 5, 4, 64, 5, BF16),
    ([1500, 40, 700], 1, 4, 4, 256, 16, BF16),
    ([1500, 40, 700], 4, 5, 2, 256, 16, E4M3),
    ([1500, 40, 700], 4, 5, 2, 256, 5, BF16),
]


@pytest.mark.parametrize("lens,Q,G,Hkv,D,page,ct", CASES)
def test_probabilities_keep_24_bits(lens, Q, G, Hkv, D, page, ct):
    """With u = 2^-24 and a the sum of the weighted values' sizes over the sum of
    the weights: an exponential is off by SCALE's error (u / 20 of it) and one
    step of the instruction (2 u), each of the few additions of the product by
    at most a step (2 u of a), four of them at the size of a and the others far
    below; the sum of the weights, the division and the last product touch the
    output by under 16 u of itself, then half a step of bf16. In all
    a 16 u + |o| (2^-8 + 16 u), and 2^-59 for the weights that are not the few's.
    Weights of 16 bits are off by up to 64 u each."""
    say(f"[attn bits] lens={lens} Q={Q} G={G} Hkv={Hkv} D={D} page={page} {ct}")
    k, v, kc, vc, table, ln = cancelling(lens, Hkv, D, page, ct, D + page + Q)
    q = torch.zeros(len(lens) * Q, G * Hkv, D, dtype=BF16)
    q[..., 0] = 1
    q[..., 1] = 1 / 64
    one = torch.ones(1, device=DEV) if ct is E4M3 else None
    got = nv.paged_attention(q.to(DEV), kc, vc, table.to(DEV), ln.to(DEV), scale=SCALE,
                             k_scale=one, v_scale=one).cpu().double()
    ref = attention(q, k, v, table, ln, SCALE)
    a = attention(q, k, v.double().abs(), table, ln, SCALE)
    assert float((ref.abs() / a).median()) < 2.0 ** -12       # they do cancel
    u = 2.0 ** -24
    tol = a * 16 * u + ref.abs() * (2.0 ** -8 + 16 * u) + 2.0 ** -59
    err = (got - ref).abs()
    say(f"  max err / tol = {float((err / tol).max()):.3f}")
    assert torch.all(err <= tol), float((err / tol).max())
    assert math.isfinite(float(got.abs().max()))
