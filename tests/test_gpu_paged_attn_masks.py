"""What no token sees, pages that do not exist and lengths outside the table, in
every form of attention over a paged cache: short tables and wide ones (whose
sequences are shared by several wavefronts and joined), one row tile and two,
pages that hold whole runs of 16 keys and pages that do not, bf16 and E4M3."""
import pytest
import torch

from gpu_util import say
from test_gpu_paged_attn import BF16, E4M3, build, check, run

pytestmark = pytest.mark.gpu

FORMS = [(ct, D, page, wide, G)
         for ct in (BF16, E4M3) for D in (64, 128, 256) for page in (16, 5)
         for wide in (False, True) for G in (2, 8)]
form = pytest.mark.parametrize("ct,D,page,wide,G", FORMS)


def bits(ct):
    """Patterns that a place may hold: NaN and infinities of the type, and all
    bits set."""
    if ct is E4M3:
        return [torch.tensor(b, dtype=torch.uint8) for b in (0x7F, 0xFF)]
    return [torch.tensor(b, dtype=torch.int16) for b in (0x7FC0, 0x7F80, -0x80, -1)]


def raw(t):
    return t.view(torch.uint8 if t.dtype is E4M3 else torch.int16)


@form
def test_what_no_token_sees(ct, D, page, wide, G):
    """Any bits behind the sequences, in pages that nobody has, before the
    window and at the later new tokens: rows that do not see them are bit for
    bit as without, and a row that does see a bad key or value is not finite."""
    say(f"[attn masks] {ct} D={D} page={page} wide={wide} G={G}")
    lens, Q, Hkv = ([1500, 70, 37, 2], 3, 2) if wide else ([200, 70, 37, 2], 3, 2)
    window = 1100 if wide else 20        # a window bounds the keys of a form, too
    q, k, v, table, ln, kc, vc, ks, vs = build(lens, Q, G * Hkv, Hkv, D, page, ct, seed=D + page)
    clean = run(q, table, ln, kc, vc, ks, vs, ct, window=window)
    check(clean, q, k, v, table, ln, D ** -0.5, window, ks, vs)
    seen = torch.zeros(k.shape[0], page, dtype=torch.bool)
    for b, n in enumerate(lens):
        j = torch.arange(max(0, n - Q - window + 1), n)
        seen[table[b].long()[j // page], j % page] = True
    for bad in bits(ct):
        def put(which):
            """The caches with `bad` where nobody looks, and at the newest token
            of sequences 0 and 1, which only its own rows see."""
            for x, c in (("k", kc), ("v", vc)):
                t = (k if x == "k" else v).clone()
                raw(t)[~seen] = bad
                for b in (0, 1) if x in which else ():
                    n = lens[b] - 1
                    raw(t)[table[b, n // page], n % page] = bad
                c.copy_(t)
        put("")
        assert torch.equal(run(q, table, ln, kc, vc, ks, vs, ct, window=window), clean)
        for which in ("k", "v", "kv"):
            put(which)
            got = run(q, table, ln, kc, vc, ks, vs, ct, window=window)
            hit = torch.zeros(len(lens) * Q, dtype=torch.bool)
            hit[Q - 1] = hit[2 * Q - 1] = True
            assert torch.equal(got[~hit], clean[~hit]), (which, int(bad))
            if which == "v" or int(bad) in (0x7F, 0xFF, 0x7FC0, -1):
                assert not torch.isfinite(got[hit]).any(), (which, int(bad))


@form
def test_pages_that_do_not_exist(ct, D, page, wide, G):
    """Holes inside a sequence that several wavefronts share, at its ends, two
    in a row, in a window's reach, and a sequence without any page. The page
    that is read in place of one that does not exist holds NaN."""
    lens, Q, Hkv = ([1500, 1100, 90, 40], 3, 2) if wide else ([200, 150, 90, 40], 3, 2)
    q, k, v, table, ln, kc, vc, ks, vs = build(lens, Q, G * Hkv, Hkv, D, page, ct, seed=D)
    table[table == 0] = -1
    for t, c in ((k, kc), (v, vc)):
        raw(t)[0] = bits(ct)[0]
        c.copy_(t)
    last = (lens[0] - 1) // page
    for j, bad in ((0, -1), (3, k.shape[0]), (last // 2, 0x7FFFFFFF), (last // 2 + 1, -0x80000000),
                   (last, -7)):
        table[0, j] = bad
    table[1, 1] = k.shape[0] + 5
    table[3, :] = -2
    for window in (0, 1050 if wide else 60):
        got = run(q, table, ln, kc, vc, ks, vs, ct, window=window)
        k2, v2 = k.clone(), v.clone()
        raw(k2)[0], raw(v2)[0] = 0, 0                     # not seen by the reference either
        check(got, q, k2, v2, table, ln, D ** -0.5, window, ks, vs)
        assert torch.all(got[3 * Q:] == 0)


@form
def test_lengths_outside_the_table(ct, D, page, wide, G):
    """Longer than the table's row counts as the row, negative as empty."""
    n = 1300 if wide else 60
    n = n // page * page                                  # the row's whole width
    q, k, v, table, ln, kc, vc, ks, vs = build([n] * 5, 3, G, 1, D, page, ct, seed=D + 1)
    ln = torch.tensor([1000000, -5, 0x7FFFFFFF, -0x80000000, 0], dtype=torch.int32)
    got = run(q, table, ln, kc, vc, ks, vs, ct)
    check(got, q, k, v, table, ln, D ** -0.5, 0, ks, vs)
    for b in (1, 3, 4):
        assert torch.all(got[3 * b:3 * b + 3] == 0)
