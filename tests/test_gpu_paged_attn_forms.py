"""Attention over a paged cache on both sides of the border between its forms
(a workgroup for each sequence and head, or runs of tiles that a second launch
joins): tables of as many keys as the border and one page more, few sequences
and many, one row for each head and many."""
import pytest

from gpu_util import say
from test_gpu_paged_attn import BF16, E4M3, build, check, run

pytestmark = pytest.mark.gpu

# (sequences, tokens, query heads, key-value heads, D, type): 2^16 bytes of a
# head's keys; twice that from 256 rows; 1024 keys from 256 workgroups, or 128
# with 16 rows each; many workgroups of one row, which never take the first form
CASES = [(1, 1, 8, 2, 128, BF16, 256), (1, 1, 8, 2, 64, E4M3, 1024), (2, 2, 8, 4, 64, BF16, 512),
         (8, 1, 32, 8, 128, BF16, 512), (4, 5, 16, 4, 128, E4M3, 1024),
         (32, 1, 8, 8, 64, BF16, 1024), (16, 4, 32, 8, 128, BF16, 1024),
         (40, 1, 8, 8, 64, BF16, 512), (100, 1, 8, 8, 64, E4M3, 32), (257, 1, 2, 1, 128, BF16, 256)]


@pytest.mark.parametrize("B,Q,Hq,Hkv,D,ct,border", CASES)
@pytest.mark.parametrize("page", [16, 8])
def test_both_sides_of_the_border(B, Q, Hq, Hkv, D, ct, border, page):
    say(f"[attn forms] B={B} Q={Q} heads {Hq}/{Hkv} of {D} {ct} keys {border} page={page}")
    for keys in (border, border + page):
        lens = [keys] + [(37 * i) % min(keys, 90) for i in range(1, B)]
        q, k, v, table, ln, kc, vc, ks, vs = build(lens, Q, Hq, Hkv, D, page, ct, seed=B + keys)
        got = run(q, table, ln, kc, vc, ks, vs, ct)
        check(got, q, k, v, table, ln, D ** -0.5, 0, ks, vs)
