"""Rotation and append around and past the 256 tokens from where a workgroup
takes a whole token or several: heads that fill a workgroup, and that do not,
in both layouts and cache types."""
import pytest

import test_gpu_rope as rope
from test_gpu_rope import BF16, E4M3, F32

pytestmark = pytest.mark.gpu

CASES = [
    (256, 28, 4, 128, 128, 16, F32, BF16, False, "nhd", 5),
    (257, 28, 4, 128, 128, 16, F32, BF16, False, "nhd", 5),
    (256, 2, 1, 64, 32, 7, BF16, E4M3, True, "hnd", 100),
    (258, 2, 1, 64, 32, 7, BF16, E4M3, True, "hnd", 100),
    (300, 8, 8, 256, 256, 256, BF16, BF16, False, "nhd", 9),
    (263, 32, 8, 128, 64, 64, BF16, E4M3, True, "wide", 1 << 20),
    (400, 1, 1, 16, 16, 3, F32, BF16, True, "nhd", 0),
    (289, 7, 1, 80, 32, 16, BF16, E4M3, False, "beside", 1 << 26),
    (270, 28, 4, 128, 0, 32, F32, BF16, False, "nhd", 3),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: f"{c[0]}-{c[1]}-{c[2]}-{c[3]}")
def test_many_tokens(case):
    rope.test_rope_append(*case)
