"""The measured cases of perf/more_operators.py and a few drawn ones: the library's
outputs are no further from the 64-bit definition than the plain 32-bit form's."""
import importlib.util
import os
import random

import pytest
import torch

from gpu_util import say

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def load():
    spec = importlib.util.spec_from_file_location("operator_cases",
                                                  os.path.join(ROOT, "perf", "more_operators.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def cases():
    m = load()
    out = m.listed()
    rng = random.Random(11)
    for i in range(16):
        c = m.draw(rng)
        c["name"] = f"drawn {i}"
        out.append(c)
    return out


def distance(a, e):
    return float((a.double() - e).norm())


def as_list(x):
    return list(x) if isinstance(x, (list, tuple)) else [x]


@pytest.mark.parametrize("case", cases(), ids=lambda c: c["name"].replace(" ", "-"))
def test_as_near_as_the_plain_form(case):
    """Outputs of 16 bits or fewer: both forms compute in 32 bits and round once,
    so their distances to the exact outputs are the roundings', sqrt(r^2 + e^2) with
    a rounding's rms r and 32-bit errors of rms e < r / 8: within 1 % of each other.
    Outputs of 32 bits (adapters): every product is exact and each sum of K, of
    rank and of a few terms rounds by 2^-24 of partial sums: K / 32 + 40 roundings in
    the longest chain of matrix instructions and additions, random in sign, come
    to 2^-24 sqrt(K / 32 + 40) of the terms' root mean square sum, which is the
    output's: 2^-24 * 21 = 1.2e-6 at K 12288; as a whole within 2^-19."""
    say(f"[cases] {case}")
    m = load()
    plain = as_list(m.run(m.prepare(case, 3)))
    m.own = True
    own = as_list(m.run(m.prepare(case, 3)))       # its own buffers, not the plain form's
    exact = as_list(m.exact(case, 3))
    assert len(own) == len(plain) == len(exact)
    for o, p, e in zip(own, plain, exact):
        assert o.shape == p.shape and o.dtype is p.dtype
        if e is None:      # 4-bit values: a border may fall the other way
            assert float((o.float() != p.float()).float().mean()) < 1e-3
        elif o.dtype is torch.float32:
            assert distance(o, e) <= 2.0 ** -19 * float(e.norm())
        else:
            a, b = distance(o, e), distance(p, e)
            say(f"  {tuple(o.shape)} {o.dtype}: {a / float(e.norm()):.6f}, plain "
                f"{b / float(e.norm()):.6f}")
            assert a <= 1.01 * b
