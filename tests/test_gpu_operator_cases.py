"""The measured cases of perf/operators.py and a few drawn ones: the library's
outputs are no further from the 64-bit definition than the plain 32-bit form's,
and equal where they are whole numbers."""
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
                                                  os.path.join(ROOT, "perf", "operators.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def cases():
    m = load()
    out = m.listed()
    rng = random.Random(7)
    for i in range(12):
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
    """Both forms compute in 32 bits and round once to the output's type, so
    their distances to the exact outputs are the roundings'. With a rounding's
    rms r and 32-bit errors of rms e before it, the distance is sqrt(r^2 + e^2)
    and a few values rounded the other way; e is below r / 8 for every type of 16
    bits or fewer at these sizes (the sums' errors, 2^-24 of the terms' sizes
    times the square root of their number over 2^-9 of the output), so the two
    forms' distances are within 1 % of each other. Outputs of 32 bits (scales,
    a residual) have to be within 2^-18 of the exact ones."""
    say(f"[cases] {case}")
    m = load()
    plain = as_list(m.run(m.prepare(case, 3)))
    m.own = True
    own = as_list(m.run(m.prepare(case, 3)))       # its own buffers, not the plain form's
    exact = m.exact(case, 3)
    exact = [None] * len(own) if exact is None else as_list(exact)
    assert len(own) == len(plain) == len(exact)
    for o, p, e in zip(own, plain, exact):
        assert o.shape == p.shape and o.dtype is p.dtype
        if not o.dtype.is_floating_point:
            assert torch.equal(o, p)
        elif e is None:      # 4-bit values: a border may fall the other way
            assert float((o.float() != p.float()).float().mean()) < 1e-3
        elif o.dtype is torch.float32:
            assert torch.all((o.double() - e).abs() <= e.abs() * 2.0 ** -18 + 1e-30)
        else:
            a, b = distance(o, e), distance(p, e)
            say(f"  {tuple(o.shape)} {o.dtype}: {a / float(e.norm()):.6f}, plain "
                f"{b / float(e.norm()):.6f}")
            assert a <= 1.01 * b
