"""RMS norm over many rows (1024 and more, where a row takes fewer threads)
and at the edges of its 8-bit scales: every row, scale and code against the
64-bit form, with residuals of both types, in place too."""
import pytest
import torch

import nvfp4_block_scaled_gemv_amd as nv
from decode_ref import E2M1, rmsnorm
from gpu_util import DEV, say
from test_gpu_norm import BF16, EPS, F32, F32_STEPS

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M", [1, 1025])
@pytest.mark.parametrize("H,group", [(64, 32), (192, 64), (256, 128), (4096, 32)])
def test_e4m3_values_too_small_for_a_scale(M, H, group):
    """A group whose largest |y| is so small that a 448th of it is zero in fp32
    has the scale 1 and zeros, not 0 / 0."""
    say(f"[norm e4m3 tiny] M={M} H={H} group={group}")
    x = torch.zeros(M, H, device=DEV)
    x[:, ::2] = 1.0
    w = torch.zeros(H, dtype=BF16, device=DEV)
    w[group:] = 2.0 ** -133               # the smallest bf16
    w[2 * group:] = 0
    x[:, group + 2:2 * group] = 2.0 ** -13
    x[:, group + 1:2 * group:2] = 0
    x[:, group] = 2.0 ** -13
    y8, sc, _ = nv.add_rmsnorm_e4m3(x, w, EPS, group=group)
    y, _ = rmsnorm(x, w, EPS)
    tiny = y[:, group:2 * group]
    assert 0 < float(tiny.max()) < 448 * 2.0 ** -151
    assert torch.all(sc == 1)             # this group, and those of zeros
    assert torch.all(y8.float() == 0)
