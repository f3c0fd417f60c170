"""Checks of the Python binding of the decode operators that need no GPU: the
refusals that come before any HIP call, and the cache descriptors."""
import pytest
import torch

import nvfp4_block_scaled_gemv_amd as nv

BF16, E4M3 = torch.bfloat16, torch.float8_e4m3fn


@pytest.mark.parametrize("H,group", [(192, 128), (96, 64), (128, 48), (64, 33), (4096, 16),
                                     (4096, 256), (64, 128), (128, -32), (40, 32)])
def test_e4m3_groups_that_are_none(H, group):
    """A group that is not 32, 64 or 128 dividing H is refused by name. (The
    number of columns of the scales alone does not tell: H // group of these is
    1, 2 or another number that divides H, and stands for another group.)"""
    x, w = torch.zeros(2, H), torch.ones(H, dtype=BF16)
    with pytest.raises(ValueError, match="group"):
        nv.add_rmsnorm_e4m3(x, w, 1e-6, group=group)
