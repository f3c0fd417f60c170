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


def descriptor(k, v):
    c = nv._kv_cache(k, v, None, None)
    return (c.num_blocks, c.page, c.n_kv_heads, c.D, c.stride_block, c.stride_token, c.stride_head)


def test_strides_of_dimensions_of_one_say_nothing():
    """k and v that lie in memory alike fit, whatever strides torch notes for a
    dimension of one: one head in both orders of heads and tokens, one token a
    page, one page of a larger buffer."""
    nhd = torch.zeros(4, 16, 1, 64, dtype=BF16)
    hnd = torch.zeros(4, 1, 16, 64, dtype=BF16).transpose(1, 2)
    assert nhd.stride() != hnd.stride()
    assert descriptor(nhd, hnd) == descriptor(nhd, nhd) == (4, 16, 1, 64, 1024, 64, 64)
    a = torch.zeros(4, 1, 2, 64, dtype=BF16)
    b = torch.zeros(4, 2, 1, 64, dtype=BF16).transpose(1, 2)
    assert a.stride() != b.stride()
    assert descriptor(a, b) == descriptor(a, a)
    c = torch.zeros(1, 16, 2, 64, dtype=BF16)
    d = torch.zeros(1, 2, 16, 2, 64, dtype=BF16)[:, 1]
    assert c.stride() != d.stride()
    assert descriptor(c, d) == descriptor(c, c)
    # strides that do say something still have to be the same
    for x, y in ((torch.zeros(4, 16, 2, 64), torch.zeros(4, 2, 16, 64).transpose(1, 2)),
                 (torch.zeros(4, 16, 2, 64), torch.zeros(4, 16, 2, 96)[..., :64]),
                 (torch.zeros(4, 16, 2, 64), torch.zeros(4, 16, 2, 128)[..., ::2])):
        with pytest.raises(ValueError, match="strides"):
            nv._kv_cache(x.to(BF16), y.to(BF16) if y.is_contiguous() else
                         torch.empty_strided(y.shape, y.stride(), dtype=BF16), None, None)
