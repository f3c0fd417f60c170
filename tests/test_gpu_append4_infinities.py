"""An infinite element in a block of either tensor scale, appended to an NVFP4 cache:
the block's scale is the largest, and every code is the oracle's of the block with
that element at the end of the range."""
import pytest
import torch

import nvfp4_block_scaled_gemv_amd as nv
from decode_ref import gen, normal
from gpu_util import DEV
from serving_ref import encode4
from test_gpu_rope_nvfp4 import GK, GV, fresh

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("at,sign", [(3, 1.0), (20, -1.0), (63, 1.0)])
def test_codes_beside_an_infinity(at, sign):
    D = 64
    x = normal(gen(4), 1, 1, D)
    x[0, 0, at] = sign * float("inf")
    got = fresh("nhd", 1, 1, 1, D)
    z = torch.zeros(1, dtype=torch.int64, device=DEV)
    nv.rope_append_nvfp4(None, x.to(DEV), x.to(DEV), z, z, torch.empty(0, device=DEV), *got)
    torch.cuda.synchronize()
    for (c, s, _), g in zip(got, (GK, GV)):
        y = x[0, 0].clone()
        y[at] = sign * 6 * 448 * g
        block = slice(at // 16 * 16, at // 16 * 16 + 16)
        # the largest of the block decides its scale: 448, as 6 * 448 * g gives it
        y[block] = y[block].clamp(-6 * 448 * g, 6 * 448 * g)
        codes, scales = encode4(y[None], g)
        scales[0, at // 16] = 0x7E
        assert torch.equal(c.cpu().flatten(), codes[0]), g
        assert torch.equal(s.cpu().flatten(), scales[0]), g
