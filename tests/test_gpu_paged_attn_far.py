"""Attention over a paged cache at the far end of the lengths: sequences of up
to 2^31 - 1 keys, whose table names the same few pages over and over, seen
through a window."""
import pytest
import torch

import nvfp4_block_scaled_gemv_amd as nv
from decode_ref import gen, normal
from gpu_util import DEV, say
from test_gpu_paged_attn import BF16, check

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("page", [65536, 100000])
@pytest.mark.parametrize("window,D", [(40, 64), (700, 64), (1, 128), (1500, 128), (90, 256)])
@pytest.mark.parametrize("lens", [[0x7FFFFFFF], [0x7FFFFE01, 5, 0x7FFFFFFF], [0x7FFFFF00, 0x7FFFFFE1]])
def test_windows_at_the_end(page, window, D, lens):
    say(f"[attn far] page={page} window={window} D={D} lens={lens}")
    Q, Hkv, nb = 3, 1, 3
    g = gen(D + window)
    blocks = (1 << 31) // page                        # the row names some 2^31 keys
    k, v = (normal(g, nb, page, Hkv, D, dtype=BF16) for _ in range(2))
    table = torch.arange(blocks, dtype=torch.int32).remainder(nb).repeat(len(lens), 1).contiguous()
    q = normal(g, len(lens) * Q, 4, D, dtype=BF16)
    ln = torch.tensor(lens, dtype=torch.int32)
    got = nv.paged_attention(q.to(DEV), k.to(DEV), v.to(DEV), table.to(DEV), ln.to(DEV),
                             window=window).cpu().double()
    check(got, q, k, v, table, ln, D ** -0.5, window, 1.0, 1.0)
