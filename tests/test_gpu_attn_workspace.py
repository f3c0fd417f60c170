"""Attention in exactly the workspace that it demands, with bytes behind it that stay
as they are: two heads of an NVFP4 or E4M3 cache side by side, which are all of its
heads or not, and fewer and more sequences than half of the runs; and plain attention
in what it needed by itself."""
import pytest
import torch

import nvfp4_block_scaled_gemv_amd as nv
import test_gpu_attn_nvfp4 as four
import test_gpu_attn_scored as scored
from decode_ref import gen
from gpu_util import DEV, say
from serving_ref import build4, place4, slopes_of
from test_abi_attn_workspace import plain
from test_gpu_paged_attn import BF16, E4M3, build, check as check_plain, scales

pytestmark = pytest.mark.gpu
GUARD = 1 << 16


def guarded(n):
    raw = torch.full((n + GUARD,), 0x5A, dtype=torch.uint8, device=DEV)
    return raw, raw[:n]


def lengths(B, longest, seed):
    """Of all kinds, zero and one among them."""
    x = torch.randint(0, longest + 1, (B,), generator=gen(seed)).tolist()
    x[0], x[B // 2], x[-1] = longest, 0, 1
    return x


def widened(table, Hkv, page, keys):
    width = keys // (Hkv * table.shape[0] * page) + 1
    more = torch.full((table.shape[0], max(0, width - table.shape[1])), -1, dtype=torch.int32)
    return torch.cat([table, more], 1)


# sequences, longest, new tokens, query heads a key-value head, its heads, D, page
CASES4 = [
    (3, 9000, 1, 4, 2, 128, 16), (70, 700, 2, 3, 2, 64, 20), (3, 9000, 1, 4, 4, 128, 64),
    (1000, 330, 1, 1, 2, 64, 16), (1024, 330, 1, 2, 2, 64, 16), (1025, 330, 1, 2, 2, 128, 16),
    (500, 200, 1, 1, 2, 256, 16), (513, 200, 1, 4, 2, 256, 20), (2100, 300, 1, 1, 2, 64, 64),
    (5, 3000, 5, 4, 8, 128, 64),
]


@pytest.mark.parametrize("B,longest,Q,G,Hkv,D,page", CASES4)
def test_nvfp4(B, longest, Q, G, Hkv, D, page):
    say(f"[workspace] nvfp4 B={B} longest={longest} Q={Q} G={G} Hkv={Hkv} D={D} page={page}")
    q, table, ln, parts = build4(lengths(B, longest, B), Q, G * Hkv, Hkv, D, page, seed=B + D)
    table = widened(table, Hkv, page, 1 << 18)
    cache = place4(parts, "nhd", DEV)
    raw, ws = guarded(nv.paged_attention_workspace_bytes(B, Q, G * Hkv, Hkv, D))
    got = four.run(q, cache, table, ln, workspace=ws)
    four.check(got, q, parts, table, ln)
    assert torch.all(raw[-GUARD:] == 0x5A)
    assert torch.equal(got, four.run(q, cache, table, ln, workspace=ws))   # whatever it held
    big = torch.zeros(2 * ws.numel(), dtype=torch.uint8, device=DEV)
    assert torch.equal(got, four.run(q, cache, table, ln, workspace=big))


@pytest.mark.parametrize("B,longest,Q,G,Hkv,page", [
    (3, 9000, 1, 4, 2, 16), (40, 900, 2, 3, 2, 20), (3, 9000, 1, 1, 6, 16),
    (1024, 520, 1, 1, 2, 16), (1030, 520, 1, 2, 2, 20)])
def test_e4m3_scored(B, longest, Q, G, Hkv, page):
    say(f"[workspace] e4m3 B={B} longest={longest} Q={Q} G={G} Hkv={Hkv} page={page}")
    q, k, v, table, ln, kc, vc, ks, vs = build(lengths(B, longest, B), Q, G * Hkv, Hkv, 64, page,
                                               E4M3, seed=B)
    table = widened(table, Hkv, page, 1 << 19)
    slopes = slopes_of(G * Hkv)
    raw, ws = guarded(nv.paged_attention_workspace_bytes(B, Q, G * Hkv, Hkv, 64))
    got = scored.run(q, table, ln, kc, vc, ks, vs, E4M3, slopes, softcap=9.0, workspace=ws)
    scored.check(got, q, k, v, table, ln, 0.125, 0, ks, vs, 9.0, slopes)
    assert torch.all(raw[-GUARD:] == 0x5A)
    assert torch.equal(got, scored.run(q, table, ln, kc, vc, ks, vs, E4M3, slopes, softcap=9.0,
                                       workspace=ws))


@pytest.mark.parametrize("ct", [BF16, E4M3])
@pytest.mark.parametrize("Q,G,Hkv,D,page", [(1, 4, 8, 128, 16), (5, 4, 8, 128, 16),
                                            (2, 2, 2, 64, 20), (5, 4, 2, 256, 16),
                                            (3, 7, 3, 256, 20)])
def test_plain(ct, Q, G, Hkv, D, page):
    q, k, v, table, ln, kc, vc, ks, vs = build([5000, 17, 900, 0], Q, G * Hkv, Hkv, D, page, ct,
                                               seed=D)
    raw, ws = guarded(plain(G * Q, Hkv, D))
    a, b = scales(ct, ks, vs)
    args = (q.to(DEV), kc, vc, table.to(DEV), ln.to(DEV))
    got = nv.paged_attention(*args, k_scale=a, v_scale=b, workspace=ws)
    torch.cuda.synchronize()
    check_plain(got.cpu().double(), q, k, v, table, ln, D ** -0.5, 0, ks, vs)
    assert torch.all(raw[-GUARD:] == 0x5A)
    assert torch.equal(got, nv.paged_attention(*args, k_scale=a, v_scale=b))
