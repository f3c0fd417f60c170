"""Attention in exactly the workspace that it demands, with bytes behind it that stay
as they are: two heads of an NVFP4 or E4M3 cache side by side, which are all of its
heads or not, and fewer and more sequences than half of the runs; and plain attention
in what it needed by itself."""
import re

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


def demanded(call):
    """The bytes that a call asks for when it gets too few."""
    with pytest.raises(nv.Nvfp4Error) as e:
        call(torch.empty(16, dtype=torch.uint8, device=DEV))
    assert e.value.status == 5
    return int(re.search(r"needs (\d+) bytes", str(e.value))[1])


@pytest.mark.parametrize("kind", ["bf16", "e4m3", "bf16 scored", "e4m3 scored", "nvfp4"])
@pytest.mark.parametrize("Q,G,Hkv,D,page", [(1, 4, 8, 128, 16), (1, 1, 16, 64, 20),
                                            (1, 3, 2, 64, 16), (5, 4, 8, 128, 16),
                                            (5, 4, 2, 256, 16), (3, 7, 3, 256, 20),
                                            (20, 4, 1, 64, 64)])
def test_what_a_call_demands_is_all_it_writes(kind, Q, G, Hkv, D, page):
    """Exactly that many bytes, the ones behind them untouched, the same result as with
    many more."""
    lens = [6000, 17, 900, 0, 1]
    g = gen(D + Q)
    if kind == "nvfp4":
        q, table, ln, parts = build4(lens, Q, G * Hkv, Hkv, D, page, seed=D)
        cache = place4(parts, "nhd", DEV)
    else:
        q, _, _, table, ln, kc, vc, ks, vs = build(lens, Q, G * Hkv, Hkv, D, page,
                                                   E4M3 if "e4m3" in kind else BF16, seed=D)
        a, b = scales(kc.dtype, ks, vs)
    table = widened(table, Hkv, page, 1 << 19)
    args = (q.to(DEV), table.to(DEV), ln.to(DEV))
    slopes = torch.rand(G * Hkv, generator=g).to(DEV)

    def call(ws):
        if kind == "nvfp4":
            return nv.paged_attention_nvfp4(args[0], *cache, *args[1:], workspace=ws)
        if "scored" in kind:
            return nv.paged_attention_scored(args[0], kc, vc, *args[1:], softcap=20.0,
                                             slopes=slopes, k_scale=a, v_scale=b, workspace=ws)
        return nv.paged_attention(args[0], kc, vc, *args[1:], k_scale=a, v_scale=b, workspace=ws)
    need = demanded(call)
    most = nv.paged_attention_workspace_bytes(len(lens), Q, G * Hkv, Hkv, D)
    assert need <= most
    raw, ws = guarded(need)
    got = call(ws)
    torch.cuda.synchronize()
    assert torch.all(raw[-GUARD:] == 0x5A)
    assert torch.equal(got, call(torch.zeros(2 * most, dtype=torch.uint8, device=DEV)))
    assert torch.isfinite(got.float()).all()


def test_one_pair_of_heads_captured():
    """A captured call over one pair of heads follows the lengths, its records counted by
    sequences, with other work between the replays."""
    q, table, ln, parts = build4([9000, 4000, 70, 3, 600], 1, 8, 2, 128, 16, seed=51)
    table = widened(table, 2, 16, 1 << 18)
    cache = place4(parts, "nhd", DEV)
    dq, dt, dl = q.to(DEV), table.to(DEV), ln.to(DEV)
    raw, ws = guarded(nv.paged_attention_workspace_bytes(5, 1, 8, 2, 128))
    out = torch.empty_like(dq)
    nv.paged_attention_nvfp4_into(dq, *cache, dt, dl, out, ws)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        nv.paged_attention_nvfp4_into(dq, *cache, dt, dl, out, ws)
    for lens in ([9000, 4000, 70, 3, 600], [1, 0, 33, 3, 5], [9000, 1, 0, 0, 0],
                 [100, 4000, 70, 2, 599], [8999, 3999, 69, 1, 1]):
        dl.copy_(torch.tensor(lens, dtype=torch.int32))
        g.replay()
        torch.cuda.synchronize()
        want = nv.paged_attention_nvfp4(dq, *cache, dt, dl)
        assert torch.equal(out, want), lens
        four.check(out.cpu().double(), q, parts, table, torch.tensor(lens, dtype=torch.int32))
    assert torch.all(raw[-GUARD:] == 0x5A)
