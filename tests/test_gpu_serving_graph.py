"""The NVFP4 cache's operators, scored attention and the adapters captured into
HIP graphs, on several streams at once and with shared workspaces: every replay,
with eager work and synchronisations between them and the outputs poisoned
before each, gives the eager result bit for bit; a captured call follows the
lengths, adapters and ranks on the device; wrong tensors are refused."""
import pytest
import torch

import nvfp4_block_scaled_gemv_amd as nv
from decode_ref import gen, inv_freq, normal
from gpu_util import DEV
from serving_ref import adapters, build4, place4, slopes_of
from test_gpu_attn_nvfp4 import check as check4
from test_gpu_graph import check_graph
from test_gpu_paged_attn import build

pytestmark = pytest.mark.gpu

BF16, E4M3 = torch.bfloat16, torch.float8_e4m3fn


def append_case(T, seed):
    g = gen(seed)
    q, k, v = (normal(g, T, h, 128).to(DEV) for h in (8, 2, 2))
    pos, slots = torch.arange(T, device=DEV) + 1000, torch.randperm(T + 5, generator=g)[:T].to(DEV)
    f = inv_freq(128).to(DEV)
    nb = (T + 5 + 15) // 16
    codes = torch.zeros(2, nb, 16, 2, 64, dtype=torch.uint8, device=DEV)
    scales = torch.zeros(2, nb, 16, 2, 8, dtype=torch.uint8, device=DEV)
    gs = torch.full((1,), 4.5 / 2688, device=DEV)
    out = torch.empty(T, 8, 128, dtype=BF16, device=DEV)

    def run():
        # the whole cache is compared: places without a token are cleared too
        codes.zero_()
        scales.zero_()
        nv.rope_append_nvfp4_into(q, k, v, pos, slots, f, out, (codes[0], scales[0], gs),
                                  (codes[1], scales[1], gs))
    return run, [out, codes, scales]


@pytest.mark.parametrize("T", [1, 7, 300])
def test_graph_append(T):
    run, outs = append_case(T, T)
    check_graph(f"append nvfp4 {T}", run, outs, append_case(T, T + 1)[0])


def attn_case(lens, Q, page, seed, width=None, cap=0.0, bias=False):
    q, table, ln, parts = build4(lens, Q, 8, 2, 128, page, seed=seed)
    if width:
        table = torch.cat([table, torch.full((len(lens), width - table.shape[1]), -1,
                                             dtype=torch.int32)], 1)
    cache = place4(parts, "nhd", DEV)
    dq, dt, dl = q.to(DEV), table.contiguous().to(DEV), ln.to(DEV)
    slopes = slopes_of(8).to(DEV) if bias else None
    out = torch.empty_like(dq)
    ws = torch.empty(nv.paged_attention_workspace_bytes(len(lens), Q, 8, 2, 128),
                     dtype=torch.uint8, device=DEV)

    def run(ws=ws):
        nv.paged_attention_nvfp4_into(dq, *cache, dt, dl, out, ws, softcap=cap, slopes=slopes)
    return run, out, dl, ws, (q, table, parts)


@pytest.mark.parametrize("lens,Q,page,width,cap,bias", [([300], 1, 16, None, 0.0, False),
                                                        ([300, 9, 1200], 2, 16, 100, 20.0, False),
                                                        ([5000, 1], 1, 5, None, 0.0, True),
                                                        ([5000, 1], 1, 16, 10000, 0.0, False)])
def test_graph_attention(lens, Q, page, width, cap, bias):
    run, out, _, _, _ = attn_case(lens, Q, page, 1, width, cap, bias)
    check_graph(f"attention nvfp4 {lens}", run, [out],
                attn_case(lens, Q, page, 2, width, cap, bias)[0])


def scored_case(ct, seed):
    q, k, v, table, ln, kc, vc, ks, vs = build([900, 33], 2, 8, 2, 128, 16, ct, seed=seed)
    dq, dt, dl, sl = q.to(DEV), table.to(DEV), ln.to(DEV), slopes_of(8).to(DEV)
    out = torch.empty_like(dq)
    ws = torch.empty(nv.paged_attention_workspace_bytes(2, 2, 8, 2, 128), dtype=torch.uint8,
                     device=DEV)
    sc = [torch.full((1,), s, device=DEV) if ct is E4M3 else None for s in (ks, vs)]

    def run():
        nv.paged_attention_scored_into(dq, kc, vc, dt, dl, out, ws, softcap=15.0, slopes=sl,
                                       k_scale=sc[0], v_scale=sc[1])
    return run, out


@pytest.mark.parametrize("ct", [BF16, E4M3])
def test_graph_scored(ct):
    run, out = scored_case(ct, 1)
    check_graph(f"scored {ct}", run, [out], scored_case(ct, 2)[0])


def lora_case(M, rank, seed, in_place=False):
    g = gen(seed)
    E, K, Ns = 6, 1024, (700, 64)
    mats = [(normal(g, E, rank, K, std=K ** -0.5, dtype=BF16), normal(g, E, n, rank, dtype=BF16))
            for n in Ns]
    x, base = normal(g, M, K, dtype=BF16), [normal(g, M, n) for n in Ns]
    ids = torch.randint(-1, E, (M,), generator=g, dtype=torch.int32)
    dm, dx, di = [(a.to(DEV), b.to(DEV)) for a, b in mats], x.to(DEV), ids.to(DEV)
    db, alpha = [b.to(DEV) for b in base], torch.ones(E, device=DEV)
    ranks = torch.full((E,), rank, dtype=torch.int32, device=DEV)
    ys = [torch.empty(M, n, device=DEV) for n in Ns]
    ws = torch.empty(nv.lora_workspace_bytes(M, K, rank, 2), dtype=torch.uint8, device=DEV)

    def run(ws=ws):
        if in_place:
            for y, b in zip(ys, db):
                y.copy_(b)
        nv.lora_segments_into(dm, dx, di, ys, ws, ys if in_place else db, alpha, ranks)
    return run, ys, (di, alpha, ranks), ws, (mats, x, base)


@pytest.mark.parametrize("M,rank,in_place", [(1, 16, False), (5, 64, True), (128, 16, True),
                                             (128, 8, False)])
def test_graph_lora(M, rank, in_place):
    run, ys, _, _, _ = lora_case(M, rank, 1, in_place)
    check_graph(f"lora {M} {rank}", run, ys, lora_case(M, rank, 2, in_place)[0])


@pytest.mark.parametrize("width", [None, 20000])
def test_captured_attention_follows_the_lengths(width):
    run, out, dl, _, (q, table, parts) = attn_case([2000, 700], 1, 16, 3, width)
    run()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        run()
    for lens in ([2000, 700], [1, 1], [0, 33], [1999, 512], [64, 700]):
        dl.copy_(torch.tensor(lens, dtype=torch.int32))
        out.fill_(float("nan"))
        g.replay()
        torch.cuda.synchronize()
        got = out.clone()
        run()
        torch.cuda.synchronize()
        assert torch.equal(got, out)
        check4(got.cpu().double(), q, parts, table, torch.tensor(lens, dtype=torch.int32))


@pytest.mark.parametrize("M,rank", [(3, 16), (60, 32)])
def test_captured_adapters_follow_ids_and_ranks(M, rank):
    run, ys, (di, alpha, ranks), _, (mats, x, base) = lora_case(M, rank, 4)
    run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    g = gen(40)
    for _ in range(4):
        ids = torch.randint(-2, 8, (M,), generator=g, dtype=torch.int32)
        al, rk = normal(g, 6), torch.randint(0, rank + 1, (6,), generator=g, dtype=torch.int32)
        di.copy_(ids), alpha.copy_(al), ranks.copy_(rk)
        for y in ys:
            y.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        for y, (ref, tol) in zip(ys, adapters(mats, x, ids, base, al, rk)):
            assert torch.all((y.cpu().double() - ref).abs() <= tol)


def test_two_graphs_share_a_workspace():
    run1, out1, _, ws, _ = attn_case([4000, 100], 1, 16, 4)
    run2, out2, _, _, _ = attn_case([100, 3000], 1, 16, 5)
    lora1, ys1, _, lws, _ = lora_case(100, 32, 6)
    lora2, ys2, _, _, _ = lora_case(100, 32, 7)
    run1(), run2(ws), lora1(), lora2(lws)
    torch.cuda.synchronize()
    outs = [out1, out2, *ys1, *ys2]
    ref = [o.clone() for o in outs]
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    with torch.cuda.graph(graphs[0]):
        run1()
        lora1()
    with torch.cuda.graph(graphs[1]):
        run2(ws)
        lora2(lws)
    for _ in range(3):
        for o in (*outs, ws, lws):
            o.fill_(0x7F)
        graphs[0].replay()
        graphs[1].replay()
        graphs[0].replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, ref))


def test_on_two_streams_at_once():
    cases = []
    for seed in (1, 2):
        p, po = append_case(30, seed)
        t, to, _, _, _ = attn_case([3000, 50], 2, 16, seed)
        s, so = scored_case(E4M3, seed)
        f, fo, _, _, _ = lora_case(90, 16, seed)
        cases.append(((p, t, s, f), [*po, to, so, *fo]))
    ref = []
    for runs, outs in cases:
        for r in runs:
            r()
        torch.cuda.synchronize()
        ref.append([o.clone() for o in outs])
        for o in outs:
            o.zero_()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(20):
        for s, (runs, _) in zip(streams, cases):
            with torch.cuda.stream(s):
                for r in runs:
                    r()
    torch.cuda.synchronize()
    for (_, outs), want in zip(cases, ref):
        assert all(torch.equal(a, b) for a, b in zip(outs, want))


def test_another_current_device_is_refused(monkeypatch):
    runs = [append_case(2, 1)[0], attn_case([5], 1, 16, 1)[0], scored_case(BF16, 1)[0],
            lora_case(2, 8, 1)[0]]
    monkeypatch.setattr(nv, "_current_device", lambda: 1)
    for run in runs:
        with pytest.raises(ValueError, match="current"):
            run()


def test_bindings_refuse_wrong_tensors():
    q, table, ln, parts = build4([40], 1, 4, 2, 64, 16)
    k, v = place4(parts, "nhd", DEV)
    dq, dt, dl = q.to(DEV), table.to(DEV), ln.to(DEV)

    def attn(k=k, v=v, q=dq, t=dt, n=dl, **kw):
        return nv.paged_attention_nvfp4(q, k, v, t, n, **kw)
    attn()
    for bad in (dict(q=dq.float()), dict(t=dt.long()), dict(n=dl.float())):
        with pytest.raises(TypeError):
            attn(**bad)
    for bad in (dict(q=dq[:, :, :32].contiguous()), dict(n=torch.ones(2, dtype=torch.int32, device=DEV)),
                dict(k=(k[0].cpu(), k[1], k[2])), dict(slopes=torch.ones(3, device=DEV)),
                dict(slopes=torch.ones(4))):
        with pytest.raises(ValueError):
            attn(**bad)
    with pytest.raises(nv.Nvfp4Error):
        attn(softcap=-1.0)
    with pytest.raises(nv.Nvfp4Error):
        attn(softcap=float("nan"))
    one, f = torch.zeros(2, dtype=torch.int64, device=DEV), inv_freq(64).to(DEV)
    x = torch.zeros(2, 2, 64, device=DEV)
    o = torch.empty(2, 2, 64, dtype=BF16, device=DEV)
    nv.rope_append_nvfp4_into(x, x, x, one, one + torch.arange(2, device=DEV), f, o, k, v)
    for bad in (dict(k=x.half()), dict(slots=one.int()), dict(k=x[:, :1]), dict(o=o.float())):
        a = dict(q=x, k=x, v=x, slots=one, o=o) | bad
        with pytest.raises((TypeError, ValueError)):
            nv.rope_append_nvfp4_into(a["q"], a["k"], a["v"], one, a["slots"], f, a["o"], k, v)
    with pytest.raises(ValueError):
        nv.rope_append_nvfp4_into(x, None, None, one, one, f, None, k, v)
    A = torch.zeros(3, 8, 64, dtype=BF16, device=DEV)
    B = torch.zeros(3, 5, 8, dtype=BF16, device=DEV)
    xx, ids = torch.zeros(2, 64, dtype=BF16, device=DEV), torch.zeros(2, dtype=torch.int32, device=DEV)
    nv.lora_segments([(A, B)], xx, ids)
    for bad in (dict(A=A.float()), dict(x=xx.float()), dict(ids=ids.long())):
        a = dict(A=A, B=B, x=xx, ids=ids) | bad
        with pytest.raises(TypeError):
            nv.lora_segments([(a["A"], a["B"])], a["x"], a["ids"])
    for bad in (dict(A=A[:2]), dict(B=B[:, :, :4].contiguous()), dict(ids=ids[:1]),
                dict(A=A.transpose(1, 2)), dict(x=xx.t().contiguous().t())):
        a = dict(A=A, B=B, x=xx, ids=ids) | bad
        with pytest.raises(ValueError):
            nv.lora_segments([(a["A"], a["B"])], a["x"], a["ids"])
    with pytest.raises(ValueError):
        nv.lora_segments([(A, B)], xx, ids, bases=[torch.zeros(2, 4, device=DEV)])
    with pytest.raises(ValueError):
        nv.lora_segments([(A, B)], xx, ids, alpha=torch.zeros(2, device=DEV))
    with pytest.raises(nv.Nvfp4Error):                       # ranks are multiples of 8
        nv.lora_segments([(A[:, :4].contiguous(), B[:, :, :4].contiguous())], xx, ids)
