"""The operators between the GEMVs captured into HIP graphs, on other streams
and with shared workspaces: every replay, with eager work and synchronisations
between them and the outputs poisoned before each, gives the eager result bit
for bit; a captured attention follows the lengths; two graphs that share a
workspace, replayed in turn, do not disturb each other."""
import pytest
import torch

import nvfp4_block_scaled_gemv_amd as nv
from decode_ref import gen, inv_freq, normal, rotate
from gpu_util import DEV, say
from test_gpu_graph import check_graph
from test_gpu_paged_attn import build, check

pytestmark = pytest.mark.gpu

BF16, F32, E4M3 = torch.bfloat16, torch.float32, torch.float8_e4m3fn


def norm_case(M, H, form, seed):
    g = gen(seed)
    x, r = normal(g, M, H).to(DEV), normal(g, M, H, dtype=BF16).to(DEV)
    w = (1 + normal(g, H, std=0.2)).to(BF16).to(DEV)
    ro = torch.empty_like(r)
    if form == "bf16":
        y = torch.empty(M, H, dtype=BF16, device=DEV)
        return lambda: nv.add_rmsnorm_into(x, w, 1e-6, y, r, ro), [y, ro]
    if form == "e4m3":
        y = torch.empty(M, H, dtype=torch.uint8, device=DEV)
        s = torch.empty(M, H // 64, device=DEV)
        return (lambda: nv.add_rmsnorm_e4m3_into(x, w, 1e-6, y.view(E4M3), s, r, ro)), [y, s, ro]
    c = torch.empty(M, H // 2, dtype=torch.uint8, device=DEV)
    s = torch.empty(M, H // 16, dtype=torch.uint8, device=DEV)
    gs = torch.full((1,), 0.002, device=DEV)
    return lambda: nv.add_rmsnorm_nvfp4_into(x, w, 1e-6, gs, c, s, r, ro), [c, s, ro]


@pytest.mark.parametrize("form", ["bf16", "e4m3", "nvfp4"])
@pytest.mark.parametrize("M,H", [(1, 4096), (5, 128), (33, 2048)])
def test_graph_norm(form, M, H):
    run, outs = norm_case(M, H, form, M + H)
    other, _ = norm_case(M, H, form, M + H + 1)
    check_graph(f"norm {form} {M} {H}", run, outs, other)


def append_case(T, ct, seed):
    g = gen(seed)
    q, k, v = (normal(g, T, h, 128).to(DEV) for h in (8, 2, 2))
    pos, slots = torch.arange(T, device=DEV) + 1000, torch.randperm(T + 5, generator=g)[:T].to(DEV)
    f = inv_freq(128).to(DEV)
    nb = (T + 5 + 15) // 16
    kc, vc = (torch.zeros(nb, 16, 2, 128, device=DEV).to(ct) for _ in range(2))
    sc = torch.full((1,), 0.02, device=DEV) if ct is E4M3 else None
    out = torch.empty(T, 8, 128, dtype=BF16, device=DEV)

    def run():
        # the whole cache is compared: places without a token are cleared too
        kc.view(torch.uint8).zero_()
        vc.view(torch.uint8).zero_()
        nv.rope_append_into(q, k, v, pos, slots, f, out, kc, vc, sc, sc)
    return run, [out, kc.view(torch.uint8), vc.view(torch.uint8)]


@pytest.mark.parametrize("ct", [BF16, E4M3])
@pytest.mark.parametrize("T", [1, 7, 200])
def test_graph_append(T, ct):
    run, outs = append_case(T, ct, T)
    other, _ = append_case(T, ct, T + 1)
    check_graph(f"append {T} {ct}", run, outs, other)


def attn_case(lens, Q, page, ct, seed, width=None):
    q, k, v, table, ln, kc, vc, ks, vs = build(lens, Q, 8, 2, 128, page, ct, seed=seed)
    if width:                # a wider table: the form for long sequences
        table = torch.cat([table, torch.full((len(lens), width - table.shape[1]), -1,
                                             dtype=torch.int32)], 1)
    dq, dt, dl = q.to(DEV), table.contiguous().to(DEV), ln.to(DEV)
    out = torch.empty_like(dq)
    n = nv.paged_attention_workspace_bytes(len(lens), Q, 8, 2, 128)
    ws = torch.empty(n, dtype=torch.uint8, device=DEV)
    sc = [torch.full((1,), s, device=DEV) if ct is E4M3 else None for s in (ks, vs)]

    def run(ws=ws):
        nv.paged_attention_into(dq, kc, vc, dt, dl, out, ws, k_scale=sc[0], v_scale=sc[1])
    return run, out, dl, ws, (q, k, v, table, ks, vs)


@pytest.mark.parametrize("lens,Q,page,ct,width", [([300], 1, 16, BF16, None),
                                                  ([300, 9, 1200], 2, 16, E4M3, 100),
                                                  ([5000, 1], 1, 5, BF16, None)])
def test_graph_attention(lens, Q, page, ct, width):
    run, out, _, _, _ = attn_case(lens, Q, page, ct, 1, width)
    other, _, _, _, _ = attn_case(lens, Q, page, ct, 2, width)
    check_graph(f"attention {lens}", run, [out], other)


def test_captured_attention_follows_the_lengths():
    run, out, dl, _, (q, k, v, table, ks, vs) = attn_case([2000, 700], 1, 16, BF16, 3)
    run()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        run()
    for lens in ([2000, 700], [1, 1], [0, 33], [1999, 512], [64, 2000]):
        say(f"[graph] lengths {lens}")
        dl.copy_(torch.tensor(lens, dtype=torch.int32))
        out.fill_(float("nan"))
        g.replay()
        torch.cuda.synchronize()
        got = out.clone()
        run()
        torch.cuda.synchronize()
        assert torch.equal(got, out)
        # rows past a shorter sequence's table hold its pages still; what lies
        # past its length is not seen
        lens2 = [min(n, m) for n, m in zip(lens, (2000, 700))]
        dl.copy_(torch.tensor(lens2, dtype=torch.int32))
        run()
        torch.cuda.synchronize()
        check(out.cpu().double(), q, k, v, table, torch.tensor(lens2), 128 ** -0.5, 0, ks, vs)


def test_two_graphs_share_a_workspace():
    run1, out1, _, ws, _ = attn_case([4000, 100], 1, 16, BF16, 4)
    run2, out2, _, _, _ = attn_case([100, 3000], 1, 16, BF16, 5)
    run1(), run2(ws)
    torch.cuda.synchronize()
    ref1, ref2 = out1.clone(), out2.clone()
    g1, g2 = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g1):
        run1()
    with torch.cuda.graph(g2):
        run2(ws)
    for _ in range(3):
        out1.zero_(), out2.zero_(), ws.fill_(0x7F)
        g1.replay()
        g2.replay()
        g1.replay()
        torch.cuda.synchronize()
        assert torch.equal(out1, ref1) and torch.equal(out2, ref2)


def verify_case(B, Q, V, seed):
    g = gen(seed)
    p = torch.softmax(normal(g, B, Q + 1, V, std=2.0), -1).to(DEV)
    q = torch.softmax(normal(g, B, Q, V, std=2.0), -1).to(DEV)
    d = torch.randint(0, V, (B, Q), generator=g, dtype=torch.int32).to(DEV)
    ua, us = torch.rand(B, Q, generator=g).to(DEV) * 0.5, torch.rand(B, generator=g).to(DEV)
    tok = torch.empty(B, Q + 1, dtype=torch.int32, device=DEV)
    acc = torch.empty(B, dtype=torch.int32, device=DEV)
    ws = torch.empty(nv.verify_draft_workspace_bytes(B, V), dtype=torch.uint8, device=DEV)
    return lambda: nv.verify_draft_into(p, q, d, ua, us, tok, acc, ws), [tok, acc]


@pytest.mark.parametrize("B,Q,V", [(1, 4, 151936), (5, 2, 3001)])
def test_graph_verify(B, Q, V):
    run, outs = verify_case(B, Q, V, 1)
    other, _ = verify_case(B, Q, V, 2)
    check_graph(f"verify {B} {Q} {V}", run, outs, other)


def test_on_other_streams_at_once():
    """Two streams, each its own inputs, outputs and workspaces, many calls in
    flight: the same results as one after the other."""
    cases = []
    for seed in (1, 2):
        n, no = norm_case(3, 4096, "bf16", seed)
        t, to, _, _, _ = attn_case([3000, 50], 2, 16, BF16, seed)
        f, fo = verify_case(3, 3, 50000, seed)
        cases.append(((n, t, f), [*no, to, *fo]))
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
    """The binding launches on the current device: with another one current a
    call is refused before it reaches the library."""
    monkeypatch.setattr(nv, "_current_device", lambda: 1)
    for run in (norm_case(2, 64, "bf16", 1)[0], append_case(2, BF16, 1)[0],
                attn_case([5], 1, 16, BF16, 1)[0], verify_case(1, 1, 10, 1)[0]):
        with pytest.raises(ValueError, match="current"):
            run()


def test_bindings_refuse_wrong_tensors():
    x, w = torch.zeros(2, 64, device=DEV), torch.ones(64, dtype=BF16, device=DEV)
    y = torch.empty(2, 64, dtype=BF16, device=DEV)
    with pytest.raises(ValueError):
        nv.add_rmsnorm_into(x.t().contiguous().t(), w, 1e-6, y)      # not contiguous
    with pytest.raises(TypeError):
        nv.add_rmsnorm_into(x.half(), w, 1e-6, y)
    with pytest.raises(ValueError):
        nv.add_rmsnorm_into(x, w[:32].contiguous(), 1e-6, y)
    with pytest.raises(ValueError):
        nv.add_rmsnorm_into(x, w, 1e-6, y, x.clone())                # no residual_out
    c = torch.zeros(2, 16, 2, 64, dtype=BF16, device=DEV)
    one, f = torch.zeros(2, dtype=torch.int64, device=DEV), inv_freq(64).to(DEV)
    k = torch.zeros(2, 2, 64, device=DEV)
    o = torch.empty(2, 2, 64, dtype=BF16, device=DEV)
    with pytest.raises(ValueError):
        nv.rope_append_into(k, k, k, one, one, f, o, c, c.transpose(1, 2).contiguous())
    with pytest.raises(ValueError):
        nv.rope_append_into(k, k, k, one, one.int(), f, o, c, c.clone())
    with pytest.raises(ValueError):                                   # heads not contiguous
        nv.rope_append_into(torch.zeros(2, 64, 2, device=DEV).transpose(1, 2), k, k, one, one, f,
                            o, c, c.clone())
    with pytest.raises(ValueError):
        nv.rope_append_into(k, k, k, one, one, f, o, c.to(E4M3), c.to(E4M3))   # no scales
    q = torch.zeros(3, 4, 64, dtype=BF16, device=DEV)
    t, ln = torch.zeros(2, 3, dtype=torch.int32, device=DEV), torch.ones(2, dtype=torch.int32,
                                                                         device=DEV)
    with pytest.raises(ValueError):
        nv.paged_attention(q, c, c.clone(), t, ln)                    # 3 tokens, 2 sequences
    with pytest.raises(TypeError):
        nv.paged_attention(q[:2], c, c.clone(), t.long(), ln)
    with pytest.raises(nv.Nvfp4Error) as e:
        nv.paged_attention(q[:2], c, c.clone(), t, ln,
                           workspace=torch.empty(16, dtype=torch.uint8, device=DEV))
    assert e.value.status == 5
    p = torch.ones(1, 3, 9, device=DEV)
    with pytest.raises(ValueError):
        nv.verify_draft(p, p, torch.zeros(1, 2, dtype=torch.int32, device=DEV),
                        torch.zeros(1, 2, device=DEV), torch.zeros(1, device=DEV))
