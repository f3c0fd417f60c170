"""The operators together, as a decode program uses them between the GEMVs: a
prompt, then verification steps of drafted tokens, through a small model of two
layers (norm, q|k|v GEMV, rotation and append, paged attention, o GEMV, norm,
gate|up and down W4A4, head GEMV, verification). Every step's logits against
the same model in 64 bits on the dequantised weights, which holds a plain cache
of its own; the tokens against the plain verification."""
import numpy as np
import pytest
import torch

import nvfp4_block_scaled_gemv_amd as nv
from decode_ref import attention, gen, inv_freq, normal, rmsnorm, rotate, verify
from gpu_util import DEV, say

pytestmark = pytest.mark.gpu

BF16, E4M3 = torch.bfloat16, torch.float8_e4m3fn
H, HQ, HKV, D, I, V, PAGE, EPS = 512, 8, 2, 64, 1024, 5000, 16, 1e-6
LAYERS = 2


def pack(g, N, K, std):
    c, s, gs = nv.pack(normal(g, N, K, std=std).to(DEV))
    return (c, s, gs), nv.dequant(c, s, gs).cpu().double()


class Model:
    def __init__(self, seed, ct):
        g = gen(seed)
        self.ct, self.layers = ct, []
        for _ in range(LAYERS):
            self.layers.append({
                "n1": (1 + normal(g, H, std=0.1)).to(BF16), "n2": (1 + normal(g, H, std=0.1)).to(BF16),
                "q": pack(g, HQ * D, H, 0.05), "k": pack(g, HKV * D, H, 0.05),
                "v": pack(g, HKV * D, H, 0.05), "o": pack(g, H, HQ * D, 0.05),
                "gate": pack(g, I, H, 0.05), "up": pack(g, I, H, 0.05),
                "down": pack(g, H, I, 0.03)})
        self.norm = (1 + normal(g, H, std=0.1)).to(BF16)
        self.head = pack(g, V, H, 0.08)
        self.embed = normal(g, V, H, dtype=BF16)
        self.freq = inv_freq(D, 10000.0)
        self.gx = torch.full((1,), 5.0 / 2688, device=DEV)
        self.ks, self.vs = (0.02, 0.01) if ct is E4M3 else (1.0, 1.0)


def kernel_step(m, tokens, lens, Q, table, caches):
    """tokens [B * Q] at the end of sequences of `lens` keys: logits, residual."""
    B = len(lens)
    T = B * Q
    pos = torch.cat([torch.arange(n - Q, n) for n in lens])
    b = torch.arange(T) // Q
    slots = (table[b, pos // PAGE].long() * PAGE + pos % PAGE).to(DEV)
    pos, dl, dt, f = pos.to(DEV), torch.tensor(lens, dtype=torch.int32, device=DEV), \
        table.to(DEV), m.freq.to(DEV)
    r = m.embed[tokens].to(DEV)
    ks = torch.full((1,), m.ks, device=DEV) if m.ct is E4M3 else None
    vs = torch.full((1,), m.vs, device=DEV) if m.ct is E4M3 else None
    x = None
    for layer, (kc, vc) in zip(m.layers, caches):
        if x is None:
            h, _ = nv.add_rmsnorm(r, layer["n1"].to(DEV), EPS)
        else:
            h, r = nv.add_rmsnorm(x, layer["n1"].to(DEV), EPS, r)
        q, k, v = nv.gemv_segments([layer[n][0] for n in "qkv"], h)
        qr = nv.rope_append(q.view(T, HQ, D), k.view(T, HKV, D), v.view(T, HKV, D), pos, slots, f,
                            kc, vc, ks, vs)
        a = nv.paged_attention(qr, kc, vc, dt, dl, k_scale=ks, v_scale=vs)
        x = nv.gemv(*layer["o"][0], a.view(T, HQ * D))
        c, s, r = nv.add_rmsnorm_nvfp4(x, layer["n2"].to(DEV), EPS, m.gx, r)
        gate, up = nv.gemv_w4a4_segments([layer["gate"][0], layer["up"][0]], c, s, m.gx)
        x = nv.gemv(*layer["down"][0], (torch.nn.functional.silu(gate) * up).to(BF16))
    h, r = nv.add_rmsnorm(x, m.norm.to(DEV), EPS, r)
    return nv.gemv(*m.head[0], h)


def quantized(y, g):
    """The NVFP4 grid of the W4A4 input in 64 bits: block scales to E4M3, values
    to E2M1."""
    T = y.shape[0]
    b = y.view(T, -1, 16)
    s = (b.abs().amax(-1, keepdim=True) / (6 * g)).clamp(max=448).float().to(E4M3).double()
    t = torch.where(s > 0, b / (s * g).clamp(min=1e-300), torch.zeros_like(b))
    grid = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64)
    mag = grid[(t.abs()[..., None] - grid).abs().argmin(-1)]
    return (mag * t.sign() * s * g).view(T, -1)


def plain_step(m, tokens, lens, Q, caches):
    """The same in 64 bits on plain caches (lists of [keys, heads, D] per
    sequence), its activations rounded where the kernels' are."""
    T = len(tokens)
    pos = torch.cat([torch.arange(n - Q, n) for n in lens])
    r = m.embed[tokens].double()

    def bf(x):
        return x.to(BF16).double()

    def kept(x, s):
        return (x / s).clamp(-448, 448).to(m.ct).double() * s

    x = None
    for layer, cache in zip(m.layers, caches):
        y, s = rmsnorm(r if x is None else x, layer["n1"], EPS, None if x is None else r)
        h, r = bf(y), bf(s)
        q, k, v = (h @ layer[n][1].T for n in "qkv")
        qr = bf(rotate(q.view(T, HQ, D), pos, m.freq, False))
        k = kept(rotate(k.view(T, HKV, D), pos, m.freq, False), m.ks)
        v = kept(v.view(T, HKV, D), m.vs)
        out = []
        for b, n in enumerate(lens):
            K, W = cache[b]
            K = torch.cat([K, k[b * Q:(b + 1) * Q]])
            W = torch.cat([W, v[b * Q:(b + 1) * Q]])
            cache[b] = (K, W)
            out.append(attention(qr[b * Q:(b + 1) * Q], K[None], W[None],
                                 torch.zeros(1, 1, dtype=torch.int32), torch.tensor([n]),
                                 D ** -0.5))
        x = bf(torch.cat(out)).view(T, -1) @ layer["o"][1].T
        y, s = rmsnorm(x, layer["n2"], EPS, r)
        r = bf(s)
        h = quantized(y, float(m.gx.cpu()))
        gate, up = h @ layer["gate"][1].T, h @ layer["up"][1].T
        x = bf(gate / (1 + torch.exp(-gate)) * up) @ layer["down"][1].T
    y, _ = rmsnorm(x, m.norm, EPS, r)
    return bf(y) @ m.head[1].T


@pytest.mark.parametrize("ct", [BF16, E4M3])
def test_prompt_and_verification_steps(ct):
    m = Model(3, ct)
    g = gen(17)
    B, Qd, nb = 3, 3, 40
    lens = [37, 21, 50]          # prompts, one call per sequence
    perm = torch.randperm(nb, generator=g).to(torch.int32)
    table = perm[:B * 10].view(B, 10).contiguous()
    caches = [tuple(torch.zeros(nb, PAGE, HKV, D, device=DEV).to(ct) for _ in range(2))
              for _ in range(LAYERS)]
    plain = [[(torch.zeros(0, HKV, D, dtype=torch.float64),) * 2 for _ in range(B)]
             for _ in range(LAYERS)]

    def compare(got, want, what):
        # Two paths of the same model that round at the same places differ where
        # a value lies at a border. A bf16 input that rounds the other way moves
        # the FFN's input by up to 2^-8, and a share of about 2^-8 times E2M1's
        # density of borders (about 3 per octave: 1 %) of its values then takes
        # the next step, a third of itself: 0.33 * sqrt(0.01) = 0.03 of the FFN's
        # input in a layer, half of the residual stream, twice. The logits agree
        # to 0.05 as a whole, not to a bound per element.
        got, want = got.double().cpu(), want
        rel = float((got - want).norm() / want.norm())
        say(f"[decode] {ct} {what} rel {rel:.4f}")
        assert rel < 0.05, what

    last = []
    for b in range(B):
        tok = torch.randint(0, V, (lens[b],), generator=g)
        # a prompt is one sequence with all its tokens new
        logits = kernel_step(m, tok, [lens[b]], lens[b], table[b:b + 1], caches)
        sub = [[c[b]] for c in plain]
        want = plain_step(m, tok, [lens[b]], lens[b], sub)
        for c, s in zip(plain, sub):
            c[b] = s[0]
        compare(logits, want, f"prompt {b}")
        last.append(int(logits[-1].argmax()))

    for step in range(3):
        # the last token and Qd drafts of each sequence, verified at once
        draft = torch.randint(0, V, (B, Qd), generator=g, dtype=torch.int32)
        tok = torch.cat([torch.tensor(last, dtype=torch.int32)[:, None], draft], 1).view(-1).long()
        Q = Qd + 1
        new = [n + Q for n in lens]
        logits = kernel_step(m, tok, new, Q, table, caches)
        want = plain_step(m, tok, new, Q, plain)
        compare(logits, want, f"step {step}")
        p = torch.softmax(logits.view(B, Q, V), -1).contiguous()
        # the drafts' own probabilities: some sure of a likely token, so that
        # drafts are kept as well as refused
        z = logits.view(B, Q, V)[:, :Qd] + normal(g, B, Qd, V, std=0.5).to(DEV)
        q = torch.softmax(z, -1).contiguous()
        ua, us = torch.rand(B, Qd, generator=g), torch.rand(B, generator=g)
        tokens, acc = nv.verify_draft(p, q, draft.to(DEV), ua.to(DEV), us.to(DEV))
        rt, ra, margin = verify(p.cpu(), q.cpu(), draft, ua, us)
        assert margin > 1e-13
        assert np.array_equal(acc.cpu().numpy(), ra) and np.array_equal(tokens.cpu().numpy(), rt)
        # what was not kept is taken back: the next step writes over it
        for b in range(B):
            n = int(ra[b]) + 1
            lens[b] += n
            last[b] = int(rt[b, int(ra[b])])
            for c in plain:
                c[b] = (c[b][0][:lens[b]], c[b][1][:lens[b]])
