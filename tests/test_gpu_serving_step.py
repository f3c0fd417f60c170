"""The operators together, as a program uses them that serves requests with
adapters over an NVFP4 cache: prompts, then steps of a batch, through a small
model of two layers (norm, q|k|v GEMV with adapters, rotation and append,
capped or biased attention over 4 bits, o GEMV with adapters, norm, gate|up and
down). Every step's outputs against the same model in 64 bits on the dequantised
weights, which holds a plain cache of its own in NVFP4."""
import pytest
import torch

import nvfp4_block_scaled_gemv_amd as nv
from decode_ref import gen, inv_freq, normal, rmsnorm, rotate
from gpu_util import DEV, say
from serving_ref import attention, decode4, encode4, slopes_of

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16
H, HQ, HKV, D, I, PAGE, EPS, E, RANK, LAYERS = 512, 8, 2, 64, 1024, 16, 1e-6, 4, 16, 2
GK, GV = 8.0 / 2688, 8.0 / 2688


def pack(g, N, K, std):
    c, s, gs = nv.pack(normal(g, N, K, std=std).to(DEV))
    return (c, s, gs), nv.dequant(c, s, gs).cpu().double()


class Model:
    def __init__(self, seed):
        g = gen(seed)
        self.layers = []
        for _ in range(LAYERS):
            layer = {"n1": (1 + normal(g, H, std=0.1)).to(BF16),
                     "n2": (1 + normal(g, H, std=0.1)).to(BF16)}
            for name, n, k in (("q", HQ * D, H), ("k", HKV * D, H), ("v", HKV * D, H),
                               ("o", H, HQ * D), ("gate", I, H), ("up", I, H), ("down", H, I)):
                layer[name] = pack(g, n, k, 0.04)
                if name in "qkvo":
                    layer["lora_" + name] = (normal(g, E, RANK, k, std=k ** -0.5, dtype=BF16),
                                             normal(g, E, n, RANK, std=0.1, dtype=BF16))
            self.layers.append(layer)
        self.alpha = 0.5 + torch.rand(E, generator=g)
        self.ranks = torch.tensor([16, 8, 16, 11], dtype=torch.int32)
        self.freq = inv_freq(D, 10000.0)
        self.slopes = slopes_of(HQ)


def kernel_step(m, x, ids, lens, Q, table, caches, cap):
    B = len(lens)
    T = B * Q
    pos = torch.cat([torch.arange(n - Q, n) for n in lens])
    b = torch.arange(T) // Q
    slots = (table[b, pos // PAGE].long() * PAGE + pos % PAGE).to(DEV)
    pos, dl = pos.to(DEV), torch.tensor(lens, dtype=torch.int32, device=DEV)
    dt, f, ids = table.to(DEV), m.freq.to(DEV), ids.to(DEV)
    extra = dict(alpha=m.alpha.to(DEV), ranks=m.ranks.to(DEV))
    ws = torch.empty(1 << 20, dtype=torch.uint8, device=DEV)
    r, x = x.to(DEV), None
    for layer, cache in zip(m.layers, caches):
        if x is None:
            h, _ = nv.add_rmsnorm(r, layer["n1"].to(DEV), EPS)
        else:
            h, r = nv.add_rmsnorm(x, layer["n1"].to(DEV), EPS, r)
        ys = nv.gemv_segments([layer[n][0] for n in "qkv"], h)
        dev = [tuple(t.to(DEV) for t in layer["lora_" + n]) for n in "qkv"]
        nv.lora_segments_into(dev, h, ids, ys, ws, bases=ys, **extra)          # in place
        q, k, v = ys
        qr = nv.rope_append_nvfp4(q.view(T, HQ, D), k.view(T, HKV, D), v.view(T, HKV, D), pos,
                                  slots, f, *cache)
        a = nv.paged_attention_nvfp4(qr, *cache, dt, dl, softcap=cap,
                                     slopes=None if cap else m.slopes.to(DEV)).view(T, HQ * D)
        o = nv.gemv(*layer["o"][0], a)
        x, = nv.lora_segments([tuple(t.to(DEV) for t in layer["lora_o"])], a, ids, [o], **extra)
        h, r = nv.add_rmsnorm(x, layer["n2"].to(DEV), EPS, r)
        gate, up = nv.gemv_segments([layer["gate"][0], layer["up"][0]], h)
        x = nv.gemv(*layer["down"][0], (torch.nn.functional.silu(gate) * up).to(BF16))
    return x + r.float()


def plain_step(m, x, ids, lens, Q, caches, cap):
    T = len(lens) * Q
    pos = torch.cat([torch.arange(n - Q, n) for n in lens])

    def bf(t):
        return t.to(BF16).double()

    def adapted(y, layer, name, h):
        a, b = layer["lora_" + name]
        y = y.clone()
        for t, e in enumerate(ids.tolist()):
            if 0 <= e < E:
                rk = int(m.ranks[e])
                low = a[e, :rk].double() @ h[t]
                y[t] += float(m.alpha[e]) * (b[e, :, :rk].double() @ low)
        return y

    def kept(t, g):
        return decode4(*encode4(t.float(), g), g)

    r, x = x.double(), None
    for layer, cache in zip(m.layers, caches):
        y, s = rmsnorm(r if x is None else x, layer["n1"], EPS, None if x is None else r)
        h, r = bf(y), bf(s)
        q, k, v = (adapted(h @ layer[n][1].T, layer, n, h) for n in "qkv")
        qr = bf(rotate(q.view(T, HQ, D), pos, m.freq, False))
        k, v = kept(rotate(k.view(T, HKV, D), pos, m.freq, False), GK), kept(v.view(T, HKV, D), GV)
        out = []
        for b, n in enumerate(lens):
            K = torch.cat([cache[b][0], k[b * Q:(b + 1) * Q]])
            W = torch.cat([cache[b][1], v[b * Q:(b + 1) * Q]])
            cache[b] = (K, W)
            out.append(attention(qr[b * Q:(b + 1) * Q], K[None], W[None],
                                 torch.zeros(1, 1, dtype=torch.int32), torch.tensor([n]),
                                 D ** -0.5, 0, cap, None if cap else m.slopes))
        a = bf(torch.cat(out)).view(T, -1)
        x = adapted(a @ layer["o"][1].T, layer, "o", a)
        y, s = rmsnorm(x, layer["n2"], EPS, r)
        h, r = bf(y), bf(s)
        gate, up = h @ layer["gate"][1].T, h @ layer["up"][1].T
        x = bf(gate / (1 + torch.exp(-gate)) * up) @ layer["down"][1].T
    return x + r


@pytest.mark.parametrize("cap", [20.0, 0.0])
def test_prompts_and_steps(cap):
    m = Model(3)
    g = gen(17)
    B, nb = 3, 40
    lens, who = [37, 21, 50], [2, -1, 3]
    perm = torch.randperm(nb, generator=g).to(torch.int32)
    table = perm[:B * 10].view(B, 10).contiguous()
    caches = [tuple((torch.zeros(nb, PAGE, HKV, D // 2, dtype=torch.uint8, device=DEV),
                     torch.zeros(nb, PAGE, HKV, D // 16, dtype=torch.uint8, device=DEV),
                     torch.full((1,), gs, device=DEV)) for gs in (GK, GV)) for _ in range(LAYERS)]
    plain = [[(torch.zeros(0, HKV, D, dtype=torch.float64),) * 2 for _ in range(B)]
             for _ in range(LAYERS)]

    def compare(got, want, what):
        # Two paths that round at the same places differ where a value lies at a
        # border. A bf16 input that rounds the other way moves k and v by up to 2^-8
        # and takes a share of about 2^-8 times E2M1's borders (3 per octave: 1 %) of
        # the cached values to the next step, a third of themselves: 0.33 sqrt(0.01) =
        # 0.03 of k and v in a layer at most, and of a part of the residual stream
        # twice. The outputs agree to 0.05 as a whole.
        rel = float((got.double().cpu() - want).norm() / want.norm())
        say(f"[serving] cap {cap} {what} rel {rel:.4f}")
        assert rel < 0.05, what

    for b in range(B):
        x = normal(g, lens[b], H, dtype=BF16)
        ids = torch.full((lens[b],), who[b], dtype=torch.int32)
        got = kernel_step(m, x, ids, [lens[b]], lens[b], table[b:b + 1], caches, cap)
        sub = [[c[b]] for c in plain]
        want = plain_step(m, x, ids, [lens[b]], lens[b], sub, cap)
        for c, s in zip(plain, sub):
            c[b] = s[0]
        compare(got, want, f"prompt {b}")
    for step, Q in enumerate((1, 3, 1)):
        lens = [n + Q for n in lens]
        x = normal(g, B * Q, H, dtype=BF16)
        ids = torch.tensor(who, dtype=torch.int32).repeat_interleave(Q)
        got = kernel_step(m, x, ids, lens, Q, table, caches, cap)
        want = plain_step(m, x, ids, lens, Q, plain, cap)
        compare(got, want, f"step {step}")
