"""Operators of a serving step beside those of operators.py: the append of keys
and values to a paged cache in NVFP4 (4 bits), attention over that cache,
attention over a bf16 or e4m3 cache whose scores are capped by a tanh or get a
bias by distance, and low-rank adapters of many requests on the outputs of
projections that share one input.

listed() and draw() give the cases, prepare() a case's inputs, run() one pass
(the plain form in torch, or the library's kernels where `own` is true), work()
what a pass cannot do without and exact() the result in 64 bits.
"""
import math

import torch

own = False

DEV = "cuda"
# static tensor scales of a 4-bit cache: values up to 4.5 in the full range
GK, GV = 4.5 / 2688, 4.2 / 2688


# ------------------------------------------------------------------- cases

def _append(name, T, Hq, Hkv, D, R, page, x, interleaved, far):
    return {"name": name, "op": "append4", "T": T, "Hq": Hq, "Hkv": Hkv, "D": D, "R": R,
            "page": page, "x": x, "interleaved": interleaved, "far": far}


def _attn(name, B, Q, Hq, Hkv, D, page, shortest, longest, cache, window=0, cap=0.0, bias=False):
    return {"name": name, "op": "attn", "B": B, "Q": Q, "Hq": Hq, "Hkv": Hkv, "D": D,
            "page": page, "shortest": shortest, "longest": longest, "cache": cache,
            "window": window, "cap": cap, "bias": bias}


def _lora(name, M, K, outs, E, rank, rows, base=True, mixed=False, idle=False, beside=False):
    return {"name": name, "op": "lora", "M": M, "K": K, "outs": outs, "E": E, "rank": rank,
            "rows": rows, "base": base, "mixed": mixed, "idle": idle, "beside": beside}


def listed():
    return [
        # five tokens of one verification step: rotate, quantize, append
        _append("append nvfp4 5 tokens", 5, 32, 8, 128, 128, 16, "f32", False, 32768),
        # a prompt's chunk at far positions, half of each head rotated
        _append("append nvfp4 prompt", 4099, 32, 8, 128, 64, 64, "bf16", True, 1 << 20),
        # one new token, a short conversation, 4-bit cache
        _attn("attention nvfp4 short", 1, 1, 32, 8, 128, 16, 700, 700, "nvfp4"),
        # five tokens of one verification step on a long context
        _attn("attention nvfp4 verify", 1, 5, 32, 8, 128, 64, 32773, 32773, "nvfp4"),
        # a serving batch of very different lengths, small pages
        _attn("attention nvfp4 ragged", 48, 1, 32, 8, 128, 16, 17, 16384, "nvfp4"),
        # a batch on long contexts: the cache streamed once
        _attn("attention nvfp4 long batch", 16, 1, 32, 8, 128, 256, 20000, 65536, "nvfp4"),
        # capped scores, local layers' window, a small batch of two-token steps
        _attn("attention capped window", 8, 2, 32, 8, 128, 16, 300, 9001, "bf16", 4096, 50.0),
        # bias by distance, a key-value head for each query head, 8-bit cache
        _attn("attention distance bias", 16, 1, 16, 16, 64, 20, 1000, 30000, "e4m3", 0, 0.0, True),
        # one decoded token's q|k|v
        _lora("adapters 1 token", 1, 4096, "4096,1024,1024", 16, 16, 1),
        # a batch of requests, nearly each with its own adapter, of several ranks, on gate|up
        _lora("adapters batch", 48, 4096, "12288,12288", 64, 64, 1, mixed=True, idle=True),
        # 16 sequences of 8 verified tokens each, on the down product
        _lora("adapters verify", 128, 12288, "4096", 24, 32, 8),
        # the projections and the adapters on them, one step of 8 requests
        _lora("projection with adapters", 8, 4096, "4096,1024,1024", 32, 16, 1, beside=True),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("append4", "attn4", "attn4", "scored", "lora", "lora"))
    if op == "append4":
        D = rng.choice((64, 128, 128, 192, 256))
        Hkv = rng.choice((1, 2, 4, 8))
        T = _log_int(rng, 1, 4000)
        Hq = Hkv * rng.choice((1, 2, 4, 7))
        while T * (Hq + 2 * Hkv) * D > 4099 * 48 * 128:
            T = (T + 1) // 2
        c = _append("", T, Hq, Hkv, D, rng.choice((D, D // 2)), rng.choice((1, 16, 20, 64)),
                    rng.choice(("f32", "bf16")), rng.random() < 0.5, _log_int(rng, 4096, 1 << 20))
    elif op == "lora":
        M = _log_int(rng, 1, 128)
        K = 32 * _log_int(rng, 8, 384)
        outs = [_log_int(rng, 250, 12288) for _ in range(rng.choice((1, 1, 2, 3)))]
        E, rank = _log_int(rng, 1, 64), 8 * _log_int(rng, 1, 16)
        while E * rank * (len(outs) * K + sum(outs)) > 1 << 27:
            E = (E + 1) // 2
        c = _lora("", M, K, ",".join(str(n) for n in outs), E, rank, _log_int(rng, 1, 16),
                  rng.random() < 0.7, rng.random() < 0.4, rng.random() < 0.4)
    else:
        D = rng.choice((64, 128, 128, 256))
        Hkv = rng.choice((1, 2, 4, 8, 16))
        most = 1 << 29 if op == "attn4" else 1 << 27
        longest = _log_int(rng, 1, 60000)
        shortest = rng.choice((longest, _log_int(rng, 1, longest)))
        B = _log_int(rng, 1, 64)
        Q = rng.choice((1, 1, 1, 2, 3, 5, 8))
        while B > 1 and B * longest * Hkv * D * (1 + Q) > most:
            B = (B + 1) // 2
        while longest > 1 and B * longest * Hkv * D * (1 + Q) > most:
            longest, shortest = (longest + 1) // 2, (shortest + 1) // 2
        cap, bias = rng.choice(((50.0, False), (0.0, True), (20.0, True)))
        if op == "attn4":
            cap, bias = rng.choice(((0.0, False), (0.0, False), (cap, bias)))
        c = _attn("", B, Q, Hkv * rng.choice((1, 2, 4, 5, 8)), Hkv, D,
                  rng.choice((1, 16, 20, 32, 64, 256)), shortest, longest,
                  "nvfp4" if op == "attn4" else rng.choice(("bf16", "e4m3")),
                  rng.choice((0, 0, 0, _log_int(rng, 16, 8192))), cap, bias)
    del c["name"]
    return c


# ------------------------------------------------------------------ inputs

def _lengths(case):
    """The sequences' lengths: spread evenly over the logarithm."""
    B, a, b = case["B"], case["shortest"], case["longest"]
    if B == 1:
        return [b]
    return [max(1, int(round(a * (b / a) ** (i / (B - 1))))) for i in range(B)]


def _sequences(case):
    """Adapters: per sequence of `rows` rows, whether it has one, and its rank."""
    n = (case["M"] + case["rows"] - 1) // case["rows"]
    has = [not (case["idle"] and i % 5 == 3) for i in range(n)]
    return has, [max(8, case["rank"] // (8 << i % 3) * 8) if case["mixed"] else case["rank"]
                 for i in range(n)]


def _dtype(name):
    return {"f32": torch.float32, "bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn}[name]


def _inv_freq(R):
    """Inverse frequencies of base 10^6, as a program computes them once."""
    i = torch.arange(0, R, 2, dtype=torch.float64)
    return (1e6 ** (-i / R)).to(torch.float32).to(DEV)


def _slopes(H):
    """The biases' slopes, falling geometrically over the heads."""
    return (2.0 ** (-8.0 * torch.arange(1, H + 1, dtype=torch.float64) / H)).float().to(DEV)


def _pairs():
    """The two E2M1 values of a byte, as the two bytes of an e4m3 pair."""
    v = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float32)
    v = torch.cat([v, -v]).to(torch.float8_e4m3fn).view(torch.uint8).to(torch.int32)
    b = torch.arange(256)
    return (v[b & 15] | (v[b >> 4] << 8)).to(torch.int16).to(DEV)


def _quantized(x, g):
    """x[..., D] fp32 on the NVFP4 grid of the tensor scale g (an fp32 tensor of
    one): codes u8 [..., D / 2] and E4M3 block scales [..., D / 16]."""
    b = x.unflatten(-1, (-1, 16))
    s8 = (b.abs().amax(-1) / (6 * g)).clamp(max=448).to(torch.float8_e4m3fn)
    d = (s8.float() * g)[..., None]
    t = torch.where(d > 0, b / torch.where(d > 0, d, torch.ones_like(d)), torch.zeros_like(b))
    a = t.abs()
    # E2M1, ties to the even code
    m = (a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) \
        + (a >= 3.5) + (a > 5)
    m = torch.where((t < 0) & (m > 0), m + 8, m).to(torch.uint8).flatten(-2)
    return m[..., 0::2] | (m[..., 1::2] << 4), s8


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed * 1000003 + 29)

    def normal(*shape, std=1.0, dtype=torch.float32):
        return (torch.randn(*shape, generator=g, device=DEV) * std).to(dtype)

    s = {"case": case}
    if case["op"] == "append4":
        T, Hq, Hkv, D, page = (case[k] for k in ("T", "Hq", "Hkv", "D", "page"))
        # one buffer for q, k and v, as a fused projection writes it
        qkv = normal(T, Hq + 2 * Hkv, D, dtype=_dtype(case["x"]))
        s["q"], s["k"], s["v"] = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
        start = int(torch.randint(0, case["far"], (1,), generator=g, device=DEV))
        s["positions"] = start + torch.arange(T, device=DEV)
        blocks = (T + page - 1) // page + 3
        at = torch.randperm(blocks, generator=g, device=DEV)[:(T + page - 1) // page]
        t = torch.arange(T, device=DEV)
        s["slots"] = at[t // page] * page + t % page
        s["inv_freq"] = _inv_freq(case["R"])
        s["codes"] = torch.zeros(2, blocks, page, Hkv, D // 2, dtype=torch.uint8, device=DEV)
        s["scales"] = torch.zeros(2, blocks, page, Hkv, D // 16, dtype=torch.uint8, device=DEV)
        s["gk"], s["gv"] = torch.full((1,), GK, device=DEV), torch.full((1,), GV, device=DEV)
        s["q_out"] = torch.empty(T, Hq, D, dtype=torch.bfloat16, device=DEV)
        s["pairs"] = _pairs()
    elif case["op"] == "attn":
        B, Q, Hq, Hkv, D, page = (case[k] for k in ("B", "Q", "Hq", "Hkv", "D", "page"))
        lens = torch.tensor(_lengths(case), dtype=torch.int32, device=DEV)
        lens = lens[torch.randperm(B, generator=g, device=DEV)].contiguous()
        width = (case["longest"] + page - 1) // page
        # pages lie in the order in which a running server hands them out
        used = [(n + page - 1) // page for n in lens.tolist()]
        blocks = sum(used) + 1
        order = torch.randperm(blocks, generator=g, device=DEV).to(torch.int32)
        first = torch.tensor([0] + used[:-1], device=DEV).cumsum(0)
        col = torch.arange(width, device=DEV)
        live = col[None, :] < torch.tensor(used, device=DEV)[:, None]
        s["table"] = torch.where(live, order[(first[:, None] + col).clamp(max=blocks - 1)],
                                 torch.zeros((), dtype=torch.int32, device=DEV)).contiguous()
        s["lens"] = lens
        # capped layers see scores of tens
        s["q"] = normal(B * Q, Hq, D, std=6.0 if case["cap"] else 1.0, dtype=torch.bfloat16)
        s["slopes"] = _slopes(Hq) if case["bias"] else None
        shape, eight = (blocks, page, Hkv, D), case["cache"] == "e4m3"
        n, step = blocks * page * Hkv * D, 1 << 27   # in pieces: the fp32 draw is the larger part
        for name, scale, gs in (("k", 0.013, GK), ("v", 0.011, GV)):
            if case["cache"] == "nvfp4":
                codes = torch.empty(n // 2, dtype=torch.uint8, device=DEV)
                scales = torch.empty(n // 16, dtype=torch.uint8, device=DEV)
                gt = torch.full((1,), gs, device=DEV)
                for i in range(0, n, step):
                    c, s8 = _quantized(normal(min(step, n - i)), gt)
                    codes[i // 2:(i + step) // 2] = c
                    scales[i // 16:(i + step) // 16] = s8.view(torch.uint8)
                s[name] = (codes.view(*shape[:3], D // 2), scales.view(*shape[:3], D // 16), gt)
            else:
                c = torch.empty(n, dtype=_dtype(case["cache"]), device=DEV)
                for i in range(0, n, step):
                    z = normal(min(step, n - i))
                    c[i:i + step] = ((z / scale).clamp(-448, 448) if eight else z).to(c.dtype)
                s[name] = (c.view(shape), torch.full((1,), scale, device=DEV) if eight else None)
        if case["cache"] == "nvfp4":
            v = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], device=DEV)
            v, b = torch.cat([v, -v]), torch.arange(256, device=DEV)
            s["values"] = torch.stack([v[b & 15], v[b >> 4]], -1)
        s["out"] = torch.empty(B * Q, Hq, D, dtype=torch.bfloat16, device=DEV)
    else:
        M, K, E, rank = (case[k] for k in ("M", "K", "E", "rank"))
        outs = [int(n) for n in case["outs"].split(",")]
        s["x"] = normal(M, K, dtype=torch.bfloat16)
        has, ranks = _sequences(case)
        at = torch.randperm(E, generator=g, device=DEV)
        seq = torch.arange(M, device=DEV) // case["rows"]
        s["ids"] = torch.where(torch.tensor(has, device=DEV)[seq], at[seq % E],
                               torch.full((), -1, device=DEV)).to(torch.int32)
        # sequences i, i + E, .. share an adapter, which has the first one's rank
        per = torch.full((E,), rank, dtype=torch.int32)
        m = min(E, len(ranks))
        per[at[:m].cpu()] = torch.tensor(ranks[:m], dtype=torch.int32)
        s["ranks"] = per.to(DEV) if case["mixed"] else None
        s["alpha"] = 0.5 + torch.rand(E, generator=g, device=DEV) * 2
        s["adapters"] = [(normal(E, rank, K, std=K ** -0.5, dtype=torch.bfloat16),
                          normal(E, n, rank, std=0.05, dtype=torch.bfloat16)) for n in outs]
        s["base"] = [normal(M, n) for n in outs] if case["base"] and not case["beside"] else None
        s["y"] = [torch.empty(M, n, device=DEV) for n in outs]
        if case["beside"]:
            gt = torch.full((1,), 0.1 / 2688, device=DEV)
            s["weights"] = [(*_quantized(normal(n, K, std=0.02), gt), gt) for n in outs]
            v = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], device=DEV)
            v, b = torch.cat([v, -v]), torch.arange(256, device=DEV)
            s["values"] = torch.stack([v[b & 15], v[b >> 4]], -1)
    return s


# --------------------------------------------------------------- plain forms

def _rotated(x, cos, sin, R, interleaved):
    x = x.float()
    rot, rest = x[..., :R], x[..., R:]
    if interleaved:
        a, b = rot[..., 0::2], rot[..., 1::2]
        rot = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = rot[..., :R // 2], rot[..., R // 2:]
        rot = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([rot, rest], -1)


def _appended(s):
    """What an append gives: q, and the whole cache as the values it stands for
    (in units of its scales)."""
    codes, scales = s["codes"], s["scales"].view(torch.float8_e4m3fn)
    return [s["q_out"], s["pairs"][codes.int()].view(torch.float8_e4m3fn).view(
        *codes.shape[:-1], -1), scales]


def _plain_append(s):
    case = s["case"]
    angle = s["positions"].double()[:, None, None] * s["inv_freq"].double()
    cos, sin = angle.cos().float(), angle.sin().float()
    R, inter = case["R"], case["interleaved"]
    s["q_out"].copy_(_rotated(s["q"], cos, sin, R, inter))
    kc, ks = _quantized(_rotated(s["k"], cos, sin, R, inter), s["gk"])
    vc, vs = _quantized(s["v"].float(), s["gv"])
    codes, scales = s["codes"].flatten(1, 2), s["scales"].flatten(1, 2)
    codes[:, s["slots"]] = torch.stack([kc, vc])
    scales[:, s["slots"]] = torch.stack([ks.view(torch.uint8), vs.view(torch.uint8)])
    return _appended(s)


def _paged(s, name):
    """[B, Hkv, L, D] in 32 bits."""
    table = s["table"]
    if s["case"]["cache"] == "nvfp4":
        codes, scales, g = s[name]
        x = s["values"][codes[table].int()].flatten(-2)
        f = scales[table].view(torch.float8_e4m3fn).float()[..., None]
        x = (x.unflatten(-1, (-1, 16)) * f).flatten(-2)
    else:
        c, g = s[name]
        x = (c[table] if g is None else c.view(torch.uint8)[table].view(c.dtype)).float()
    x = x.flatten(1, 2).transpose(1, 2)
    return x if g is None else x * g


def _plain_attn(s):
    case = s["case"]
    B, Q, Hq, Hkv, D = (case[k] for k in ("B", "Q", "Hq", "Hkv", "D"))
    G = Hq // Hkv
    q = s["q"].float().view(B, Q, Hkv, G, D).permute(0, 2, 1, 3, 4).reshape(B, Hkv, Q * G, D)
    k = _paged(s, "k")
    scores = torch.matmul(q * D ** -0.5, k.transpose(2, 3).contiguous())
    del k
    if case["cap"]:
        scores = case["cap"] * torch.tanh(scores / case["cap"])
    L = scores.shape[-1]
    at = torch.arange(L, device=DEV)
    pos = s["lens"].long()[:, None] - Q + torch.arange(Q, device=DEV)
    if case["bias"]:
        far = (at - pos[..., None]).float()[:, None, :, None]           # [B, 1, Q, 1, L]
        bias = far * s["slopes"].view(Hkv, 1, G, 1)
        scores = scores + bias.reshape(B, Hkv, Q * G, L)
        del bias
    live = at <= pos[..., None]
    if case["window"]:
        live &= at > pos[..., None] - case["window"]
    live = live.repeat_interleave(G, 1)[:, None]
    scores = torch.where(live, scores, torch.full((), -math.inf, device=DEV))
    top = scores.amax(-1, keepdim=True)
    p = torch.exp(scores - torch.where(top > -math.inf, top, torch.zeros_like(top)))
    del scores
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p, _paged(s, "v").contiguous())
    o = torch.where(total > 0, o / total, torch.zeros_like(o))
    return o.view(B, Hkv, Q, G, D).permute(0, 2, 1, 3, 4).reshape(B * Q, Hq, D).to(torch.bfloat16)


def _dense(s, i):
    codes, scales, g = s["weights"][i]
    w = s["values"][codes.int()].flatten(-2).unflatten(-1, (-1, 16)) * scales.float()[..., None]
    return torch.matmul(s["x"].float(), (w * g).flatten(-2).t().contiguous())


def _adapted(s, i):
    a, b = s["adapters"][i]
    ids = s["ids"].long()
    at = ids.clamp(min=0)
    f = torch.where(ids >= 0, s["alpha"][at], torch.zeros_like(s["alpha"][at]))
    t = torch.bmm(a[at].float(), s["x"].float()[..., None])              # [M, rank, 1]
    if s["ranks"] is not None:
        r = torch.arange(a.shape[1], device=DEV)
        t = torch.where(r[:, None] < s["ranks"][at][:, None, None], t, torch.zeros_like(t))
    return torch.bmm(b[at].float(), t)[..., 0] * f[:, None]


def _plain_lora(s):
    n = range(len(s["y"]))
    base = [_dense(s, i) for i in n] if s["case"]["beside"] else s["base"]
    return [_adapted(s, i) if base is None else base[i] + _adapted(s, i) for i in n]


# -------------------------------------------------------------------- passes

def _own_append(s):
    import nvfp4_block_scaled_gemv_amd as nv
    nv.rope_append_nvfp4_into(s["q"], s["k"], s["v"], s["positions"], s["slots"], s["inv_freq"],
                              s["q_out"], (s["codes"][0], s["scales"][0], s["gk"]),
                              (s["codes"][1], s["scales"][1], s["gv"]),
                              interleaved=s["case"]["interleaved"])
    return _appended(s)


def _own_attn(s):
    import nvfp4_block_scaled_gemv_amd as nv
    case = s["case"]
    if "workspace" not in s:   # a serving program keeps one for its largest batch
        n = nv.paged_attention_workspace_bytes(case["B"], case["Q"], case["Hq"], case["Hkv"],
                                               case["D"])
        s["workspace"] = torch.empty(max(n, 256), dtype=torch.uint8, device=DEV)
    if case["cache"] == "nvfp4":
        nv.paged_attention_nvfp4_into(s["q"], s["k"], s["v"], s["table"], s["lens"], s["out"],
                                      s["workspace"], window=case["window"], softcap=case["cap"],
                                      slopes=s["slopes"])
    else:
        nv.paged_attention_scored_into(s["q"], s["k"][0], s["v"][0], s["table"], s["lens"],
                                       s["out"], s["workspace"], softcap=case["cap"],
                                       slopes=s["slopes"], window=case["window"],
                                       k_scale=s["k"][1], v_scale=s["v"][1])
    return s["out"]


def _own_lora(s):
    import nvfp4_block_scaled_gemv_amd as nv
    case = s["case"]
    if "workspace" not in s:
        n = nv.lora_workspace_bytes(case["M"], case["K"], case["rank"], len(s["y"]))
        s["workspace"] = torch.empty(max(n, 256), dtype=torch.uint8, device=DEV)
    base = s["base"]
    if case["beside"]:
        nv.gemv_segments_into([(c, f.view(torch.uint8), g) for c, f, g in s["weights"]], s["x"],
                              s["y"])
        base = s["y"]          # in place, on what the projections wrote
    nv.lora_segments_into(s["adapters"], s["x"], s["ids"], s["y"], s["workspace"], bases=base,
                          alpha=s["alpha"], ranks=s["ranks"])
    return s["y"]


def run(state):
    op = state["case"]["op"]
    if own:
        return {"append4": _own_append, "attn": _own_attn, "lora": _own_lora}[op](state)
    return {"append4": _plain_append, "attn": _plain_attn, "lora": _plain_lora}[op](state)


# ---------------------------------------------------------------------- work

def work(case):
    if case["op"] == "append4":
        T, Hq, Hkv, D = (case[k] for k in ("T", "Hq", "Hkv", "D"))
        n = T * (Hq + 2 * Hkv) * D * (4 if case["x"] == "f32" else 2) + T * 16
        return {"bytes": n + T * D * (2 * Hq + 2 * Hkv * (0.5 + 1 / 16)),
                "flops": 3.0 * T * (Hq + Hkv) * case["R"]}
    if case["op"] == "attn":
        B, Q, Hq, Hkv, D, w = (case[k] for k in ("B", "Q", "Hq", "Hkv", "D", "window"))
        keys = pairs = 0
        for n in _lengths(case):
            for i in range(Q):
                pos = n - Q + i
                pairs += max(0, min(pos + 1, w) if w else pos + 1)
            keys += min(n, w + Q - 1) if w else n
        one = {"bf16": 2, "e4m3": 1, "nvfp4": 0.5 + 1 / 16}[case["cache"]]
        return {"bytes": 2 * Hkv * D * one * keys + 4 * B * Q * Hq * D + 4 * keys / case["page"],
                "flops": 4.0 * pairs * Hq * D}
    M, K = case["M"], case["K"]
    has, ranks = _sequences(case)
    E = case["E"]
    # an adapter is read once for all its rows; the first E sequences show all of them
    weights = sum(r for i, r in enumerate(ranks[:E]) if any(has[i::E]))
    rows = sum(ranks[i % E] * (min(M, (i + 1) * case["rows"]) - i * case["rows"])
               for i in range(len(ranks)) if has[i])
    N = sum(int(n) for n in case["outs"].split(","))
    S = len(case["outs"].split(","))
    bytes_ = 2.0 * M * K + 2.0 * weights * (S * K + N) + 4.0 * M * N * (2 if case["base"] else 1)
    flops = 2.0 * rows * (S * K + N)
    if case["beside"]:   # the projections write what the adapters add to: once
        bytes_ += N * K * (0.5 + 1 / 16) - 4.0 * M * N
        flops += 2.0 * M * N * K
    return {"bytes": bytes_, "flops": flops}


# --------------------------------------------------------------------- exact

def _exact_append(s, case):
    R, D = case["R"], case["D"]
    theta = torch.outer(s["positions"].double(), s["inv_freq"].double())
    turn = torch.polar(torch.ones_like(theta), theta)[:, None]

    def rotate(x):
        x = x.double()
        y = x.clone()
        first = slice(0, R, 2) if case["interleaved"] else slice(0, R // 2)
        second = slice(1, R, 2) if case["interleaved"] else slice(R // 2, R)
        z = torch.complex(x[..., first], x[..., second]) * turn
        y[..., first], y[..., second] = z.real, z.imag
        return y

    # the block scales; a 4-bit value follows from its block's rounded scale
    scales = torch.zeros(s["scales"].shape, dtype=torch.float64, device=DEV).flatten(1, 2)
    for i, (rows, g) in enumerate(((rotate(s["k"]), s["gk"]), (s["v"].double(), s["gv"]))):
        top = rows.reshape(*rows.shape[:-1], D // 16, 16).abs().max(-1).values
        scales[i, s["slots"]] = (top / (6 * g.double())).clamp(max=448)
    return [rotate(s["q"]), None, scales.view(s["scales"].shape)]


def _exact_attn(s, case):
    B, Q, Hq, Hkv, D, page = (case[k] for k in ("B", "Q", "Hq", "Hkv", "D", "page"))
    G = Hq // Hkv
    out = torch.zeros(B, Q, Hq, D, dtype=torch.float64, device=DEV)
    grid = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, 0, -.5, -1, -1.5, -2, -3, -4, -6],
                        dtype=torch.float64, device=DEV)

    def rows(name, slot):
        if case["cache"] != "nvfp4":
            c, f = s[name]
            x = c.view(-1, Hkv, D).view(torch.uint8)[slot].view(c.dtype).double()
            return x if f is None else x * f.double()
        codes, scales, g = s[name]
        c = codes.view(-1, Hkv, D // 2)[slot].long()
        x = torch.empty(*c.shape[:2], D, dtype=torch.float64, device=DEV)
        x[..., 0::2], x[..., 1::2] = grid[c % 16], grid[c // 16]
        f = scales.view(-1, Hkv, D // 16)[slot].view(torch.float8_e4m3fn).double() * g.double()
        return x * f.repeat_interleave(16, -1)

    q = s["q"].double().view(B, Q, Hkv, G, D)
    for b, n in enumerate(s["lens"].tolist()):
        t = torch.arange(n, device=DEV)
        slot = s["table"][b].long()[t // page] * page + t % page
        k, v = rows("k", slot), rows("v", slot)
        for h in range(Hkv):
            kh, vh = k[:, h].contiguous(), v[:, h].contiguous()
            for i in range(Q):
                last = n - Q + i
                first = max(0, last + 1 - case["window"]) if case["window"] else 0
                if last < 0:
                    continue
                z = q[b, i, h] @ kh[first:last + 1].t().contiguous() / math.sqrt(D)
                if case["cap"]:
                    z = case["cap"] * torch.tanh(z / case["cap"])
                if case["bias"]:
                    far = (last - t[first:last + 1]).double()
                    z = z - s["slopes"][h * G:(h + 1) * G, None].double() * far
                w = torch.exp(z - z.max(1, keepdim=True).values)
                o = w @ vh[first:last + 1] / w.sum(1, keepdim=True)
                out[b, i, h * G:(h + 1) * G] = o
    return out.view(B * Q, Hq, D)


def _exact_lora(s, case):
    grid = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, 0, -.5, -1, -1.5, -2, -3, -4, -6],
                        dtype=torch.float64, device=DEV)
    x, ids = s["x"].double(), s["ids"].tolist()
    ys = []
    for i, (a, b) in enumerate(s["adapters"]):
        y = torch.zeros(s["y"][i].shape, dtype=torch.float64, device=DEV)
        if case["beside"]:
            codes, scales, g = s["weights"][i]
            w = torch.stack([grid[(codes % 16).long()], grid[(codes // 16).long()]], -1).flatten(1)
            w = w * scales.double().repeat_interleave(16, 1) * g.double()
            y += x @ w.t().contiguous()
        elif s["base"] is not None:
            y += s["base"][i].double()
        for e in sorted(set(ids) - {-1}):
            m = torch.tensor([j for j, n in enumerate(ids) if n == e], device=DEV)
            r = case["rank"] if s["ranks"] is None else int(s["ranks"][e])
            low = x[m] @ a[e, :r].double().t().contiguous()
            y[m] += s["alpha"][e].double() * (low @ b[e, :, :r].double().t().contiguous())
        ys.append(y)
    return ys


def exact(case, seed):
    s = prepare(case, seed)
    return {"append4": _exact_append, "attn": _exact_attn, "lora": _exact_lora}[case["op"]](s, case)
