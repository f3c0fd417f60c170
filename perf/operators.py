"""The operators of a decode step that stand between the GEMVs: RMS norm with
the residual's addition (bf16, e4m3 and NVFP4 outputs), rotary positions with
the append to a paged key-value cache, attention of the new tokens over that
cache, and verification of drafted tokens.

listed() and draw() give the cases, prepare() a case's inputs, run() one pass
(the plain form in torch, or the library's kernels where `own` is true), work()
what a pass cannot do without and exact() the result in 64 bits.
"""
import math

import torch

own = False

DEV = "cuda"
VOCAB = 151936
EPS = 1e-6


# ------------------------------------------------------------------- cases

def _norm(name, M, H, x, residual, out, group=0):
    return {"name": name, "op": "norm", "M": M, "H": H, "x": x, "residual": residual,
            "out": out, "group": group}


def _append(name, T, Hq, Hkv, D, R, page, x, cache, interleaved, far):
    return {"name": name, "op": "append", "T": T, "Hq": Hq, "Hkv": Hkv, "D": D, "R": R,
            "page": page, "x": x, "cache": cache, "interleaved": interleaved, "far": far}


def _attn(name, B, Q, Hq, Hkv, D, page, shortest, longest, cache, window=0):
    return {"name": name, "op": "attn", "B": B, "Q": Q, "Hq": Hq, "Hkv": Hkv, "D": D,
            "page": page, "shortest": shortest, "longest": longest, "cache": cache,
            "window": window}


def _verify(name, B, Q, V, draft_p):
    return {"name": name, "op": "verify", "B": B, "Q": Q, "V": V, "draft_p": draft_p}


def listed():
    return [
        # the norm before q|k|v for one decoded token: x is the previous GEMV's fp32 output
        _norm("norm 1 token", 1, 4096, "f32", "bf16", "bf16"),
        # the same for a batch of tokens whose next product takes NVFP4 activations
        _norm("norm W4A4 batch", 8, 4096, "f32", "bf16", "nvfp4"),
        # a prompt's rows, 8-bit output with a scale for each 128 values, fp32 residual stream
        _norm("norm prompt 8 bits", 2048, 7168, "bf16", "f32", "e4m3", 128),
        # five tokens of one verification step: rotate and append
        _append("append 5 tokens", 5, 32, 8, 128, 128, 16, "f32", "bf16", False, 32768),
        # a prompt's chunk at far positions, half of each head rotated, 8-bit cache
        _append("append prompt", 4099, 32, 8, 128, 64, 64, "bf16", "e4m3", True, 1 << 20),
        # one new token, a short conversation
        _attn("attention short", 1, 1, 32, 8, 128, 16, 700, 700, "bf16"),
        # five tokens of one verification step on a long context
        _attn("attention verify", 1, 5, 32, 8, 128, 64, 32773, 32773, "bf16"),
        # a serving batch of very different lengths, 8-bit cache, small pages
        _attn("attention ragged 8 bits", 48, 1, 32, 8, 128, 16, 17, 16384, "e4m3"),
        # one key-value head for each query head, small heads, a window, pages that no tile fits
        _attn("attention window", 8, 2, 16, 16, 64, 20, 900, 9001, "bf16", 2048),
        # a batch on long contexts: the cache streamed once
        _attn("attention long batch", 16, 1, 32, 8, 128, 256, 20000, 65536, "bf16"),
        # one verification step of four drafts
        _verify("verify 4 drafts", 1, 4, VOCAB, True),
        # a batch of verification steps (128 rows of the LM head)
        _verify("verify batch", 16, 7, VOCAB, True),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("norm", "norm", "append", "attn", "attn", "verify"))
    if op == "norm":
        out = rng.choice(("bf16", "e4m3", "nvfp4"))
        H = 8 * _log_int(rng, 16, 2048)
        group = rng.choice((0, 32, 64, 128)) if out == "e4m3" else 0
        unit = group if group else 32 if out == "nvfp4" else 8
        H = max(unit, H // unit * unit)
        M = _log_int(rng, 1, 3000)
        while M * H > 1 << 24:
            M = (M + 1) // 2
        c = _norm("", M, H, rng.choice(("f32", "bf16")), rng.choice(("none", "bf16", "f32")),
                  out, group)
    elif op == "append":
        D = rng.choice((64, 96, 128, 256))
        Hkv = rng.choice((1, 2, 4, 8))
        T = _log_int(rng, 1, 4000)
        Hq = Hkv * rng.choice((1, 2, 4, 7))
        while T * (Hq + 2 * Hkv) * D > 4099 * 48 * 128:
            T = (T + 1) // 2
        c = _append("", T, Hq, Hkv, D, rng.choice((D, D // 2)), rng.choice((1, 16, 20, 64)),
                    rng.choice(("f32", "bf16")), rng.choice(("bf16", "e4m3")),
                    rng.random() < 0.5, _log_int(rng, 4096, 1 << 20))
    elif op == "attn":
        D = rng.choice((64, 128, 128, 256))
        Hkv = rng.choice((1, 2, 4, 8, 16))
        longest = _log_int(rng, 1, 60000)
        shortest = rng.choice((longest, _log_int(rng, 1, longest)))
        B = _log_int(rng, 1, 64)
        Q = rng.choice((1, 1, 1, 2, 3, 5, 8))
        while B > 1 and B * longest * Hkv * D * (1 + Q) > 1 << 29:
            B = (B + 1) // 2
        while longest > 1 and B * longest * Hkv * D * (1 + Q) > 1 << 29:
            longest, shortest = (longest + 1) // 2, (shortest + 1) // 2
        c = _attn("", B, Q, Hkv * rng.choice((1, 2, 4, 5, 8)), Hkv, D,
                  rng.choice((1, 16, 20, 32, 64, 256)), shortest, longest,
                  rng.choice(("bf16", "e4m3")), rng.choice((0, 0, 0, _log_int(rng, 16, 8192))))
    else:
        V = _log_int(rng, 1000, 200000)
        Q = rng.randint(1, 8)
        B = _log_int(rng, 1, 32)
        while B * (2 * Q + 1) * V > 16 * 15 * VOCAB:
            B = (B + 1) // 2
        c = _verify("", B, Q, V, rng.random() < 0.7)
    del c["name"]
    return c


# ------------------------------------------------------------------ inputs

def _lengths(case):
    """The sequences' lengths: spread evenly over the logarithm."""
    B, a, b = case["B"], case["shortest"], case["longest"]
    if B == 1:
        return [b]
    return [max(1, int(round(a * (b / a) ** (i / (B - 1))))) for i in range(B)]


def _dtype(name):
    return {"f32": torch.float32, "bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn}[name]


def _inv_freq(R):
    """Inverse frequencies of base 10^6, as a program computes them once."""
    i = torch.arange(0, R, 2, dtype=torch.float64)
    return (1e6 ** (-i / R)).to(torch.float32).to(DEV)


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed * 1000003 + 17)

    def normal(*shape, std=1.0, dtype=torch.float32):
        return (torch.randn(*shape, generator=g, device=DEV) * std).to(dtype)

    s = {"case": case}
    if case["op"] == "norm":
        M, H = case["M"], case["H"]
        s["x"] = normal(M, H, std=0.5, dtype=_dtype(case["x"]))
        s["residual"] = s["residual_out"] = None
        if case["residual"] != "none":
            s["residual"] = normal(M, H, std=2.0, dtype=_dtype(case["residual"]))
            s["residual_out"] = torch.empty_like(s["residual"])
        s["weight"] = (1 + normal(H, std=0.2)).to(torch.bfloat16)
        if case["out"] == "bf16":
            s["y"] = torch.empty(M, H, dtype=torch.bfloat16, device=DEV)
        elif case["out"] == "e4m3":
            s["y"] = torch.empty(M, H, dtype=torch.float8_e4m3fn, device=DEV)
            s["scales"] = torch.empty(M, H // (case["group"] or H), device=DEV)
        else:
            s["gscale"] = torch.full((1,), 4.5 / 2688, device=DEV)
            s["codes"] = torch.empty(M, H // 2, dtype=torch.uint8, device=DEV)
            s["scales"] = torch.empty(M, H // 16, dtype=torch.uint8, device=DEV)
            # the two E2M1 values of a byte, as the two bytes of an e4m3 pair
            v = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float32)
            v = torch.cat([v, -v]).to(torch.float8_e4m3fn).view(torch.uint8).to(torch.int32)
            b = torch.arange(256)
            s["pairs"] = (v[b & 15] | (v[b >> 4] << 8)).to(torch.int16).to(DEV)
    elif case["op"] == "append":
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
        cache = torch.zeros(2, blocks, page, Hkv, D, device=DEV).to(_dtype(case["cache"]))
        s["k_cache"], s["v_cache"] = cache[0], cache[1]
        eight = case["cache"] == "e4m3"
        s["k_scale"] = torch.full((1,), 0.013, device=DEV) if eight else None
        s["v_scale"] = torch.full((1,), 0.011, device=DEV) if eight else None
        s["q_out"] = torch.empty(T, Hq, D, dtype=torch.bfloat16, device=DEV)
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
        s["q"] = normal(B * Q, Hq, D, dtype=torch.bfloat16)
        eight = case["cache"] == "e4m3"
        s["k_scale"] = torch.full((1,), 0.013, device=DEV) if eight else None
        s["v_scale"] = torch.full((1,), 0.011, device=DEV) if eight else None
        kv = []
        for scale in (0.013, 0.011):
            c = torch.empty(blocks, page, Hkv, D, dtype=_dtype(case["cache"]), device=DEV)
            flat, n, step = c.view(-1), c.numel(), 1 << 28
            for i in range(0, n, step):   # in pieces: the fp32 draw is the larger part
                z = normal(min(step, n - i))
                flat[i:i + step] = ((z / scale).clamp(-448, 448) if eight else z).to(c.dtype)
            kv.append(c)
        s["k_cache"], s["v_cache"] = kv
        s["out"] = torch.empty(B * Q, Hq, D, dtype=torch.bfloat16, device=DEV)
    else:
        B, Q, V = case["B"], case["Q"], case["V"]
        logits = normal(B, Q + 1, V, std=2.5)
        s["p"] = torch.softmax(logits, -1)
        q = torch.softmax(logits[:, :Q] + normal(B, Q, V, std=0.7), -1)
        # the drafts are drawn from the draft's own probabilities
        u = torch.rand(B, Q, 1, generator=g, device=DEV, dtype=torch.float64)
        cdf = q.double().cumsum(-1)
        draft = torch.searchsorted(cdf, u * cdf[..., -1:], right=True).clamp(max=V - 1)
        s["draft"] = draft[..., 0].to(torch.int32).contiguous()
        s["q"] = q if case["draft_p"] else None
        s["u_accept"] = torch.rand(B, Q, generator=g, device=DEV)
        s["u_sample"] = torch.rand(B, generator=g, device=DEV)
        s["tokens"] = torch.empty(B, Q + 1, dtype=torch.int32, device=DEV)
        s["accepted"] = torch.empty(B, dtype=torch.int32, device=DEV)
    return s


# --------------------------------------------------------------- plain forms

def _plain_norm(s):
    case = s["case"]
    v = s["x"].float()
    out = []
    if s["residual"] is not None:
        v = v + s["residual"].float()
        out.append(v.to(s["residual"].dtype))
    y = v * torch.rsqrt((v * v).mean(-1, keepdim=True) + EPS) * s["weight"].float()
    if case["out"] == "bf16":
        return [y.to(torch.bfloat16)] + out
    M, H = y.shape
    if case["out"] == "e4m3":
        y = y.view(M, -1, case["group"] or H)
        amax = y.abs().amax(-1, keepdim=True)
        scale = torch.where(amax > 0, amax / 448, torch.ones_like(amax))
        y8 = (y / scale).clamp(-448, 448).to(torch.float8_e4m3fn)
        return [y8.view(M, H), scale[..., 0]] + out
    y = y.view(M, H // 16, 16)
    r = y.abs().amax(-1, keepdim=True) / (6 * s["gscale"])
    s8 = r.clamp(max=448).to(torch.float8_e4m3fn)
    d = s8.float() * s["gscale"]
    t = torch.where(d > 0, y / torch.where(d > 0, d, torch.ones_like(d)), torch.zeros_like(y))
    a = t.abs()
    # E2M1, ties to the even code
    m = 0.5 * (a > 0.25) + 0.5 * (a >= 0.75) + 0.5 * (a > 1.25) + 0.5 * (a >= 1.75) \
        + 1.0 * (a > 2.5) + 1.0 * (a >= 3.5) + 2.0 * (a > 5)
    q = torch.where((t < 0) & (m > 0), -m, m).to(torch.float8_e4m3fn)
    return [q.view(M, H), s8[..., 0]] + out


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


def _store(cache, slots, rows, scale):
    flat = cache.view(-1, *cache.shape[2:])
    if scale is None:
        flat[slots] = rows.to(cache.dtype)
    else:
        rows = (rows / scale).clamp(-448, 448).to(cache.dtype)
        flat.view(torch.uint8)[slots] = rows.view(torch.uint8)


def _plain_append(s):
    case = s["case"]
    angle = s["positions"].double()[:, None, None] * s["inv_freq"].double()
    cos, sin = angle.cos().float(), angle.sin().float()
    R, inter = case["R"], case["interleaved"]
    q = _rotated(s["q"], cos, sin, R, inter).to(torch.bfloat16)
    _store(s["k_cache"], s["slots"], _rotated(s["k"], cos, sin, R, inter), s["k_scale"])
    _store(s["v_cache"], s["slots"], s["v"].float(), s["v_scale"])
    return [q, s["k_cache"], s["v_cache"]]


def _paged(cache, table, scale):
    """[B, Hkv, L, D] in 32 bits."""
    x = cache.view(torch.uint8)[table].view(cache.dtype) if scale is not None else cache[table]
    B, n, page, Hkv, D = x.shape
    x = x.view(B, n * page, Hkv, D).permute(0, 2, 1, 3).float()
    return x if scale is None else x * scale


def _plain_attn(s):
    case = s["case"]
    B, Q, Hq, Hkv, D = (case[k] for k in ("B", "Q", "Hq", "Hkv", "D"))
    G = Hq // Hkv
    q = s["q"].float().view(B, Q, Hkv, G, D).permute(0, 2, 1, 3, 4).reshape(B, Hkv, Q * G, D)
    k = _paged(s["k_cache"], s["table"], s["k_scale"])
    scores = torch.matmul(q * D ** -0.5, k.transpose(2, 3).contiguous())
    del k
    L = scores.shape[-1]
    at = torch.arange(L, device=DEV)
    pos = s["lens"].long()[:, None] - Q + torch.arange(Q, device=DEV)
    live = at <= pos[..., None]
    if case["window"]:
        live &= at > pos[..., None] - case["window"]
    live = live.repeat_interleave(G, 1)[:, None]
    scores = torch.where(live, scores, torch.full((), -math.inf, device=DEV))
    top = scores.amax(-1, keepdim=True)
    p = torch.exp(scores - torch.where(top > -math.inf, top, torch.zeros_like(top)))
    del scores
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p, _paged(s["v_cache"], s["table"], s["v_scale"]).contiguous())
    o = torch.where(total > 0, o / total, torch.zeros_like(o))
    return o.view(B, Hkv, Q, G, D).permute(0, 2, 1, 3, 4).reshape(B * Q, Hq, D).to(torch.bfloat16)


def _plain_verify(s):
    B, Q, V = (s["case"][k] for k in ("B", "Q", "V"))
    at = s["draft"].long()[..., None]
    pt = s["p"][:, :Q].gather(-1, at)[..., 0].double()
    qt = torch.ones_like(pt) if s["q"] is None else s["q"].gather(-1, at)[..., 0].double()
    ok = s["u_accept"].double() * qt < pt
    n = ok.long().cumprod(-1).sum(-1)
    row = torch.arange(B, device=DEV)
    p = s["p"][row, n].double()
    j = n.clamp(max=Q - 1)
    if s["q"] is None:
        q = torch.zeros_like(p).scatter(1, s["draft"].long()[row, j][:, None], math.inf)
    else:
        q = s["q"][row, j].double()
    rest = torch.where((n < Q)[:, None], (p - q).clamp(min=0), p)
    rest = torch.where(rest.sum(-1, keepdim=True) > 0, rest, p)
    cdf = rest.cumsum(-1)
    new = (cdf <= s["u_sample"].double()[:, None] * cdf[:, -1:]).sum(-1).clamp(max=V - 1)
    col = torch.arange(Q + 1, device=DEV)
    draft = torch.cat([s["draft"].long(), torch.zeros_like(n)[:, None]], 1)
    tokens = torch.where(col < n[:, None], draft,
                         torch.where(col == n[:, None], new[:, None], torch.full_like(draft, -1)))
    return [tokens.to(torch.int32), n.to(torch.int32)]


# -------------------------------------------------------------------- passes

def _own_norm(s):
    import nvfp4_block_scaled_gemv_amd as nv
    case = s["case"]
    out = [] if s["residual"] is None else [s["residual_out"]]
    if case["out"] == "bf16":
        nv.add_rmsnorm_into(s["x"], s["weight"], EPS, s["y"], s["residual"], s["residual_out"])
        return [s["y"]] + out
    if case["out"] == "e4m3":
        nv.add_rmsnorm_e4m3_into(s["x"], s["weight"], EPS, s["y"], s["scales"], s["residual"],
                                 s["residual_out"])
        return [s["y"], s["scales"]] + out
    nv.add_rmsnorm_nvfp4_into(s["x"], s["weight"], EPS, s["gscale"], s["codes"], s["scales"],
                              s["residual"], s["residual_out"])
    M, H = s["x"].shape
    values = s["pairs"][s["codes"].int()].view(torch.float8_e4m3fn).view(M, H)
    return [values, s["scales"].view(torch.float8_e4m3fn)] + out


def _own_append(s):
    import nvfp4_block_scaled_gemv_amd as nv
    nv.rope_append_into(s["q"], s["k"], s["v"], s["positions"], s["slots"], s["inv_freq"],
                        s["q_out"], s["k_cache"], s["v_cache"], k_scale=s["k_scale"],
                        v_scale=s["v_scale"], interleaved=s["case"]["interleaved"])
    return [s["q_out"], s["k_cache"], s["v_cache"]]


def _own_attn(s):
    import nvfp4_block_scaled_gemv_amd as nv
    case = s["case"]
    if "workspace" not in s:   # a serving program keeps one for its largest batch
        n = nv.paged_attention_workspace_bytes(case["B"], case["Q"], case["Hq"], case["Hkv"],
                                               case["D"])
        s["workspace"] = torch.empty(max(n, 256), dtype=torch.uint8, device=DEV)
    nv.paged_attention_into(s["q"], s["k_cache"], s["v_cache"], s["table"], s["lens"], s["out"],
                            s["workspace"], window=case["window"], k_scale=s["k_scale"],
                            v_scale=s["v_scale"])
    return s["out"]


def _own_verify(s):
    import nvfp4_block_scaled_gemv_amd as nv
    if "workspace" not in s:
        n = nv.verify_draft_workspace_bytes(s["case"]["B"], s["case"]["V"])
        s["workspace"] = torch.empty(max(n, 256), dtype=torch.uint8, device=DEV)
    nv.verify_draft_into(s["p"], s["q"], s["draft"], s["u_accept"], s["u_sample"], s["tokens"],
                         s["accepted"], s["workspace"])
    return [s["tokens"], s["accepted"]]


def run(state):
    op = state["case"]["op"]
    if own:
        return {"norm": _own_norm, "append": _own_append, "attn": _own_attn,
                "verify": _own_verify}[op](state)
    return {"norm": _plain_norm, "append": _plain_append, "attn": _plain_attn,
            "verify": _plain_verify}[op](state)


# ---------------------------------------------------------------------- work

_BYTES = {"f32": 4, "bf16": 2, "e4m3": 1, "none": 0}


def work(case):
    if case["op"] == "norm":
        M, H = case["M"], case["H"]
        one = _BYTES[case["x"]] + 2 * _BYTES[case["residual"]]
        y = {"bf16": 2.0, "e4m3": 1 + 4 / (case["group"] or H), "nvfp4": 0.5 + 1 / 16}[case["out"]]
        return {"bytes": M * H * (one + y) + 2 * H, "flops": 6.0 * M * H}
    if case["op"] == "append":
        T, Hq, Hkv, D = (case[k] for k in ("T", "Hq", "Hkv", "D"))
        n = T * (Hq + 2 * Hkv) * D * _BYTES[case["x"]] + T * 16
        return {"bytes": n + T * D * (2 * Hq + 2 * Hkv * _BYTES[case["cache"]]),
                "flops": 3.0 * T * (Hq + Hkv) * case["R"]}
    if case["op"] == "attn":
        B, Q, Hq, Hkv, D, w = (case[k] for k in ("B", "Q", "Hq", "Hkv", "D", "window"))
        keys = pairs = 0
        for n in _lengths(case):
            for i in range(Q):
                pos = n - Q + i
                pairs += max(0, min(pos + 1, w) if w else pos + 1)
            keys += min(n, w + Q - 1) if w else n
        kv = 2 * Hkv * D * _BYTES[case["cache"]] * keys
        return {"bytes": kv + 4 * B * Q * Hq * D + 4 * keys / case["page"],
                "flops": 4.0 * pairs * Hq * D}
    B, V = case["B"], case["V"]
    rows = 2 if case["draft_p"] else 1
    return {"bytes": 4.0 * B * V * rows, "flops": 2.0 * B * V * rows}


# --------------------------------------------------------------------- exact

def _exact_norm(s, case):
    M, H = case["M"], case["H"]
    v = s["x"].double()
    tail = []
    if s["residual"] is not None:
        v = v + s["residual"].double()
        tail = [v]
    y = v / ((v ** 2).sum(1, keepdim=True) / H + EPS).sqrt() * s["weight"].double()
    if case["out"] == "bf16":
        return [y] + tail
    if case["out"] == "e4m3":
        width = case["group"] or H
        scale = y.abs().reshape(M, H // width, width).max(2).values / 448
        scale = torch.where(scale == 0, torch.ones_like(scale), scale)
        return [y / scale.repeat_interleave(width, 1), scale] + tail
    # the block scales; a 4-bit value follows from its block's rounded scale
    r = y.abs().reshape(M, H // 16, 16).max(2).values / (6 * s["gscale"].double())
    return [None, r.clamp(max=448)] + tail


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

    def cached(like, rows, scale):
        c = torch.zeros(like.shape[0] * like.shape[1], *like.shape[2:], dtype=torch.float64,
                        device=DEV)
        c[s["slots"]] = rows if scale is None else (rows / scale.double()).clamp(-448, 448)
        return c.view(like.shape)

    return [rotate(s["q"]), cached(s["k_cache"], rotate(s["k"]), s["k_scale"]),
            cached(s["v_cache"], s["v"].double(), s["v_scale"])]


def _exact_attn(s, case):
    B, Q, Hq, Hkv, D, page = (case[k] for k in ("B", "Q", "Hq", "Hkv", "D", "page"))
    out = torch.zeros(B, Q, Hq, D, dtype=torch.float64, device=DEV)
    ks = 1.0 if s["k_scale"] is None else s["k_scale"].double()
    vs = 1.0 if s["v_scale"] is None else s["v_scale"].double()
    q = s["q"].double().view(B, Q, Hkv, Hq // Hkv, D)
    for b, n in enumerate(s["lens"].tolist()):
        t = torch.arange(n, device=DEV)
        slot = s["table"][b].long()[t // page] * page + t % page
        k, v = (c.view(-1, Hkv, D).view(torch.uint8)[slot].view(c.dtype)
                for c in (s["k_cache"], s["v_cache"]))
        for h in range(Hkv):
            kh, vh = k[:, h].double() * ks, v[:, h].double() * vs
            for i in range(Q):
                last = n - Q + i
                first = max(0, last + 1 - case["window"]) if case["window"] else 0
                if last < 0:
                    continue
                z = q[b, i, h] @ kh[first:last + 1].t().contiguous() / math.sqrt(D)
                w = torch.exp(z - z.max(1, keepdim=True).values)
                o = w @ vh[first:last + 1] / w.sum(1, keepdim=True)
                out[b, i, h * (Hq // Hkv):(h + 1) * (Hq // Hkv)] = o
    return out.view(B * Q, Hq, D)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm":
        return _exact_norm(s, case)
    if case["op"] == "append":
        return _exact_append(s, case)
    if case["op"] == "attn":
        return _exact_attn(s, case)
    return None   # whole numbers only: they have to be equal
