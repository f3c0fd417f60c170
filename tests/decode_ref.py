"""Plain 64-bit forms of the operators of a decode step between the GEMVs, on
the CPU, and their inputs. Written from the formulas of the header, token by
token and head by head; the tests compare the kernels with them."""
import math

import numpy as np
import torch

E4M3_MAX = 448.0
E2M1 = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])


def gen(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


def normal(g, *shape, std=1.0, dtype=torch.float32):
    return (torch.randn(*shape, generator=g) * std).to(dtype)


def rmsnorm(x, weight, eps, residual=None):
    """(y, s) in 64 bits."""
    s = x.double()
    if residual is not None:
        s = s + residual.double()
    y = s / (s.pow(2).mean(-1, keepdim=True) + eps).sqrt() * weight.double()
    return y, s


def inv_freq(R, base=1e6):
    i = torch.arange(0, R, 2, dtype=torch.float64)
    return (base ** (-i / R)).float()


def rotate(x, positions, freq, interleaved, scale=1.0):
    """x [T, heads, D] turned, in 64 bits."""
    y = x.double().clone()
    R = 2 * freq.numel()
    a = positions.double()[:, None, None] * freq.double()
    c, s = a.cos() * scale, a.sin() * scale
    i0 = torch.arange(0, R, 2) if interleaved else torch.arange(R // 2)
    i1 = i0 + (1 if interleaved else R // 2)
    x0, x1 = x.double()[..., i0], x.double()[..., i1]
    y[..., i0] = x0 * c - x1 * s
    y[..., i1] = x1 * c + x0 * s
    return y


def attention(q, k_cache, v_cache, table, lens, scale, window=0, k_scale=1.0, v_scale=1.0):
    """out [T, Hq, D] in 64 bits, one (token, head) at a time over the keys that
    it sees (those of pages that exist)."""
    T, Hq, D = q.shape
    nb, page, Hkv, _ = k_cache.shape
    B, width = table.shape
    Q, G = T // B, Hq // Hkv
    kc, vc = k_cache.double() * k_scale, v_cache.double() * v_scale
    out = torch.zeros(T, Hq, D, dtype=torch.float64)
    for b in range(B):
        n = min(max(int(lens[b]), 0), width * page)
        for i in range(Q):
            p = n - Q + i
            lo = max(0, p - window + 1) if window else 0
            keys = [j for j in range(lo, p + 1) if 0 <= int(table[b, j // page]) < nb]
            if not keys:
                continue
            at = torch.tensor(keys)
            pages, places = table[b].long()[at // page], at % page
            for h in range(Hkv):
                kh, vh = kc[pages, places, h], vc[pages, places, h]
                z = scale * (q[b * Q + i, h * G:(h + 1) * G].double() @ kh.T)
                w = torch.exp(z - z.max(-1, keepdim=True).values)
                out[b * Q + i, h * G:(h + 1) * G] = (w @ vh) / w.sum(-1, keepdim=True)
    return out


def verify(p, q, draft, u_accept, u_sample, n_draft=None):
    """(tokens, accepted, margin): margin is how near a comparison came to its
    border, relative to the sums compared."""
    B, Q1, V = p.shape
    Q = Q1 - 1
    p = p.double().numpy()
    q = None if q is None else q.double().numpy()
    tokens, accepted, margin = np.full((B, Q1), -1, np.int32), np.zeros(B, np.int32), math.inf
    for b in range(B):
        nd = Q if n_draft is None else min(max(int(n_draft[b]), 0), Q)
        n = 0
        while n < nd:
            d = int(draft[b, n])
            if not 0 <= d < V:
                break
            qd = 1.0 if q is None else q[b, n, d]
            if not float(u_accept[b, n]) * qd < p[b, n, d]:
                break
            tokens[b, n] = d
            n += 1
        r = p[b, n].copy()
        if n < nd and q is not None:
            r = np.maximum(r - q[b, n], 0)
        elif n < nd and 0 <= int(draft[b, n]) < V:
            r[int(draft[b, n])] = 0
        if not r.sum() > 0:
            r = p[b, n]
        c = np.array([math.fsum([x]) for x in np.cumsum(r.astype(np.longdouble))])
        target = float(u_sample[b]) * c[-1]
        hit = np.nonzero(c > target)[0]
        tokens[b, n] = hit[0] if len(hit) else V - 1
        accepted[b] = n
        if c[-1] > 0:
            margin = min(margin, float(np.min(np.abs(c[r > 0] - target)) / c[-1]))
    return tokens, accepted, margin
