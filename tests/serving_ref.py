"""Plain 64-bit forms of the NVFP4 cache, of attention with capped or biased
scores and of low-rank adapters, on the CPU, and their inputs. Written from the
formulas of the header; the tests compare the kernels with them."""
import numpy as np
import torch

import oracle
from decode_ref import gen, normal

BF16, E4M3 = torch.bfloat16, torch.float8_e4m3fn
_E2M1 = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, 0, -.5, -1, -1.5, -2, -3, -4, -6],
                     dtype=torch.float64)


def encode4(x, g):
    """x[..., D] fp32 in NVFP4 with the tensor scale g, by the oracle: (codes u8
    [..., D / 2], scales u8 [..., D / 16])."""
    D = x.shape[-1]
    c, s, _ = oracle.pack(x.reshape(-1, D).float().numpy(), np.float32(g))
    return (torch.from_numpy(c).view(*x.shape[:-1], D // 2),
            torch.from_numpy(s).view(*x.shape[:-1], D // 16))


def decode4(codes, scales, g):
    """The values of codes [..., D / 2] and scale bytes [..., D / 16], 64 bits."""
    c = codes.long()
    x = torch.stack([_E2M1[c & 15], _E2M1[c >> 4]], -1).flatten(-2)
    return x * scales.view(E4M3).double().repeat_interleave(16, -1) * float(np.float32(g))


def attention(q, kc, vc, table, lens, scale, window=0, softcap=0.0, slopes=None, weigh=None):
    """out [T, Hq, D] in 64 bits over caches [blocks, page, Hkv, D] of any type,
    one (token, key-value head) at a time over the keys it sees. weigh(z, w, v):
    called for each, with the final scores, the weights and the values."""
    T, Hq, D = q.shape
    nb, page, Hkv, _ = kc.shape
    B, width = table.shape
    Q, G = T // B, Hq // Hkv
    kc, vc = kc.double(), vc.double()
    out = torch.zeros(T, Hq, D, dtype=torch.float64)
    for b in range(B):
        n = min(max(int(lens[b]), 0), width * page)
        for i in range(Q):
            p = n - Q + i
            lo = max(0, p - window + 1) if window else 0
            at = torch.arange(lo, p + 1) if p >= lo else torch.zeros(0, dtype=torch.long)
            ids = table[b].long()[at // page]
            ok = (ids >= 0) & (ids < nb)
            at, ids = at[ok], ids[ok]
            if not len(at):
                continue
            places = at % page
            for h in range(Hkv):
                kh, vh = kc[ids, places, h], vc[ids, places, h]
                z = scale * (q[b * Q + i, h * G:(h + 1) * G].double() @ kh.T)
                if softcap:
                    z = softcap * torch.tanh(z / softcap)
                if slopes is not None:
                    z = z + slopes[h * G:(h + 1) * G, None].double() * (at - p).double()
                w = torch.exp(z - z.max(-1, keepdim=True).values)
                if weigh is not None:
                    weigh(z, w, vh)
                out[b * Q + i, h * G:(h + 1) * G] = (w @ vh) / w.sum(-1, keepdim=True)
    return out


def slopes_of(H):
    return (2.0 ** (-8.0 * torch.arange(1, H + 1, dtype=torch.float64) / H)).float()


def adapters(mats, x, ids, bases=None, alpha=None, ranks=None):
    """Per projection (y, bound): y in 64 bits, and what fp32 sums may be off by.
    t = A x of K products: 2 K 2^-24 sum |a x| (each product is exact, each of at
    most K additions rounds by 2^-24 of partial sums of at most sum |a x|, twice
    that for the inside of a matrix instruction). y: that through |B|, then 2
    rank 2^-24 of sum |B t| in the same way, and three roundings of alpha's
    product, the base's addition and y."""
    out = []
    for i, (a, b) in enumerate(mats):
        E, rank, K = a.shape
        N = b.shape[1]
        base = torch.zeros(x.shape[0], N, dtype=torch.float64) if bases is None \
            else bases[i].double()
        y, bound = base.clone(), base.abs() * 2.0 ** -24
        for m, e in enumerate(ids.tolist()):
            if not 0 <= e < E:
                continue
            r = rank if ranks is None else min(max(int(ranks[e]), 0), rank)
            f = 1.0 if alpha is None else float(alpha[e])
            ae, be, xm = a[e, :r].double(), b[e, :, :r].double(), x[m].double()
            t, size = ae @ xm, ae.abs() @ xm.abs()
            d = be @ t
            y[m] += f * d
            off = be.abs() @ (size * 2 * K * 2.0 ** -24) + (be.abs() @ t.abs()) * (
                2 * rank * 2.0 ** -24)
            bound[m] += abs(f) * (off + d.abs() * 2.0 ** -23) + y[m].abs() * 2.0 ** -23
        out.append((y, bound + 1e-38))
    return out


def build4(lens, Q, Hq, Hkv, D, page, order="nhd", seed=1, spare=3, gk=4.5 / 2688, gv=4.2 / 2688,
           q_std=1.0):
    """Inputs of attention over an NVFP4 cache: q, table, lens on the CPU, the
    cache's codes and scales (CPU, [blocks, page, Hkv, ..]) and its values in 64
    bits; every sequence's pages scattered, unused table entries out of range."""
    g = gen(seed)
    B = len(lens)
    used = [(max(n, 0) + page - 1) // page for n in lens]
    nb = sum(used) + spare
    perm = torch.randperm(nb, generator=g)
    table = torch.full((B, max(max(used), 1)), -7, dtype=torch.int32)
    at = 0
    for b, n in enumerate(used):
        table[b, :n] = perm[at:at + n].to(torch.int32)
        at += n
    q = normal(g, B * Q, Hq, D, std=q_std, dtype=BF16)
    parts = []
    for gs in (gk, gv):
        c, s = encode4(normal(g, nb, page, Hkv, D), gs)
        parts.append((c, s, gs))
    return q, table, torch.tensor(lens, dtype=torch.int32), parts


def place4(parts, order, device):
    """The cache's triples on the device, in a memory order: [page, heads, D],
    [heads, page, D], k's pages beside v's, or heads in a wider row."""
    def put(x, unit):
        nb, page, H, n = x[0].shape
        raw = torch.full((2, nb, H, page, n) if order == "hnd" else
                         (nb, 2, page, H, n) if order == "beside" else
                         (2, nb, page, H, n + unit) if order == "wide" else (2, nb, page, H, n),
                         0x7F, dtype=torch.uint8, device=device)
        k, v = (raw[:, 0], raw[:, 1]) if order == "beside" else (raw[0], raw[1])
        if order == "hnd":
            k, v = k.transpose(1, 2), v.transpose(1, 2)
        k, v = k[..., :n], v[..., :n]
        k.copy_(x[0])
        v.copy_(x[1])
        return k, v
    codes = put([p[0] for p in parts], 16)
    scales = put([p[1] for p in parts], 4)
    return tuple((c, s, torch.full((1,), p[2], device=device))
                 for c, s, p in zip(codes, scales, parts))
