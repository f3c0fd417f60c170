"""Attention over a paged NVFP4 cache on the GPU against a plain 64-bit form:
head layouts and sizes, pages that fit tiles and that do not, several new
tokens, windows, caps and biases, lengths from zero to many workgroups per
sequence, missing pages, and what no token sees."""
import pytest
import torch

import nvfp4_block_scaled_gemv_amd as nv
from gpu_util import DEV, say
from serving_ref import attention, build4, decode4, place4, slopes_of

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


def run(q, cache, table, lens, **kw):
    out = nv.paged_attention_nvfp4(q.to(DEV), *cache, table.to(DEV), lens.to(DEV), **kw)
    torch.cuda.synchronize()
    return out.cpu().double()


def check(got, q, parts, table, lens, scale=None, window=0, softcap=0.0, slopes=None):
    """The bound. Scores: D exact products summed in fp32, off by at most 2 D
    2^-24 |q| |k| scale; the cap adds 2^-21 of them, the scale's products, the bias
    and the factors of log2 six roundings of 2^-24: 2^-20 of the largest in all. q enters
    within 2^-39 of its largest element, far below the sums' 2^-24. A weight is
    off by twice the score's error and 2^-24 (its two fp16), or 2^-36 of the
    row's largest: sum_j 2^-36 |v_j| in all, the sum of weights being at least
    the largest. Sums over the keys in fp32 add 2^-24 per addition of the longest
    chain, taken as 2^-14. The output is rounded by 2^-8 of it."""
    D = q.shape[-1]
    scale = D ** -0.5 if scale is None else scale
    k, v = (decode4(*p) for p in parts)
    k, v = torch.nan_to_num(k), torch.nan_to_num(v)   # where NaN, not compared
    top = [0.0]

    def weigh(z, w, vh):
        top[0] = max(top[0], float(z.abs().max()))
    ref = attention(q, k, v, table, lens, scale, window, softcap, slopes, weigh)
    a = attention(q, k, v.abs(), table, lens, scale, window, softcap, slopes)
    size = float(q.double().norm(dim=-1).max() * k.norm(dim=-1).max()) * abs(scale)
    dz = 2 * D * 2.0 ** -24 * size + 2.0 ** -20 * top[0]
    n = min(int(lens.max()), table.shape[1] * parts[0][0].shape[1])
    tol = a * (2 * dz + 2.0 ** -24 + 2.0 ** -14) + n * 2.0 ** -36 * float(v.abs().max()) \
        + ref.abs() * 2.0 ** -8 + 1e-30
    err = (got - ref).abs()
    bad = ~(err <= tol)
    assert not bad.any(), (int(bad.sum()), float((err / tol).max()), torch.nonzero(bad)[0].tolist())
    return float((err / tol).max())


CASES = [
    # lens, Q, Hq, Hkv, D, page, window, order, softcap, bias
    ([1], 1, 4, 1, 64, 16, 0, "nhd", 0.0, False),
    ([33], 1, 32, 8, 128, 16, 0, "nhd", 0.0, False),
    ([700], 1, 32, 8, 128, 16, 0, "nhd", 0.0, False),
    ([700], 1, 32, 8, 128, 16, 0, "hnd", 30.0, True),
    ([5000], 1, 8, 2, 128, 256, 0, "beside", 0.0, False),
    ([129, 0, 1, 64, 128, 500, 31], 1, 8, 2, 64, 32, 0, "nhd", 0.0, False),
    ([1000, 3, 777], 5, 32, 8, 128, 64, 0, "nhd", 0.0, False),
    ([1000, 3, 777], 5, 32, 8, 128, 64, 0, "wide", 0.0, True),
    ([300, 2], 3, 16, 16, 64, 20, 100, "nhd", 0.0, False),
    ([300, 2], 3, 16, 16, 64, 20, 7, "hnd", 4.0, False),
    ([260, 515], 2, 4, 4, 256, 16, 0, "nhd", 0.0, False),
    ([260, 515], 2, 4, 4, 256, 1, 0, "nhd", 0.0, False),
    ([97, 200], 1, 6, 2, 128, 1, 0, "hnd", 0.0, True),
    ([97, 200], 8, 8, 1, 128, 7, 0, "nhd", 0.0, False),
    ([150], 5, 16, 1, 256, 48, 0, "wide", 0.0, False),
    ([400, 90, 1], 1, 64, 1, 64, 16, 33, "nhd", 0.0, False),
    ([150, 1300], 5, 16, 2, 256, 20, 0, "nhd", 10.0, True),
    ([150, 1300], 5, 16, 2, 256, 16, 90, "hnd", 0.0, False),
    ([700, 20], 3, 32, 2, 128, 3, 0, "nhd", 0.0, False),
    ([1025, 513, 512], 1, 8, 8, 128, 16, 0, "hnd", 0.0, False),
    ([63] * 70, 1, 2, 1, 64, 16, 0, "nhd", 0.0, False),
    ([1, 2, 3, 4, 5, 6, 7, 8] * 17, 2, 4, 2, 64, 16, 0, "beside", 0.0, False),
    ([2049], 64, 1, 1, 64, 128, 500, "nhd", 0.0, False),
    ([40000], 1, 5, 1, 64, 16, 0, "nhd", 0.0, False),
]


@pytest.mark.parametrize("lens,Q,Hq,Hkv,D,page,window,order,cap,bias", CASES)
def test_attention(lens, Q, Hq, Hkv, D, page, window, order, cap, bias):
    say(f"[attn4] lens={lens[:8]} x{len(lens)} Q={Q} Hq={Hq} Hkv={Hkv} D={D} page={page} "
        f"window={window} {order} cap={cap} bias={bias}")
    q, table, ln, parts = build4(lens, Q, Hq, Hkv, D, page, seed=D + page)
    slopes = slopes_of(Hq) if bias else None
    got = run(q, place4(parts, order, DEV), table, ln, window=window, softcap=cap,
              slopes=None if slopes is None else slopes.to(DEV))
    r = check(got, q, parts, table, ln, None, window, cap, slopes)
    say(f"  max err / tol = {r:.3f}")


WIDE_CASES = [
    # lens, Q, Hq, Hkv, D, page, window, order, softcap, bias: rows of a head that fit
    # beside another's, tables of 2^18 keys of all heads and more
    ([1], 1, 2, 2, 64, 16, 0, "nhd", 0.0, False),
    ([700, 33, 0, 64], 1, 32, 8, 128, 16, 0, "nhd", 0.0, False),
    ([700, 33, 0, 64], 1, 32, 8, 128, 64, 0, "hnd", 20.0, True),
    ([129, 5000], 1, 16, 2, 128, 256, 0, "beside", 0.0, False),   # 8 rows
    ([1000, 3, 777], 2, 16, 4, 128, 32, 0, "wide", 0.0, True),    # 8 rows, two tokens
    ([300, 2, 95], 3, 4, 4, 64, 20, 100, "nhd", 0.0, False),
    ([300, 2, 95], 8, 2, 2, 64, 7, 30, "hnd", 4.0, False),
    ([260, 515], 2, 12, 4, 256, 16, 0, "nhd", 0.0, False),
    ([260, 515], 1, 14, 2, 256, 20, 0, "wide", 0.0, True),
    ([97, 200], 5, 6, 6, 256, 64, 48, "beside", 0.0, False),
    ([63] * 70, 1, 4, 4, 64, 16, 0, "nhd", 0.0, False),
    ([20000, 17], 1, 8, 2, 128, 16, 0, "nhd", 0.0, False),
    ([20000, 17], 1, 8, 2, 128, 1, 0, "nhd", 0.0, True),
    # and rows that do not: one head a wavefront on the same tables
    ([700, 33], 1, 18, 2, 128, 16, 0, "nhd", 0.0, False),
    ([700, 33], 1, 3, 3, 128, 64, 0, "nhd", 0.0, False),
    ([700, 1033], 5, 32, 8, 128, 32, 600, "hnd", 0.0, False),
]


@pytest.mark.parametrize("lens,Q,Hq,Hkv,D,page,window,order,cap,bias", WIDE_CASES)
def test_wide_tables(lens, Q, Hq, Hkv, D, page, window, order, cap, bias):
    say(f"[attn4 wide] lens={lens[:8]} x{len(lens)} Q={Q} Hq={Hq} Hkv={Hkv} D={D} page={page} "
        f"window={window} {order} cap={cap} bias={bias}")
    q, table, ln, parts = build4(lens, Q, Hq, Hkv, D, page, seed=D + page + 1)
    width = -(-(1 << 18) // (len(lens) * Hkv * page)) + 1
    table = torch.cat([table, torch.full((len(lens), max(0, width - table.shape[1])), -5,
                                         dtype=torch.int32)], 1)
    slopes = slopes_of(Hq) if bias else None
    got = run(q, place4(parts, order, DEV), table, ln, window=window, softcap=cap,
              slopes=None if slopes is None else slopes.to(DEV))
    r = check(got, q, parts, table, ln, None, window, cap, slopes)
    say(f"  max err / tol = {r:.3f}")


@pytest.mark.parametrize("scale", [0.0, -0.3, 1e-38, -1e-30])
@pytest.mark.parametrize("width", [4, 40000])
def test_scales_of_any_sign(scale, width):
    """A negative factor turns the order of the keys, zero and the smallest make
    all that are seen alike; those that are not seen stay out."""
    q, table, ln, parts = build4([50, 3, 0], 2, 8, 2, 64, 16, seed=21)
    table = torch.cat([table, torch.full((3, width - table.shape[1] + 4), -1, dtype=torch.int32)], 1)
    got = run(q, place4(parts, "nhd", DEV), table, ln, scale=scale)
    check(got, q, parts, table, ln, scale)
    got = run(q, place4(parts, "nhd", DEV), table, ln, scale=scale, softcap=2.0)
    check(got, q, parts, table, ln, scale, 0, 2.0)


@pytest.mark.parametrize("D", [64, 128, 256])
def test_large_and_ascending_scores(D):
    """Scores of hundreds, and scores that grow from key to key: the reference of
    the exponentials moves by far more than the slack."""
    q, table, ln, parts = build4([900, 130], 1, 8, 2, D, 16, seed=5, q_std=40.0)
    cache = place4(parts, "nhd", DEV)
    got = run(q, cache, table, ln)
    check(got, q, parts, table, ln)
    # every element of key j is +-0.5 .. 6 times a scale that grows with j
    kc, ks, gk = parts[0]
    kc.fill_(0x22)                                       # 1.0
    for b, n in ((0, 900), (1, 130)):
        for j in range(n):
            ks[table[b, j // 16], j % 16] = 8 + j * 100 // n   # E4M3 bytes, ascending
    q = torch.full_like(q, 2.0)
    got = run(q, place4(parts, "nhd", DEV), table, ln)
    check(got, q, parts, table, ln)


@pytest.mark.parametrize("exponent", [-126, -60, 0, 60, 100])
def test_queries_of_any_size(exponent):
    """bf16's whole range in q: a row's power of two takes it into fp16 and back."""
    q, table, ln, parts = build4([200], 2, 8, 2, 128, 16, seed=6)
    q = (q.double() * 2.0 ** exponent).to(BF16)
    q[0, 0] = 0
    q[1, 1, 5] = 2.0 ** -130                             # below bf16's normal numbers
    scale = float(2.0 ** min(max(-exponent, -100), 100)) * 128 ** -0.5
    got = run(q, place4(parts, "nhd", DEV), table, ln, scale=scale)
    check(got, q, parts, table, ln, scale)


def test_small_elements_of_a_query_count():
    """An element 2^-30 of the row's largest, times a key that is zero where the
    largest is: the score is that element's alone."""
    q, table, ln, parts = build4([64], 1, 4, 1, 128, 16, seed=7)
    q.zero_()
    q[..., 0], q[..., 100] = 2.0 ** 20, 1.40625 * 2.0 ** -10
    kc = parts[0][0]
    kc[..., 0] = kc[..., 0] & 0xF0                        # element 0 of every key
    scale = 2.0 ** 10 * 4
    got = run(q, place4(parts, "nhd", DEV), table, ln, scale=scale)
    # the score is exact but for its factors: the bound with |q||k| of that element
    k, v = (decode4(*p) for p in parts)
    ref = attention(q, k, v, table, ln, scale)
    a = attention(q, k, v.abs(), table, ln, scale)
    assert torch.all((got - ref).abs() <= a * 2.0 ** -14 + ref.abs() * 2.0 ** -8)


@pytest.mark.parametrize("keys", [600, 5000])
def test_weights_of_24_bits(keys):
    """Many equal weights p that fp16 does not hold, against values that cancel
    all but 2^-11 of their sum: one fp16 of p would be off by up to 2^-12 of each,
    all the same way. Scores are one product each (q and k have one element), so
    a weight is off by 2^-20 at most (two roundings of a score of at most 6), two
    fp16 by 2^-24 more, sums over the keys by 2^-24 for each of at most 2^7
    additions in a chain: 2^-16 of sum p |v| in all, and the output's 2^-8."""
    q, table, ln, parts = build4([keys], 1, 2, 1, 128, 16, seed=8, gk=1.0, gv=1.0)
    q.zero_()
    q[..., 0] = 1.0
    for p in parts:
        p[0].zero_()
        p[1].fill_(0x38)                                  # 1.0
    order = table[0].long()
    j = torch.arange(keys)
    page, place = order[j // 16], j % 16
    w = float(torch.exp(torch.tensor(-1.5, dtype=torch.float64)))   # scores 0 and -1.5
    n1 = int(keys / (1 + w))
    low = torch.zeros(keys, dtype=torch.bool)
    low[torch.randperm(keys)[:n1]] = True
    kc, vc = parts[0][0], parts[1][0]
    kc[page[low], place[low], 0, 0] = 0xB                 # -1.5
    vc[page[low], place[low]] = 0x22                      # 1.0
    vc[page[~low], place[~low]] = 0xAA                    # -1.0
    got = run(q, place4(parts, "nhd", DEV), table, ln, scale=1.0)
    k, v = (decode4(*p) for p in parts)
    ref = attention(q, k, v, table, ln, 1.0)
    assert float(ref.abs().max()) < 2.0 ** -7
    assert torch.all((got - ref).abs() <= 2.0 ** -16 + ref.abs() * 2.0 ** -8)


@pytest.mark.parametrize("D,page,Q,Hkv", [(64, 16, 3, 2), (128, 5, 3, 2), (128, 16, 1, 1),
                                          (256, 16, 2, 2), (128, 32, 20, 1)])
@pytest.mark.parametrize("wide", [0, 3000, 60000])
def test_what_no_token_sees_does_not_reach_it(D, page, Q, Hkv, wide):
    """NaN scales and other codes behind each sequence, in pages that nobody has
    and before the window leave every row as it was, bit for bit; at the newest
    token they reach its own row only."""
    lens, window = [70, 37, 2], 20
    q, table, ln, parts = build4(lens, Q, 4 * Hkv, Hkv, D, page, seed=9)
    if wide:   # wider tables: the form for long sequences, with one head a wavefront and two
        table = torch.cat([table, torch.full((3, wide // page), -1, dtype=torch.int32)], 1)
    clean = run(q, place4(parts, "nhd", DEV), table, ln, window=window)
    check(clean, q, parts, table, ln, None, window)
    nb = parts[0][0].shape[0]
    seen = torch.zeros(nb, page, dtype=torch.bool)
    for b, n in enumerate(lens):
        for j in range(max(0, n - Q - window + 1), n):
            seen[table[b, j // page], j % page] = True
    for byte in (0x7F, 0xFF, 0x7E):
        dirty = [(c.clone(), s.clone(), g) for c, s, g in parts]
        for c, s, _ in dirty:
            c[~seen], s[~seen] = 0x9E, byte
        got = run(q, place4(dirty, "nhd", DEV), table, ln, window=window)
        assert torch.equal(got, clean)
        n = lens[0]
        for c, s, _ in dirty:
            s[table[0, (n - 1) // page], (n - 1) % page] = byte
        got = run(q, place4(dirty, "nhd", DEV), table, ln, window=window)
        assert torch.equal(got[:Q - 1], clean[:Q - 1]) and torch.equal(got[Q:], clean[Q:])
        if byte != 0x7E:
            assert torch.isnan(got[Q - 1]).all()


@pytest.mark.parametrize("wide", [0, 60000])
def test_nan_scale_stays_in_its_head_and_sequence(wide):
    q, table, ln, parts = build4([1500, 700, 90], 2, 4, 2, 128, 16, seed=11)
    table = torch.cat([table, torch.full((3, wide // 16), -1, dtype=torch.int32)], 1)
    clean = run(q, place4(parts, "nhd", DEV), table, ln)
    parts[1][1][table[1, 20], 3, 1, 5] = 0x7F            # dims 80 .. 95 of head 1
    got = run(q, place4(parts, "nhd", DEV), table, ln)
    assert torch.equal(got[:2], clean[:2]) and torch.equal(got[4:], clean[4:])
    assert torch.equal(got[2:4, :2], clean[2:4, :2])
    assert torch.isnan(got[2:4, 2:, 80:96]).all()
    # its dimensions, or all of them for those that see it
    same = got[2:4, 2:] == clean[2:4, 2:]
    assert torch.all(same | torch.isnan(got[2:4, 2:]))
    if not wide:
        assert torch.equal(got[2:4, 2:, :80], clean[2:4, 2:, :80])


@pytest.mark.parametrize("page", [16, 6])
@pytest.mark.parametrize("D,Q", [(64, 2), (128, 2), (256, 9)])
def test_missing_pages_and_lengths(page, D, Q):
    q, table, ln, parts = build4([200, 90, 40], Q, 8, 2, D, page, seed=3)
    nb = parts[0][0].shape[0]
    table[0, 2], table[0, 5], table[1, 0] = -1, nb, 0x7FFFFFFF
    table[2, :] = -0x80000000                            # a sequence with no page at all
    cache = place4(parts, "nhd", DEV)
    got = run(q, cache, table, ln)
    check(got, q, parts, table, ln)
    assert torch.all(got[2 * Q:] == 0)
    more = torch.cat([table, torch.full((3, 60000 // page), nb, dtype=torch.int32)], 1)
    got = run(q, cache, more, ln)                        # the form for long sequences
    check(got, q, parts, more, ln)
    assert torch.all(got[2 * Q:] == 0)
    ln = torch.tensor([1000000, -5, 0x7FFFFFFF], dtype=torch.int32)
    got = run(q, cache, table, ln)
    check(got, q, parts, table, ln)
    assert torch.all(got[Q:] == 0)


def test_no_pages_at_all():
    q = torch.ones(2, 4, 64, dtype=BF16, device=DEV)
    one, ln = torch.ones(1, device=DEV), torch.tensor([5, 9], dtype=torch.int32, device=DEV)

    def cache(nb):
        return [(torch.full((nb, 16, 2, 32), 0x22, dtype=torch.uint8, device=DEV),
                 torch.full((nb, 16, 2, 4), 0x38, dtype=torch.uint8, device=DEV), one)
                for _ in range(2)]
    out = nv.paged_attention_nvfp4(q, *cache(0), torch.zeros(2, 3, dtype=torch.int32, device=DEV),
                                   ln)
    assert torch.all(out == 0)
    out = nv.paged_attention_nvfp4(q, *cache(1), torch.zeros(2, 0, dtype=torch.int32, device=DEV),
                                   ln)
    assert torch.all(out == 0)


@pytest.mark.parametrize("lens", [[9000, 100, 4000], [12000, 100, 4000]])   # a head a wavefront, two
def test_the_same_bits_whatever_the_workspace_held(lens):
    q, table, ln, parts = build4(lens, 1, 32, 8, 128, 16, seed=6)
    cache = place4(parts, "nhd", DEV)
    n = nv.paged_attention_workspace_bytes(3, 1, 32, 8, 128)
    dq, dt, dl = q.to(DEV), table.to(DEV), ln.to(DEV)
    outs = []
    for fill in (0, 0x7F, 0xFF):
        ws = torch.full((n,), fill, dtype=torch.uint8, device=DEV)
        outs.append(nv.paged_attention_nvfp4(dq, *cache, dt, dl, workspace=ws))
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])
    check(outs[0].cpu().double(), q, parts, table, ln)


def test_codes_past_4_gib():
    """Pages whose byte offset passes 2^32, in codes: 90000 pages of 64 KiB."""
    nb, page, Hkv, D = 90000, 128, 8, 128
    q, table, ln, parts = build4([500], 1, 8, Hkv, D, page, seed=8, spare=0)
    ids = torch.tensor([[nb - 1, 0, nb // 2, 77777]], dtype=torch.int32)
    cache = []
    for c, s, g in parts:
        cd = torch.empty(nb, page, Hkv, D // 2, dtype=torch.uint8, device=DEV)
        sd = torch.empty(nb, page, Hkv, D // 16, dtype=torch.uint8, device=DEV)
        at = ids[0].long().to(DEV)
        cd[at], sd[at] = c[table[0].long()].to(DEV), s[table[0].long()].to(DEV)
        cache.append((cd, sd, torch.full((1,), g, device=DEV)))
    got = run(q, cache, ids, ln)
    check(got, q, parts, table, ln)


@pytest.mark.parametrize("page,D", [(65536, 64), (100000, 128), (65536, 256)])
@pytest.mark.parametrize("window", [1, 40, 700])
def test_windows_at_the_end(page, D, window):
    """Sequences of up to 2^31 - 1 keys whose table names the same pages over and
    over, seen through a window."""
    Q, nb = 3, 3
    blocks = (1 << 31) // page
    q, _, _, parts = build4([page * nb] * 1, Q, 4, 1, D, page, seed=D, spare=0)
    table = torch.arange(blocks, dtype=torch.int32).remainder(nb)[None].contiguous()
    for n in (0x7FFFFFFF, 0x7FFFFE01):
        ln = torch.tensor([n], dtype=torch.int32)
        got = run(q, place4(parts, "nhd", DEV), table, ln, window=window)
        check(got, q, parts, table, ln, None, window)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("width", [0, 20000])
def test_far_strides(D, width):
    """Tokens and heads hundreds of kilobytes to 32 MB apart: a tile's offsets come
    near 2^32 bytes."""
    q, table, ln, parts = build4([61], 2, 4, 2, D, 16, seed=31, spare=0)
    table = torch.cat([table, torch.full((1, width), -1, dtype=torch.int32)], 1)
    nb = parts[0][0].shape[0]
    cache = []
    for c, s, g in parts:
        far = []
        for x, token in ((c, 1 << 25), (s, (1 << 25) - 64)):
            n = x.shape[-1]
            raw = torch.empty(16 * token + 2 * 300000 * 16, dtype=torch.uint8, device=DEV)
            view = torch.as_strided(raw, (nb, 16, 2, n), (4096, token, 300000 * 16, 1))
            view.copy_(x)
            far.append(view)
        cache.append((*far, torch.full((1,), g, device=DEV)))
    got = run(q, cache, table, ln)
    check(got, q, parts, table, ln)
