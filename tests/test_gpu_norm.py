"""RMS norm with the residual's addition on the GPU against a plain 64-bit
form: bf16, E4M3 and NVFP4 outputs, every type of x and residual, rows of one
wavefront and of many, in place, odd row counts."""
import numpy as np
import pytest
import torch

import nvfp4_block_scaled_gemv_amd as nv
import oracle
from decode_ref import E2M1, gen, normal, rmsnorm
from gpu_util import DEV, say

pytestmark = pytest.mark.gpu

EPS = 1e-6
# fp32 arithmetic before the last rounding: the sum of H squares (at most 33
# sequential additions per lane, 6 + 16 across, each 2^-24 relative), the mean,
# the root, the division and two products: under 64 steps of 2^-24.
F32_STEPS = 64 * 2.0 ** -24
BF16 = torch.bfloat16
F32 = torch.float32

# (M, H): one wavefront per row (up to 512) with rows that leave a workgroup
# part empty, 2 to 16 wavefronts, two and four groups per lane, the largest row
SHAPES = [(1, 8), (5, 64), (7, 128), (4, 504), (3, 512), (2, 520), (3, 1000), (1, 4096), (2, 8192),
          (2, 8200), (1, 16384), (2, 16392), (1, 32768), (301, 128), (130, 2048)]


def case(M, H, xt, rt, seed):
    g = gen(seed)
    x = normal(g, M, H, std=0.7, dtype=xt)
    r = None if rt is None else normal(g, M, H, std=2.0, dtype=rt)
    w = (1 + normal(g, H, std=0.3)).to(BF16)
    return x, r, w


def dev(t):
    return None if t is None else t.to(DEV)


def check_residual(out, s, rt):
    if rt is None:
        assert out is None
        return
    got = out.cpu().double()
    # one fp32 addition, then one rounding to the type
    tol = s.abs() * (2.0 ** -24 + (2.0 ** -8 if rt is BF16 else 0)) + 1e-37
    assert torch.all((got - s).abs() <= tol)


@pytest.mark.parametrize("M,H", SHAPES)
@pytest.mark.parametrize("xt,rt", [(F32, BF16), (BF16, F32), (BF16, None), (F32, F32), (BF16, BF16),
                                   (F32, None)])
def test_bf16(M, H, xt, rt):
    say(f"[norm] M={M} H={H} {xt} {rt}")
    x, r, w = case(M, H, xt, rt, M * 7 + H)
    y, ro = nv.add_rmsnorm(dev(x), dev(w), EPS, dev(r))
    yr, s = rmsnorm(x, w, EPS, r)
    assert torch.all((y.cpu().double() - yr).abs() <= yr.abs() * (2.0 ** -8 + F32_STEPS) + 1e-37)
    check_residual(ro, s, rt)


@pytest.mark.parametrize("M,H,group", [(1, 64, 0), (3, 128, 128), (5, 192, 64), (2, 96, 32),
                                       (2, 4096, 0), (3, 4096, 128), (2, 7168, 64), (1, 16640, 128),
                                       (2, 32768, 0), (2, 20480, 32), (6, 512, 32), (3, 72, 0)])
@pytest.mark.parametrize("xt,rt", [(F32, BF16), (BF16, F32), (BF16, None)])
def test_e4m3(M, H, group, xt, rt):
    say(f"[norm e4m3] M={M} H={H} group={group} {xt} {rt}")
    x, r, w = case(M, H, xt, rt, M * 5 + H)
    y8, sc, ro = nv.add_rmsnorm_e4m3(dev(x), dev(w), EPS, dev(r), group=group)
    yr, s = rmsnorm(x, w, EPS, r)
    check_residual(ro, s, rt)
    n = group or H
    blocks = yr.view(M, H // n, n)
    scale = blocks.abs().amax(-1) / 448
    got = sc.cpu().double()
    assert torch.all((got - scale).abs() <= scale * (F32_STEPS + 2.0 ** -24))
    # the value that the byte stands for: half a step of E4M3 (2^-4 relative,
    # 2^-10 among its subnormal numbers) around y / scale, which is itself
    # rounded in fp32
    q = y8.cpu().float().double().view(M, H // n, n)
    t = blocks / scale[..., None]
    tol = torch.maximum(t.abs() * 2.0 ** -4, torch.tensor(2.0 ** -10, dtype=torch.float64))
    assert torch.all((q - t).abs() <= tol + t.abs() * 3 * F32_STEPS)
    assert torch.all(q.abs().amax(-1) == 448)       # the largest value of a group


@pytest.mark.parametrize("M,H", [(1, 32), (3, 64), (5, 512), (2, 544), (8, 4096), (2, 8224),
                                 (1, 16416), (1, 32768)])
@pytest.mark.parametrize("xt,rt", [(F32, BF16), (BF16, F32), (BF16, None)])
def test_nvfp4(M, H, xt, rt):
    say(f"[norm nvfp4] M={M} H={H} {xt} {rt}")
    x, r, w = case(M, H, xt, rt, M * 3 + H)
    g = 4.5 / 2688
    codes, sc, ro = nv.add_rmsnorm_nvfp4(dev(x), dev(w), EPS, torch.full((1,), g, device=DEV),
                                         dev(r))
    g = float(np.float32(g))
    yr, s = rmsnorm(x, w, EPS, r)
    check_residual(ro, s, rt)
    blocks = yr.view(M, H // 16, 16)
    sv = sc.cpu().view(torch.float8_e4m3fn).float().double()
    ratio = (blocks.abs().amax(-1) / (6 * g)).clamp(max=448)
    tol = torch.maximum(ratio * 2.0 ** -4, torch.tensor(2.0 ** -10, dtype=torch.float64))
    assert torch.all((sv - ratio).abs() <= tol + ratio * 3 * F32_STEPS)
    c = codes.cpu().numpy()
    nib = np.stack([c & 15, c >> 4], -1).reshape(M, H // 16, 16)
    val = torch.from_numpy(np.where(nib & 8, -1.0, 1.0) * E2M1[nib & 7])
    t = torch.where(sv[..., None] > 0, blocks / (sv[..., None] * g).clamp(min=1e-300),
                    torch.zeros_like(blocks))
    # E2M1: steps of 0.5 below 2, 1 below 4, 2 below 6, saturating
    a = t.abs()
    half = torch.where(a <= 2, 0.25, torch.where(a <= 4, 0.5, 1.0)).double()
    over = (a - 6).clamp(min=0)
    assert torch.all((val - t).abs() <= half + over + a * 3 * F32_STEPS)


@pytest.mark.parametrize("M,H", [(3, 256), (2, 4096)])
def test_nvfp4_equals_the_quantizer_on_exact_rows(M, H):
    """Where y is exact in bf16 the fused output is nvfp4_quantize_act's and
    the oracle's, bit for bit: rows of +-2^k with a mean square of 1."""
    say(f"[norm nvfp4 exact] M={M} H={H}")
    g = gen(H)
    x = torch.where(torch.rand(M, H, generator=g) < 0.5, -1.0, 1.0)
    w = (2.0 ** torch.randint(-3, 4, (H,), generator=g)).to(BF16)
    y = (x * w.float()).to(BF16)
    gs = torch.full((1,), 0.01, device=DEV)
    codes, sc, _ = nv.add_rmsnorm_nvfp4(dev(x), dev(w), 0.0, gs)
    c2, s2 = nv.quantize_act(dev(y), gs)
    assert torch.equal(codes, c2) and torch.equal(sc, s2)
    c3, s3 = oracle.quantize_act(y.view(torch.int16).numpy().view(np.uint16), np.float32(0.01))
    assert np.array_equal(codes.cpu().numpy(), c3) and np.array_equal(sc.cpu().numpy(), s3)


@pytest.mark.parametrize("rt", [BF16, F32])
def test_in_place_residual(rt):
    x, r, w = case(3, 4096, F32, rt, 11)
    y, ro = nv.add_rmsnorm(dev(x), dev(w), EPS, dev(r))
    rd = dev(r)
    y2 = torch.empty_like(y)
    nv.add_rmsnorm_into(dev(x), dev(w), EPS, y2, rd, rd)
    assert torch.equal(y, y2) and torch.equal(ro, rd)


def test_rows_do_not_touch_each_other():
    """A row's result does not depend on the rows beside it; a row of NaN, one
    with an infinity and one of zeros stay theirs."""
    x, r, w = case(6, 512, F32, None, 12)
    y, _ = nv.add_rmsnorm(dev(x), dev(w), EPS)
    x2 = x.clone()
    x2[1] = float("nan")
    x2[3, 100] = float("inf")
    x2[4] = 0.0
    y2, _ = nv.add_rmsnorm(dev(x2), dev(w), EPS)
    for i in (0, 2, 5):
        assert torch.equal(y[i], y2[i])
    assert torch.isnan(y2[1]).all() and torch.isnan(y2[3, 100])
    assert torch.all(y2[4] == 0)
    y8, sc, _ = nv.add_rmsnorm_e4m3(dev(x2), dev(w), EPS)
    assert torch.all(y8[4].float() == 0) and sc[4, 0] == 1
    assert torch.isnan(y8[1].float()).all()


def test_empty_calls():
    w = torch.ones(64, dtype=BF16, device=DEV)
    y, _ = nv.add_rmsnorm(torch.empty(0, 64, device=DEV), w, EPS)
    assert y.shape == (0, 64)


@pytest.mark.parametrize("M,H", [(70001, 64), (1024, 2056), (1025, 4104), (1500, 8192),
                                 (1030, 16640)])
def test_many_rows(M, H):
    """More rows than a grid of one round, the last workgroup part empty, and
    the shapes of 1024 rows and more."""
    x = torch.randn(M, H, device=DEV, generator=torch.Generator(DEV).manual_seed(3))
    w = (1 + 0.2 * torch.randn(H, device=DEV, generator=torch.Generator(DEV).manual_seed(4))).to(BF16)
    y, _ = nv.add_rmsnorm(x, w, EPS)
    yr, _ = rmsnorm(x, w, EPS)
    assert torch.all((y.double() - yr).abs() <= yr.abs() * (2.0 ** -8 + F32_STEPS) + 1e-37)
    if H % 128 == 0:
        y8, sc, _ = nv.add_rmsnorm_e4m3(x, w, EPS, group=128)
        t = yr.view(M, -1, 128)
        scale = t.abs().amax(-1, keepdim=True) / 448
        tol = torch.maximum((t / scale).abs() * 2.0 ** -4,
                            torch.tensor(2.0 ** -10, dtype=torch.float64, device=DEV))
        q = y8.float().double().view(M, -1, 128)
        assert torch.all((q - t / scale).abs() <= tol + (t / scale).abs() * 3 * F32_STEPS)
        one, s1, _ = nv.add_rmsnorm_nvfp4(x, w, EPS, torch.full((1,), 0.0017, device=DEV))
        few, s2, _ = nv.add_rmsnorm_nvfp4(x[:7].contiguous(), w, EPS,
                                          torch.full((1,), 0.0017, device=DEV))
        # fewer rows take another shape, whose sum may round the other way:
        # a code in a thousand may lie on the other side of a border
        assert float((one[:7] != few).float().mean()) < 1e-3
        assert float((s1[:7] != s2).float().mean()) < 1e-3


@pytest.mark.parametrize("M,H", [(1, 64), (3, 4096), (1100, 4096)])
@pytest.mark.parametrize("big", [1e6, 1e30, 3e38, float("inf")])
def test_nvfp4_saturates(M, H, big):
    """Values far above what the static scale covers take the largest code,
    whatever the quotient, infinite ones too."""
    x = torch.ones(M, H, device=DEV)
    x[:, 1::2] = -1
    w = torch.ones(H, dtype=BF16, device=DEV)
    w[16:32] = big
    q, s, _ = nv.add_rmsnorm_nvfp4(x, w, EPS, torch.full((1,), 2.0 ** -9, device=DEV))
    assert torch.all(s[:, 1] == 0x7E)
    assert torch.all(q.view(torch.uint8)[:, 8:16] == 0xF7)
    s1 = s[:, :1].clone()
    assert torch.all(s[:, 2:] == s1) and torch.all(s[:, 0] == s1[:, 0])
    assert torch.all(q.view(torch.uint8)[:, :8] == 0xF7)
