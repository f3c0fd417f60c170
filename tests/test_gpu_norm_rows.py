"""RMS norm over many rows (1024 and more, where a row takes fewer threads)
and at the edges of its 8-bit scales: every row, scale and code against the
64-bit form, with residuals of both types, in place too."""
import pytest
import torch

import nvfp4_block_scaled_gemv_amd as nv
from decode_ref import E2M1, rmsnorm
from gpu_util import DEV, say
from test_gpu_norm import BF16, EPS, F32, F32_STEPS

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M", [1, 1025])
@pytest.mark.parametrize("H,group", [(64, 32), (192, 64), (256, 128), (4096, 32)])
def test_e4m3_values_too_small_for_a_scale(M, H, group):
    """A group whose largest |y| is so small that a 448th of it is zero in fp32
    has the scale 1 and zeros, not 0 / 0."""
    say(f"[norm e4m3 tiny] M={M} H={H} group={group}")
    x = torch.zeros(M, H, device=DEV)
    x[:, ::2] = 1.0
    w = torch.zeros(H, dtype=BF16, device=DEV)
    w[group:] = 2.0 ** -133               # the smallest bf16
    w[2 * group:] = 0
    x[:, group + 2:2 * group] = 2.0 ** -13
    x[:, group + 1:2 * group:2] = 0
    x[:, group] = 2.0 ** -13
    y8, sc, _ = nv.add_rmsnorm_e4m3(x, w, EPS, group=group)
    y, _ = rmsnorm(x, w, EPS)
    tiny = y[:, group:2 * group]
    assert 0 < float(tiny.max()) < 448 * 2.0 ** -151
    assert torch.all(sc == 1)             # this group, and those of zeros
    assert torch.all(y8.float() == 0)


def check_residual(out, s, rt):
    if rt is None:
        assert out is None
        return
    # one fp32 addition, then one rounding to the type
    tol = s.abs() * (2.0 ** -24 + (2.0 ** -8 if rt is BF16 else 0)) + 1e-37
    assert torch.all((out.double() - s).abs() <= tol)


def check_e4m3(y8, sc, y, n):
    """Scales and the values that the bytes stand for: half a step of E4M3
    (2^-4 relative, 2^-10 among its subnormal numbers) around y / scale, which
    fp32 leaves within F32_STEPS each for y, the scale and the quotient."""
    blocks = y.view(y.shape[0], -1, n)
    scale = blocks.abs().amax(-1) / 448
    assert torch.all((sc.double() - scale).abs() <= scale * (F32_STEPS + 2.0 ** -24))
    t = blocks / scale[..., None]
    tol = torch.maximum(t.abs() * 2.0 ** -4, torch.full((), 2.0 ** -10, device=DEV).double())
    assert torch.all((y8.float().double().view_as(t) - t).abs() <= tol + t.abs() * 3 * F32_STEPS)


def check_nvfp4(codes, sc, y, g):
    """Block scales within half a step of E4M3 of max|y| / (6 g), and E2M1 codes
    within half a step of y / (scale g) under the block's own scale."""
    blocks = y.view(y.shape[0], -1, 16)
    s = sc.view(torch.float8_e4m3fn).float().double()
    ratio = (blocks.abs().amax(-1) / (6 * g)).clamp(max=448)
    tol = torch.maximum(ratio * 2.0 ** -4, torch.full((), 2.0 ** -10, device=DEV).double())
    assert torch.all((s - ratio).abs() <= tol + ratio * 3 * F32_STEPS)
    nib = torch.stack([codes & 15, codes >> 4], -1).view_as(blocks).long()
    val = torch.tensor(E2M1, device=DEV)[nib & 7] * torch.where(nib & 8 > 0, -1.0, 1.0)
    t = torch.where(s[..., None] > 0, blocks / (s[..., None] * g).clamp(min=1e-300),
                    torch.zeros_like(blocks))
    a = t.abs()
    half = torch.where(a <= 2, 0.25, torch.where(a <= 4, 0.5, 1.0)).double()
    assert torch.all((val - t).abs() <= half + (a - 6).clamp(min=0) + a * 3 * F32_STEPS)


# from 1024, 2048 or 4096 rows on, by the types, fewer threads take a row
@pytest.mark.parametrize("M,H", [(1023, 4096), (1024, 2048), (1027, 4096), (1024, 7168),
                                 (2048, 8192), (1031, 16384), (4097, 4096), (4096, 8224)])
@pytest.mark.parametrize("xt,rt,in_place", [(F32, None, False), (F32, BF16, False),
                                            (BF16, F32, True), (F32, BF16, True), (F32, F32, False)])
def test_many_rows_in_every_form(M, H, xt, rt, in_place):
    """Rows of other sizes side by side, so that a row or block in another's
    place would show."""
    say(f"[norm rows] M={M} H={H} {xt} {rt} in_place={in_place}")
    g = torch.Generator(DEV).manual_seed(M + H)
    x = (torch.randn(M, H, device=DEV, generator=g) *
         torch.exp2(torch.randint(-3, 4, (M, 1), device=DEV, generator=g))).to(xt)
    w = (1 + 0.3 * torch.randn(H, device=DEV, generator=g)).to(BF16)
    r = None if rt is None else (2 * torch.randn(M, H, device=DEV, generator=g)).to(rt)
    y, s = rmsnorm(x, w, EPS, r)

    def call(f, *outs):
        rr = None if r is None else r.clone()
        ro = rr if in_place else None if r is None else torch.empty_like(r)
        f(x, w, EPS, *outs, residual=rr, residual_out=ro)
        check_residual(ro, s, rt)

    out = torch.empty(M, H, dtype=BF16, device=DEV)
    call(nv.add_rmsnorm_into, out)
    assert torch.all((out.double() - y).abs() <= y.abs() * (2.0 ** -8 + F32_STEPS) + 1e-37)
    for n in (H, 128, 32) if H % 128 == 0 else (H, 32):
        y8 = torch.empty(M, H, dtype=torch.float8_e4m3fn, device=DEV)
        sc = torch.empty(M, H // n, device=DEV)
        call(nv.add_rmsnorm_e4m3_into, y8, sc)
        check_e4m3(y8, sc, y, n)
    gs = torch.full((1,), 4.5 / 2688, device=DEV)
    codes = torch.empty(M, H // 2, dtype=torch.uint8, device=DEV)
    sc = torch.empty(M, H // 16, dtype=torch.uint8, device=DEV)
    call(nv.add_rmsnorm_nvfp4_into, gs, codes, sc)
    check_nvfp4(codes, sc, y, float(gs))
