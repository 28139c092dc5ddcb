"""Layer norm on the GPU where the mean is large against the deviations.

Tolerances, with u = 2^-24.  The first mean is off by at most 256 u top (top: the
row's largest magnitude).  Deviations from it, each rounded by u of itself, give the correction of the
mean and the squares, their sums off by 256 u of the terms: the mean is then off by its own rounding
and 260 u of the mean deviation, the squares' mean by 264 u of itself, of which the square of the
correction is a part."""
import math

import pytest
import torch

import bwd_tbe_fwd_amd as tbe
from gpu_util import flush_print
from test_gpu_tower_norm import U, UNIT, check, vector

pytestmark = pytest.mark.gpu
F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16

WIDTHS = [5, 100, 128, 1000, 1024, 4096, 5000, 14001, 40000]


@pytest.mark.parametrize("dtype", [F32, F16])
@pytest.mark.parametrize("width", WIDTHS)
def test_constant_rows_give_the_shift(dtype, width):
    flush_print("norm of constant rows", dtype, width)
    values = torch.tensor([0.1, 0.3, 1 / 3, 0.7, -0.7, 3.3, 1000.1, -12345.6, 2.5, 0.0], device="cuda")
    x = values.to(dtype)[:, None].expand(-1, width).contiguous()
    w, b = vector(width, F32, 1, 1.0), vector(width, F32, 2, 0.0)
    for eps in (1e-5, 1e-12):
        y = torch.empty(x.shape, device="cuda")
        mean, rstd = torch.empty(len(x), device="cuda"), torch.empty(len(x), device="cuda")
        tbe.tbe_layer_norm_forward(x, w, b, eps, y, mean, rstd)
        assert torch.equal(mean, x[:, 0].float())
        assert torch.equal(y, b.expand_as(y))
        # the deviations' mean square is zero but for the rounding of the correction's square
        c = 256 * U * x[:, 0].double().abs()
        assert (rstd.double() <= (1 + 4 * U) / math.sqrt(eps)).all()
        assert (rstd.double() >= (1 - 4 * U) / (eps + 264 * U * c * c).sqrt()).all()


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("width", [131072, 1 << 20, 1 << 22])
def test_very_wide_constant_rows_give_the_shift(dtype, width):
    flush_print("norm of wide constant rows", dtype, width)
    x = torch.tensor([0.1, 1000.1, -12345.6], device="cuda").to(dtype)[:, None].expand(-1, width).contiguous()
    b = vector(width, F32, 2, 0.0)
    y = torch.empty(x.shape, device="cuda")
    tbe.tbe_layer_norm_forward(x, None, b, 1e-12, y)
    assert torch.equal(y, b.expand_as(y))


@pytest.mark.parametrize("yt", [F32, BF16])
@pytest.mark.parametrize("width", WIDTHS)
def test_means_far_above_the_deviations(yt, width):
    flush_print("norm of rows far from zero", yt, width)
    g = torch.Generator().manual_seed(width)
    scale = torch.tensor([1e-3, 1e-2, 1.0, 1e-3])[:, None]
    middle = torch.tensor([1000.0, -3.0, 1e5, 7.0])[:, None]
    x = (torch.randn(48, width, generator=g) * scale.repeat(12, 1) + middle.repeat(12, 1)).cuda()
    w, b = vector(width, F32, 1, 1.0), vector(width, F32, 2, 0.0)
    for eps in (1e-5, 1e-9):
        y = torch.empty(x.shape, dtype=yt, device="cuda")
        mean, rstd = torch.empty(48, device="cuda"), torch.empty(48, device="cuda")
        tbe.tbe_layer_norm_forward(x, w, b, eps, y, mean, rstd)
        xd, wd, bd = x.double(), w.double(), b.double()
        m = xd.mean(1, keepdim=True)
        var = (xd - m).square().mean(1, keepdim=True)
        r = 1 / (var + eps).sqrt()
        c = 256 * U * xd.abs().amax(1, keepdim=True)  # the first mean's error
        mean_tol = U * m.abs() + 260 * U * ((xd - m).abs().mean(1, keepdim=True) + c)
        rel = 264 * U * (var + c * c) * r * r + 4 * U
        check("mean", mean, m[:, 0], mean_tol[:, 0])
        check("rstd", rstd, r[:, 0], (rel * r)[:, 0])
        exp = (xd - m) * r * wd + bd
        tol = UNIT[yt] * exp.abs() + wd.abs() * r * mean_tol + (rel + 4 * U) * ((xd - m) * r * wd).abs() + \
            2 * U * (exp.abs() + bd.abs())
        check("y", y, exp, tol)
