"""Layer norm on the GPU against its definition in 64 bits.

Tolerances, with u = 2^-24 (fp32 unit roundoff) and t the unit roundoff of the stored type:
  * a row's sums run over at most 70 elements a lane and then a tree of 10 levels, a column's over
    at most 100 rows a lane group, 64 partial rows and 16 sums: both depths are below 256, so a
    sum is off by at most 256 u times the sum of its |terms|;
  * h = (x - mean) * rstd carries the rounding of x - mean: its terms count with
    rstd * (|x| + |mean|), not with |h|;
  * the stored result adds t times its magnitude."""
import pytest
import torch

import bwd_tbe_fwd_amd as tbe
from gpu_util import flush_print

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
UNIT = {torch.float32: U, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
LEAST = {torch.float32: 0.0, torch.float16: 2.0 ** -25, torch.bfloat16: 0.0}  # half a subnormal step
F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16


def rows_of(rows, width, dtype, seed, stride=None, shift=0.5):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, width, generator=g) + shift * torch.randn(rows, 1, generator=g)
    buf = torch.full((rows, stride or width), float("nan"), dtype=dtype)
    buf[:, :width] = x.to(dtype)
    return buf.cuda()[:, :width]


def vector(width, dtype, seed, shift):
    return (torch.randn(width, generator=torch.Generator().manual_seed(seed)) * 0.3 + shift).to(dtype).cuda()


def check(what, got, exp, tol):
    got, exp, tol = got.double().cpu(), exp.double().cpu(), tol.double().cpu()
    bad = ~((got - exp).abs() <= tol)
    bad &= ~(got.isnan() & exp.isnan())
    if bad.any():
        i = tuple(bad.nonzero()[0].tolist())
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} off; first at {i}: {got[i]!r}, "
                             f"exact {exp[i]!r}, tolerance {tol[i]!r}")


def check_forward(x, w, b, eps, y, mean, rstd):
    xd = x.double()
    m = xd.mean(1, keepdim=True)
    r = 1 / ((xd - m).square().mean(1, keepdim=True) + eps).sqrt()
    wd = torch.ones_like(xd[0]) if w is None else w.double()
    bd = torch.zeros_like(xd[0]) if b is None else b.double()
    exp = (xd - m) * r * wd + bd
    top = xd.abs().amax(1, keepdim=True)
    mean_tol = 256 * U * xd.abs().mean(1, keepdim=True)
    # squares of deviations that are each off by u |x|, their sum off by 256 u
    rstd_rel = U * (260 + 4 * top * r)
    if mean is not None:
        check("mean", mean, m[:, 0], mean_tol[:, 0])
        check("rstd", rstd, r[:, 0], (rstd_rel * r)[:, 0])
    tol = UNIT[y.dtype] * exp.abs() + LEAST[y.dtype] + wd.abs() * r * (mean_tol + 4 * U * top) + \
        (rstd_rel + 4 * U) * ((xd - m) * r * wd).abs() + 2 * U * (exp.abs() + bd.abs())
    check("y", y, exp, tol)


def run_forward(rows, width, xt, yt, wt=F32, stride=None, eps=1e-5, weight=True, bias=True, stats=True, seed=1, shift=0.5):
    x = rows_of(rows, width, xt, seed, stride, shift)
    w = vector(width, wt, seed + 1, 1.0) if weight else None
    b = vector(width, wt, seed + 2, 0.0) if bias else None
    y = torch.full((rows, (stride or width) + 3), float("nan"), dtype=yt, device="cuda")
    mean, rstd = (torch.full((rows,), float("nan"), device="cuda") if stats else None for _ in range(2))
    tbe.tbe_layer_norm_forward(x, w, b, eps, y[:, 1:1 + width], mean, rstd)
    torch.cuda.synchronize()
    assert torch.isnan(y[:, 0]).all() and torch.isnan(y[:, 1 + width:]).all(), "wrote beside the rows"
    check_forward(x, w, b, eps, y[:, 1:1 + width], mean, rstd)


@pytest.mark.parametrize("xt", [F32, F16, BF16])
@pytest.mark.parametrize("yt", [F32, F16, BF16])
@pytest.mark.parametrize("width", [1, 7, 64, 130, 1001, 4096])
def test_forward(xt, yt, width):
    flush_print("norm forward", xt, yt, width)
    run_forward(67, width, xt, yt)


# every width at which the lanes or vectors of a row change, and one to each side of it
@pytest.mark.parametrize("xt", [F32, BF16])
@pytest.mark.parametrize("vectors", [16, 32, 64, 128, 256, 512, 1024, 2048, 4096])
def test_forward_widths(xt, vectors):
    edge = vectors * (4 if xt == F32 else 8)
    for width in (edge - 1, edge, edge + 1):
        flush_print("norm forward", xt, width)
        run_forward(9, width, xt, xt, wt=xt, seed=width)


def test_forward_rows_and_options():
    for rows in (1, 3, 15, 16, 17, 5000):
        flush_print("norm forward rows", rows)
        run_forward(rows, 96, BF16, BF16, seed=rows)
    run_forward(33, 200, F32, BF16, stride=211)
    run_forward(33, 200, BF16, F32, weight=False)
    run_forward(33, 200, F16, F16, wt=F16, bias=False)
    run_forward(33, 200, BF16, BF16, wt=BF16, weight=False, bias=False, stats=False)
    run_forward(12, 70001, F32, BF16)
    run_forward(12, 70001, BF16, BF16, wt=BF16, stride=70003)
    # a mean far above the deviations: taken off before the squares
    run_forward(40, 512, F32, F32, shift=3000.0)


# rows whose last vector overlaps the one before it, for each number of lanes and vectors
@pytest.mark.parametrize("xt,yt", [(F32, BF16), (BF16, BF16), (F16, F32), (F32, F32)])
@pytest.mark.parametrize("width", [3, 5, 9, 100, 361, 1100, 1535, 2100, 3071, 5001, 9001, 12287, 14001])
def test_ragged_widths(xt, yt, width):
    flush_print("norm ragged", xt, yt, width)
    run_forward(37, width, xt, yt, stride=width + 8 - width % 8, seed=width)
    run_backward(37, width, xt, yt, seed=width)


@pytest.mark.parametrize("width", [7, 131, 1001, 2047, 9001])
def test_ragged_in_place(width):
    for xt in (F32, BF16):
        x = rows_of(1100, width, xt, 3)
        w, b = vector(width, F32, 4, 1.0), vector(width, F32, 5, 0.0)
        y = torch.empty_like(x)
        tbe.tbe_layer_norm_forward(x, w, b, 1e-5, y)
        tbe.tbe_layer_norm_forward(x, w, b, 1e-5, x)
        assert torch.equal(x, y)


def test_no_rows_and_in_place():
    e = torch.empty(0, 64, device="cuda")
    tbe.tbe_layer_norm_forward(e, None, None, 1e-5, e, torch.empty(0, device="cuda"), torch.empty(0, device="cuda"))
    for width in (48, 3000, 40000):
        x = rows_of(20, width, BF16, 3)
        w, b = vector(width, F32, 4, 1.0), vector(width, F32, 5, 0.0)
        y = torch.empty_like(x)
        tbe.tbe_layer_norm_forward(x, w, b, 1e-5, y)
        tbe.tbe_layer_norm_forward(x, w, b, 1e-5, x)
        assert torch.equal(x.view(torch.int16), y.view(torch.int16))


def test_special_rows_stay_by_themselves():
    """A row with an infinity or a NaN gives NaN there and nowhere else; a constant row gives the shift."""
    for width in (8, 100, 1000, 5000, 40000):
        x = rows_of(40, width, F32, 6)
        x[3, width // 2] = float("inf")
        x[7, 0] = float("nan")
        x[11] = 2.5
        w, b = vector(width, F32, 7, 1.0), vector(width, F32, 8, 0.0)
        y = torch.empty_like(x)
        tbe.tbe_layer_norm_forward(x, w, b, 1e-5, y)
        bad = y.isnan().any(1).nonzero()[:, 0].tolist()
        assert bad == [3, 7] and y[7].isnan().all()
        assert torch.equal(y[11], b)
        gy = rows_of(40, width, F32, 9)
        gx, gw, gb, mean, rstd = run_backward_on(x, gy, w, 1e-5)
        assert gx.isnan().any(1).nonzero()[:, 0].tolist() == [3, 7]
        assert not gb.isnan().any() and gw.isnan().any()


# -------------------------------------------------------------------------------------------------
def run_backward_on(x, gy, w, eps, wt=F32, want=(True, True, True), pad=0, extra=0):
    rows, width = x.shape
    xf = x.float()
    mean = xf.mean(1)
    rstd = 1 / ((xf - mean[:, None]).square().mean(1) + eps).sqrt()
    buf = torch.full((rows, width + pad), float("nan"), dtype=x.dtype, device="cuda")
    gx = buf[:, :width] if want[0] else None
    gw = torch.full((width,), float("nan"), dtype=wt, device="cuda") if want[1] else None
    gb = torch.full((width,), float("nan"), dtype=wt, device="cuda") if want[2] else None
    ws = tbe.workspace(tbe.tbe_layer_norm_backward_workspace_bytes(rows, width) + extra)
    ws.view(torch.uint8).fill_(255)  # NaN where a partial is read but not written
    tbe.tbe_layer_norm_backward(x, gy, mean, rstd, w, gx, gw, gb, ws)
    torch.cuda.synchronize()
    assert pad == 0 or buf[:, width:].isnan().all()
    return gx, gw, gb, mean, rstd


def check_backward(x, gy, w, gx, gw, gb, mean, rstd):
    xd, gd, m, r = x.double(), gy.double(), mean.double()[:, None], rstd.double()[:, None]
    wd = torch.ones_like(xd[0]) if w is None else w.double()
    h, d = (xd - m) * r, gd * wd
    exp = r * (d - d.mean(1, keepdim=True) - h * (d * h).mean(1, keepdim=True))
    big_h, big_d = r * (xd.abs() + m.abs()), d.abs()
    if gx is not None:
        tol = UNIT[gx.dtype] * exp.abs() + LEAST[gx.dtype] + 256 * U * r * (
            big_d + big_d.mean(1, keepdim=True) + big_h * (big_d * big_h).mean(1, keepdim=True))
        check("grad_x", gx, exp, tol)
    if gw is not None:
        e = (gd * h).sum(0)
        check("grad_weight", gw, e, UNIT[gw.dtype] * e.abs() + LEAST[gw.dtype] + 256 * U * (gd.abs() * big_h).sum(0))
    if gb is not None:
        e = gd.sum(0)
        check("grad_bias", gb, e, UNIT[gb.dtype] * e.abs() + LEAST[gb.dtype] + 256 * U * gd.abs().sum(0))


def run_backward(rows, width, xt, yt, wt=F32, stride=None, weight=True, want=(True, True, True), seed=1, pad=0):
    x, gy = rows_of(rows, width, xt, seed, stride), rows_of(rows, width, yt, seed + 1, stride)
    w = vector(width, wt, seed + 2, 1.0) if weight else None
    check_backward(x, gy, w, *run_backward_on(x, gy, w, 1e-5, wt, want, pad))


@pytest.mark.parametrize("xt", [F32, F16, BF16])
@pytest.mark.parametrize("yt", [F32, F16, BF16])
@pytest.mark.parametrize("width", [1, 7, 64, 130, 1001, 4096])
def test_backward(xt, yt, width):
    flush_print("norm backward", xt, yt, width)
    run_backward(67, width, xt, yt, pad=5)


@pytest.mark.parametrize("xt", [F32, BF16])
@pytest.mark.parametrize("vectors", [16, 32, 64, 128, 256, 512, 1024, 2048, 4096])
def test_backward_widths(xt, vectors):
    edge = vectors * (4 if xt == F32 else 8)
    for width in (edge - 1, edge, edge + 1):
        flush_print("norm backward", xt, width)
        run_backward(9, width, xt, xt, wt=xt, seed=width)


def test_backward_rows_and_options():
    for rows in (1, 3, 15, 16, 17, 20000):
        flush_print("norm backward rows", rows)
        run_backward(rows, 96, BF16, BF16, seed=rows)
    run_backward(3000, 1500, F32, BF16, seed=5)
    run_backward(33, 200, F32, BF16, stride=211)
    run_backward(33, 200, BF16, F32, weight=False)
    for want in ((True, False, False), (False, True, False), (False, False, True), (True, True, False)):
        run_backward(33, 200, F16, F16, wt=F16, want=want)
        run_backward(5, 70001, BF16, BF16, wt=F32, want=want)
    run_backward(12, 70001, F32, BF16)


def test_backward_without_rows_is_zero():
    x = torch.empty(0, 40, device="cuda")
    gw, gb = (torch.full((40,), 3.0, device="cuda") for _ in range(2))
    s = torch.empty(0, device="cuda")
    tbe.tbe_layer_norm_backward(x, x, s, s, None, x, gw, gb, None)
    assert not gw.any() and not gb.any()


def test_backward_repeats_bit_for_bit():
    x, gy = rows_of(7001, 520, BF16, 11), rows_of(7001, 520, BF16, 12)
    w = vector(520, F32, 13, 1.0)
    a, b = run_backward_on(x, gy, w, 1e-5), run_backward_on(x, gy, w, 1e-5)
    for p, q in zip(a, b):
        assert torch.equal(p, q)


def test_backward_against_differences():
    """The gradients' products with a direction against the change of <gy, y> along it, in 64 bits."""
    x, gy = rows_of(6, 300, F32, 21), rows_of(6, 300, F32, 22)
    w, b = vector(300, F32, 23, 1.0), vector(300, F32, 24, 0.0)
    gx, gw, gb, _, _ = run_backward_on(x, gy, w, 1e-5)
    dx, dw, db = rows_of(6, 300, F32, 25), vector(300, F32, 26, 0.0), vector(300, F32, 27, 0.0)

    def loss(h):
        xd, wd, bd = x.double() + h * dx.double(), w.double() + h * dw.double(), b.double() + h * db.double()
        m = xd.mean(1, keepdim=True)
        return (gy.double() * ((xd - m) / ((xd - m).square().mean(1, keepdim=True) + 1e-5).sqrt() * wd + bd)).sum()

    h = 1e-5
    change = (loss(h) - loss(-h)) / (2 * h)
    terms = [gx.double() * dx.double(), gw.double() * dw.double(), gb.double() * db.double()]
    # fp32 gradients, 256 u of their terms; the difference's own error is h^2 and 2^-53 / h
    size = float(sum(t.abs().sum() for t in terms))
    assert abs(float(change - sum(t.sum() for t in terms))) <= (256 * U + 1e-8) * size


def test_norm_on_a_side_stream_and_in_a_graph():
    x, gy = rows_of(300, 700, F32, 31), rows_of(300, 700, BF16, 32)
    w, b = vector(700, F32, 33, 1.0), vector(700, F32, 34, 0.0)
    y = torch.empty(300, 700, dtype=BF16, device="cuda")
    mean, rstd, gx = torch.empty(300, device="cuda"), torch.empty(300, device="cuda"), torch.empty_like(x)
    gw, gb = torch.empty(700, device="cuda"), torch.empty(700, device="cuda")
    ws = tbe.workspace(tbe.tbe_layer_norm_backward_workspace_bytes(300, 700))

    def step():
        tbe.tbe_layer_norm_forward(x, w, b, 1e-5, y, mean, rstd)
        tbe.tbe_layer_norm_backward(x, gy, mean, rstd, w, gx, gw, gb, ws)

    outs = (y, mean, rstd, gx, gw, gb)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    eager = [t.clone() for t in outs]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    scratch = torch.randn(1 << 20, device="cuda")
    for k in range(3):
        for t in outs:
            t.zero_()
        g.replay()
        scratch.mul_(1.5).add_(float(k))
        torch.cuda.synchronize()
        for t, e in zip(outs, eager):
            assert torch.equal(t, e)
