"""Softmax cross entropy over all items, and its gradients, on the GPU against their definitions in 64 bits.

Tolerances, with u = 2^-24 and t the unit roundoff of the stored 16-bit type:
  * a logit is a sum of D exact products in fp32, off by at most (D + 4) u times s sum |x w| + |b| (call it e);
  * an exponential is off by its argument's rounding, 3 u |l - lse|, and 4 u; the sums of a row's V exponentials, all positive,
    have chains of fewer than 256 + V / 2048 additions; the logarithm and the last sum add 2 u |lse|;
  * z = p - [v = t] is off by p (e + 3 u |l - lse| + 4 u + 2 u |lse|), its rounding by t |z| (fp16: at least half a subnormal
    step over 2^15); sums of K products of it by K u times the sum of their magnitudes; x * g / largest is rounded by t |x g|
    (fp16: at least half a subnormal step times the largest); the result by t;
  * fp32 has nothing between 0 and 2^-149, and an exponential, a product or a sum below 2^-126 may become 0: each
    probability, each of the K products and the result count 2^-126 more (a probability of 1e-113 is 0 in 32 bits)."""
import pytest
import torch

import bwd_tbe_fwd_amd as tbe
from gpu_util import flush_print

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
F16, BF16 = torch.float16, torch.bfloat16
UNIT = {F16: 2.0 ** -11, BF16: 2.0 ** -8}
LEAST = {F16: 2.0 ** -25, BF16: 0.0}
INF = float("inf")
TINY = 2.0 ** -126


def matrix(rows, width, dtype, seed, scale=1.0, stride=None, offset=0):
    g = torch.Generator().manual_seed(seed)
    stride = stride or width
    buf = torch.full((offset + rows * stride,), float("nan"), dtype=dtype)
    buf[offset:].view(rows, stride)[:, :width].copy_(torch.randn(rows, width, generator=g) * scale)
    return buf.cuda()[offset:].view(rows, stride)[:, :width]


def some_targets(rows, items, pad, seed, dtype=torch.int64):
    g = torch.Generator().manual_seed(seed)
    t = torch.randint(0, items, (rows,), generator=g)
    t[torch.rand(rows, generator=g) < pad] = -1
    t[torch.rand(rows, generator=g) < pad / 3] = items
    return t.to(dtype).cuda()


def check(what, got, exp, tol):
    got, exp, tol = got.double(), exp.double(), tol.double()
    bad = ~((got - exp).abs() <= tol)
    bad &= ~((got == exp) | (got.isnan() & exp.isnan()))
    if bool(bad.any()):
        i = tuple(bad.nonzero()[0].tolist())
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} off; first at {i}: {got[i]!r}, exact {exp[i]!r}, "
                             f"tolerance {tol[i]!r}")


class Exact:
    """The definition in 64 bits, with what each value may be off by."""

    def __init__(self, x, w, bias, targets, scale):
        s = float(torch.tensor(scale, dtype=torch.float32))
        self.x, self.w, self.s, self.dtype = x.double(), w.double(), s, x.dtype
        rows, items = x.shape[0], w.shape[0]
        self.there = (targets >= 0) & (targets < items)
        self.t = torch.where(self.there, targets, 0).long()
        self.x = torch.where(self.there[:, None], self.x, 0.0)
        b = torch.zeros(items, dtype=torch.float64, device="cuda") if bias is None else bias.double()
        self.l = self.x @ self.w.t() * s + b
        size = self.x.abs() @ self.w.abs().t() * abs(s) + b.abs().nan_to_num(posinf=0.0)
        self.e = (x.shape[1] + 4) * U * size
        self.lse = self.l.logsumexp(1)
        far = (self.l - self.lse[:, None]).abs().nan_to_num(nan=0.0, posinf=0.0)
        self.p = (self.l - self.lse[:, None]).exp().nan_to_num(nan=0.0)
        rel = self.e + 3 * U * far + 4 * U
        self.rel = rel + 2 * U * self.lse.abs().nan_to_num(posinf=0.0)[:, None]
        self.lse_tol = (self.p * rel).sum(1) + (256 + items / 2048) * U + 2 * U * self.lse.abs().nan_to_num(posinf=0.0)
        at = self.l.gather(1, self.t[:, None])[:, 0]
        self.loss = torch.where(at == -INF, INF, self.lse - at)
        self.loss_tol = self.lse_tol + self.e.gather(1, self.t[:, None])[:, 0] + 2 * U * self.loss.abs().nan_to_num(posinf=0.0)

    def check_forward(self, loss, lse):
        check("lse", lse, torch.where(self.there, self.lse, 0.0), self.lse_tol)
        check("loss", loss, torch.where(self.there, self.loss, 0.0), self.loss_tol)

    def check_backward(self, grad_loss, gx, gw, gb):
        t, least, rows, items = UNIT[self.dtype], LEAST[self.dtype], *self.l.shape
        g = torch.where(self.there, grad_loss.double(), 0.0)[:, None]
        z = self.p.clone()
        z.scatter_add_(1, self.t[:, None], -torch.ones(rows, 1, dtype=torch.float64, device="cuda"))
        exact_off = self.p * self.rel + TINY
        off = exact_off + t * (z.abs() + exact_off) + least / 32768
        if gx is not None:
            exp = z @ self.w * self.s * g
            tol = (off + items * U * z.abs()) @ self.w.abs() * abs(self.s) * g.abs()
            check("grad_x", gx, exp, tol * 1.01 + (t + 4 * U) * exp.abs() + least + (items + 1) * TINY)
        if gw is not None:
            exp = (z * g).t() @ self.x * self.s
            tol = (off * g.abs()).t() @ self.x.abs() + ((t + rows * U) * z.abs() * g.abs()).t() @ self.x.abs()
            tol += least * float(g.abs().max()) * z.abs().sum(0)[:, None]
            check("grad_weight", gw, exp, 1.01 * tol * abs(self.s) + (t + 4 * U) * exp.abs() + least + (rows + 1) * TINY)
        if gb is not None:
            exp = (z * g).sum(0)
            check("grad_bias", gb, exp, 1.01 * ((exact_off + (rows + 4) * U * z.abs()) * g.abs()).sum(0))


def forward(x, w, bias, targets, scale):
    rows, items = x.shape[0], w.shape[0]
    need = tbe.tbe_cross_entropy_forward_workspace_bytes(rows, items, x.shape[1])
    ws = torch.full((need + 4096,), 0xA5, dtype=torch.uint8, device="cuda")
    loss, lse = (torch.full((rows + 7,), 77.0, device="cuda") for _ in range(2))
    tbe.tbe_cross_entropy_forward(x, w, bias, targets, scale, loss[:rows], lse[:rows], ws[:need])
    assert bool((ws[need:] == 0xA5).all()) and bool((loss[rows:] == 77).all()) and bool((lse[rows:] == 77).all())
    return loss[:rows], lse[:rows]


def backward(x, w, bias, targets, scale, lse, grad_loss, like_x=None, like_w=None, with_bias=True):
    rows, items = x.shape[0], w.shape[0]
    need = tbe.tbe_cross_entropy_backward_workspace_bytes(rows, items, x.shape[1])
    ws = torch.full((need + 4096,), 0xA5, dtype=torch.uint8, device="cuda")
    gx = torch.empty_like(x) if like_x is None else like_x
    gw = torch.empty_like(w) if like_w is None else like_w
    gb = torch.full((items + 5,), 77.0, device="cuda") if with_bias else None
    tbe.tbe_cross_entropy_backward(x, w, bias, targets, scale, lse, grad_loss, gx, gw, None if gb is None else gb[:items], ws[:need])
    assert bool((ws[need:] == 0xA5).all()) and (gb is None or bool((gb[items:] == 77).all()))
    return gx, gw, None if gb is None else gb[:items]


CASES = [(1, 1, 1, BF16), (1, 7, 8, F16), (2, 257, 3, BF16), (8, 1000, 64, BF16), (16, 5000, 128, F16), (33, 20000, 24, BF16),
         (65, 300, 40, F16), (64, 256, 64, BF16), (100, 3000, 256, BF16), (130, 515, 1024, BF16), (257, 129, 16, F16),
         (300, 4097, 200, F16), (517, 10007, 515, BF16), (1000, 65, 128, BF16), (1025, 2049, 136, F16), (2000, 9000, 128, BF16),
         (3, 300001, 8, BF16), (700, 1300, 1100, F16), (5, 40, 4096, BF16)]


@pytest.mark.parametrize("rows,items,width,dtype", CASES)
def test_forward_and_backward(rows, items, width, dtype):
    for k, (stride, offset, pad, scale, with_bias, itype) in enumerate((
            (width, 0, 0.0, 1.0, False, torch.int64), ((width + 15) // 8 * 8, 8, 0.3, 0.7, True, torch.int32),
            (width + 3, 1, 0.6, -1.3, True, torch.int64))):
        flush_print(f"loss {rows} {items} {width} {dtype} variant {k}")
        x, w = matrix(rows, width, dtype, 1, 1.0, stride, offset), matrix(items, width, dtype, 2, 2 * width ** -0.5, stride, offset)
        bias = matrix(1, items, torch.float32, 3, 1.5)[0] if with_bias else None
        t = some_targets(rows, items, pad, 4, itype)
        x[~((t >= 0) & (t < items))] = float("nan")  # rows without a target are not looked at
        exact = Exact(x, w, bias, t, scale)
        loss, lse = forward(x, w, bias, t, scale)
        exact.check_forward(loss, lse)
        grad = torch.full((rows,), 1.0 / rows, device="cuda") if k < 2 else matrix(1, rows, torch.float32, 5)[0]
        if dtype == F16:
            grad = grad * 1024
        gx, gw, gb = backward(x, w, bias, t, scale, lse, grad, matrix(rows, width, dtype, 6, 1.0, stride, offset),
                              matrix(items, width, dtype, 7, 1.0, stride, offset))
        exact.check_backward(grad, gx, gw, gb)
        assert bool((gx[~exact.there] == 0).all())
        again = forward(x, w, bias, t, scale) + backward(x, w, bias, t, scale, lse, grad)
        for a, b in zip(again, (loss, lse, gx, gw, gb)):
            assert torch.equal(a, b), "another result for the same inputs"
        # each gradient alone, the others left out
        need = tbe.tbe_cross_entropy_backward_workspace_bytes(rows, items, width)
        for i, one in enumerate((gx, gw, gb)):
            outs = [None, None, None]
            outs[i] = torch.empty_like(one)
            tbe.tbe_cross_entropy_backward(x, w, bias, t, scale, lse, grad, *outs, tbe.workspace(need))
            assert torch.equal(outs[i], one)


def test_several_pieces_of_the_items():
    rows, items, width = 70000, 8000, 16
    x, w, t = matrix(rows, width, BF16, 1), matrix(items, width, BF16, 2, 0.6), some_targets(rows, items, 0.2, 3)
    bias, grad = matrix(1, items, torch.float32, 4)[0], matrix(1, rows, torch.float32, 5)[0] / rows
    exact = Exact(x, w, bias, t, 1.0)
    loss, lse = forward(x, w, bias, t, 1.0)
    exact.check_forward(loss, lse)
    exact.check_backward(grad, *backward(x, w, bias, t, 1.0, lse, grad))


def test_masked_items():
    rows, items, width = 40, 700, 64
    x, w = matrix(rows, width, BF16, 1), matrix(items, width, BF16, 2, 0.2)
    t = some_targets(rows, items, 0.1, 3)
    grad = torch.full((rows,), 0.05, device="cuda")
    bias = torch.zeros(items, device="cuda")
    bias[::3] = -INF
    bias[1::3] = torch.finfo(torch.float32).min  # no probability beside others
    exact = Exact(x, w, bias, t, 1.0)
    loss, lse = forward(x, w, bias, t, 1.0)
    masked = exact.there & (t % 3 == 0)
    assert bool((loss[masked] == INF).all()) and int(masked.sum()) > 0
    far = exact.there & (t % 3 == 1)
    assert bool((loss[far] > 3e38).all())
    near = exact.there & (t % 3 == 2)
    check("loss", loss[near], exact.loss[near], exact.loss_tol[near])
    check("lse", lse, torch.where(exact.there, exact.lse, 0.0), exact.lse_tol)
    gx, gw, gb = backward(x, w, bias, t, 1.0, lse, grad)
    assert bool(gx.isfinite().all()) and bool(gw.isfinite().all()) and bool(gb.isfinite().all())
    untouched = torch.ones(items, dtype=torch.bool, device="cuda")
    untouched[t[exact.there]] = False
    untouched[2::3] = False
    assert bool((gw[untouched] == 0).all()) and bool((gb[untouched] == 0).all())
    exact.check_backward(grad, gx, gw, gb)


def test_every_item_masked():
    rows, items, width = 5, 300, 32
    x, w, t = matrix(rows, width, F16, 1), matrix(items, width, F16, 2), some_targets(rows, items, 0.0, 3)
    bias, grad = torch.full((items,), -INF, device="cuda"), torch.ones(rows, device="cuda")
    loss, lse = forward(x, w, bias, t, 1.0)
    assert bool((lse == -INF).all()) and bool((loss == INF).all())
    gx, gw, gb = backward(x, w, bias, t, 1.0, lse, grad)  # p is 0: only the targets' -1 is left
    assert torch.equal(gx, -w[t])
    assert torch.equal(gb, -torch.bincount(t, minlength=items).float())
    # the lowest value everywhere is no mask: all items are alike
    bias.fill_(torch.finfo(torch.float32).min)
    loss, lse = forward(x, w, bias, t, 1.0)
    gx, gw, gb = backward(x, w, bias, t, 1.0, lse, grad)
    assert bool(lse.isfinite().all()) and bool(gx.isfinite().all())


def test_no_row_has_a_target():
    for rows in (0, 9, 300):
        items, width = 500, 72
        x, w = matrix(rows, width, BF16, 1), matrix(items, width, BF16, 2)
        t = torch.full((rows,), -1, device="cuda")
        if rows:
            loss, lse = forward(x, w, None, t, 1.0)
            assert bool((loss == 0).all()) and bool((lse == 0).all())
        gx, gw, gb = backward(x, w, None, t, 1.0, torch.zeros(rows, device="cuda"), torch.ones(rows, device="cuda"))
        assert bool((gx == 0).all()) and bool((gw == 0).all()) and bool((gb == 0).all())


def test_values_that_are_not_finite_stay_in_their_rows():
    rows, items, width = 20, 400, 40
    x, w, t = matrix(rows, width, BF16, 1), matrix(items, width, BF16, 2), some_targets(rows, items, 0.0, 3)
    good = forward(x, w, None, t, 1.0)
    x[3, 5], x[11, 0] = float("nan"), INF
    loss, lse = forward(x, w, None, t, 1.0)
    keep = torch.ones(rows, dtype=torch.bool, device="cuda")
    keep[3], keep[11] = False, False
    assert torch.equal(loss[keep], good[0][keep]) and torch.equal(lse[keep], good[1][keep])
    assert not bool(loss[~keep].isfinite().any())
    gx, _, _ = backward(x, w, None, t, 1.0, lse, torch.ones(rows, device="cuda"))
    assert bool(gx[keep].isfinite().all()) and not bool(gx[~keep].isfinite().any())


def test_large_logits():
    """Logits of thousands: nothing overflows, and probabilities of 0 and 1 are that."""
    rows, items, width = 70, 1000, 64
    x, w, t = matrix(rows, width, BF16, 1, 30.0), matrix(items, width, BF16, 2, 20.0), some_targets(rows, items, 0.0, 3)
    exact = Exact(x, w, None, t, 1.0)
    loss, lse = forward(x, w, None, t, 1.0)
    exact.check_forward(loss, lse)
    assert float(exact.loss.max()) > 1000
    gx, gw, gb = backward(x, w, None, t, 1.0, lse, torch.ones(rows, device="cuda"))
    exact.check_backward(torch.ones(rows, device="cuda"), gx, gw, gb)


def test_weights_far_apart():
    """Rows of items past 2^31 elements: 40000 items 65544 apart, 2.6e9 elements."""
    rows, items, width, stride = 12, 40000, 8, 65544
    buf = torch.empty(items * stride, dtype=BF16, device="cuda")
    w = buf.view(items, stride)[:, :width]
    w.copy_(matrix(items, width, BF16, 2))
    x, t = matrix(rows, width, BF16, 1), some_targets(rows, items, 0.0, 3)
    t[0], t[1] = items - 1, 0
    close = w.contiguous()
    loss, lse = forward(x, w, None, t, 1.0)
    Exact(x, close, None, t, 1.0).check_forward(loss, lse)
    grad = torch.ones(rows, device="cuda")
    gx, gw, _ = backward(x, w, None, t, 1.0, lse, grad, like_w=torch.empty_like(close))
    Exact(x, close, None, t, 1.0).check_backward(grad, gx, gw, None)


def test_gradients_against_differences():
    rows, items, width = 6, 50, 24
    x, w, t = matrix(rows, width, F16, 1), matrix(items, width, F16, 2, 0.3), some_targets(rows, items, 0.3, 3)
    bias = matrix(1, items, torch.float32, 4, 0.5)[0]
    weights = torch.rand(rows, generator=torch.Generator().manual_seed(5)).cuda() + 0.5
    lse = forward(x, w, bias, t, 1.0)[1]
    gx, gw, gb = backward(x, w, bias, t, 1.0, lse, weights)

    def value(x, w, b):
        return float((forward(x, w, b, t, 1.0)[0].double() * weights.double()).sum())

    # steps h that the 16-bit values hold exactly; the third derivative of a logsumexp along one coordinate is below
    # 2 max |slope|^3; losses are off by a few 1e-6
    h = 2.0 ** -6
    for i, d in ((0, 0), (2, 7), (5, 23)):
        up, down = x.clone(), x.clone()
        up[i, d] = (x[i, d].float() / h).round() * h + h
        down[i, d] = up[i, d] - 2 * h
        mid = x.clone()
        mid[i, d] = up[i, d] - h
        lse_mid = forward(mid, w, bias, t, 1.0)[1]
        g = backward(mid, w, bias, t, 1.0, lse_mid, weights)[0]
        slope = float(w.float().abs().max())
        assert abs((value(up, w, bias) - value(down, w, bias)) / (2 * h) - float(g[i, d])) <= \
            2 * slope ** 3 * h * h + 1e-5 / h + 2 ** -10 * slope * 2
    for v in (0, 17, int(t[t >= 0][0])):
        up, down = bias.clone(), bias.clone()
        up[v] += h
        down[v] -= h
        assert abs((value(x, w, up) - value(x, w, down)) / (2 * h) - float(gb[v])) <= 2 * h * h * rows * 1.5 + 1e-5 / h


def test_captured_and_replayed_beside_eager_work():
    for rows, items, width, dtype in ((10, 3000, 64, BF16), (400, 2000, 136, F16)):
        x, w = matrix(rows, width, dtype, 1), matrix(items, width, dtype, 2, width ** -0.5)
        t = some_targets(rows, items, 0.2, 3)
        bias, grad = matrix(1, items, torch.float32, 4)[0], torch.full((rows,), 0.5, device="cuda")
        loss, lse = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
        gx, gw, gb = torch.empty_like(x), torch.empty_like(w), torch.empty_like(bias)
        fws = tbe.workspace(tbe.tbe_cross_entropy_forward_workspace_bytes(rows, items, width))
        bws = tbe.workspace(tbe.tbe_cross_entropy_backward_workspace_bytes(rows, items, width))
        stream = torch.cuda.Stream()
        stream.wait_stream(torch.cuda.current_stream())
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            tbe.tbe_cross_entropy_forward(x, w, bias, t, 0.9, loss, lse, fws)
            tbe.tbe_cross_entropy_backward(x, w, bias, t, 0.9, lse, grad, gx, gw, gb, bws)
        for seed in range(4):
            t.copy_(some_targets(rows, items, (0.0, 0.9, 0.3, 1.0)[seed], 30 + seed))
            x.copy_(matrix(rows, width, dtype, 40 + seed))
            graph.replay()
            torch.cuda.synchronize()
            e_loss, e_lse = forward(x, w, bias, t, 0.9)
            e = (e_loss, e_lse) + backward(x, w, bias, t, 0.9, e_lse, grad)
            for name, a, b in zip(("loss", "lse", "grad_x", "grad_weight", "grad_bias"), (loss, lse, gx, gw, gb), e):
                assert torch.equal(a, b), f"replay {seed}: {name}"


def test_on_another_stream_with_a_smaller_batch_in_the_same_workspace():
    rows, items, width = 900, 1500, 72
    need = tbe.tbe_cross_entropy_backward_workspace_bytes(rows, items, width)
    ws, side = tbe.workspace(need), torch.cuda.Stream()
    w = matrix(items, width, BF16, 2)
    for n in (900, 17, 400):
        x, t = matrix(n, width, BF16, n), some_targets(n, items, 0.2, n)
        grad, lse = torch.ones(n, device="cuda"), forward(x, w, None, t, 1.0)[1]
        gx, gw = torch.empty_like(x), torch.empty_like(w)
        torch.cuda.synchronize()
        tbe.tbe_cross_entropy_backward(x, w, None, t, 1.0, lse, grad, gx, gw, None, ws, stream=side)
        torch.cuda.synchronize()
        alone = backward(x, w, None, t, 1.0, lse, grad, with_bias=False)
        assert torch.equal(gx, alone[0]) and torch.equal(gw, alone[1])
