"""Logits past 2^20, where fp32 holds no digits behind the point: the largest one's probability is 1 all the same, the others' 0."""
import pytest
import torch

from gpu_util import flush_print
from test_gpu_items_loss import BF16, F16, LEAST, U, UNIT, backward, forward, matrix, some_targets

pytestmark = pytest.mark.gpu

WIDTHS = [16, 64, 96, 128, 136, 200, 328]


def check_one_hot(x, w, t, scale, top, certain, lse, grad):
    """Gradients where p is 1 for `top` in the `certain` rows and 0 elsewhere: z is then 1, 0 and -1, all exact."""
    rows, items = x.shape[0], w.shape[0]
    gx, gw, gb = backward(x, w, None, t, scale, lse, grad)
    there = (t >= 0) & (t < items)
    u, least = UNIT[x.dtype], LEAST[x.dtype]
    for g in (gx, gw, gb):
        assert bool(g.isfinite().all())
    at = torch.where(there, t, 0).long()
    exp = (w[top].double() - w[at].double()) * scale * torch.where(there, grad, 0.0).double()[:, None]
    size = (w[top].double().abs() + w[at].double().abs()) * abs(scale) * grad.abs().double()[:, None]
    off = (gx.double() - exp).abs() - (u * exp.abs() + 8 * U * size + least)
    assert bool((off[certain | ~there] <= 0).all()), f"grad_x: {float(off[certain | ~there].max())}"
    assert int(certain.sum()) > rows // 2
    if bool((certain | ~there).all()):
        z = torch.zeros(items, rows, dtype=torch.float64, device="cuda")
        z[top[there], there.nonzero()[:, 0]] += 1
        terms = z.clone()  # p and [v = t], each off for itself: they do not cancel in what z may be off by
        z[t[there].long(), there.nonzero()[:, 0]] -= 1
        terms[t[there].long(), there.nonzero()[:, 0]] += 1
        # p |g| / largest may be taken as a power of two of its logarithm, off by 3 roundings of that and 4 of its own; sums of rows
        part = grad.double().abs() / grad.double().abs().max()
        rel = (rows + 8 + 3 * part.log2().abs().nan_to_num(posinf=0.0)) * U
        exp_b = z @ grad.double()
        assert bool(((gb.double() - exp_b).abs() <= terms @ (grad.double().abs() * rel)).all())
        exp_w = z @ (x.double() * grad.double()[:, None]).nan_to_num(nan=0.0) * scale
        # x * grad / largest is rounded once more
        size = z.abs() @ (x.double() * grad.double()[:, None]).abs().nan_to_num(nan=0.0) * abs(scale)
        off = terms @ (x.double() * (grad.double() * rel)[:, None]).abs().nan_to_num(nan=0.0) * abs(scale)
        least_w = least * (1 + terms.sum(1) * float(grad.abs().max()) * abs(scale))
        assert bool(((gw.double() - exp_w).abs() <= u * exp_w.abs() + 1.01 * (u * size + off) + least_w[:, None]).all())


@pytest.mark.parametrize("width", WIDTHS)
@pytest.mark.parametrize("power", [18, 21, 24, 27, 32, 45, 64])
def test_one_logit_above_all_others(width, power):
    """Item i % items is along row i and the others are not: no two logits of a row are near each other."""
    for rows, items, dtype in ((70, 500, BF16), (300, 1000, BF16), (20, 300, F16)):
        if dtype == F16 and power > 24:
            continue
        for sign in (1, -1):
            flush_print(f"far logits: {rows} {items} {width} {dtype} 2^{power} sign {sign}")
            scale = sign * 2.0 ** power
            x, w = matrix(rows, width, dtype, 1), matrix(items, width, dtype, 2, 0.5 * width ** -0.5)
            top = torch.arange(rows, device="cuda") * 3 % items
            w[top] = x * sign * 0.25
            t = some_targets(rows, items, 0.1, 3)
            t[::4] = top[::4]
            there = (t >= 0) & (t < items)
            logits = x.double() @ w.double().t() * scale
            best = logits.topk(2, 1)
            error = (width + 4) * U * (x.double().abs() @ w.double().abs().t() * abs(scale)).max(1)[0]
            certain = (best.values[:, 0] - best.values[:, 1] > 2 * error + 200) & there
            loss, lse = forward(x, w, None, t, scale)
            assert bool(((lse.double() - best.values[:, 0]).abs()[certain] <= error[certain] + 2 * U * lse.abs()[certain]).all())
            hit = certain & (t == best.indices[:, 0])
            # the target's logit is summed in another order than the matrix instructions'
            assert bool((loss[hit].abs() <= 2 * error[hit] + 4 * U * lse[hit].abs()).all())
            grad = torch.full((rows,), 2.0 ** -power, device="cuda")
            check_one_hot(x, w, t, scale, best.indices[:, 0], certain, lse, grad)
            if dtype == BF16:
                grad = matrix(1, rows, torch.float32, 5, 2.0 ** -power)[0]  # of either sign
                check_one_hot(x, w, t, scale, best.indices[:, 0], certain, lse, grad)


@pytest.mark.parametrize("width", WIDTHS)
def test_biases_far_out(width):
    """All biases far out on either side: probabilities are those of their differences."""
    rows, items = 130, 700
    x, w, t = matrix(rows, width, BF16, 1), matrix(items, width, BF16, 2, 0.05 * width ** -0.5), some_targets(rows, items, 0.1, 3)
    grad = torch.ones(rows, device="cuda")
    there = (t >= 0) & (t < items)
    for far in (2.0 ** 22, -2.0 ** 22, 2.0 ** 33, -2.0 ** 33, 1e30, -1e30, 9e37, -9e37):
        flush_print(f"far biases: {width} {far}")
        step = max(abs(far) * 2.0 ** -16, 64.0)
        bias = far - step * (torch.arange(items, device="cuda") * 9 % items).float()  # item 0 alone is the highest: 9 and 700 have no common divisor
        loss, lse = forward(x, w, bias, t, 1.0)
        assert bool(((lse[there].double() - float(bias[0])).abs() <= 4 * U * abs(far) + 1).all())
        _, _, gb = backward(x, w, bias, t, 1.0, lse, grad)
        exp = -torch.bincount(t[there], minlength=items).double()
        exp[0] += int(there.sum())
        # logits of item 0 differ from its bias by what fp32 cannot hold or by less than 0.05 * 8
        assert bool(((gb.double() - exp).abs() <= (rows + 4) * U * rows + 1e-6 * rows).all())


@pytest.mark.parametrize("width", WIDTHS)
@pytest.mark.parametrize("high", [3e38, 1.2e38, 9e37])
def test_one_bias_near_the_largest_value(width, high):
    """Its item's probability is 1, whatever the target."""
    rows, items = 90, 600
    x, w, t = matrix(rows, width, BF16, 1), matrix(items, width, BF16, 2, width ** -0.5), some_targets(rows, items, 0.1, 3)
    t[::3] = 7
    there = (t >= 0) & (t < items)
    bias = matrix(1, items, torch.float32, 4)[0]
    bias[7] = high
    for scale in (1.0, -3.0):
        loss, lse = forward(x, w, bias, t, scale)
        # narrow rows' biases are divided by the scale and multiplied again: 3 roundings, and the target's own
        assert bool((loss >= 0).all()) and bool((loss[there & (t == 7)] <= (0 if width > 128 else 8 * U * high)).all())
        _, _, gb = backward(x, w, bias, t, scale, lse, torch.ones(rows, device="cuda"))
        exp = -torch.bincount(t[there], minlength=items).double()
        exp[7] += int(there.sum())
        assert torch.equal(gb.double(), exp)
