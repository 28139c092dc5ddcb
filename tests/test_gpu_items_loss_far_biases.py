"""Biases of the largest and the lowest values: where |scale| is below 1, finite ones count as no higher than the largest value times
|scale|, for the probabilities and for the target's logit alike, at every width."""
import pytest
import torch

from gpu_util import flush_print
from test_gpu_items_loss import BF16, U, backward, forward, matrix, some_targets

pytestmark = pytest.mark.gpu

LARGEST = torch.finfo(torch.float32).max
WIDTHS = [16, 64, 128, 136, 200]


@pytest.mark.parametrize("width", WIDTHS)
@pytest.mark.parametrize("scale", [1.0, 0.25, -0.25, 3.0, 20.0, 0.0])
@pytest.mark.parametrize("high", [LARGEST, 3e38, 2e38])
def test_an_item_of_the_largest_bias(width, scale, high):
    """Its probability is 1, the others' are 0."""
    for rows, items in ((70, 500), (300, 1000)):
        flush_print(f"largest bias: {rows} {items} {width} scale {scale} {high}")
        x, w, t = matrix(rows, width, BF16, 1), matrix(items, width, BF16, 2, width ** -0.5), some_targets(rows, items, 0.2, 3)
        t[:5] = 7
        there = (t >= 0) & (t < items)
        bias = matrix(1, items, torch.float32, 4)[0]
        bias[7], bias[9] = high, torch.finfo(torch.float32).min
        loss, lse = forward(x, w, bias, t, scale)
        counts_as = min(high, LARGEST * min(1.0, abs(scale) or 1.0))
        # lse is that but for the roundings of the scale's inverse, the bias over the scale and the product
        assert bool(((lse[there].double() - counts_as).abs() <= 16 * U * counts_as).all())
        assert bool((loss[there & (t == 7)].abs() <= 16 * U * counts_as).all())
        assert bool((loss >= 0).all()) and bool(loss.isfinite().all())
        other = there & (t != 7) & (t != 9)
        assert bool(((loss[other].double() - counts_as).abs() <= 16 * U * counts_as).all())
        grad = torch.ones(rows, device="cuda")
        gx, gw, gb = backward(x, w, bias, t, scale, lse, grad)
        # p is 1 for item 7 and 0 for the others, so z is 1, 0 and -1
        assert bool(gx.isfinite().all()) and bool(gw.isfinite().all())
        exp = -torch.bincount(t[there], minlength=items).double()
        exp[7] += int(there.sum())
        assert torch.equal(gb.double(), exp)
        exp_x = torch.where(there[:, None], (w[7].double() - w[torch.where(there, t, 0)].double()) * scale, 0.0)
        size = (w[7].double().abs() + w[torch.where(there, t, 0)].double().abs()) * abs(scale)
        assert bool(((gx.double() - exp_x).abs() <= 2.0 ** -8 * exp_x.abs() + 8 * U * size).all())


@pytest.mark.parametrize("width", WIDTHS)
def test_a_table_of_two(width):
    """One row, one item near the largest value: its target's loss and gradients are 0."""
    x, w = torch.zeros(1, width, dtype=BF16, device="cuda"), matrix(2, width, BF16, 2)
    t = torch.zeros(1, dtype=torch.int64, device="cuda")
    for scale in (1.0, 0.5, 8.0, 3.0):
        for high in (3e38, LARGEST, 1e38):
            bias = torch.tensor([high, 0.0], device="cuda")
            loss, lse = forward(x, w, bias, t, scale)
            counts_as = min(high, LARGEST * min(1.0, scale))
            assert abs(float(lse) - counts_as) <= 16 * U * counts_as and 0 <= float(loss) <= 16 * U * counts_as
            _, _, gb = backward(x, w, bias, t, scale, lse, torch.ones(1, device="cuda"))
            assert bool((gb == 0).all())


@pytest.mark.parametrize("width", WIDTHS)
@pytest.mark.parametrize("low", [-1e38, -2e38, -1e30, -9e36])
def test_the_same_low_bias_everywhere(width, low):
    """No item is masked against the others: lse is that bias, and every probability exp(logit - lse), at most 1."""
    rows, items = 90, 300
    x, w, t = matrix(rows, width, BF16, 1), matrix(items, width, BF16, 2, width ** -0.5), some_targets(rows, items, 0.0, 3)
    for scale in (1.0, 0.75, 8.0, -3.0):
        bias = torch.full((items,), low, device="cuda")
        loss, lse = forward(x, w, bias, t, scale)
        assert bool(((lse.double() - low).abs() <= 16 * U * abs(low)).all())
        assert bool((loss >= 0).all()) and bool((loss <= 16 * U * abs(low)).all())
        gx, gw, gb = backward(x, w, bias, t, scale, lse, torch.ones(rows, device="cuda"))
        assert all(bool(g.isfinite().all()) for g in (gx, gw, gb)) and bool((gb.abs() <= rows).all())


@pytest.mark.parametrize("width", WIDTHS)
@pytest.mark.parametrize("scale", [0.5, -0.125, 2.0 ** -40])
@pytest.mark.parametrize("low", [-LARGEST, -2e38, -1e38, -1e30])
def test_only_low_biases_below_a_scale_of_one(width, scale, low):
    """Over the scale such biases are past the lowest value.  Every item has the same one, so lse is that and the losses are 0 but
    for roundings."""
    for rows, items in ((90, 300), (5, 1), (300, 5000)):
        x, w, t = matrix(rows, width, BF16, 1), matrix(items, width, BF16, 2, width ** -0.5), some_targets(rows, items, 0.2, 3)
        there = (t >= 0) & (t < items)
        bias = torch.full((items,), low, device="cuda")
        loss, lse = forward(x, w, bias, t, scale)
        assert bool(((lse[there].double() - low).abs() <= 16 * U * abs(low)).all())
        assert bool((loss >= 0).all()) and bool((loss <= 16 * U * abs(low)).all())
        gx, gw, gb = backward(x, w, bias, t, scale, lse, torch.ones(rows, device="cuda"))
        assert all(bool(g.isfinite().all()) for g in (gx, gw, gb)) and bool((gb.abs() <= rows).all())
        if items > 1:  # one item that is open takes all of the probability
            bias[items // 2] = 0.0
            loss, lse = forward(x, w, bias, t, scale)
            assert bool((lse.abs() <= 20).all())
            far = there & (t != items // 2)
            assert bool(((loss[far].double() + low).abs() <= 16 * U * abs(low)).all())
            gb = backward(x, w, bias, t, scale, lse, torch.ones(rows, device="cuda"))[2]
            exp = -torch.bincount(t[there], minlength=items).double()
            exp[items // 2] += int(there.sum())
            assert bool(((gb.double() - exp).abs() <= 8 * U * rows).all())
