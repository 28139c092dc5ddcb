"""Biases of the largest and the lowest values: finite ones count as no higher than 1e38 and 1e38 |scale|, for the
probabilities and for the target's logit alike, at every width."""
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
        counts_as = 1e38 * min(1.0, abs(scale) or 1.0)
        # lse is that but for its roundings, the reference's step of 2^-22 among them
        assert bool(((lse[there].double() - counts_as).abs() <= 16 * U * counts_as).all())
        assert bool((loss[there & (t == 7)].abs() <= 16 * U * counts_as).all())
        assert bool((loss >= 0).all()) and bool(loss.isfinite().all())
        other = there & (t != 7) & (t != 9)
        assert bool(((loss[other].double() - counts_as).abs() <= 16 * U * counts_as).all())
        grad = torch.ones(rows, device="cuda")
        gx, gw, gb = backward(x, w, bias, t, scale, lse, grad)
        # z is 1 for item 7 and -1 for the target: p as far as the roundings of numbers so far out allow, 8 units of them
        assert bool(gb.isfinite().all()) and bool(gx.isfinite().all()) and bool(gw.isfinite().all())
        hits = torch.bincount(t[there], minlength=items).float()
        rest = torch.arange(items, device="cuda") != 7
        assert torch.equal(gb[rest], -hits[rest])


@pytest.mark.parametrize("width", WIDTHS)
def test_the_same_rule_at_every_width(width):
    """One row with one item above 1e38 in a table of two: its target's loss is 0 and its gradients are too, but for roundings."""
    x, w = torch.zeros(1, width, dtype=BF16, device="cuda"), matrix(2, width, BF16, 2)
    t = torch.zeros(1, dtype=torch.int64, device="cuda")
    for scale in (1.0, 0.5, 8.0):
        bias = torch.tensor([3e38, 0.0], device="cuda")
        loss, lse = forward(x, w, bias, t, scale)
        counts_as = 1e38 * min(1.0, scale)
        assert abs(float(lse) - counts_as) <= 16 * U * counts_as and 0 <= float(loss) <= 16 * U * counts_as
        _, _, gb = backward(x, w, bias, t, scale, lse, torch.ones(1, device="cuda"))
        assert bool(gb.isfinite().all()) and float(gb[1]) == 0
