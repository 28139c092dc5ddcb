"""Rows with a NaN or an infinity stay alone: the rows beside them, in the same wave and in the same lane of it, have their own
losses and gradients.  Tolerances as in test_gpu_items_loss.py."""
import pytest
import torch

from gpu_util import flush_print
from test_gpu_items_loss import BF16, INF, Exact, backward, forward, matrix, some_targets

pytestmark = pytest.mark.gpu

NAN = float("nan")


def rising(rows, items, width):
    """Rows whose logits rise by several hundred over the items."""
    x, w = matrix(rows, width, BF16, 1), matrix(items, width, BF16, 2, width ** -0.5)
    x[:, 0] = 8.0
    w[:, 0] = torch.linspace(-40.0, 60.0, items, device="cuda").to(BF16)
    return x, w


@pytest.mark.parametrize("width", [40, 128, 200])
@pytest.mark.parametrize("rows,items", [(20, 3000), (200, 3000), (1000, 5000)])
@pytest.mark.parametrize("scale", [1.0, 4.0])
def test_rows_that_are_not_finite(rows, items, width, scale):
    kinds = {"a NaN in 16 adjacent rows": (range(2, 18), NAN), "in every fourth": (range(0, rows, 4), NAN),
             "in the first": ((0,), NAN), "in all but one": (range(1, rows), NAN), "an infinity in 16 adjacent rows": (range(2, 18), INF),
             "in every row of an even number": (range(0, rows, 2), -INF)}
    for what, (bad, value) in kinds.items():
        flush_print(f"not finite: {rows} {items} {width} scale {scale} {what}")
        x, w = rising(rows, items, width)
        x[1::3, 0] = -8.0  # falling ones too
        t, grad = some_targets(rows, items, 0.0, 3), torch.rand(rows, generator=torch.Generator().manual_seed(5)).cuda() + 0.25
        keep = torch.ones(rows, dtype=torch.bool, device="cuda")
        keep[list(bad)] = False
        x[~keep, 3] = value
        loss, lse = forward(x, w, None, t, scale)
        exact = Exact(x[keep], w, None, t[keep], scale)
        exact.check_forward(loss[keep], lse[keep])
        assert not bool(loss[~keep].isfinite().any())
        gx, _, _ = backward(x, w, None, t, scale, lse, grad, with_bias=False)
        exact.check_backward(grad[keep], gx[keep], None, None)
        assert not bool(gx[~keep].isfinite().all(1).any())


@pytest.mark.parametrize("width", [40, 128, 200])
def test_a_row_that_rises_alone(width):
    """All rows are zeros but a few whose logits rise by 12800 over the items, 200 in the ranges of ten tiles that a wave takes, so
    no other lane asks for what such a row needs; a row of its own lane holds a NaN."""
    rows, items = 2000, 40000
    x, w = rising(rows, items, width)
    bad, alone = [0, 300, 1048, 1900], [16, 268, 1000, 1932]
    x[:] = 0.0
    x[alone, 0] = torch.tensor([128.0, -128.0, 128.0, 128.0], dtype=BF16, device="cuda")
    x[bad, 1] = NAN
    t = some_targets(rows, items, 0.0, 3)
    loss, lse = forward(x, w, None, t, 1.0)
    keep = torch.ones(rows, dtype=torch.bool, device="cuda")
    keep[bad] = False
    Exact(x[keep], w, None, t[keep], 1.0).check_forward(loss[keep], lse[keep])
    assert bool(loss[bad].isnan().all()) and bool(lse[bad].isnan().all())


@pytest.mark.parametrize("width", [64, 200])
def test_an_item_that_is_not_finite(width):
    """Every row that scores it is NaN or infinite, whatever else it holds."""
    rows, items = 150, 900
    x, w = rising(rows, items, width)
    w[517, 2] = NAN
    loss, lse = forward(x, w, None, some_targets(rows, items, 0.0, 3), 1.0)
    assert bool(loss.isnan().all()) and bool(lse.isnan().all())
