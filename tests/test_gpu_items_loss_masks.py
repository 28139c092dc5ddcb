"""Softmax cross entropy with masked items at scales other than 1: a scaled cosine's 1 / temperature, and far ones.

Whole ranges of the items masked by -infinity or by the lowest value, last tiles of few items, every item masked.  Tolerances
as in test_gpu_items_loss.py."""
import pytest
import torch

from gpu_util import flush_print
from test_gpu_items_loss import BF16, F16, INF, U, Exact, backward, forward, matrix, some_targets

pytestmark = pytest.mark.gpu

LOWEST = torch.finfo(torch.float32).min


def rows_and_items(rows, items, width, scale, dtype=BF16, seed=1):
    """Logits of a few units, whatever the scale."""
    w = matrix(items, width, dtype, seed + 1, 2 * width ** -0.5)
    if dtype == BF16:
        return matrix(rows, width, dtype, seed), w / abs(scale)
    return matrix(rows, width, dtype, seed) * abs(scale) ** -0.5, w * abs(scale) ** -0.5


def one_case(rows, items, width, scale, bias, dtype=BF16):
    """Targets among the items that are not masked."""
    x, w = rows_and_items(rows, items, width, scale, dtype)
    t = some_targets(rows, items, 0.1, 4)
    if bias is not None:
        open_ = (bias > -1e30).nonzero()[:, 0]
        t = torch.where((t >= 0) & (t < items), open_[t.clamp(0, items - 1) % len(open_)], t)
    exact = Exact(x, w, bias, t, scale)
    loss, lse = forward(x, w, bias, t, scale)
    assert bool(loss.isfinite().all()) and bool(lse.isfinite().all())
    exact.check_forward(loss, lse)
    grad = torch.rand(rows, generator=torch.Generator().manual_seed(5)).cuda() + 0.25
    exact.check_backward(grad, *backward(x, w, bias, t, scale, lse, grad))


@pytest.mark.parametrize("width", [16, 64, 128, 200])
@pytest.mark.parametrize("scale", [2.4, 4.0, -20.0, 100.0])
def test_last_tiles_of_few_items(width, scale):
    for rows in (20, 200):
        for items in (1, 8, 65, 87, 64 * 9 + 24, 10007):
            flush_print(f"few items in the last tile: {rows} {items} {width} scale {scale}")
            one_case(rows, items, width, scale, None)


@pytest.mark.parametrize("mask", [-INF, LOWEST])
@pytest.mark.parametrize("width", [64, 128, 200])
@pytest.mark.parametrize("scale", [1.0, 3.0, 20.0, -4.0, 2.0 ** 40, -2.0 ** 64])
def test_runs_of_masked_items(width, scale, mask):
    # the first 8, 32 and 64 items of a range, whole ranges of them, all but the last
    for rows, items, first, end in ((20, 4097, 0, 8), (20, 4097, 0, 64), (20, 4097, 64, 1088), (200, 5000, 0, 32),
                                    (200, 5000, 0, 1000), (200, 5000, 2000, 4999), (70, 300, 0, 299), (2000, 9000, 0, 4000)):
        flush_print(f"masked items: {rows} {items} {width} scale {scale} mask {mask} {first} {end}")
        bias = matrix(1, items, torch.float32, 3, 1.5)[0]
        bias[first:end] = mask
        one_case(rows, items, width, scale, bias)


@pytest.mark.parametrize("scale", [4.0, -20.0])
def test_masked_items_in_half_precision(scale):
    for rows, items, width in ((20, 1000, 64), (200, 3000, 128), (100, 3000, 200)):
        bias = torch.zeros(items, device="cuda")
        bias[:40] = -INF
        bias[64:200] = LOWEST
        one_case(rows, items, width, scale, bias, F16)


@pytest.mark.parametrize("width", [40, 128, 200])
@pytest.mark.parametrize("scale", [1.0, 3.0, -10.0, 20.0, 2.0 ** 40])
def test_every_item_masked(width, scale):
    for rows, items in ((5, 300), (200, 1000), (70, 1)):
        flush_print(f"every item masked: {rows} {items} {width} scale {scale}")
        x, w = rows_and_items(rows, items, width, scale)
        t, grad = some_targets(rows, items, 0.0, 3), torch.ones(rows, device="cuda")
        bias = torch.full((items,), -INF, device="cuda")
        loss, lse = forward(x, w, bias, t, scale)
        assert bool((lse == -INF).all()) and bool((loss == INF).all())
        gx, _, gb = backward(x, w, bias, t, scale, lse, grad)  # p is 0: only the targets' -1 is left
        assert bool(gx.isfinite().all())
        assert torch.equal(gb, -torch.bincount(t, minlength=items).float())
        # the lowest value everywhere: all items are alike, and lse is that value but for its roundings (the scale's inverse, the
        # bias over the scale, times the scale: 3, and the step to the nearest)
        bias.fill_(LOWEST)
        loss, lse = forward(x, w, bias, t, scale)
        assert bool(((lse.double() - LOWEST).abs() <= 4 * 2 * U * abs(LOWEST)).all())
        assert bool((loss.abs() <= 8 * U * abs(LOWEST)).all())
        assert all(bool(g.isfinite().all()) for g in backward(x, w, bias, t, scale, lse, grad))
