"""Softmax cross entropy at the sizes and calls where its plan changes: weights copied a piece at a time, many rows, few
rows of a large vocabulary, shares of the rows, a single item, two streams.  Tolerances as in test_gpu_items_loss.py."""
import pytest
import torch

import bwd_tbe_fwd_amd as tbe
from gpu_util import flush_print
from test_gpu_items_loss import BF16, F16, Exact, backward, forward, matrix, some_targets

pytestmark = pytest.mark.gpu


def one_case(rows, items, width, dtype, stride=None, offset=0, pad=0.2, scale=1.0, grad=None):
    flush_print(f"loss {rows} {items} {width} {dtype} stride {stride} scale {scale}")
    x, w = matrix(rows, width, dtype, 1), matrix(items, width, dtype, 2, 2 * width ** -0.5, stride, offset)
    bias, t = matrix(1, items, torch.float32, 3, 1.5)[0], some_targets(rows, items, pad, 4)
    exact = Exact(x, w, bias, t, scale)
    loss, lse = forward(x, w, bias, t, scale)
    exact.check_forward(loss, lse)
    grad = torch.rand(rows, generator=torch.Generator().manual_seed(5)).cuda() + 0.25 if grad is None else grad
    out = backward(x, w, bias, t, scale, lse, grad)
    exact.check_backward(grad, *out)
    return out


# pieces of 131072 items of 127 and of 16640 of 1001: the last has few, whose rows are then shared among many workgroups
@pytest.mark.parametrize("rows,items,width", [(2000, 131072 + 70, 127), (2000, 131072 + 1, 125), (100, 16640 + 33, 1001)])
def test_copied_weights_whose_last_piece_is_small(rows, items, width):
    one_case(rows, items, width, BF16, stride=width, offset=1)


@pytest.mark.parametrize("rows,items,width,dtype", [(33000, 40, 24, BF16), (140000, 33, 8, F16), (132000, 9, 136, BF16),
                                                    (40000, 300, 64, F16)])
def test_many_rows(rows, items, width, dtype):
    one_case(rows, items, width, dtype)


@pytest.mark.parametrize("rows,items,width,dtype", [(3, 70000, 264, BF16), (64, 66001, 1000, F16), (20, 200000, 136, BF16),
                                                    (300, 30000, 512, BF16)])
def test_few_rows_of_a_large_vocabulary(rows, items, width, dtype):
    one_case(rows, items, width, dtype)


@pytest.mark.parametrize("rows,items,width", [(9000, 10000, 128), (8000, 52000, 96), (5000, 3000, 64), (6000, 49152, 128)])
def test_shares_of_the_rows(rows, items, width):
    one_case(rows, items, width, BF16)


@pytest.mark.parametrize("rows,width", [(50, 8), (70, 200), (1, 128)])
def test_one_item(rows, width):
    """The only item's probability is 1: losses are 0, and so are the gradients."""
    gx, gw, gb = one_case(rows, 1, width, F16, pad=0.0)
    assert float(gb.abs().max()) < 1e-4 * rows and gx.shape == (rows, width) and gw.shape == (1, width)


def test_scale_of_zero_and_gradients_of_zero():
    for width in (64, 200):
        gx, gw, gb = one_case(90, 700, width, BF16, scale=0.0)
        assert bool((gx == 0).all()) and bool((gw == 0).all()) and bool((gb != 0).any())
        for out in one_case(90, 700, width, BF16, grad=torch.zeros(90, device="cuda")):
            assert bool((out == 0).all())


def test_one_target_for_every_row():
    for width in (40, 328):
        rows, items = 500, 900
        x, w = matrix(rows, width, F16, 1), matrix(items, width, F16, 2, width ** -0.5)
        t = torch.full((rows,), 899, dtype=torch.int32, device="cuda")
        exact = Exact(x, w, None, t, 1.0)
        loss, lse = forward(x, w, None, t, 1.0)
        exact.check_forward(loss, lse)
        grad = torch.ones(rows, device="cuda")
        exact.check_backward(grad, *backward(x, w, None, t, 1.0, lse, grad))


def test_two_streams_with_a_workspace_each():
    side = [torch.cuda.Stream() for _ in range(2)]
    for rows, items, width in ((700, 9000, 64), (600, 5000, 264)):
        w, grad = matrix(items, width, BF16, 2, width ** -0.5), torch.ones(rows, device="cuda")
        need = (tbe.tbe_cross_entropy_forward_workspace_bytes(rows, items, width),
                tbe.tbe_cross_entropy_backward_workspace_bytes(rows, items, width))
        x = [matrix(rows, width, BF16, 10 + k) for k in range(2)]
        t = [some_targets(rows, items, 0.2, 20 + k) for k in range(2)]
        loss, lse = [[torch.empty(rows, device="cuda") for _ in range(2)] for _ in range(2)]
        gx, gw = [torch.empty_like(v) for v in x], [torch.empty_like(w) for _ in range(2)]
        ws = [[tbe.workspace(n) for n in need] for _ in range(2)]
        torch.cuda.synchronize()
        for _ in range(5):
            for k, s in enumerate(side):
                tbe.tbe_cross_entropy_forward(x[k], w, None, t[k], 1.0, loss[k], lse[k], ws[k][0], stream=s)
                tbe.tbe_cross_entropy_backward(x[k], w, None, t[k], 1.0, lse[k], grad, gx[k], gw[k], None, ws[k][1], stream=s)
        torch.cuda.synchronize()
        for k in range(2):
            e_loss, e_lse = forward(x[k], w, None, t[k], 1.0)
            e_gx, e_gw, _ = backward(x[k], w, None, t[k], 1.0, e_lse, grad, with_bias=False)
            for a, b in zip((loss[k], lse[k], gx[k], gw[k]), (e_loss, e_lse, e_gx, e_gw)):
                assert torch.equal(a, b)


@pytest.mark.parametrize("width", [64, 200])
def test_scales_and_biases_at_their_ends(width):
    rows, items = 70, 500
    x, w, t = matrix(rows, width, BF16, 1), matrix(items, width, BF16, 2, width ** -0.5), some_targets(rows, items, 0.2, 3)
    grad = torch.ones(rows, device="cuda")
    for scale, size in ((2.0 ** -64, 1.0), (-2.0 ** -40, 0.1), (2.0 ** 12, 500.0)):
        bias = matrix(1, items, torch.float32, 4, size)[0]
        exact = Exact(x, w, bias, t, scale)
        loss, lse = forward(x, w, bias, t, scale)
        exact.check_forward(loss, lse)
        exact.check_backward(grad, *backward(x, w, bias, t, scale, lse, grad))
    for scale in (2.0 ** 64, -2.0 ** 45, 2.0 ** 31, 2.0 ** 25, 2.0 ** 20):  # logits without digits behind the point
        exact = Exact(x, w, None, t, scale)
        loss, lse = forward(x, w, None, t, scale)
        exact.check_forward(loss, lse)
        gx, gw, gb = backward(x, w, None, t, scale, lse, grad)
        # a probability is 1 but for the roundings of lse and the logit, 8 units of it at most
        assert bool(gb.isfinite().all()) and float(gb.abs().max()) <= rows * 2
        if abs(scale) < 2.0 ** 40:
            assert bool(gx.isfinite().all()) and bool(gw.isfinite().all())
    # biases that are out of range once divided by the scale count as 1e38 of it
    bias = torch.zeros(items, device="cuda")
    bias[7], bias[9] = torch.finfo(torch.float32).max, torch.finfo(torch.float32).min
    loss, lse = forward(x, w, bias, t, 0.25)
    assert bool(loss.isfinite().all()) and bool(lse.isfinite().all()) and bool((lse[(t >= 0) & (t < items)] >= 2.4e37).all())


def test_items_past_the_threads_of_a_launch():
    """2^28 + 70 items: their biases' gradients take more than a launch of a workgroup for every 64."""
    rows, items, width = 3, (1 << 28) + 70, 8
    w = torch.empty(items, width, dtype=BF16, device="cuda").normal_(generator=torch.Generator("cuda").manual_seed(1))
    x, t = matrix(rows, width, BF16, 2), torch.tensor([items - 1, 0, 5], device="cuda")
    grad = torch.tensor([1.0, -2.0, 0.5], device="cuda")
    loss, lse = forward(x, w, None, t, 1.0)
    gb = torch.empty(items, device="cuda")
    ws = tbe.workspace(tbe.tbe_cross_entropy_backward_workspace_bytes(rows, items, width))
    tbe.tbe_cross_entropy_backward(x, w, None, t, 1.0, lse, grad, None, None, gb, ws)
    part = 1 << 25
    total = torch.zeros(rows, dtype=torch.float64, device="cuda")
    for v in range(0, items, part):
        total += (w[v:v + part].double() @ x.double().t()).exp().sum(0)
    exact = total.log()
    # sums of e^l with chains of fewer than 256 + items / 2048 additions of values off by 4 + 3 |l - lse| < 100 roundings
    assert bool(((lse.double() - exact).abs() <= (400 + items / 2048) * 2.0 ** -24).all())
    for v in (0, part, 5 * part, items - 70):
        some = w[v:v + 4096].double()
        p = (some @ x.double().t() - exact).exp()
        z = p.clone()
        for i in range(rows):
            if v <= int(t[i]) < v + 4096:
                z[int(t[i]) - v, i] -= 1
        z *= grad.double()
        tol = (p * grad.abs().double()).sum(1) * (600 + items / 2048) * 2.0 ** -24 + 8 * 2.0 ** -24 * z.abs().sum(1) + 1e-37
        assert bool(((gb[v:v + 4096].double() - z.sum(1)).abs() <= tol).all())


@pytest.mark.parametrize("rows,items,width,dtype,stride", [
    (17, 69351, 13, BF16, 13), (1, 200000, 5, F16, 7), (1024, 40000, 20, F16, 24), (1025, 40000, 20, BF16, 21),
    (40, 90001, 1000, BF16, 1000), (256, 9001, 301, F16, 301), (257, 9001, 301, F16, 301), (30, 40003, 1024, BF16, 1027),
    (30, 40003, 1030, BF16, 1030)])
def test_many_shares_of_the_items(rows, items, width, dtype, stride):
    one_case(rows, items, width, dtype, stride=stride)


@pytest.mark.parametrize("rows,width", [(20, 200), (300, 200), (20, 72)])
def test_rows_further_apart_than_a_tile_reaches(rows, width):
    """Strides past 2^21 elements, of weights, rows and both gradients."""
    items, stride = 700, (1 << 21) + 8
    w, gw = [torch.empty(items * stride, dtype=BF16, device="cuda").view(items, stride)[:, :width] for _ in range(2)]
    x, gx = [torch.empty(rows * stride, dtype=BF16, device="cuda").view(rows, stride)[:, :width] for _ in range(2)]
    w.copy_(matrix(items, width, BF16, 2, 2 * width ** -0.5))
    x.copy_(matrix(rows, width, BF16, 1))
    t, grad = some_targets(rows, items, 0.2, 3), torch.full((rows,), 0.25, device="cuda")
    exact = Exact(x.contiguous(), w.contiguous(), None, t, 1.0)
    loss, lse = forward(x, w, None, t, 1.0)
    exact.check_forward(loss, lse)
    exact.check_backward(grad, *backward(x, w, None, t, 1.0, lse, grad, gx, gw))


def test_captured_with_copies_and_shares():
    """Captured and replayed at sizes with copied weights, shares of the items and of the rows, beside eager calls."""
    for rows, items, width in ((30, 40003, 13), (9000, 3000, 100), (70, 9001, 301), (20, 9001, 301)):
        x, w = matrix(rows, width, F16, 1), matrix(items, width, F16, 2, width ** -0.5)
        t, bias = some_targets(rows, items, 0.2, 3), matrix(1, items, torch.float32, 4)[0]
        grad, loss, lse = torch.full((rows,), 0.5, device="cuda"), torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
        gx, gw, gb = torch.empty_like(x), torch.empty_like(w), torch.empty_like(bias)
        fws = tbe.workspace(tbe.tbe_cross_entropy_forward_workspace_bytes(rows, items, width))
        bws = tbe.workspace(tbe.tbe_cross_entropy_backward_workspace_bytes(rows, items, width))
        stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
        stream.wait_stream(torch.cuda.current_stream())
        with torch.cuda.graph(graph, stream=stream):
            tbe.tbe_cross_entropy_forward(x, w, bias, t, 1.1, loss, lse, fws)
            tbe.tbe_cross_entropy_backward(x, w, bias, t, 1.1, lse, grad, gx, gw, gb, bws)
        for seed in range(3):
            t.copy_(some_targets(rows, items, (0.0, 0.9, 1.0)[seed], 30 + seed))
            w.copy_(matrix(items, width, F16, 40 + seed, width ** -0.5))
            graph.replay()
            torch.cuda.synchronize()
            e_loss, e_lse = forward(x, w, bias, t, 1.1)
            e = (e_loss, e_lse) + backward(x, w, bias, t, 1.1, e_lse, grad)
            for name, a, b in zip(("loss", "lse", "grad_x", "grad_weight", "grad_bias"), (loss, lse, gx, gw, gb), e):
                assert torch.equal(a, b), f"{rows} {items} {width} replay {seed}: {name}"
