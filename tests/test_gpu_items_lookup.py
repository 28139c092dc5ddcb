"""Scaled lookup and the table's dense gradient on the GPU, against their definitions in 64 bits.

Tolerances, with u = 2^-24 and t the unit roundoff of the stored type: a product is off by u, a stored result by t (fp16
below its normal range by half a subnormal step).  A gradient's sum of m terms in fp32 is off by at most d u times the sum
of their |terms|, where d is the longest chain of additions: m, or at most 128 positions of a share and 64 taken over, a
sixteenth of a row's shares one after the other (70000 positions of one id in shares of 16: 274) and 16 such sums."""
import pytest
import torch

import bwd_tbe_fwd_amd as tbe
from gpu_util import flush_print

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
UNIT = {torch.float32: U, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
LEAST = {torch.float32: 0.0, torch.float16: 2.0 ** -25, torch.bfloat16: 0.0}
F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16


def matrix(rows, width, dtype, seed, stride=None, scale=1.0, offset=0):
    """Rows `stride` apart, from `offset` elements into their buffer on; NaN between the rows."""
    g = torch.Generator().manual_seed(seed)
    stride = stride or width
    buf = torch.full((offset + rows * stride,), float("nan"), dtype=dtype)
    m = buf[offset:].view(rows, stride)[:, :width]
    m.copy_(torch.randn(rows, width, generator=g) * scale)
    buf = buf.cuda()
    return buf[offset:].view(rows, stride)[:, :width]


def some_ids(n, E, kind, seed, dtype=torch.int64):
    g = torch.Generator().manual_seed(seed)
    ids = torch.randint(0, E, (n,), generator=g)
    if kind == "padded":
        ids[torch.rand(n, generator=g) < 0.3] = -1
        ids[torch.rand(n, generator=g) < 0.1] = E
        ids[torch.rand(n, generator=g) < 0.05] = 2 ** 31 - 1 if dtype == torch.int32 else 2 ** 40 + 1
    elif kind == "hot":
        ids[torch.rand(n, generator=g) < 0.6] = E // 2
    elif kind == "one":
        ids[:] = E - 1
    elif kind == "none":
        ids[:] = -7
    elif kind == "low":  # popular ids side by side
        ids = (E * torch.rand(n, generator=g) ** 8).long().clamp(max=E - 1)
    return ids.to(dtype)


def check(what, got, exp, tol):
    got, exp, tol = got.double().cpu(), exp.double().cpu(), tol.double().cpu()
    bad = ~((got - exp).abs() <= tol)
    if bad.any():
        i = tuple(bad.nonzero()[0].tolist())
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} off; first at {i}: {got[i]!r}, exact {exp[i]!r}, "
                             f"tolerance {tol[i]!r}")


def scale32(scale):
    return float(torch.tensor(scale, dtype=torch.float32))


@pytest.mark.parametrize("n,E,width,tt,yt,itype,kind", [
    (1, 1, 1, F32, F32, torch.int64, "any"), (64, 1000, 1024, BF16, BF16, torch.int32, "any"),
    (63, 100, 8, F16, BF16, torch.int64, "padded"), (517, 3001, 515, F32, BF16, torch.int32, "padded"),
    (4097, 77, 100, BF16, F32, torch.int64, "hot"), (1000, 50, 1500, F16, F16, torch.int64, "padded"),
    (33, 9, 4096, F32, F16, torch.int64, "any"), (20011, 500, 4, F32, F32, torch.int32, "padded"),
    (300, 40, 129, BF16, F16, torch.int64, "none"), (257, 31, 3, BF16, BF16, torch.int64, "padded")])
def test_forward(n, E, width, tt, yt, itype, kind):
    flush_print(f"lookup forward {n} {E} {width} {tt} {yt} {kind}")
    for stride, offset, scale in ((width, 0, 1.0), (width + 8, 8, width ** 0.5), (width + 3, 1, -0.37)):
        table = matrix(E, width, tt, 1, stride, offset=offset)
        ids = some_ids(n, E, kind, 2, itype).cuda()
        y = matrix(n, width, yt, 3, stride, offset=offset)
        full = y.as_strided((n * stride,), (1,), y.storage_offset())[:(n - 1) * stride + width]
        before = full.clone()
        tbe.tbe_lookup_forward(table, ids, scale, y)
        there = (ids >= 0) & (ids < E)
        exp = torch.where(there[:, None], table[torch.where(there, ids, 0).long()].double() * scale32(scale), 0.0)
        check("y", y, exp, (UNIT[yt] + 1.01 * U) * exp.abs() + LEAST[yt])
        after, keep = full.clone(), torch.ones(full.numel(), dtype=torch.bool, device="cuda")
        for k in (before, after, keep):
            k.as_strided((n, width), (stride, 1)).fill_(0)
        assert torch.equal(before.isnan() & keep, after.isnan() & keep), "values between the rows were written"


def gradient(ids, gy, scale, E):
    there = (ids >= 0) & (ids < E)
    k, g = ids[there].long(), gy[there].double() * scale32(scale)
    exp = torch.zeros(E, gy.shape[1], dtype=torch.float64, device="cuda").index_put_((k,), g, accumulate=True)
    mag = torch.zeros_like(exp).index_put_((k,), g.abs(), accumulate=True)
    count = torch.bincount(k, minlength=E).double()[:, None]
    return exp, mag, count


BACKWARD = [
    (1, 1, 1, F32, F32, torch.int64, "any"), (1, 5, 8, BF16, BF16, torch.int64, "any"), (0, 37, 24, BF16, F32, torch.int64, "any"),
    (64, 1000, 1024, BF16, BF16, torch.int32, "any"), (65, 3, 40, F16, BF16, torch.int64, "any"),
    (517, 3001, 515, BF16, F32, torch.int32, "padded"), (4096, 1000, 128, F16, F16, torch.int64, "hot"),
    (4097, 1000, 128, F16, F16, torch.int64, "hot"), (4095, 20, 100, F32, F32, torch.int32, "one"),
    (9000, 50021, 16, BF16, F32, torch.int64, "low"), (30000, 70, 72, F32, BF16, torch.int64, "padded"),
    (70000, 513, 8, F32, F32, torch.int64, "one"), (20011, 5000, 1001, BF16, F16, torch.int64, "hot"),
    (129, 17, 1500, F16, F32, torch.int64, "padded"), (3000, 11, 4096, BF16, BF16, torch.int64, "hot"),
    (5000, 2, 33, F32, F32, torch.int64, "none"), (12000, 1 << 21, 4, BF16, BF16, torch.int64, "low"),
    (777, 1, 260, BF16, F32, torch.int32, "padded")]


@pytest.mark.parametrize("add", [False, True])
@pytest.mark.parametrize("n,E,width,yt,tt,itype,kind", BACKWARD)
def test_backward(n, E, width, yt, tt, itype, kind, add):
    flush_print(f"lookup backward {n} {E} {width} {yt} {tt} {kind} add={add}")
    for stride, offset, scale in ((width, 0, 1.0), (width + 5, 3, 2.3)):
        ids = some_ids(n, E, kind, 5, itype).cuda()
        gy = matrix(n, width, yt, 6, stride, offset=offset)
        there = (ids >= 0) & (ids < E)
        gy[~there] = float("nan")  # what padded positions hold does not matter
        grad = matrix(E, width, tt, 7, stride, 0.5, offset)
        old = grad.clone()
        need = tbe.tbe_lookup_backward_workspace_bytes(n, E, width)
        ws = torch.full((need + 4096,), 0xA5, dtype=torch.uint8, device="cuda")
        tbe.tbe_lookup_backward(ids, gy, scale, grad, ws[:need], accumulate=add)
        exp, mag, count = gradient(ids, gy, scale, E)
        chain = torch.minimum(count, torch.tensor(512.0, device="cuda", dtype=torch.float64)) + 3
        tol = chain * U * mag
        if add:
            exp = exp + old.double()
            tol = tol + 2 * U * old.double().abs()
        check("grad", grad, exp, tol + UNIT[tt] * (exp.abs() + tol) + LEAST[tt])
        if add:  # rows that no id names keep their bits
            untouched = (count == 0)[:, 0]
            assert torch.equal(grad[untouched], old[untouched])
        assert bool((ws[need:] == 0xA5).all()), "bytes behind the workspace were written"
        again = old.clone() if add else torch.empty_like(old)
        tbe.tbe_lookup_backward(ids, gy, scale, again, ws[:need], accumulate=add)
        assert torch.equal(again, grad), "another result for the same inputs"


def test_added_rows_that_no_id_names_keep_what_they_hold():
    E, width = 300, 64
    grad = torch.full((E, width), float("nan"), dtype=BF16, device="cuda")
    ids = torch.arange(0, E, 3, device="cuda").repeat(3)
    grad[::3] = 1.0
    gy = torch.ones(ids.numel(), width, dtype=BF16, device="cuda")
    ws = tbe.workspace(tbe.tbe_lookup_backward_workspace_bytes(ids.numel(), E, width))
    tbe.tbe_lookup_backward(ids, gy, 2.0, grad, ws, accumulate=True)
    assert bool((grad[::3] == 7.0).all()) and bool(grad[1::3].isnan().all()) and bool(grad[2::3].isnan().all())


def test_values_that_are_not_finite_stay_in_their_rows():
    E, width = 50, 24
    table = matrix(E, width, F32, 1)
    table[7, 3], table[8, 0] = float("inf"), float("nan")
    ids = torch.tensor([7, 8, 9, -1, 7], device="cuda")
    y = torch.empty(5, width, device="cuda")
    tbe.tbe_lookup_forward(table, ids, float("inf"), y)  # padding is zero whatever the scale is
    assert bool((y[3] == 0).all())
    tbe.tbe_lookup_forward(table, ids, 0.5, y)
    assert y[0, 3] == float("inf") and bool(y[1, 0].isnan()) and int((~y.isfinite()).sum()) == 3
    grad = torch.empty(E, width, device="cuda")
    ws = tbe.workspace(tbe.tbe_lookup_backward_workspace_bytes(5, E, width))
    tbe.tbe_lookup_backward(ids, y, 1.0, grad, ws)
    assert int((~grad.isfinite()).sum()) == 2 and bool((grad[10:] == 0).all())


def test_rows_past_32_bits():
    E, width, stride = 70001, 8, 65544  # the last row starts 4.59e9 elements behind the first
    buf = torch.empty(E * stride, dtype=F16, device="cuda")
    table = buf.view(E, stride)[:, :width]
    ids = torch.tensor([0, E - 1, 65535, 65536, E - 1], device="cuda")
    table[ids] = torch.arange(1, 6, device="cuda").half()[:, None].expand(5, width)
    y = torch.empty(5, width, dtype=F16, device="cuda")
    tbe.tbe_lookup_forward(table, ids, 2.0, y)
    assert torch.equal(y, table[ids] * 2)
    table[ids] = 1.0
    ws = tbe.workspace(tbe.tbe_lookup_backward_workspace_bytes(5, E, width))
    tbe.tbe_lookup_backward(ids, y, 1.0, table, ws, accumulate=True)
    assert torch.equal(table[ids[2:4]], y[2:4] + 1) and torch.equal(table[E - 1], y[1] + y[4] + 1)


def test_gradient_against_differences():
    """The sum of y * c over all positions changes by the gradient times a step of the table."""
    E, width, n = 13, 20, 90
    table, ids = matrix(E, width, F32, 1), some_ids(n, E, "padded", 2).cuda()
    c = matrix(n, width, F32, 3)
    grad, y = torch.empty(E, width, device="cuda"), torch.empty(n, width, device="cuda")
    ws = tbe.workspace(tbe.tbe_lookup_backward_workspace_bytes(n, E, width))
    tbe.tbe_lookup_backward(ids, c, 1.7, grad, ws)

    def value(t):
        tbe.tbe_lookup_forward(t, ids, 1.7, y)
        return float((y.double() * c.double()).sum())

    for v, d in ((0, 0), (5, 7), (12, 19)):
        step = torch.zeros_like(table)
        step[v, d] = 0.5
        # linear: the difference is exact but for the roundings of y, u |y| |c| each
        tol = 4 * U * float((table.abs().max() + 1) * 1.7 * c.abs().sum())
        assert abs(value(table + step) - value(table - step) - float(grad[v, d])) <= tol


def test_captured_and_replayed_beside_eager_work():
    E, width = 4000, 136
    for n in (300, 9000):
        ids, table = some_ids(n, E, "hot", 1).cuda(), matrix(E, width, BF16, 2)
        gy = matrix(n, width, BF16, 3)
        y, grad = torch.empty(n, width, dtype=BF16, device="cuda"), torch.empty(E, width, dtype=F32, device="cuda")
        ws = tbe.workspace(tbe.tbe_lookup_backward_workspace_bytes(n, E, width))
        stream = torch.cuda.Stream()
        stream.wait_stream(torch.cuda.current_stream())
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            tbe.tbe_lookup_forward(table, ids, 3.0, y)
            tbe.tbe_lookup_backward(ids, gy, 3.0, grad, ws)
        eager_ws = tbe.workspace(tbe.tbe_lookup_backward_workspace_bytes(n, E, width))
        for seed in range(4):
            ids.copy_(some_ids(n, E, ("hot", "padded", "low", "one")[seed], 10 + seed))
            gy.copy_(matrix(n, width, BF16, 20 + seed))
            graph.replay()
            torch.cuda.synchronize()
            ye, ge = torch.empty_like(y), torch.empty_like(grad)
            tbe.tbe_lookup_forward(table, ids, 3.0, ye)
            tbe.tbe_lookup_backward(ids, gy, 3.0, ge, eager_ws)
            assert torch.equal(y, ye) and torch.equal(grad, ge), f"replay {seed}"


def test_two_streams_with_a_workspace_each():
    E, width, n = 3000, 256, 6000
    side = [torch.cuda.Stream() for _ in range(2)]
    ids = [some_ids(n, E, k, 1).cuda() for k in ("hot", "low")]
    gy = [matrix(n, width, BF16, 2 + i) for i in range(2)]
    grad = [torch.empty(E, width, device="cuda") for _ in range(2)]
    ws = [tbe.workspace(tbe.tbe_lookup_backward_workspace_bytes(n, E, width)) for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(3):
        for i in range(2):
            tbe.tbe_lookup_backward(ids[i], gy[i], 1.0, grad[i], ws[i], stream=side[i])
    torch.cuda.synchronize()
    for i in range(2):
        alone = torch.empty_like(grad[i])
        tbe.tbe_lookup_backward(ids[i], gy[i], 1.0, alone, ws[0])
        assert torch.equal(alone, grad[i])
