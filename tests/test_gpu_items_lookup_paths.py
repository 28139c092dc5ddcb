"""The lookup's gradient where its sort changes, and tables of the largest number of rows.  Tolerances as in
test_gpu_items_lookup.py."""
import pytest
import torch

import bwd_tbe_fwd_amd as tbe
from gpu_util import flush_print
from test_gpu_items_lookup import BF16, F16, F32, LEAST, U, UNIT, check, gradient, matrix, some_ids

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n,E,width,yt,tt,itype,kind", [
    (8191, 59276, 8, F16, F16, torch.int64, "padded"), (8192, 300, 64, BF16, F32, torch.int32, "hot"),
    (8193, 300, 64, BF16, F32, torch.int32, "hot"), (6000, 5000000, 4, F32, F32, torch.int64, "low"),
    (8192, 9, 24, F32, BF16, torch.int64, "one"), (8192, 100, 16, BF16, BF16, torch.int64, "none"),
    (1023, 40, 12, F16, F32, torch.int32, "any"), (1025, 40, 12, F16, F32, torch.int32, "any")])
def test_ids_sorted_by_counting(n, E, width, yt, tt, itype, kind):
    flush_print(f"lookup backward {n} {E} {width} {yt} {tt} {kind}")
    for add in (False, True):
        ids, gy, grad = some_ids(n, E, kind, 5, itype).cuda(), matrix(n, width, yt, 6), matrix(E, width, tt, 7, scale=0.5)
        gy[~((ids >= 0) & (ids < E))] = float("nan")
        old = grad.clone()
        tbe.tbe_lookup_backward(ids, gy, 1.5, grad, tbe.workspace(tbe.tbe_lookup_backward_workspace_bytes(n, E, width)), accumulate=add)
        exp, mag, count = gradient(ids, gy, 1.5, E)
        tol = (torch.minimum(count, torch.tensor(512.0, device="cuda", dtype=torch.float64)) + 3) * U * mag
        if add:
            exp, tol = exp + old.double(), tol + 2 * U * old.double().abs()
        check("grad", grad, exp, tol + UNIT[tt] * (exp.abs() + tol) + LEAST[tt])


def test_the_largest_table():
    """2^31 - 2 rows of one value."""
    items, n = (1 << 31) - 2, 5000
    table = torch.empty(items, 1, dtype=BF16, device="cuda").normal_(generator=torch.Generator("cuda").manual_seed(1))
    ids = torch.randint(0, items, (n,), generator=torch.Generator().manual_seed(2))
    ids[:4] = torch.tensor([items - 1, 0, items, items - 1])
    ids = ids.cuda()
    there = ids < items
    y = torch.empty(n, 1, dtype=F32, device="cuda")
    tbe.tbe_lookup_forward(table, ids, 2.0, y)
    assert torch.equal(y[there], table[ids[there]].float() * 2) and bool((y[~there] == 0).all())
    gy = matrix(n, 1, BF16, 3)
    named, which = torch.unique(ids[there], return_inverse=True)
    exp = torch.zeros(len(named), 1, dtype=torch.float64, device="cuda").index_put_((which,), gy[there].double(), accumulate=True)
    ws = tbe.workspace(tbe.tbe_lookup_backward_workspace_bytes(n, items, 1))
    old = table[named].double()
    for add in (True, False):
        tbe.tbe_lookup_backward(ids, gy, 1.0, table, ws, accumulate=add)
        want = exp + old if add else exp
        assert bool(((table[named].double() - want).abs() <= 2.0 ** -8 * want.abs() + 8 * U * (exp.abs() + old.abs()) + 1e-38).all())
    there = 0
    for v in range(0, items, 1 << 28):
        there += int(torch.count_nonzero(table[v:v + (1 << 28)]))
    assert there == int(torch.count_nonzero(table[named])) and there > n * 0.99


def test_the_largest_number_of_items():
    rows, items = 2, (1 << 31) - 2
    w = torch.empty(items, 1, dtype=BF16, device="cuda").normal_(generator=torch.Generator("cuda").manual_seed(1))
    x, t = torch.tensor([[0.5], [-1.0]], dtype=BF16, device="cuda"), torch.tensor([items - 1, 3], device="cuda")
    loss, lse = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    tbe.tbe_cross_entropy_forward(x, w, None, t, 1.0, loss, lse, tbe.workspace(tbe.tbe_cross_entropy_forward_workspace_bytes(rows, items, 1)))
    total, mean = [torch.zeros(rows, dtype=torch.float64, device="cuda") for _ in range(2)]
    for v in range(0, items, 1 << 26):
        some = w[v:v + (1 << 26)].double()
        p = (some * x.double()[:, 0]).exp()
        total += p.sum(0)
        mean += (p * some).sum(0)
    exact = total.log()
    # sums of e^l: chains of fewer than 4096 additions of values off by 100 roundings, in each of the pieces and over them
    assert bool(((lse.double() - exact).abs() <= 4500 * U).all())
    assert bool(((loss.double() - (exact - (w[t].double() * x.double())[:, 0])).abs() <= 4600 * U).all())
    gx, gw = torch.empty_like(x), torch.empty_like(w)
    grad = torch.ones(rows, device="cuda")
    tbe.tbe_cross_entropy_backward(x, w, None, t, 1.0, lse, grad, gx, gw, None,
                                   tbe.workspace(tbe.tbe_cross_entropy_backward_workspace_bytes(rows, items, 1)))
    # p around 2^-31 rounded to bf16 one by one, without a bias of their sum beyond 2^-8 of the sum of |w| p (below 1.2)
    want = mean / total - w[t].double()[:, 0]
    assert bool(((gx.double()[:, 0] - want).abs() <= 2.0 ** -8 * (1.2 + want.abs()) + 1e-3).all())
    for v in (0, items - 4096, 1 << 30):
        p = (w[v:v + 4096].double() * x.double()[:, 0] - exact).exp()
        for i in range(rows):
            if v <= int(t[i]) < v + 4096:
                p[int(t[i]) - v, i] -= 1
        z = p * x.double()[:, 0]
        assert bool(((gw[v:v + 4096, 0].double() - z.sum(1)).abs() <= 2.0 ** -7 * z.abs().sum(1) + 1e-12).all())
