"""Grouped products with far more experts than rows, and wide results: as many tiles as the experts that have rows
take, not as all experts could."""
import pytest
import torch

import bwd_tbe_fwd_amd as tbe
from test_gpu_tower_norm import U, UNIT, check

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


def test_few_rows_of_very_many_experts():
    E, outer, rows, owners = 65535, 16400, 3, (5, 40000, 65534)
    g = torch.Generator(device="cuda").manual_seed(1)
    w = torch.randn(E, outer, 1, generator=g, device="cuda", dtype=BF16)
    x = torch.randn(rows, 1, generator=g, device="cuda", dtype=BF16)
    gy = torch.randn(rows, outer, generator=g, device="cuda", dtype=BF16)
    counts = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    for e in owners:
        counts[e + 1] = 1
    off = torch.cumsum(counts, 0).to(torch.int32)
    y = torch.full((rows, outer), float("nan"), dtype=BF16, device="cuda")
    tbe.tbe_grouped_linear_forward(x, w, None, off, y)
    own = w[list(owners), :, 0].double()
    exp = own * x.double()
    check("y", y, exp, (UNIT[BF16] + 2 * U) * exp.abs())
    gx = torch.full((rows, 1), float("nan"), dtype=BF16, device="cuda")
    tbe.tbe_grouped_linear_backward_input(gy, w, off, gx)
    exp = (gy.double() * own).sum(1, keepdim=True)
    terms = (gy.double() * own).abs().sum(1, keepdim=True)
    check("grad_x", gx, exp, UNIT[BF16] * exp.abs() + 2 * U * (outer / 8 + 32) * terms)
    gw, gb = torch.full_like(w, float("nan")), torch.full((E, outer), float("nan"), dtype=BF16, device="cuda")
    ws = tbe.workspace(tbe.tbe_grouped_linear_backward_weight_workspace_bytes(rows, E, 1, outer))
    tbe.tbe_grouped_linear_backward_weight(x, gy, off, gw, gb, ws)
    exp = gy.double() * x.double()
    check("grad_weight", gw[list(owners), :, 0], exp, (UNIT[BF16] + 2 * U) * exp.abs())
    assert torch.equal(gb[list(owners)], gy)
    gw[list(owners)], gb[list(owners)] = 0, 0
    assert not gw.any() and not gb.any()
