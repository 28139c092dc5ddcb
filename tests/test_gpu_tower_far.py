"""The tower's operators where element offsets pass 32 bits: a few rows far apart in one buffer, and a
tensor of more than 2^32 values."""
import pytest
import torch

import bwd_tbe_fwd_amd as tbe
from gpu_util import flush_print
from test_gpu_tower_adamw import BLOCK, Tensor, opened, pack, plan_of
from test_gpu_tower_grouped import Case
from test_gpu_tower_norm import check_backward, check_forward, rows_of, vector

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16


def far(rows, like):
    """The rows of `like` with the largest stride that the operators take, over 2^32 bytes apart."""
    buf = torch.empty((rows - 1) * 2 ** 31 + like.shape[1], dtype=like.dtype, device="cuda")
    view = buf.as_strided((rows, like.shape[1]), (2 ** 31, 1))
    view.copy_(like)
    return view


def test_norm_rows_far_apart():
    flush_print("norm, rows 2^31 elements apart")
    x, gy = far(3, rows_of(3, 1000, BF16, 1)), far(3, rows_of(3, 1000, BF16, 2))
    w, b = vector(1000, F32, 3, 1.0), vector(1000, F32, 4, 0.0)
    y, mean, rstd = far(3, torch.zeros_like(x)), torch.empty(3, device="cuda"), torch.empty(3, device="cuda")
    tbe.tbe_layer_norm_forward(x, w, b, 1e-5, y, mean, rstd)
    check_forward(x.contiguous(), w, b, 1e-5, y.contiguous(), mean, rstd)
    gw, gb = torch.empty(1000, device="cuda"), torch.empty(1000, device="cuda")
    ws = tbe.workspace(tbe.tbe_layer_norm_backward_workspace_bytes(3, 1000))
    tbe.tbe_layer_norm_backward(x, gy, mean, rstd, w, y, gw, gb, ws)
    check_backward(x.contiguous(), gy.contiguous(), w, y.contiguous(), gw, gb, mean, rstd)


def test_grouped_rows_far_apart():
    flush_print("grouped, rows 2^31 elements apart")
    c = Case([2, 0, 1], 136, 72, BF16)
    c.x, c.gy = far(3, c.x), far(3, c.gy)
    c.all()
    y = far(3, torch.zeros(3, 72, dtype=BF16, device="cuda"))
    tbe.tbe_grouped_linear_forward(c.x, c.w, c.b, c.off, y)
    near = torch.empty(3, 72, dtype=BF16, device="cuda")
    tbe.tbe_grouped_linear_forward(c.x, c.w, c.b, c.off, near)
    assert torch.equal(y, near)


def test_adamw_past_32_bits():
    """The last blocks of a tensor of 2^32 + 900 values step as a small tensor of their own."""
    flush_print("adamw, 2^32 + 900 values")
    n, tail = 2 ** 32 + 900, 900
    t = Tensor(tail, BF16, BF16, True, False, 0.01, 11)
    big = {k: torch.zeros(m, dtype=d, device="cuda") for k, m, d in (
        ("dp", n, BF16), ("dg", n, BF16), ("dm", n, torch.uint8), ("dv", n, torch.uint8),
        ("dme", -(-n // BLOCK), torch.uint8), ("dve", -(-n // BLOCK), torch.uint8))}
    for k, v in big.items():  # 2^32 is a whole number of blocks
        part = getattr(t, k)
        v[v.numel() - part.numel():] = part
    plan = tbe.AdamWTensors([big["dp"]], [big["dg"]], [big["dm"]], [big["dv"]], weight_decay=0.01,
                            exp_avg_scales=[big["dme"]], exp_avg_sq_scales=[big["dve"]])
    tbe.tbe_adamw_step(plan, 3, 1e-2)
    tbe.tbe_adamw_step(plan_of([t]), 3, 1e-2)
    torch.cuda.synchronize()
    for k, v in big.items():
        assert torch.equal(v[v.numel() - getattr(t, k).numel():], getattr(t, k)), k
    assert not big["dp"][:2 ** 32].any() and not big["dm"][:2 ** 32].any()
    out = [torch.empty(n, dtype=BF16, device="cuda") for _ in range(2)]
    tbe.tbe_adamw_state_read(plan, [out[0]], [out[1]])
    t.expect(3, 1e-2, 0.9, 0.999, 1e-8)
    for got, x, second in ((out[0], t.m, False), (out[1], t.v, True)):
        assert torch.equal(got[-tail:].float().cpu(), opened(*pack(x, second), second))
