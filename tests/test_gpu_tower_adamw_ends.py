"""AdamW's states of 8 bits at the ends of their range, on the GPU: bit for bit against a quantiser in
64 bits."""
import pytest
import torch

import bwd_tbe_fwd_amd as tbe
from test_gpu_tower_adamw import BLOCK, Tensor, pack, plan_of

pytestmark = pytest.mark.gpu
F32 = torch.float32


def stepped(g, b1, b2, **kw):
    """One step from zero states of 8 bits; the codes against the quantiser in 64 bits."""
    t = Tensor(g.numel(), F32, F32, True, False, 0.0, 5)
    t.g = g
    t.dg.copy_(g)
    for buf in (t.dm, t.dv, t.dme, t.dve):
        buf.zero_()
    t.m, t.v = torch.zeros(g.numel()), torch.zeros(g.numel())
    tbe.tbe_adamw_step(plan_of([t]), 1, 1e-3, b1, b2, **kw)
    torch.cuda.synchronize()
    t.expect(1, 1e-3, b1, b2, 1e-8)
    return t


def test_second_moments_of_a_wide_block_stay_above_zero():
    """Values a factor of 2^149 and more below their block's largest."""
    g = torch.zeros(3 * BLOCK)
    g[0], g[1], g[2], g[100] = 3.2e5, 3.2e-19, 1e-15, 0.0      # 1e8, 1e-40, 1e-33
    g[BLOCK:2 * BLOCK] = 2.0 ** -torch.arange(BLOCK).float()   # 2^0 down to 2^-127
    g[BLOCK] = 2.0 ** 60
    g[2 * BLOCK:] = 1e-20
    t = stepped(g, 0.9, 0.999)
    code, e = pack(t.v, True)
    assert (t.v[[0, 1, 2]] > 0).all()
    assert torch.equal(t.dve.cpu(), e) and torch.equal(t.dv.cpu(), code)
    assert (t.dv.cpu()[t.v > 0] > 0).all() and not t.dv.cpu()[t.v == 0].any()
