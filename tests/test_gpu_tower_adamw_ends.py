"""AdamW's states of 8 bits at the ends of their range, and the roundings of a step with states of 32 bits,
on the GPU: bit for bit against a quantiser in 64 bits and fp32 operations on the CPU."""
import math

import pytest
import torch

import bwd_tbe_fwd_amd as tbe
from gpu_util import flush_print
from test_gpu_tower_adamw import BLOCK, Tensor, opened, pack, plan_of

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16


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


def test_finite_moments_beyond_the_codes_range_take_its_ends():
    """The scale byte stops at 250: larger finite moments take the largest code, and do not become NaN."""
    g = torch.zeros(3 * BLOCK)
    g[:8] = torch.tensor([3e38, -3e38, 1e38, -5e37, 2.5e37, 3.7e37, 3.75e37, 1.0])
    g[BLOCK:BLOCK + 4] = torch.tensor([1.8e19, 1.6e19, 4e18, -1e10])
    t = stepped(g, 0.0, 0.0)
    for got, scale, x, second in ((t.dm, t.dme, t.m, False), (t.dv, t.dve, t.v, True)):
        code, e = pack(torch.where(x.isfinite(), x, 0.0), second)
        assert torch.equal(scale.cpu(), e)
        keep = x.isfinite()
        assert torch.equal(got.cpu()[keep], code[keep])
    m = torch.empty(3 * BLOCK, device="cuda")
    v = torch.empty(3 * BLOCK, device="cuda")
    tbe.tbe_adamw_state_read(plan_of([t]), [m], [v])
    assert m.isfinite().all() and torch.equal(v.isfinite().cpu(), t.v.isfinite())
    assert float(m[0]) == 448 * 2.0 ** 116 and float(m[1]) == -448 * 2.0 ** 116 and float(v[BLOCK]) == 3.5 * 2.0 ** 123


def test_reading_every_code_in_16_bits():
    """bf16 holds every value from 2^-126 on; smaller second moments are rounded to nearest, above zero all."""
    code = torch.arange(256, dtype=torch.uint8).repeat(6)
    e = torch.tensor([24, 24, 25, 25, 26, 26, 27, 27, 40, 40, 250, 250], dtype=torch.uint8)
    n = code.numel()
    flat = torch.zeros(n, device="cuda")
    plan = tbe.AdamWTensors([flat], [flat], [code.cuda()], [code.cuda()], exp_avg_scales=[e.cuda()], exp_avg_sq_scales=[e.cuda()])
    m, v = (torch.empty(n, dtype=BF16, device="cuda") for _ in range(2))
    tbe.tbe_adamw_state_read(plan, [m], [v])
    for got, second in ((m.cpu(), False), (v.cpu(), True)):
        exp = opened(code, e, second)
        assert torch.equal(got.isnan(), exp.isnan())
        ok = ~exp.isnan()
        assert torch.equal(got[ok], exp[ok].bfloat16())
        held = ok & (exp.abs() >= 2.0 ** -126)
        assert torch.equal(got[held].float(), exp[held])
        assert ((got != 0) == (exp != 0))[ok].all()


@pytest.mark.parametrize("p,g", [(F32, F32), (BF16, F32), (BF16, BF16)])
def test_each_operation_of_a_32_bit_step_is_rounded_by_itself(p, g):
    """Weights bit for bit against fp32 operations on the CPU, one rounding each (fp32 weights or masters)."""
    flush_print("adamw rounding", p, g)
    n, step, lr, b1, b2, eps = 20011, 17, 3e-3, 0.9, 0.99, 1e-8
    f = lambda x: torch.tensor(x, dtype=torch.float32)  # noqa: E731
    for decay in (0.0, 0.1):
        t = Tensor(n, p, g, False, p != F32, decay, 700)
        p0, m0, v0 = t.p0.clone(), t.m.clone(), t.v.clone()
        v0[:4000] *= 1e-42  # among them roots of subnormal numbers
        t.dv[:4000] = v0[:4000].cuda()
        t.dg[:2000] = 0
        gr = t.dg.cpu().float()
        tbe.tbe_adamw_step(plan_of([t]), step, lr, b1, b2, eps)
        torch.cuda.synchronize()
        m = m0 * f(b1) + gr * f(1 - b1)
        v = v0 * f(b2) + gr * gr * f(1 - b2)
        keep = f(1.0) - f(lr) * f(decay)
        size, root = f(lr / (1 - b1 ** step)), f(1 / math.sqrt(1 - b2 ** step))
        # (the root through 64 bits, which rounds to the nearest fp32; torch's fp32 one on the CPU does not always)
        w = p0 * keep - size * m / (v.double().sqrt().float() * root + f(eps))
        assert torch.equal(t.dm.cpu(), m) and torch.equal(t.dv.cpu(), v)
        got = t.dp if t.dw is None else t.dw
        assert torch.equal(got.cpu(), w)
        assert torch.equal(t.dp.cpu(), w.to(p))
