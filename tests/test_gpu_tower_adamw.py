"""AdamW on the GPU: moments and their 8-bit codes bit for bit against fp32 operations rounded one
by one on the CPU and a quantiser written on floats in 64 bits, weights against the step in 64 bits.

Tolerance of a weight, with u = 2^-24 and t its type's unit roundoff: the step's terms pass through
at most 8 roundings each, and sqrt and the division through one of at most 2 u:
t |p| + 16 u (|p| + |step terms|)."""
import math

import pytest
import torch

import bwd_tbe_fwd_amd as tbe
from gpu_util import flush_print
from test_gpu_tower_norm import LEAST, U, UNIT, check

pytestmark = pytest.mark.gpu
F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16
BLOCK = tbe.TBE_ADAMW_BLOCK


def randn(n, seed, scale=1.0):
    return torch.randn(n, generator=torch.Generator().manual_seed(seed)) * scale


def code_values_m():
    """The 256 values of an e4m3 byte."""
    out = []
    for c in range(256):
        s, e, f = c >> 7, (c >> 3) & 15, c & 7
        v = math.nan if (e, f) == (15, 7) else (f / 8 * 2.0 ** -6 if e == 0 else (1 + f / 8) * 2.0 ** (e - 7))
        out.append(-v if s else v)
    return torch.tensor(out, dtype=torch.float64)


def code_values_v():
    """The 256 values of an unsigned byte of 5 exponent and 3 mantissa bits: (1 + f/8) 2^(e - 30)."""
    out = [0.0] + [(1 + (c & 7) / 8) * 2.0 ** ((c >> 3) - 30) for c in range(1, 255)] + [math.nan]
    return torch.tensor(out, dtype=torch.float64)


M_VALUES, V_VALUES = code_values_m(), code_values_v()


def blocks_of(x):
    pad = -x.numel() % BLOCK
    return torch.cat([x, x.new_zeros(pad)]).view(-1, BLOCK)


def pack(x, second):
    """Codes and scale bytes of fp32 values x, by search for the nearest value (ties to even codes)."""
    b = blocks_of(x).double()
    top = b.abs().amax(1)
    e = torch.where(top > 0, torch.frexp(top)[1] - 1 + 127, 0).clamp(24, 250)
    unit = torch.pow(2.0, e.double() - (127 if second else 134))[:, None]
    r = b / unit
    values = V_VALUES[:255] if second else M_VALUES[:127]  # ascending, not negative
    a = r.abs()
    hi = torch.searchsorted(values, a.contiguous()).clamp(1, len(values) - 1)
    lo = hi - 1
    dl, dh = a - values[lo], values[hi] - a
    code = torch.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
    if second:
        code = torch.where(a > 0, code.clamp(min=1), 0)
    else:
        code = torch.where(torch.signbit(r), code + 128, code)
    return code.to(torch.uint8).view(-1)[:x.numel()].clone(), e.to(torch.uint8)


def opened(code, e, second):
    v = (V_VALUES if second else M_VALUES)[code.long()]
    unit = torch.pow(2.0, e.double() - (127 if second else 134)).repeat_interleave(BLOCK)[:code.numel()]
    return (v * unit).float()  # exact


class Tensor:
    """One tensor of a step: its host values and its device buffers."""

    def __init__(self, n, p, g, eight, master, decay, seed, shift=0):
        self.p0 = randn(n, seed, 0.1)
        self.p0 = self.p0 if master else self.p0.to(p).float()
        self.g = randn(n, seed + 1, 1e-2).to(g)
        self.m, self.v = randn(n, seed + 2, 3e-3), randn(n, seed + 3, 1e-2).square()
        self.eight, self.decay, self.p_dtype = eight, decay, p
        if eight:
            self.mc, self.me = pack(self.m, False)
            self.vc, self.ve = pack(self.v, True)
            self.m, self.v = opened(self.mc, self.me, False), opened(self.vc, self.ve, True)

        def dev(t):  # `shift` elements into a larger buffer: aligned to the element only
            buf = torch.zeros(t.numel() + shift + 3, dtype=t.dtype, device="cuda")
            buf[shift:shift + t.numel()] = t.cuda()
            return buf[shift:shift + t.numel()]

        self.dp, self.dg = dev(self.p0.to(p)), dev(self.g)
        self.dw = dev(self.p0) if master else None
        if eight:
            self.dm, self.dv, self.dme, self.dve = dev(self.mc), dev(self.vc), dev(self.me), dev(self.ve)
        else:
            self.dm, self.dv, self.dme, self.dve = dev(self.m), dev(self.v), None, None

    def expect(self, step, lr, b1, b2, eps, factor=1.0):
        g = self.g.float() * factor
        self.m = self.m * b1 + g * (1 - b1)
        self.v = self.v * b2 + g * g * (1 - b2)
        md, vd, p = self.m.double(), self.v.double(), self.p0.double()
        upd = lr / (1 - b1 ** step) * md / (vd.sqrt() / math.sqrt(1 - b2 ** step) + eps)
        self.p = p * (1 - lr * self.decay) - upd
        self.tol = 16 * U * (p.abs() + upd.abs())

    def check(self, what):
        got = self.dp if self.dw is None else self.dw
        t = got.dtype
        check(what + " weights", got, self.p, UNIT[t] * self.p.abs() + LEAST[t] + self.tol)
        if self.dw is not None:
            assert torch.equal(self.dp, self.dw.to(self.p_dtype)), what
        if self.eight:
            for got, (code, e) in ((
                    (self.dm, self.dme), pack(self.m, False)), ((self.dv, self.dve), pack(self.v, True))):
                assert torch.equal(got[1].cpu(), e), what + ": scales"
                assert torch.equal(got[0].cpu(), code), what + ": codes"
        else:
            assert torch.equal(self.dm.cpu(), self.m) and torch.equal(self.dv.cpu(), self.v), what + ": moments"


def plan_of(ts):
    return tbe.AdamWTensors([t.dp for t in ts], [t.dg for t in ts], [t.dm for t in ts], [t.dv for t in ts],
                            weight_decay=[t.decay for t in ts], masters=[t.dw for t in ts],
                            exp_avg_scales=[t.dme for t in ts], exp_avg_sq_scales=[t.dve for t in ts])


SIZES = [1, 7, 8, 9, 127, 128, 129, 2047, 2048, 2049, 8191, 8192, 8193, 20000]


@pytest.mark.parametrize("eight", [False, True])
@pytest.mark.parametrize("p,g,master", [(F32, F32, False), (F32, BF16, False), (BF16, BF16, False), (BF16, F32, True),
                                        (BF16, BF16, True), (F16, F16, True), (F16, F32, False)])
def test_step(p, g, master, eight):
    flush_print("adamw", p, g, master, eight)
    ts = [Tensor(n, p, g, eight, master, 0.01 * (i % 2), 100 + 10 * i, shift=i % 3) for i, n in enumerate(SIZES)]
    plan = plan_of(ts)
    tbe.tbe_adamw_step(plan, 7, 1e-2, 0.9, 0.99, 1e-8)
    torch.cuda.synchronize()
    for t in ts:
        t.expect(7, 1e-2, 0.9, 0.99, 1e-8)
        t.check(f"n = {t.p0.numel()}")


def test_many_tensors_of_mixed_kinds():
    """More tensors than one launch takes, of several types, some without values."""
    kinds = [(F32, F32, False, False), (BF16, BF16, True, False), (BF16, BF16, True, True), (F32, F32, True, False)]
    ts = [Tensor([0, 5, 300, 9000, 128][i % 5], *[kinds[i % 4][k] for k in (0, 1)], kinds[i % 4][2], kinds[i % 4][3],
                 0.1, 1000 + 10 * i) for i in range(230)]
    tbe.tbe_adamw_step(plan_of(ts), 1, 1e-3)
    torch.cuda.synchronize()
    for i, t in enumerate(ts):
        t.expect(1, 1e-3, 0.9, 0.999, 1e-8)
        t.check(f"tensor {i}")


def test_several_steps_in_8_bits():
    ts = [Tensor(n, F32, F32, True, False, 0.01, 50 + n) for n in (300, 5000)]
    plan = plan_of(ts)
    for step in range(1, 6):
        tbe.tbe_adamw_step(plan, step, 1e-3)
        torch.cuda.synchronize()
        for t in ts:
            t.expect(step, 1e-3, 0.9, 0.999, 1e-8)
            t.check(f"step {step}")
            t.p0 = t.dp.cpu()  # the next step starts from the device's weights and the codes' values
            t.m, t.v = opened(*pack(t.m, False), False), opened(*pack(t.v, True), True)


def test_extreme_moments_in_8_bits():
    """Blocks of zeros, of one value, over 40 powers of two, at both ends of fp32's range."""
    n = 8 * BLOCK
    t = Tensor(n, F32, F32, True, False, 0.0, 5)
    g = torch.zeros(n)
    g[BLOCK] = 1.0
    g[2 * BLOCK:3 * BLOCK] = 2.0 ** -torch.arange(BLOCK).float().mul(0.25)
    g[3 * BLOCK:4 * BLOCK] = 1e-19
    g[4 * BLOCK:5 * BLOCK] = 1e18 * randn(BLOCK, 6)
    g[5 * BLOCK:6 * BLOCK] = 1e-30
    g[6 * BLOCK:] = 0.25
    t.g = g
    t.dg.copy_(g)
    for buf in (t.dm, t.dv, t.dme, t.dve):
        buf.zero_()  # zeroed bytes are zero states
    t.m, t.v = torch.zeros(n), torch.zeros(n)
    tbe.tbe_adamw_step(plan_of([t]), 1, 1e-3, eps=1e-12)
    torch.cuda.synchronize()
    t.expect(1, 1e-3, 0.9, 0.999, 1e-12)
    t.check("extreme")
    positive = t.v > 0
    assert (t.dv.cpu()[positive] > 0).all() and not t.dv.cpu()[~positive].any()


def test_state_read():
    for dtype in (F32, BF16):
        ts = [Tensor(n, BF16, BF16, True, False, 0.0, 70 + n, shift=n % 2) for n in [0] + SIZES] * 5
        plan = plan_of(ts)
        m = [torch.full((t.p0.numel(),), float("nan"), dtype=dtype, device="cuda") for t in ts]
        v = [torch.full((t.p0.numel(),), float("nan"), dtype=dtype, device="cuda") for t in ts]
        tbe.tbe_adamw_state_read(plan, m, v)
        torch.cuda.synchronize()
        for t, a, b in zip(ts, m, v):
            assert torch.equal(a.float().cpu(), t.m) and torch.equal(b.float().cpu(), t.v)
    # every code, at several scales
    n = 256 * 4
    code = torch.arange(256, dtype=torch.uint8).repeat(4)
    e = torch.tensor([0, 24, 24, 100, 127, 200, 250, 250], dtype=torch.uint8)
    flat = torch.zeros(n, device="cuda")
    plan = tbe.AdamWTensors([flat], [flat], [code.cuda()], [code.cuda()], exp_avg_scales=[e.cuda()], exp_avg_sq_scales=[e.cuda()])
    m, v = torch.empty(n, device="cuda"), torch.empty(n, device="cuda")
    tbe.tbe_adamw_state_read(plan, [m], [v])
    rest = e.repeat_interleave(BLOCK) > 0  # scale byte 0 only goes with zero codes
    for got, second in ((m, False), (v, True)):
        exp = opened(code, e, second)
        got = got.cpu()
        assert torch.equal(got.isnan()[rest], exp.isnan()[rest])
        ok = rest & ~exp.isnan()
        assert torch.equal(got[ok], exp[ok])


def test_bad_gradients_stay_visible():
    """An infinity or a NaN in a gradient leaves a NaN in its 8-bit moments, and none elsewhere."""
    t = Tensor(4 * BLOCK, F32, F32, True, False, 0.0, 9)
    t.dg[5] = float("nan")
    t.dg[2 * BLOCK + 1] = float("inf")
    tbe.tbe_adamw_step(plan_of([t]), 3, 1e-3)
    m, v = (torch.empty(4 * BLOCK, device="cuda") for _ in range(2))
    tbe.tbe_adamw_state_read(plan_of([t]), [m], [v])
    for x in (m, v, t.dp):
        assert x.isnan().nonzero()[:, 0].tolist() == [5, 2 * BLOCK + 1]
    t.expect(3, 1e-3, 0.9, 0.999, 1e-8)
    keep = torch.ones(4 * BLOCK, dtype=torch.bool)
    keep[[5, 2 * BLOCK + 1]] = False
    t.m[~keep], t.v[~keep] = 0.0, 0.0
    for got, second in ((t.dm, False), (t.dv, True)):
        assert torch.equal(got.cpu()[keep], pack(t.v if second else t.m, second)[0][keep])


def test_control():
    """The step, the factors and the skip from the device, in a graph whose replays see other values."""
    for eight in (False, True):
        ts = [Tensor(n, F32, F32, eight, False, 0.05, 300 + n) for n in (100, 9000)]
        control = torch.tensor([3.0, 0.5, 0.25, 0.0], dtype=torch.float64, device="cuda")
        plan = plan_of(ts)
        warm = plan_of([Tensor(64, F32, F32, eight, False, 0.0, 1)])
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            tbe.tbe_adamw_step(warm, 0, 1e-2, control=control)
        torch.cuda.current_stream().wait_stream(side)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            tbe.tbe_adamw_step(plan, 0, 1e-2, control=control)
        scratch = torch.randn(1 << 20, device="cuda")
        for step, lr, factor, skip in ((3, 0.5, 0.25, 0), (4, 0.25, 2.0, 0), (5, 1.0, 1.0, 1), (1000000, 1.0, 1.0, 0)):
            control.copy_(torch.tensor([step, lr, factor, skip], dtype=torch.float64))
            before = [t.dp.clone() for t in ts]
            g.replay()
            scratch.mul_(1.5).add_(float(step))
            torch.cuda.synchronize()
            for t, p in zip(ts, before):
                if skip:
                    assert torch.equal(t.dp, p)
                    continue
                t.expect(step, 1e-2 * lr, 0.9, 0.999, 1e-8, factor)
                t.check(f"step {step}")
                t.p0 = t.dp.cpu()
                if eight:
                    t.m, t.v = opened(*pack(t.m, False), False), opened(*pack(t.v, True), True)


def test_training_with_8_bits_follows_32():
    """A quadratic loss falls as it does with states of 32 bits."""
    n = 1000
    target, start = randn(n, 1).cuda(), randn(n, 2).cuda()
    losses = []
    for eight in (False, True):
        p, g = start.clone(), torch.empty(n, device="cuda")
        kw, dt = {}, torch.float32
        if eight:
            dt = torch.uint8
            kw = {k: [torch.zeros(-(-n // BLOCK), dtype=dt, device="cuda")] for k in ("exp_avg_scales", "exp_avg_sq_scales")}
        plan = tbe.AdamWTensors([p], [g], [torch.zeros(n, dtype=dt, device="cuda")],
                                [torch.zeros(n, dtype=dt, device="cuda")], **kw)
        for step in range(1, 201):
            torch.sub(p, target, out=g)
            tbe.tbe_adamw_step(plan, step, 2e-2)
        losses.append(float((p - target).square().sum()))
    first = float((start - target).square().sum())
    flush_print("adamw losses", first, losses)
    assert losses[0] < 0.02 * first and losses[1] < 0.02 * first
