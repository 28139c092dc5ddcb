"""New gradient tensors for the same AdamW plan, as a program has them that frees its gradients at every step."""
import pytest
import torch

import bwd_tbe_fwd_amd as tbe
from test_gpu_tower_adamw import BLOCK, Tensor, opened, pack, plan_of

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16


def test_each_step_takes_its_own_gradients():
    ts = [Tensor(n, F32, F32, eight, False, 0.01, 40 + n) for n, eight in ((300, False), (5000, True), (129, False))]
    plan = plan_of(ts)
    for step in range(1, 4):
        dtype = BF16 if step == 2 else F32  # another type may come too
        grads = [(torch.randn(t.p0.numel(), generator=torch.Generator().manual_seed(100 * step + i)) * 1e-2).to(dtype)
                 for i, t in enumerate(ts)]
        plan.set_gradients([g.cuda() for g in grads])  # kept alive by the plan alone
        tbe.tbe_adamw_step(plan, step, 1e-3)
        torch.cuda.synchronize()
        for t, g in zip(ts, grads):
            t.g = g
            t.expect(step, 1e-3, 0.9, 0.999, 1e-8)
            t.check(f"step {step}")
            t.p0 = t.dp.cpu()
            if t.eight:
                t.m, t.v = opened(*pack(t.m, False), False), opened(*pack(t.v, True), True)


def test_refused_gradients_leave_the_old_ones():
    ts = [Tensor(n, F32, F32, False, False, 0.0, 60 + n) for n in (BLOCK, 40)]
    plan = plan_of(ts)
    new = [torch.zeros(BLOCK, device="cuda"), torch.zeros(40, device="cuda")]
    for bad, word in ((new[:1], "as many"), ([new[0], new[0]], "gradient"), ([new[0], new[1].double()], "float64"),
                      ([new[0], torch.zeros(40)], "not on the current GPU"), ([new[0], torch.zeros(80, device="cuda")[::2]], "gradient")):
        with pytest.raises(tbe.TbeError, match=word):
            plan.set_gradients(bad)
    tbe.tbe_adamw_step(plan, 1, 1e-3)
    torch.cuda.synchronize()
    for t in ts:
        t.expect(1, 1e-3, 0.9, 0.999, 1e-8)
        t.check("old gradients")
