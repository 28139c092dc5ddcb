"""The example model of examples/next_item.py: lookup, layer norms, a linear layer and the cross entropy together, with one
table at both ends.  One step's losses and gradients equal the same model's in 64 bits up to its bf16 activations.

Tolerance: on the longest path (the table's gradient through the lookup) 12 activations and gradients are stored in bf16 one
after the other (five forward, z and six backward), each off by at most t = 2^-8 of its value; a tensor's relative error
(2-norm) stays below their sum, 12 t = 0.047."""
import os
import sys

import pytest
import torch

import bwd_tbe_fwd_amd as tbe
from gpu_util import flush_print

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, os.path.join(ROOT, "examples"))
import next_item  # noqa: E402

pytestmark = pytest.mark.gpu


def rel(got, exp):
    return float((got.double() - exp).norm() / exp.norm())


@pytest.mark.parametrize("positions,items,dim", [(1000, 700, 64), (333, 1501, 136), (70, 90, 40)])
def test_one_step_against_64_bits(positions, items, dim):
    model = next_item.Model(positions=positions, items=items, dim=dim, seed=3)
    ids, targets = next_item.sequences(positions, items, 12, 7)
    for k, (name, p) in enumerate(model.p.items()):
        if "norm" in name or "bias" in name:
            p.add_((torch.randn(p.shape, generator=torch.Generator().manual_seed(k)) * 0.1).to(p))
    p = {n: w.double().requires_grad_() for n, w in model.p.items()}
    loss = model.forward(ids, targets).clone()
    model.backward(ids, targets)
    torch.cuda.synchronize()

    there = targets >= 0
    assert 0 < int(there.sum()) < positions

    def norm(x, w, b):
        m = x.mean(1, keepdim=True)
        return (x - m) / ((x - m).square().mean(1, keepdim=True) + next_item.EPS).sqrt() * w + b

    h = p["table"][ids[there]] * model.scale_in
    a = norm(h, p["norm1.weight"], p["norm1.bias"])
    lin = a @ p["layer.weight"][0].t() + p["layer.bias"][0]
    side = model.lin[there] > 0  # relu's side as the model has it: where it differs, within the rounding of zero
    assert (lin.detach()[side != (lin > 0)].abs() <= 0.02 * lin.detach().square().mean().sqrt()).all()
    x = norm(a + lin * side, p["norm2.weight"], p["norm2.bias"])
    logits = model.scale_out * x @ p["table"].t() + p["bias"]
    exact = torch.nn.functional.cross_entropy(logits, targets[there], reduction="none")
    exact.mean().backward()
    errors = {"loss": rel(loss[there], exact.detach())}
    errors.update({n: rel(model.g[n], p[n].grad) for n in p})
    flush_print({n: f"{e:.2g}" for n, e in errors.items()})
    assert all(e <= 12 * 2.0 ** -8 for e in errors.values()), errors
    assert bool((loss[~there] == 0).all())


def test_training_steps_run():
    model = next_item.Model(positions=2000, items=800, dim=64)
    for k in range(4):
        ids, targets = next_item.sequences(2000, 800, 16, k)
        loss = model.train_step(ids, targets)
        assert bool(loss.isfinite().all())
    for name, p in model.p.items():
        assert bool(p.isfinite().all()), name
        if model.master[name] is not None:
            assert torch.equal(p, model.master[name].bfloat16()), name
