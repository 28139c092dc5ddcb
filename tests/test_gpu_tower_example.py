"""The example model of examples/expert_tower.py: its losses fall, and one step's logits and gradients
equal the same model's in 64 bits up to its bf16 activations.

Tolerance: every activation and gradient between two operators is stored in bf16, t = 2^-8 of its
value, five of them one after the other on the longest path, each followed by sums whose errors add
up at random; a whole tensor's relative error (2-norm) stays below 5 t = 0.02."""
import os
import sys

import pytest
import torch

import bwd_tbe_fwd_amd as tbe
from gpu_util import flush_print

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, os.path.join(ROOT, "examples"))
import expert_tower  # noqa: E402

pytestmark = pytest.mark.gpu


def rel(got, exp):
    return float((got.double() - exp).norm() / exp.norm())


def test_one_step_against_64_bits():
    model = expert_tower.Model(B=777, tables=3, rows=200, dim=32, hidden=136, markets=5, seed=3)
    ids, offsets, labels = model.batch(7)
    tower = model.tower
    # scales and shifts that are not 1 and 0, as after some training
    for k, (name, p) in enumerate(tower.p.items()):
        if "norm" in name or "bias" in name:
            p.add_((torch.randn(p.shape, generator=torch.Generator().manual_seed(k)) * 0.1).to(p))
    params = {n: p.double().requires_grad_() for n, p in tower.p.items()}
    weights = model.weights.clone()
    model.train_step(ids, offsets, labels)
    torch.cuda.synchronize()

    table = weights.double().view(3, 200, 32)
    pooled = torch.cat([table[t][ids.view(3, 777, -1)[t]].sum(1) for t in range(3)], 1).requires_grad_()

    def norm(x, w, b):
        m = x.mean(1, keepdim=True)
        return (x - m) / ((x - m).square().mean(1, keepdim=True) + expert_tower.EPS).sqrt() * w + b

    def experts(x, w, b):
        at = offsets.tolist()
        return torch.cat([x[at[e]:at[e + 1]] @ w[e].t() + b[e] for e in range(5)])

    p = params
    # relu's derivative jumps at zero, where a rounded activation may lie on the other side: the model's
    # own side is taken (and lies within the rounding of the exact one)
    pre = experts(norm(pooled, p["norm1.weight"], p["norm1.bias"]), p["layer1.weight"], p["layer1.bias"])
    side = tower.a > 0
    assert (pre.detach()[side != (pre > 0)].abs() <= 0.02 * pre.detach().square().mean().sqrt()).all()
    a = pre * side
    logit = experts(norm(a, p["norm2.weight"], p["norm2.bias"]), p["layer2.weight"], p["layer2.bias"])
    torch.nn.functional.binary_cross_entropy_with_logits(logit, labels.double()).backward()
    errors = {"pooled": rel(model.pooled, pooled.detach()), "logit": rel(tower.logit, logit.detach()),
              "grad_pooled": rel(tower.grad_pooled, pooled.grad)}
    errors.update({n: rel(tower.g[n], p[n].grad) for n in p})
    flush_print({n: f"{e:.2g}" for n, e in errors.items()})
    assert all(e <= 0.02 for e in errors.values()), errors


def test_loss_falls():
    model = expert_tower.Model(B=2048)
    losses = [float(model.train_step(*model.batch(1000 + k))) for k in range(60)]
    flush_print("losses", losses[0], losses[-1])
    assert model.counts.tolist() == [0, 0]
    first, last = sum(losses[:5]) / 5, sum(losses[-5:]) / 5
    assert 0.6 < first < 0.9 and last < 0.85 * first
    # the bf16 weights are their masters' rounded copies
    for name, p in model.tower.p.items():
        assert torch.equal(p, model.tower.master[name].bfloat16()), name
