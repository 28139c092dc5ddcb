"""A ranking model trained end to end: embedding tables, layer norm, one expert per market, AdamW.

Each sample belongs to a market (a country, a surface, a domain) and a batch holds its samples grouped
by market, so that the tower's linear layers are one expert per market on consecutive rows:

  pooled [B, W] fp32 = tables (pooled sums)           tbe_forward_hoisted
  h      [B, W] bf16 = layer norm of pooled           tbe_layer_norm_forward
  a      [B, H] bf16 = relu(expert layer 1 of h)      tbe_grouped_linear_forward
  g      [B, H] bf16 = layer norm of a                tbe_layer_norm_forward
  logit  [B, 1] fp32 = expert layer 2 of g            tbe_grouped_linear_forward

and back: the pooled rows' gradient comes out of the first layer norm in fp32, as the tables' backward
takes it.  The tables take one exact row-wise Adagrad step a row, the tower one AdamW step on fp32
master weights, with states of 8 bits for the experts' weights and of 32 bits for the vectors.

Run:  python examples/expert_tower.py [--steps 60]        (needs an MI355X and the built library)
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import bwd_tbe_fwd_amd as tbe  # noqa: E402

EPS = 1e-5


class Tower:
    """The dense part: its bf16 weights with fp32 masters, its gradients, and every buffer of a step."""

    def __init__(self, B: int, width: int, hidden: int, markets: int, seed: int, lr: float = 3e-3, device="cuda"):
        gen = torch.Generator().manual_seed(seed)
        shapes = {"norm1.weight": (width,), "norm1.bias": (width,), "layer1.weight": (markets, hidden, width),
                  "layer1.bias": (markets, hidden), "norm2.weight": (hidden,), "norm2.bias": (hidden,),
                  "layer2.weight": (markets, 1, hidden), "layer2.bias": (markets, 1)}
        self.master, self.p, self.g, self.lr, self.step = {}, {}, {}, lr, 0
        for name, shape in shapes.items():
            if "norm" in name:
                w = torch.full(shape, 1.0 if "weight" in name else 0.0)
            elif "bias" in name:
                w = torch.zeros(shape)
            else:
                w = torch.randn(shape, generator=gen) * shape[-1] ** -0.5
            self.master[name] = w.to(device)
            self.p[name] = self.master[name].bfloat16()
            self.g[name] = torch.empty_like(self.p[name])
        moments, scales = [[], []], [[], []]
        for name, w in self.master.items():
            blocks = -(-w.numel() // tbe.TBE_ADAMW_BLOCK)
            eight = w.dim() == 3  # the experts' weights
            for k in range(2):
                moments[k].append(torch.zeros(w.numel(), dtype=torch.uint8 if eight else torch.float32, device=device))
                scales[k].append(torch.zeros(blocks, dtype=torch.uint8, device=device) if eight else None)
        names = list(self.p)
        self.plan = tbe.AdamWTensors([self.p[n] for n in names], [self.g[n] for n in names], moments[0], moments[1],
                                     weight_decay=[0.01 if self.p[n].dim() == 3 else 0.0 for n in names],
                                     masters=[self.master[n] for n in names], exp_avg_scales=scales[0],
                                     exp_avg_sq_scales=scales[1])

        def empty(*shape, dtype=torch.bfloat16):
            return torch.empty(*shape, dtype=dtype, device=device)

        f32 = torch.float32
        self.h, self.a, self.n2 = empty(B, width), empty(B, hidden), empty(B, hidden)
        self.logit = empty(B, 1, dtype=f32)
        self.stats = [empty(B, dtype=f32) for _ in range(4)]
        self.grad_n2, self.grad_a, self.grad_h = empty(B, hidden), empty(B, hidden), empty(B, width)
        self.grad_pooled = empty(B, width, dtype=f32)
        need = [tbe.tbe_layer_norm_backward_workspace_bytes(B, width), tbe.tbe_layer_norm_backward_workspace_bytes(B, hidden),
                tbe.tbe_grouped_linear_backward_weight_workspace_bytes(B, markets, width, hidden),
                tbe.tbe_grouped_linear_backward_weight_workspace_bytes(B, markets, hidden, 1)]
        self.workspace = tbe.workspace(max(need), device)  # the calls run one after the other on one stream

    def forward(self, pooled: torch.Tensor, offsets: torch.Tensor) -> torch.Tensor:
        p, (m1, r1, m2, r2) = self.p, self.stats
        tbe.tbe_layer_norm_forward(pooled, p["norm1.weight"], p["norm1.bias"], EPS, self.h, m1, r1)
        tbe.tbe_grouped_linear_forward(self.h, p["layer1.weight"], p["layer1.bias"], offsets, self.a)
        self.a.relu_()
        tbe.tbe_layer_norm_forward(self.a, p["norm2.weight"], p["norm2.bias"], EPS, self.n2, m2, r2)
        tbe.tbe_grouped_linear_forward(self.n2, p["layer2.weight"], p["layer2.bias"], offsets, self.logit)
        return self.logit

    def backward(self, pooled: torch.Tensor, offsets: torch.Tensor, grad_logit: torch.Tensor) -> torch.Tensor:
        """Fills the weights' gradients and returns the pooled rows'."""
        p, g, ws, (m1, r1, m2, r2) = self.p, self.g, self.workspace, self.stats
        tbe.tbe_grouped_linear_backward_weight(self.n2, grad_logit, offsets, g["layer2.weight"], g["layer2.bias"], ws)
        tbe.tbe_grouped_linear_backward_input(grad_logit, p["layer2.weight"], offsets, self.grad_n2)
        tbe.tbe_layer_norm_backward(self.a, self.grad_n2, m2, r2, p["norm2.weight"], self.grad_a, g["norm2.weight"],
                                    g["norm2.bias"], ws)
        self.grad_a.mul_(self.a > 0)
        tbe.tbe_grouped_linear_backward_weight(self.h, self.grad_a, offsets, g["layer1.weight"], g["layer1.bias"], ws)
        tbe.tbe_grouped_linear_backward_input(self.grad_a, p["layer1.weight"], offsets, self.grad_h)
        tbe.tbe_layer_norm_backward(pooled, self.grad_h, m1, r1, p["norm1.weight"], self.grad_pooled, g["norm1.weight"],
                                    g["norm1.bias"], ws)
        return self.grad_pooled

    def update(self):
        self.step += 1
        tbe.tbe_adamw_step(self.plan, self.step, self.lr)


class Model:
    """Tables of pooled embeddings under the tower."""

    def __init__(self, B=2048, tables=4, rows=1000, dim=64, lookups=5, hidden=256, markets=6, seed=1, device="cuda"):
        self.B, self.T, self.rows, self.lookups, self.markets = B, tables, rows, lookups, markets
        gen = torch.Generator().manual_seed(seed)
        self.tables = tbe.Tables([rows] * tables, [dim] * tables, B, torch.float16, device=device)
        self.weights = (torch.rand(tables * rows * dim, generator=gen) * 0.2 - 0.1).half().to(device)
        self.momentum = torch.zeros(tables * rows, device=device)
        self.pooled = torch.empty(B, tables * dim, device=device)
        n = B * tables * lookups
        self.cfg, self.bcfg = tbe.make_config(), tbe.make_config(pretransposed=1)
        self.counts = torch.zeros(2, dtype=torch.int64, device=device)
        self.bounds = tbe.workspace(tbe.tbe_bounds_check_workspace_bytes(self.tables), device)
        self.ws = tbe.workspace(tbe.tbe_backward_workspace_bytes(self.tables, n, False, self.cfg), device)
        self.bag_offsets = (torch.arange(B * tables + 1, dtype=torch.int64) * lookups).to(device)
        # what the labels follow: a value for each row of each table, seen differently by each market
        self.teacher = torch.randn(markets, tables, rows, generator=gen)
        self.tower = Tower(B, tables * dim, hidden, markets, seed + 1, device=device)

    def batch(self, seed: int):
        """Ids [T * B * L], market offsets [markets + 1] and labels [B, 1] of one batch, grouped by market."""
        gen = torch.Generator().manual_seed(seed)
        market = torch.sort(torch.randint(0, self.markets, (self.B,), generator=gen))[0]
        offsets = torch.searchsorted(market, torch.arange(self.markets + 1)).to(torch.int32)
        ids = torch.randint(0, self.rows, (self.T, self.B, self.lookups), generator=gen)
        score = sum(self.teacher[market[:, None], t, ids[t]].sum(1) for t in range(self.T))
        labels = (score > 0).float()[:, None]
        dev = self.pooled.device
        return ids.view(-1).to(dev), offsets.to(dev), labels.to(dev)

    def train_step(self, ids: torch.Tensor, offsets: torch.Tensor, labels: torch.Tensor, lr: float = 0.05):
        tower = self.tower
        tbe.tbe_forward_hoisted(self.tables, self.weights, ids, self.bag_offsets, None, self.pooled, self.counts, self.bounds,
                                self.ws, self.cfg)
        logit = tower.forward(self.pooled, offsets)
        loss = torch.nn.functional.binary_cross_entropy_with_logits(logit, labels)
        grad_logit = ((torch.sigmoid(logit) - labels) / self.B).bfloat16()
        grad_pooled = tower.backward(self.pooled, offsets, grad_logit)
        tbe.tbe_backward_rowwise_adagrad(self.tables, self.weights, self.momentum, ids, self.bag_offsets, None, grad_pooled,
                                         lr, 1e-8, self.ws, self.bcfg)
        tower.update()
        return loss


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--steps", type=int, default=60)
    ap.add_argument("--batch", type=int, default=2048)
    a = ap.parse_args()
    model = Model(B=a.batch)
    for step in range(a.steps):
        loss = model.train_step(*model.batch(1000 + step))
        if step % 10 == 0 or step == a.steps - 1:
            print(f"step {step:4d}  loss {float(loss):.4f}", flush=True)


if __name__ == "__main__":
    main()
