"""A next-item model trained end to end: one table at both ends, a small tower between them.

Sequences of items are read position by position and each position predicts the item that comes next:

  h      [n, D] bf16 = sqrt(D) * table[item]                   tbe_lookup_forward
  a      [n, D] bf16 = layer norm of h                         tbe_layer_norm_forward
  u      [n, D] bf16 = a W^T + b, relu, added to a             tbe_grouped_linear_forward (one expert)
  x      [n, D] bf16 = layer norm of u                         tbe_layer_norm_forward
  loss   [n]    fp32 = cross entropy of x table^T + bias       tbe_cross_entropy_forward

and back.  The loss's gradient of the table is overwritten first (every item is scored by every position), the lookup's is
added to it (the positions' own items).  Sequences are padded with -1: such positions have no row, no target and no
gradient.  AdamW steps on fp32 master weights, the table's states in 8 bits.

Run:  python examples/next_item.py [--steps 60]        (needs an MI355X and the built library)
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


class Model:
    """Its weights with fp32 masters, their gradients and every buffer of a step of `positions` positions."""

    def __init__(self, positions=4096, items=5000, dim=128, seed=1, lr=3e-3, device="cuda"):
        gen = torch.Generator().manual_seed(seed)
        self.n, self.items, self.dim, self.lr, self.step = positions, items, dim, lr, 0
        self.scale_in, self.scale_out = dim ** 0.5, 1.0
        start = {"table": torch.randn(items, dim, generator=gen) * dim ** -0.5, "norm1.weight": torch.ones(dim),
                 "norm1.bias": torch.zeros(dim), "layer.weight": torch.randn(1, dim, dim, generator=gen) * dim ** -0.5,
                 "layer.bias": torch.zeros(1, dim), "norm2.weight": torch.ones(dim), "norm2.bias": torch.zeros(dim)}
        self.master = {k: w.to(device) for k, w in start.items()}
        self.p = {k: w.bfloat16() for k, w in self.master.items()}
        self.g = {k: torch.empty_like(w) for k, w in self.p.items()}
        # the items' biases are fp32 throughout
        self.p["bias"], self.g["bias"] = torch.zeros(items, device=device), torch.empty(items, device=device)
        self.master["bias"] = None
        names = list(self.p)
        states, scales = [[], []], [[], []]
        for k in names:
            n = self.p[k].numel()
            eight = k == "table"
            for i in range(2):
                states[i].append(torch.zeros(n, dtype=torch.uint8 if eight else torch.float32, device=device))
                scales[i].append(torch.zeros(-(-n // tbe.TBE_ADAMW_BLOCK), dtype=torch.uint8, device=device) if eight else None)
        self.plan = tbe.AdamWTensors([self.p[k] for k in names], [self.g[k] for k in names], states[0], states[1],
                                     weight_decay=[0.01 if self.p[k].dim() > 1 else 0.0 for k in names],
                                     masters=[self.master[k] for k in names], exp_avg_scales=scales[0],
                                     exp_avg_sq_scales=scales[1])

        def rows(count, dtype=torch.bfloat16):
            return [torch.empty(positions, dim, dtype=dtype, device=device) for _ in range(count)]

        self.h, self.a, self.lin, self.u, self.x = rows(5)
        self.grad_x, self.grad_u, self.grad_lin, self.grad_a, self.grad_h = rows(5)
        self.stats = [torch.empty(positions, device=device) for _ in range(4)]
        self.loss, self.lse, self.grad_loss = (torch.empty(positions, device=device) for _ in range(3))
        self.offsets = torch.tensor([0, positions], dtype=torch.int32, device=device)
        sizes = (positions, items, dim)
        self.workspace = tbe.workspace(max(  # the calls follow each other on one stream
            tbe.tbe_lookup_backward_workspace_bytes(*sizes), tbe.tbe_cross_entropy_forward_workspace_bytes(*sizes),
            tbe.tbe_cross_entropy_backward_workspace_bytes(*sizes), tbe.tbe_layer_norm_backward_workspace_bytes(positions, dim),
            tbe.tbe_grouped_linear_backward_weight_workspace_bytes(positions, 1, dim, dim)), device)

    def forward(self, ids: torch.Tensor, targets: torch.Tensor) -> torch.Tensor:
        """The loss of each position; 0 where there is no target."""
        p, (m1, r1, m2, r2) = self.p, self.stats
        tbe.tbe_lookup_forward(p["table"], ids, self.scale_in, self.h)
        tbe.tbe_layer_norm_forward(self.h, p["norm1.weight"], p["norm1.bias"], EPS, self.a, m1, r1)
        tbe.tbe_grouped_linear_forward(self.a, p["layer.weight"], p["layer.bias"], self.offsets, self.lin)
        torch.add(self.a, torch.relu(self.lin), out=self.u)
        tbe.tbe_layer_norm_forward(self.u, p["norm2.weight"], p["norm2.bias"], EPS, self.x, m2, r2)
        tbe.tbe_cross_entropy_forward(self.x, p["table"], p["bias"], targets, self.scale_out, self.loss, self.lse, self.workspace)
        return self.loss

    def backward(self, ids: torch.Tensor, targets: torch.Tensor):
        """The gradients of the mean loss over the positions that have a target, into self.g."""
        p, g, ws, (m1, r1, m2, r2) = self.p, self.g, self.workspace, self.stats
        there = (targets >= 0) & (targets < self.items)
        self.grad_loss.copy_(there / there.sum().clamp(min=1))
        tbe.tbe_cross_entropy_backward(self.x, p["table"], p["bias"], targets, self.scale_out, self.lse, self.grad_loss,
                                       self.grad_x, g["table"], g["bias"], ws)
        tbe.tbe_layer_norm_backward(self.u, self.grad_x, m2, r2, p["norm2.weight"], self.grad_u, g["norm2.weight"],
                                    g["norm2.bias"], ws)
        torch.mul(self.grad_u, self.lin > 0, out=self.grad_lin)
        tbe.tbe_grouped_linear_backward_weight(self.a, self.grad_lin, self.offsets, g["layer.weight"], g["layer.bias"], ws)
        tbe.tbe_grouped_linear_backward_input(self.grad_lin, p["layer.weight"], self.offsets, self.grad_a)
        self.grad_a.add_(self.grad_u)
        tbe.tbe_layer_norm_backward(self.h, self.grad_a, m1, r1, p["norm1.weight"], self.grad_h, g["norm1.weight"],
                                    g["norm1.bias"], ws)
        tbe.tbe_lookup_backward(ids, self.grad_h, self.scale_in, g["table"], ws, accumulate=True)

    def update(self):
        self.step += 1
        tbe.tbe_adamw_step(self.plan, self.step, self.lr)

    def train_step(self, ids: torch.Tensor, targets: torch.Tensor) -> torch.Tensor:
        loss = self.forward(ids, targets)
        self.backward(ids, targets)
        self.update()
        return loss


def sequences(positions: int, items: int, length: int, seed: int, device="cuda"):
    """Padded sequences in which item i is followed by (7 i + a small step) mod items: ids and targets, one after the other."""
    gen = torch.Generator().manual_seed(seed)
    count = -(-positions // length)
    ids = torch.full((count, length + 1), -1, dtype=torch.int64)
    ids[:, 0] = torch.randint(0, items, (count,), generator=gen)
    for k in range(1, length + 1):
        ids[:, k] = (7 * ids[:, k - 1] + torch.randint(0, 3, (count,), generator=gen)) % items
    keep = torch.randint(2, length + 2, (count, 1), generator=gen)
    ids[torch.arange(length + 1) >= keep] = -1
    targets = ids[:, 1:].clone()
    ids = ids[:, :-1].clone()
    ids[targets < 0] = -1  # a sequence's last item predicts nothing
    return ids.reshape(-1)[:positions].to(device), targets.reshape(-1)[:positions].to(device)


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--steps", type=int, default=60)
    ap.add_argument("--positions", type=int, default=4096)
    a = ap.parse_args()
    model = Model(positions=a.positions)
    for step in range(a.steps):
        ids, targets = sequences(a.positions, model.items, 32, 1000 + step)
        loss = model.train_step(ids, targets)
        if step % 10 == 0 or step == a.steps - 1:
            print(f"step {step:4d}  loss {float(loss.sum() / (targets >= 0).sum()):.4f}", flush=True)


if __name__ == "__main__":
    main()
