"""A mixture-of-experts layer trained on the logical ranks of one GPU.

p ranks hold their own tokens, a replica of the router and experts / p
experts each. A step goes through the operators in the order a training
program meets them:

    vcoll_moe_route                       logits -> experts and weights of every token
    vcoll_moe_sort, vcoll_moe_dispatch    token rows to their experts, one run of rows per expert
    (one matrix product per expert)
    vcoll_moe_combine_weighted            rows back to their tokens
    vcoll_moe_combine_weighted_backward   gradients of the experts' outputs and of the weights
    vcoll_moe_combine_weighted(None)      gradient of the dispatched tokens
    vcoll_moe_route_backward              gradient of the logits
    vcoll_allreduce                       the router's gradient, summed over the ranks by a ring
    vcoll_adamw                           router and experts in one call

    python examples/moe_training_step.py [--steps N] [--bits 8|32]
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import collective_communication_algorithms_vcoll_amd as vc  # noqa: E402


class MoeLayer:
    """y_t = sum_k w_tk (x_t W_e(t,k)), w the router's softmax over the chosen experts."""

    def __init__(self, p: int, hidden: int, experts: int, topk: int, seed: int = 0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.p, self.topk, self.per_rank = p, topk, experts // p
        self.router = torch.randn((hidden, experts), device="cuda", generator=g) / hidden ** 0.5
        self.experts = torch.randn((experts, hidden, hidden), device="cuda", generator=g) / hidden ** 0.5

    def _each_expert(self):
        """(rank, its rows of each of its experts, the expert) for the current offsets."""
        for j, row in enumerate(self.offsets.tolist()):
            for l in range(self.per_rank):
                if row[l + 1] > row[l]:
                    yield j, slice(row[l], row[l + 1]), j * self.per_rank + l

    def forward(self, x: torch.Tensor) -> torch.Tensor:
        """x [p, tokens, hidden] -> y of the same shape."""
        self.x, T = x, x.shape[1]
        self.logits = x @ self.router
        self.ids, self.weights = vc.vcoll_moe_route(self.logits, self.topk)
        self.slots, self.offsets = vc.vcoll_moe_sort(self.ids, self.per_rank)
        rows = self.offsets[:, -1].tolist()
        self.recv = vc.vcoll_moe_dispatch(list(x), list(self.slots), rows, self.topk)
        self.out = [torch.empty_like(r) for r in self.recv]
        for j, rows, e in self._each_expert():
            torch.mm(self.recv[j][rows], self.experts[e], out=self.out[j][rows])
        return vc.vcoll_moe_combine_weighted(self.out, self.slots, self.weights, T, self.topk)

    def backward(self, dy: torch.Tensor):
        """Gradients (of x, of the router summed over the ranks, of the experts) from that of y."""
        T = dy.shape[1]
        d_out, d_weights = vc.vcoll_moe_combine_weighted_backward(dy, self.out, self.slots, self.weights, self.topk)
        d_experts = torch.zeros_like(self.experts)
        d_recv = [torch.zeros_like(r) for r in self.recv]
        for j, rows, e in self._each_expert():
            torch.mm(self.recv[j][rows].t(), d_out[j][rows], out=d_experts[e])
            torch.mm(d_out[j][rows], self.experts[e].t(), out=d_recv[j][rows])
        dx = vc.vcoll_moe_combine_weighted(d_recv, self.slots, None, T, self.topk)
        d_logits = vc.vcoll_moe_route_backward(self.logits, self.ids, self.weights, d_weights)
        dx += d_logits @ self.router.t()
        # every rank's contribution, then the sum that a ring leaves on all of them
        d_router = torch.stack([self.x[i].t() @ d_logits[i] for i in range(self.p)])
        vc.vcoll_allreduce("ring", d_router.view(self.p, -1), d_router.view(self.p, -1))
        return dx, d_router[0], d_experts


def train(steps: int = 60, bits: int = 8, p: int = 4, tokens: int = 256, hidden: int = 64, experts: int = 16,
          topk: int = 2, say=print) -> list:
    """Fits the layer to another one of the same shape; returns the loss of every step."""
    teacher, layer = MoeLayer(p, hidden, experts, topk, seed=1), MoeLayer(p, hidden, experts, topk, seed=2)
    layer.router.copy_(teacher.router)
    params = [layer.router, layer.experts]
    grads = [torch.empty_like(t) for t in params]
    update = vc.prepare_adamw(params, grads, **vc.adamw_state(params, bits))
    g = torch.Generator(device="cuda").manual_seed(3)
    losses = []
    for step in range(1, steps + 1):
        x = torch.randn((p, tokens, hidden), device="cuda", generator=g)
        difference = layer.forward(x) - teacher.forward(x)
        losses.append(float(difference.square().mean()))
        _, d_router, d_experts = layer.backward(2 * difference / difference.numel())
        grads[0].copy_(d_router)
        grads[1].copy_(d_experts)
        update(lr=1e-2, step=step, weight_decay=0.0, seed=step)
        if say and (step == 1 or step % 10 == 0):
            say(f"step {step:4d}  loss {losses[-1]:.5f}")
    return losses


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__.split("\n\n")[0])
    ap.add_argument("--steps", type=int, default=60)
    ap.add_argument("--bits", type=int, default=8, choices=(8, 32))
    a = ap.parse_args()
    train(a.steps, a.bits)
