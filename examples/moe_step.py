"""A mixture-of-experts block trained with the layer operators and the Muon step.

    python examples/moe_step.py [--steps 30]

One block on one GPU, in bf16:

    h = linear(x, w_mix, b_mix, "silu", residual=x)            dense layer
    r = route(top-k of h w_router)                             entries sorted by expert
    u = expert_linear(dispatch(h, r), w_in, r.offsets, b_in, "gelu")
    y = combine(expert_linear(u, w_out, r.offsets), r, weights, residual=h)
    out = linear(dropout(y, p, seed, step), w_out2)

The 3-D expert weights and the 2-D dense ones are stepped by one ``MuonPlan``
on the gradients that autograd leaves; biases and the router by plain gradient
descent.  Data are synthetic: a fixed random two-layer map of Gaussian inputs.
"""

from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import muon_newton_schulz_05_amd as muon  # noqa: E402


class Block:
    def __init__(self, h, hidden, experts, top, device, seed=0):
        g = torch.Generator(device=device).manual_seed(seed)

        def weight(*shape):
            return (torch.randn(shape, generator=g, device=device) * shape[-2] ** -0.5).bfloat16().requires_grad_()

        def bias(*shape):
            return torch.zeros(shape, device=device, dtype=torch.bfloat16, requires_grad=True)

        self.experts, self.top = experts, top
        self.w_mix, self.b_mix = weight(h, h), bias(h)
        self.w_in, self.b_in = weight(experts, h, hidden), bias(experts, hidden)
        self.w_out = weight(experts, hidden, h)
        self.w_head = weight(h, h)
        self.w_router = weight(h, experts)
        self.matrices = [self.w_mix, self.w_in, self.w_out, self.w_head]
        self.others = [self.b_mix, self.b_in, self.w_router]

    def forward(self, x, p, seed, step):
        h = muon.linear(x, self.w_mix, self.b_mix, activation="silu", residual=x)
        scores, ids = torch.topk(muon.linear(h, self.w_router).float(), self.top, dim=1)
        r = muon.route(ids, self.experts)
        u = muon.expert_linear(muon.dispatch(h, r), self.w_in, r.offsets, self.b_in, activation="gelu")
        y = muon.combine(muon.expert_linear(u, self.w_out, r.offsets), r, torch.softmax(scores, 1), residual=h)
        if p:
            y = muon.dropout(y, p, seed=seed, offset=step)
        return muon.linear(y, self.w_head)


def train(steps=30, tokens=2048, h=256, hidden=512, experts=8, top=2, p=0.05, lr=0.02, seed=0, device="cuda"):
    """The losses of every step."""
    block = Block(h, hidden, experts, top, device, seed)
    momenta = [torch.zeros(w.shape, device=device) for w in block.matrices]
    plan = muon.MuonPlan([w.detach() for w in block.matrices], grad_dtypes=[torch.bfloat16] * len(block.matrices),
                         update_scale="aspect")
    g = torch.Generator(device=device).manual_seed(seed + 1)
    a = torch.randn(h, 2 * h, generator=g, device=device) * h ** -0.5
    b = torch.randn(2 * h, h, generator=g, device=device) * (2 * h) ** -0.5
    losses = []
    for step in range(steps):
        x = torch.randn(tokens, h, generator=g, device=device)
        target = torch.relu(x @ a) @ b
        loss = (block.forward(x.bfloat16(), p, seed, step).float() - target).square().mean()
        loss.backward()
        plan.step([w.grad.contiguous() for w in block.matrices], momenta, lr=lr, beta=0.9)
        with torch.no_grad():
            for t in block.others:
                t -= lr * t.grad
            for t in block.matrices + block.others:
                t.grad = None
        losses.append(loss.detach())
    losses = torch.stack(losses).tolist()
    if plan.status() != 0:
        raise RuntimeError("the plan's device error word is set")
    plan.close()
    return losses


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=30)
    args = ap.parse_args()
    for i, loss in enumerate(train(args.steps)):
        print(f"step {i:3d}  loss {loss:.4f}")


if __name__ == "__main__":
    main()
