"""A pre-norm mixture-of-experts block: norms, gate, balance loss, routed experts, the Muon step, and four-bit evaluation.

    python examples/moe_prenorm.py [--steps 30]

One block on one GPU, in bf16:

    x1 = linear(rms_norm(x, g1), w_mix, b_mix, "silu", residual=x)
    h = rms_norm(x1, g2);  logits = linear(h, w_router)
    weights, ids = gate(logits, top);  balance = balance_loss(logits, ids)
    r = route(ids);  u = expert_linear(dispatch(h, r), w_in, r.offsets, b_in, "gelu")
    y = combine(expert_linear(u, w_out, r.offsets), r, weights, residual=x1)
    out = linear(layer_norm(y, g3, b3), w_head)

Matrices are stepped by one ``MuonPlan``, norms, biases and the router by plain gradient
descent, on the squared error plus a share of the balance loss.  Afterwards the same block is evaluated with its matrices
in four bits.  Data are synthetic: a fixed random two-layer map of Gaussian inputs.
"""

from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import muon_newton_schulz_05_amd as muon  # noqa: E402


class Block:
    def __init__(self, h, hidden, experts, top, device="cuda", dtype=torch.bfloat16, seed=0):
        g = torch.Generator(device=device).manual_seed(seed)

        def weight(*shape):
            return (torch.randn(shape, generator=g, device=device) * shape[-2] ** -0.5).to(dtype).requires_grad_()

        def vector(*shape, value=0.0):
            return torch.full(shape, value, device=device, dtype=dtype, requires_grad=True)

        self.experts, self.top = experts, top
        self.w_mix, self.w_in, self.w_out, self.w_head = (weight(h, h), weight(experts, h, hidden),
                                                          weight(experts, hidden, h), weight(h, h))
        self.w_router = weight(h, experts)
        self.b_mix, self.b_in, self.b3 = vector(h), vector(experts, hidden), vector(h)
        self.g1, self.g2, self.g3 = (vector(h, value=1.0) for _ in range(3))
        self.matrices = [self.w_mix, self.w_in, self.w_out, self.w_head]
        self.others = [self.w_router, self.b_mix, self.b_in, self.b3, self.g1, self.g2, self.g3]

    def forward(self, x, layer=muon.linear, expert_layer=muon.expert_linear, matrices=None):
        """The block's output and its ``Balance``; layers and matrices may be others than the trained ones."""
        w_mix, w_in, w_out, w_head = matrices or self.matrices
        x1 = layer(muon.rms_norm(x, self.g1), w_mix, self.b_mix, activation="silu", residual=x)
        h = muon.rms_norm(x1, self.g2)
        logits = muon.linear(h, self.w_router)
        weights, ids = muon.gate(logits, self.top)
        balance = muon.balance_loss(logits, ids)
        r = muon.route(ids, self.experts)
        u = expert_layer(muon.dispatch(h, r), w_in, r.offsets, self.b_in, activation="gelu")
        y = muon.combine(expert_layer(u, w_out, r.offsets), r, weights, residual=x1)
        return layer(muon.layer_norm(y, self.g3, self.b3), w_head), balance

    @torch.no_grad()
    def forward_four_bits(self, x):
        held = [muon.mx_quantize(w) for w in self.matrices]
        return self.forward(x, muon.mx_linear, muon.mx_expert_linear, held)


def train(steps=30, tokens=2048, h=256, hidden=512, experts=8, top=2, share=0.01, lr=0.02, seed=0, device="cuda"):
    """The losses and expert counts of every step, and the last batch's loss evaluated in bf16 and in four bits."""
    block = Block(h, hidden, experts, top, device, seed=seed)
    momenta = [torch.zeros(w.shape, device=device) for w in block.matrices]
    plan = muon.MuonPlan([w.detach() for w in block.matrices], grad_dtypes=[torch.bfloat16] * len(block.matrices),
                         update_scale="aspect")
    g = torch.Generator(device=device).manual_seed(seed + 1)
    a = torch.randn(h, 2 * h, generator=g, device=device) * h ** -0.5
    b = torch.randn(2 * h, h, generator=g, device=device) * (2 * h) ** -0.5
    losses, counts = [], []
    for _ in range(steps):
        x = torch.randn(tokens, h, generator=g, device=device)
        target, x = torch.relu(x @ a) @ b, x.bfloat16()
        out, balance = block.forward(x)
        loss = (out.float() - target).square().mean()
        (loss + share * balance.loss).backward()
        plan.step([w.grad.contiguous() for w in block.matrices], momenta, lr=lr, beta=0.9)
        with torch.no_grad():
            for t in block.others:
                t -= lr * t.grad
            for t in block.matrices + block.others:
                t.grad = None
        losses.append(loss.detach())
        counts.append(balance.counts)
    with torch.no_grad():
        full = (block.forward(x)[0].float() - target).square().mean()
        four = (block.forward_four_bits(x)[0].float() - target).square().mean()
    if plan.status() != 0:
        raise RuntimeError("the plan's device error word is set")
    plan.close()
    return torch.stack(losses).tolist(), torch.stack(counts).tolist(), full.item(), four.item()


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=30)
    losses, counts, full, four = train(ap.parse_args().steps)
    for i, (loss, c) in enumerate(zip(losses, counts)):
        print(f"step {i:3d}  loss {loss:.4f}  rows of the experts {c}")
    print(f"evaluated: bf16 {full:.4f}, four bits {four:.4f}")


if __name__ == "__main__":
    main()
