"""The pre-norm example block: it runs, repeats itself, and its gradients are those of the formulas."""

from __future__ import annotations

import importlib.util
import math
import os

import pytest
import torch

from ops_reference import U32

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("moe_prenorm", os.path.join(ROOT, "examples", "moe_prenorm.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_block_runs_and_repeats(example):
    args = dict(steps=4, tokens=512, h=128, hidden=192, experts=6)
    losses, counts, full, four = example.train(**args)
    assert all(math.isfinite(v) for v in (*losses, full, four))
    assert all(sum(c) == 2 * 512 for c in counts)
    assert example.train(**args) == (losses, counts, full, four)        # the same seed gives the same bits


def test_block_gradients(example):
    h, hidden, e, top, t = 48, 72, 6, 2, 90
    block = example.Block(h, hidden, e, top, dtype=torch.float32, seed=3)
    g = torch.Generator().manual_seed(4)
    x, dy = torch.randn(t, h, generator=g), torch.randn(t, h, generator=g)
    leaves = block.matrices + block.others
    out, balance = block.forward(x.cuda())
    got = torch.autograd.grad((out, balance.loss), leaves, (dy.cuda(), torch.tensor(0.5, device="cuda")))

    w_mix, w_in, w_out, w_head, w_router, b_mix, b_in, b3, g1, g2, g3 = d = [
        v.detach().double().cpu().requires_grad_() for v in leaves]
    rms = lambda v, w: v * torch.rsqrt(v.square().mean(1, keepdim=True) + 1e-6) * w  # noqa: E731
    x = x.double()
    x1 = torch.nn.functional.silu(rms(x, g1) @ w_mix + b_mix) + x
    n = rms(x1, g2)
    logits = n @ w_router
    z, ids = torch.topk(logits, top, dim=1)
    w = torch.softmax(z, 1)
    each = torch.stack([torch.nn.functional.gelu(n @ w_in[i] + b_in[i]) @ w_out[i] for i in range(e)], 1)
    y = (w[:, :, None] * each.gather(1, ids[:, :, None].expand(-1, -1, h))).sum(1) + x1
    want = torch.nn.functional.layer_norm(y, (h,), g3, b3, 1e-5) @ w_head
    counts = torch.stack([(ids == i).sum() for i in range(e)])
    assert torch.equal(balance.counts.cpu().long(), counts)
    loss = e * (counts.double() / (t * top) * torch.softmax(logits, 1).mean(0)).sum()
    ref = torch.autograd.grad((want, loss), d, (dy.double(), torch.tensor(0.5).double()))
    # float32 throughout: six layers and four norms of sums over at most 90 terms, each step a few U32 off.
    assert float((out.detach().double().cpu() - want.detach()).norm() / want.detach().norm()) < 300 * U32
    for a, b in zip(got, ref):
        assert float((a.double().cpu() - b).norm() / b.norm()) < 600 * U32
