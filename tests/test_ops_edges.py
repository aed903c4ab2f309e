"""Host-side tests (no GPU) of what the layer operators refuse: the binding's kernel call is reached or not."""

from __future__ import annotations

import os

import pytest
import torch
from torch.autograd import forward_ad

INVALID = 1
CALLS = ("linear", "linear, residual", "expert_linear", "dispatch", "combine", "combine, residual", "dropout")


@pytest.fixture(scope="module")
def ops():
    import muon_newton_schulz_05_amd as pkg
    if not os.path.exists(pkg.LIB_PATH):
        pytest.skip("libmuon.so not built (run __graft_entry__.build())")
    from muon_newton_schulz_05_amd import ops as o
    o.load_ops()
    return o


@pytest.fixture
def on_cpu(ops, monkeypatch):
    """The binding taking CPU tensors, so that a call goes all the way to the kernels'."""
    monkeypatch.setattr(ops, "_check_linear", lambda *a: None)
    monkeypatch.setattr(ops, "_gpu", lambda *a: None)
    return ops


def operator_calls(ops, x=None, ys=None):
    """{name: call} of every differentiable operator, with its first tensor replaced where given."""
    x = torch.randn(3, 8) if x is None else x
    ys = torch.randn(6, 8) if ys is None else ys
    w, e = torch.randn(8, 4), torch.randn(2, 8, 4)
    position, offsets = torch.arange(6, dtype=torch.int32).view(3, 2), torch.tensor([0, 3, 6], dtype=torch.int32)
    r = ops.Routing(offsets, torch.arange(6, dtype=torch.int32), position)
    return {"linear": lambda: ops.linear(x, w), "linear, residual": lambda: ops.linear(torch.randn(3, 4), torch.randn(4, 8),
                                                                                      residual=x),
            "expert_linear": lambda: ops.expert_linear(ys, e, offsets), "dispatch": lambda: ops.dispatch(x, r),
            "combine": lambda: ops.combine(ys, r, torch.rand(3, 2)),
            "combine, residual": lambda: ops.combine(torch.randn(6, 8), r, torch.rand(3, 2), x),
            "dropout": lambda: ops.dropout(x, 0.5)}


@pytest.mark.parametrize("name", CALLS)
@pytest.mark.parametrize("grad", [False, True])
def test_forward_mode_is_refused(on_cpu, monkeypatch, name, grad):
    """A tangent is not dropped without a word: the call raises as it does for a leaf that requires grad."""
    monkeypatch.setattr(on_cpu, "_call", lambda *a: None)
    with forward_ad.dual_level(), torch.set_grad_enabled(grad):
        operator_calls(on_cpu)[name]()                       # no tangent: nothing to refuse
        x, ys = (forward_ad.make_dual(torch.randn(n, 8), torch.ones(n, 8)) for n in (3, 6))
        with pytest.raises((RuntimeError, NotImplementedError), match="forward"):
            operator_calls(on_cpu, x, ys)[name]()


@pytest.mark.parametrize("name", CALLS)
@pytest.mark.parametrize("how", ["make_fx", "make_fx, pre-dispatch", "jit.trace"])
def test_tracing_is_refused(on_cpu, name, how):
    """A tracer sees none of the kernels: it would record a program that returns memory nobody wrote."""
    from torch.fx.experimental.proxy_tensor import make_fx
    x, ys = torch.randn(3, 8), torch.randn(6, 8)

    def program(x, ys):
        return operator_calls(on_cpu, x, ys)[name]()
    with pytest.raises(RuntimeError, match="cannot be traced"):
        if how == "jit.trace":
            torch.jit.trace(program, (x, ys))
        else:
            make_fx(program, pre_dispatch=how != "make_fx")(x, ys)


def test_tracing_of_a_sort_is_refused(on_cpu):
    from torch.fx.experimental.proxy_tensor import make_fx
    with pytest.raises(RuntimeError, match="cannot be traced"):
        make_fx(lambda ids: on_cpu.route(ids, 4).order)(torch.zeros(3, 2, dtype=torch.int64))
