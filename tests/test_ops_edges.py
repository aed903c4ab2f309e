"""Host-side tests (no GPU) of what the layer operators refuse: the binding's kernel call is reached or not."""

from __future__ import annotations

import ctypes
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


def _desc(ops, **kw):
    d = dict(dtype=1, act=2, groups=0, w_layout=0, rows=4, k=8, n=8, ldx=0, ldw=0, w_stride=0, ldr=8, ldg=0)
    d.update(kw)
    d.update(ldx=d["k"], ldw=d["n"], ldg=d["n"])
    return ops.LinearDesc(*[d[f[0]] for f in ops.LinearDesc._fields_])


# What a call that got past its checks says here, where there is no GPU to launch on.
LAUNCHED = 3
BACKWARD_SHAPES = [dict(rows=4), dict(rows=64, k=64, n=16384), dict(rows=200, k=64, n=16384), dict(rows=2100, k=1001, n=2003),
                   dict(rows=300, act=0, k=64, n=4096), dict(dtype=0, rows=300, k=640, n=520),
                   dict(rows=40, groups=3, w_stride=64), dict(rows=4000, groups=3, k=64, n=72, w_stride=64 * 72)]


@pytest.mark.skipif(torch.cuda.is_available(), reason="the pointers are made up: nothing may be launched on them")
@pytest.mark.parametrize("kw", BACKWARD_SHAPES, ids=str)
def test_backward_checks_before_it_launches(ops, kw):
    """Whatever is wrong with a pointer or the workspace is said before the first launch, for any outputs asked for."""
    lib, d, need = ops.load_ops(), _desc(ops, **kw), ctypes.c_uint64(0)
    assert lib.muon_linear_workspace(ctypes.byref(d), 4, ctypes.byref(need)) == 0
    a = 1 << 32                                              # never read

    def call(offsets=a if d.groups else None, x=a, w=a, z=a, dy=a, dx=a, dw=a, db=a, ws=a, size=need.value):
        return lib.muon_linear_backward(ctypes.byref(d), offsets, x, w, z, dy, dx, dw, db, ws, size, None)
    assert call() == LAUNCHED
    bad = [dict(w=None), dict(x=None), dict(dy=None), dict(w=a + 1), dict(x=a + 1), dict(dy=a + 1), dict(dx=a + 1),
           dict(dw=a + 1), dict(db=a + 1), dict(offsets=None if d.groups else a), dict(ws=a + 8)]
    bad += [dict(z=None)] if d.act else []
    bad += [dict(ws=None), dict(size=0)] if need.value else []
    for one in bad:
        assert call(**one) == INVALID, one
    # Only what the asked outputs need has to be there.
    assert call(x=None, dw=None) == LAUNCHED and call(w=None, dx=None) == LAUNCHED
    assert call(x=None, w=None, dx=None, dw=None) == LAUNCHED
    # One byte less than is told is too little for pointers of some alignment, and no pointers need more.
    worst = [call(x=a + p, w=a + q, dy=a + r, size=max(need.value - 1, 0)) for p in (0, 4) for q in (0, 4) for r in (0, 4)]
    if d.dtype == 1:
        worst += [call(x=a + p, w=a + q, dy=a + r, size=max(need.value - 1, 0)) for p in (0, 2) for q in (0, 2)
                  for r in (0, 2)]
    assert set(worst) <= {INVALID, LAUNCHED} and (INVALID in worst or not need.value)
    for off in (0, 4):
        assert call(x=a + off, w=a + off, dy=a + off) == LAUNCHED


class Elsewhere(torch.Tensor):
    """A tensor that says it lives on a GPU and has no memory: for the binding's checks."""

    @staticmethod
    def __new__(cls, *shape, dtype=torch.float32):
        return torch.Tensor._make_wrapper_subclass(cls, shape, dtype=dtype, device="cuda")

    @classmethod
    def __torch_dispatch__(cls, func, types, args=(), kwargs=None):
        raise NotImplementedError(str(func))


def test_routing_with_offsets_on_the_host_is_refused(ops):
    """The kernels would read them through a host pointer."""
    r = ops.Routing(torch.tensor([0, 3, 6], dtype=torch.int32), Elsewhere(6, dtype=torch.int32),
                    Elsewhere(3, 2, dtype=torch.int32))
    x, ys, w = Elsewhere(3, 8), Elsewhere(6, 8), Elsewhere(3, 2)
    for call in [lambda: ops.dispatch(x, r), lambda: ops.dispatch_forward(x, r), lambda: ops.dispatch_backward(ys, r),
                 lambda: ops.combine(ys, r, w), lambda: ops.combine_forward(ys, r, w),
                 lambda: ops.combine_backward(x, ys, r, w)]:
        with pytest.raises(ValueError, match="offsets"):
            call()


@pytest.mark.parametrize("size", ["rows", "k", "n"])
def test_linear_sizes_end_short_of_32_bits(ops, size):
    """The kernels step a block past a size in 32 bits: the last sizes below 2^31 are refused."""
    lib, need = ops.load_ops(), ctypes.c_uint64(0)
    for value, rc in (((1 << 31) - 1024, 0), ((1 << 31) - 1023, INVALID), ((1 << 31) - 1, INVALID)):
        d = _desc(ops, **{**dict(rows=1, k=1, n=1), size: value})
        for op in range(5):
            assert lib.muon_linear_workspace(ctypes.byref(d), op, ctypes.byref(need)) == rc, (value, op)
        if rc:
            a = 1 << 32
            assert lib.muon_linear_backward(ctypes.byref(d), None, a, a, a, a, a, a, a, a, 1 << 40, None) == INVALID


def test_backward_of_few_rows_carries_the_rest_of_dz_where_there_is_one(ops):
    """relu's slope is 0 or 1: dz is exact in bf16, and takes no more than for many rows."""
    lib, need = ops.load_ops(), ctypes.c_uint64(0)

    def bytes_of(**kw):
        assert lib.muon_linear_workspace(ctypes.byref(_desc(ops, rows=64, k=24, n=72, **kw)), 4, ctypes.byref(need)) == 0
        return need.value
    assert bytes_of(act=2) >= 2 * 64 * (2 * 72 + 2 * 24)
    assert bytes_of(act=1) < 2 * 64 * 72 + 64 * 72


def test_backward_of_experts_counts_the_rows_of_each(ops):
    """The rest of dz is carried up to 16 rows an expert on average, and up to 64 in all."""
    lib, need = ops.load_ops(), ctypes.c_uint64(0)
    for groups, rows, on in ((0, 64, True), (0, 65, False), (2, 64, True), (2, 65, False), (8, 128, True), (8, 129, False),
                             (64, 1024, True), (64, 1025, False)):
        d = _desc(ops, rows=rows, groups=groups, k=24, n=72, w_stride=24 * 72)
        assert lib.muon_linear_workspace(ctypes.byref(d), 4, ctypes.byref(need)) == 0
        assert (need.value >= 2 * rows * (2 * 72 + 2 * 24 + 4 * 24)) == on, (groups, rows)


def test_optional_tensors_without_memory_are_refused(ops):
    """A wrapper's null address would read as "not given" behind the C interface: a bias left out without a word."""
    assert ops._ptr(None) is None and ops._ptr(torch.empty(0)) == 0 and ops._ptr(torch.zeros(1)) != 0
    with pytest.raises(ValueError, match="memory"):
        ops._ptr(Elsewhere(8))
