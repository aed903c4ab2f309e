"""Host-side tests of the operators around a block's products (no GPU): exported symbols, layouts, refusals and their
codes, workspaces, the references' own pins."""

from __future__ import annotations

import ctypes
import os
import re
import subprocess
import tempfile

import pytest
import torch
from torch.autograd import forward_ad

import block_reference as ref

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "muon_block.h")
INVALID, LAUNCHED = 1, 3          # LAUNCHED: past all checks, where there is no GPU to launch on
A = 1 << 32                       # an address that is never read
no_gpu = pytest.mark.skipif(torch.cuda.is_available(), reason="the pointers are made up: nothing may be launched on them")


@pytest.fixture(scope="module")
def block():
    import muon_newton_schulz_05_amd as pkg
    if not os.path.exists(pkg.LIB_PATH):
        pytest.skip("libmuon.so not built (run __graft_entry__.build())")
    from muon_newton_schulz_05_amd import block as b
    b.load_block()
    return b


@pytest.fixture(scope="module")
def mx(block):
    from muon_newton_schulz_05_amd import mx as m
    return m


def test_exports_every_declared_function(block):
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    declared = set(re.findall(r"\b(muon_[a-z_]+)\s*\(", text))
    assert declared == set(block.EXPORTED_BLOCK)
    for name in declared:
        assert getattr(block.load_block(), name).argtypes, name


def test_public_names_resolve():
    import muon_newton_schulz_05_amd as pkg
    for name in pkg._BLOCK + pkg._MX:
        assert callable(getattr(pkg, name))


def test_struct_layout_matches_c(block):
    lines = "".join(f'  printf("%zu %zu\\n", sizeof({c}), offsetof({c}, {f}));\n' for c, f in (
        ("muon_norm_desc_t", "rows"), ("muon_norm_desc_t", "eps"), ("muon_gate_desc_t", "tokens"),
        ("muon_gate_desc_t", "ldz"), ("muon_mx_desc_t", "rows"), ("muon_mx_desc_t", "ldr")))
    src = f'#include <stddef.h>\n#include <stdio.h>\n#include "muon_block.h"\nint main(void) {{\n{lines}  return 0;\n}}\n'
    with tempfile.TemporaryDirectory() as d:
        c, exe = os.path.join(d, "t.c"), os.path.join(d, "t")
        open(c, "w").write(src)
        subprocess.run(["gcc", "-std=c99", "-I", os.path.join(ROOT, "include"), c, "-o", exe], check=True)
        got = [int(v) for v in subprocess.run([exe], capture_output=True, text=True, check=True).stdout.split()]
    want = []
    for s, f in ((block.NormDesc, "rows"), (block.NormDesc, "eps"), (block.GateDesc, "tokens"), (block.GateDesc, "ldz"),
                 (block.MxDesc, "rows"), (block.MxDesc, "ldr")):
        want += [ctypes.sizeof(s), getattr(s, f).offset]
    assert got == want


def _desc(cls, defaults, kw):
    v = {**defaults, **kw}
    return cls(*[v[f[0]] for f in cls._fields_])


def norm_desc(block, **kw):
    return _desc(block.NormDesc, dict(dtype=1, kind=0, rows=4, cols=8, ldx=8, ldr=8, ldg=8, ldd=8, eps=1e-5), kw)


def gate_desc(block, **kw):
    return _desc(block.GateDesc, dict(dtype=1, experts=8, top=2, normalize=1, tokens=4, ldz=8), kw)


def mx_desc(block, **kw):
    return _desc(block.MxDesc, dict(dtype=1, act=0, groups=0, w_layout=0, rows=4, k=64, n=32, ldx=64, ldw=32, w_stride=0,
                                    ldr=32), kw)


def norm_calls(lib, d):
    p = ctypes.byref(d)
    need = ctypes.c_uint64(0)
    return [lambda: lib.muon_norm_workspace(p, ctypes.byref(need)),
            lambda: lib.muon_norm_forward(p, A, None, None, None, A, None, None, None),
            lambda: lib.muon_norm_backward(p, A, A, None, None, A, None, A, None, None, None, 0, None)]


def gate_calls(lib, d):
    p = ctypes.byref(d)
    return [lambda: lib.muon_gate_forward(p, A, None, A, A, None),
            lambda: lib.muon_gate_backward(p, A, None, A, A, A, A, None)]


def balance_calls(lib, d):
    p, need = ctypes.byref(d), ctypes.c_uint64(0)
    return [lambda: lib.muon_balance_workspace(p, ctypes.byref(need)),
            lambda: lib.muon_balance_forward(p, A, A, 4, None, A, A, A, A, 1 << 40, None),
            lambda: lib.muon_balance_backward(p, A, None, A, A, A, None)]


def mx_calls(lib, d):
    p, a, b = ctypes.byref(d), ctypes.c_uint64(0), ctypes.c_uint64(0)
    return [lambda: lib.muon_mx_sizes(p, ctypes.byref(a), ctypes.byref(b)),
            lambda: lib.muon_mx_quantize(p, A, A, A, None), lambda: lib.muon_mx_dequantize(p, A, A, A, None),
            lambda: lib.muon_mx_linear_workspace(p, ctypes.byref(a)),
            lambda: lib.muon_mx_linear(p, None if d.groups <= 0 else A, A, A, A, None, None, A, A, 1 << 40, None)]


BIG = 1 << 31


@pytest.mark.parametrize("kw", [dict(dtype=7), dict(kind=2), dict(kind=-1), dict(rows=-1), dict(rows=BIG - 1023),
                                dict(cols=-1), dict(cols=(1 << 24) + 1), dict(ldx=-8), dict(ldr=-1), dict(ldg=-1), dict(ldd=-1),
                                dict(eps=-1e-9), dict(eps=float("nan")), dict(eps=float("inf"))], ids=str)
def test_norm_refuses_bad_descriptors(block, kw):
    for call in norm_calls(block.load_block(), norm_desc(block, **kw)):
        assert call() == INVALID


@pytest.mark.parametrize("kw", [dict(dtype=2), dict(experts=0), dict(experts=1025), dict(top=0), dict(top=-1),
                                dict(tokens=-1), dict(tokens=BIG - 1023), dict(ldz=-1)], ids=str)
def test_gate_and_balance_refuse_bad_descriptors(block, kw):
    lib, d = block.load_block(), gate_desc(block, **kw)
    for call in gate_calls(lib, d) + balance_calls(lib, d):
        assert call() == INVALID
    assert lib.muon_gate_forward(ctypes.byref(gate_desc(block, top=9)), A, None, A, A, None) == INVALID
    for call in balance_calls(lib, gate_desc(block, tokens=1 << 28, top=8)):   # 2^31 entries
        assert call() == INVALID


@pytest.mark.parametrize("kw", [dict(dtype=-1), dict(act=5), dict(act=-1), dict(groups=-1), dict(groups=65536),
                                dict(w_layout=2), dict(rows=-1), dict(rows=BIG - 1023), dict(k=(1 << 23) + 1), dict(k=-1),
                                dict(n=(1 << 23) + 1), dict(n=-3), dict(ldx=-1), dict(ldw=-1), dict(w_stride=-1),
                                dict(ldr=-1)], ids=str)
def test_mx_refuses_bad_descriptors(block, kw):
    for call in mx_calls(block.load_block(), mx_desc(block, **kw)):
        assert call() == INVALID


def test_null_descriptors_are_refused(block):
    lib, need = block.load_block(), ctypes.c_uint64(0)
    assert lib.muon_norm_workspace(None, ctypes.byref(need)) == INVALID
    assert lib.muon_norm_workspace(ctypes.byref(norm_desc(block)), None) == INVALID
    assert lib.muon_balance_workspace(None, ctypes.byref(need)) == INVALID
    assert lib.muon_gate_forward(None, A, None, A, A, None) == INVALID
    assert lib.muon_mx_linear_workspace(None, ctypes.byref(need)) == INVALID
    assert lib.muon_mx_sizes(ctypes.byref(mx_desc(block)), None, None) == INVALID


def _refused(call, good, bad):
    """call(**good) gets past its checks, and not with any one of `bad` in place of its own."""
    assert call(**good) == LAUNCHED
    for one in bad:
        assert call(**{**good, **one}) == INVALID, one


@no_gpu
def test_norm_checks_every_pointer(block):
    lib, d = block.load_block(), norm_desc(block)

    def forward(x, r, w, b, y, s, stats):
        return lib.muon_norm_forward(ctypes.byref(d), x, r, w, b, y, s, stats, None)
    _refused(forward, dict(x=A, r=A, w=A, b=A, y=A, s=A, stats=A),
             [dict(x=None), dict(y=None), dict(s=None), dict(r=None)] + [{n: A + 1} for n in ("x", "r", "w", "b", "y", "s")]
             + [dict(stats=A + 2)])
    need = ctypes.c_uint64(0)
    assert lib.muon_norm_workspace(ctypes.byref(d), ctypes.byref(need)) == 0 and need.value

    def backward(dy, x, r, w, stats, ds, dx, dw, db, ws, size):
        return lib.muon_norm_backward(ctypes.byref(d), dy, x, r, w, stats, ds, dx, dw, db, ws, size, None)
    good = dict(dy=A, x=A, r=A, w=A, stats=A, ds=A, dx=A, dw=A, db=A, ws=A, size=need.value)
    _refused(backward, good, [dict(dy=None), dict(x=None), dict(stats=None), dict(ws=None), dict(size=need.value - 1),
                              dict(ws=A + 8), dict(stats=A + 2)] + [{n: A + 1} for n in ("dy", "x", "r", "w", "ds", "dx", "dw", "db")])
    assert backward(**{**good, "dw": None, "db": None, "ws": None, "size": 0}) == LAUNCHED   # dx alone needs none
    assert backward(**{**good, "dx": None, "dw": None, "db": None, "dy": None}) == 0         # nothing is asked for


@no_gpu
def test_gate_checks_every_pointer(block):
    lib, d, dense = block.load_block(), gate_desc(block), gate_desc(block, normalize=0)

    def forward(z, w, i):
        return lib.muon_gate_forward(ctypes.byref(d), z, None, w, i, None)
    _refused(forward, dict(z=A, w=A, i=A), [dict(z=None), dict(w=None), dict(i=None), dict(z=A + 1), dict(w=A + 2), dict(i=A + 2)])

    def backward(z, w, i, dw, dz, d=dense):
        return lib.muon_gate_backward(ctypes.byref(d), z, None, w, i, dw, dz, None)
    good = dict(z=A, w=A, i=A, dw=A, dz=A)
    _refused(backward, good, [{n: None} for n in good] + [dict(z=A + 1), dict(w=A + 2), dict(i=A + 1), dict(dw=A + 2), dict(dz=A + 1)])
    assert backward(**{**good, "z": None, "d": d}) == LAUNCHED     # normalised weights need no logits


@no_gpu
def test_balance_checks_every_pointer(block):
    lib, d, need = block.load_block(), gate_desc(block, top=12), ctypes.c_uint64(0)   # more entries than experts
    assert lib.muon_balance_workspace(ctypes.byref(d), ctypes.byref(need)) == 0 and need.value

    def forward(z, i, ib, loss, counts, shares, ws, size):
        return lib.muon_balance_forward(ctypes.byref(d), z, i, ib, None, loss, counts, shares, ws, size, None)
    good = dict(z=A, i=A, ib=8, loss=A, counts=A, shares=A, ws=A, size=need.value)
    _refused(forward, good, [{n: None} for n in ("z", "i", "loss", "counts", "shares", "ws")] + [
        dict(ib=2), dict(i=A + 4), dict(z=A + 1), dict(loss=A + 2), dict(counts=A + 2), dict(shares=A + 2), dict(ws=A + 4),
        dict(size=need.value - 1)])

    def backward(z, shares, dloss, dz):
        return lib.muon_balance_backward(ctypes.byref(d), z, None, shares, dloss, dz, None)
    good = dict(z=A, shares=A, dloss=A, dz=A)
    _refused(backward, good, [{n: None} for n in good] + [dict(z=A + 1), dict(shares=A + 2), dict(dloss=A + 2), dict(dz=A + 1)])


@no_gpu
@pytest.mark.parametrize("groups", [0, 3])
def test_mx_checks_every_pointer(block, groups):
    lib, d = block.load_block(), mx_desc(block, groups=groups, w_stride=64 * 32, rows=200)
    need = ctypes.c_uint64(0)
    for f in (lib.muon_mx_quantize, lib.muon_mx_dequantize):
        order = (lambda w, v, s: (w, v, s)) if f is lib.muon_mx_quantize else (lambda w, v, s: (v, s, w))

        def call(w, v, s):
            return f(ctypes.byref(d), *order(w, v, s), None)
        _refused(call, dict(w=A, v=A, s=A), [dict(w=None), dict(v=None), dict(s=None), dict(w=A + 1), dict(v=A + 8), dict(s=A + 8)])
    assert lib.muon_mx_linear_workspace(ctypes.byref(d), ctypes.byref(need)) == 0 and need.value

    def linear(o, x, v, s, b, r, y, ws, size):
        return lib.muon_mx_linear(ctypes.byref(d), o, x, v, s, b, r, y, ws, size, None)
    good = dict(o=A if groups else None, x=A, v=A, s=A, b=A, r=None if groups else A, y=A, ws=A, size=need.value)
    _refused(linear, good, [dict(x=None), dict(v=None), dict(s=None), dict(y=None), dict(ws=None), dict(x=A + 1), dict(v=A + 4),
                            dict(s=A + 4), dict(b=A + 1), dict(y=A + 1), dict(ws=A + 8), dict(size=need.value - 1),
                            dict(o=None if groups else A), dict(r=A if groups else A + 1)])


def test_sizes_without_anything_to_do_launch_nothing(block):
    lib = block.load_block()
    assert lib.muon_norm_forward(ctypes.byref(norm_desc(block, rows=0)), None, None, None, None, None, None, None, None) == 0
    assert lib.muon_norm_forward(ctypes.byref(norm_desc(block, cols=0)), None, None, None, None, None, None, None, None) == 0
    assert lib.muon_gate_forward(ctypes.byref(gate_desc(block, tokens=0)), None, None, None, None, None) == 0
    assert lib.muon_mx_quantize(ctypes.byref(mx_desc(block, n=0)), None, None, None, None) == 0
    assert lib.muon_mx_linear(ctypes.byref(mx_desc(block, rows=0)), None, None, A, A, None, None, None, None, 0, None) == 0


@pytest.mark.parametrize("layout", [0, 1])
@pytest.mark.parametrize("groups, k, n", [(65535, 1000 * 512, 1), (1, 1 << 23, 4096), (4096, 1 << 13, 1 << 10)])
def test_weights_that_no_launch_holds_are_refused(block, groups, k, n, layout):
    """A launch holds fewer than 2^32 threads; one column of many weights takes a workgroup of 256 for 512 values each."""
    lib = block.load_block()
    d = mx_desc(block, groups=groups, k=k, n=n, w_layout=layout)
    assert lib.muon_mx_quantize(ctypes.byref(d), A, A, A, None) == INVALID
    assert lib.muon_mx_dequantize(ctypes.byref(d), A, A, A, None) == INVALID


def test_mx_sizes(block):
    lib, v, s = block.load_block(), ctypes.c_uint64(0), ctypes.c_uint64(0)
    for groups, k, n in ((0, 1, 1), (0, 32, 5), (0, 33, 5), (2, 257, 3), (0, 0, 4), (7, 4096, 16384)):
        assert lib.muon_mx_sizes(ctypes.byref(mx_desc(block, groups=groups, k=k, n=n)), ctypes.byref(v), ctypes.byref(s)) == 0
        e = max(groups, 1)
        assert v.value == e * n * -(-k // 128) * 64 and s.value == e * -(-k // 512) * n * 16


# ------------------------------------------------------------------ the binding


@pytest.fixture
def on_cpu(block, mx, monkeypatch):
    """The binding taking CPU tensors, so that a call goes all the way to the kernels'."""
    for m in (block, mx):
        monkeypatch.setattr(m, "_gpu", lambda *a: None)
    monkeypatch.setattr(mx, "_check_linear", lambda *a: None)
    return block


def calls(x):
    import muon_newton_schulz_05_amd as muon
    w = torch.ones(8)
    ids = torch.zeros(len(x), 2, dtype=torch.int32)
    return {"layer_norm": lambda: muon.layer_norm(x, w, w), "layer_norm, residual": lambda: muon.layer_norm(
        torch.ones_like(x.detach()), w, residual=x), "rms_norm": lambda: muon.rms_norm(x, w),
        "gate": lambda: muon.gate(x, 2), "balance_loss": lambda: muon.balance_loss(x, ids),
        "mx_linear": lambda: muon.mx_linear(x, muon.MxWeight(torch.zeros(1, 4, 64, dtype=torch.uint8),
                                                             torch.zeros(1, 4, 16, dtype=torch.uint8), 8))}


def stand_in(block, mx, monkeypatch):
    """In the place of the module that launches: something of the right number of results."""
    class Nodes:
        def __getattr__(self, name):
            return lambda *a: (a[0],) * (1 if name == "mx_linear" else 2)
    for m in (block, mx):
        monkeypatch.setattr(m, "_nodes", lambda what: Nodes())


NAMES = ("layer_norm", "layer_norm, residual", "rms_norm", "gate", "balance_loss", "mx_linear")


@pytest.mark.parametrize("name", NAMES)
@pytest.mark.parametrize("grad", [False, True])
def test_forward_mode_is_refused(on_cpu, mx, monkeypatch, name, grad):
    stand_in(on_cpu, mx, monkeypatch)
    with forward_ad.dual_level(), torch.set_grad_enabled(grad):
        calls(torch.randn(3, 8))[name]()
        x = forward_ad.make_dual(torch.randn(3, 8), torch.ones(3, 8))
        with pytest.raises((RuntimeError, NotImplementedError), match="forward"):
            calls(x)[name]()


@pytest.mark.parametrize("name", NAMES)
@pytest.mark.parametrize("how", ["make_fx", "jit.trace"])
def test_tracing_is_refused(on_cpu, name, how):
    from torch.fx.experimental.proxy_tensor import make_fx
    x = torch.randn(3, 8)
    with pytest.raises(RuntimeError, match="cannot be traced"):
        (make_fx(lambda x: calls(x)[name]()) if how == "make_fx" else lambda x: torch.jit.trace(
            lambda x: calls(x)[name](), (x,)))(x)


@pytest.mark.parametrize("name", NAMES)
@pytest.mark.parametrize("transform", [torch.func.functionalize, torch.func.vmap])
def test_tensors_without_memory_are_refused(on_cpu, name, transform):
    """A view inside functionalization reports its place in a storage of nothing as an address."""
    x = torch.randn(*(() if transform is torch.func.functionalize else (2,)), 4, 8)
    with torch.no_grad(), pytest.raises(RuntimeError, match="no memory|torage"):
        transform(lambda t: calls(t[1:])[name]())(x)


def test_four_bits_refuse_a_gradient(on_cpu, mx, monkeypatch):
    stand_in(on_cpu, mx, monkeypatch)
    x = torch.randn(3, 8, requires_grad=True)
    with pytest.raises(RuntimeError, match="no gradient"):
        calls(x)["mx_linear"]()
    with torch.no_grad():
        calls(x)["mx_linear"]()
    import muon_newton_schulz_05_amd as muon
    muon.mx_quantize(torch.randn(8, 4, requires_grad=True))        # takes the value


class Elsewhere(torch.Tensor):
    """A tensor that says it lives on a GPU and has no memory: for the binding's checks."""

    @staticmethod
    def __new__(cls, *shape, dtype=torch.float32):
        return torch.Tensor._make_wrapper_subclass(cls, shape, dtype=dtype, device="cuda")

    @classmethod
    def __torch_dispatch__(cls, func, types, args=(), kwargs=None):
        raise NotImplementedError(str(func))


def test_the_binding_refuses_what_does_not_fit(block):
    import muon_newton_schulz_05_amd as muon
    G, I32, BF = Elsewhere, torch.int32, torch.bfloat16
    x, z, ids = G(3, 8), G(3, 8), G(3, 2, dtype=I32)
    host = torch.zeros(3, 8)
    bad = [
        lambda: muon.layer_norm(host), lambda: muon.layer_norm(x, G(7)), lambda: muon.layer_norm(x, G(8), G(9)),
        lambda: muon.layer_norm(x, G(8, dtype=BF)), lambda: muon.layer_norm(x, residual=G(3, 7)),
        lambda: muon.layer_norm(x, residual=host), lambda: muon.rms_norm(G(3, 8, dtype=torch.float16)),
        lambda: muon.layer_norm(G()), lambda: muon.norm_forward(x, kind="batch"),
        lambda: muon.norm_backward(x, x, None, G(3, 2), kind="x"), lambda: muon.norm_backward(x, x, None, G(2, 2)),
        lambda: muon.norm_backward(x, x, None, G(3, 2, dtype=BF)), lambda: muon.norm_backward(G(2, 8), x, None, G(3, 2)),
        lambda: muon.norm_backward(x, x, None, G(3, 2), ds=G(3, 9)),
        lambda: muon.norm_backward(x, x, None, G(3, 2), residual=G(3, 9)), lambda: muon.norm_backward(x, x, None, G(3, 2), ds=host), lambda: muon.norm_backward(x, x, G(9), G(3, 2)),
        lambda: muon.gate(host, 2), lambda: muon.gate(z, 0), lambda: muon.gate(z, 9), lambda: muon.gate(G(8), 2),
        lambda: muon.gate(G(3, 1025), 2), lambda: muon.gate(G(3, 0), 1), lambda: muon.gate(G(3, 8, dtype=torch.float64), 2),
        lambda: muon.gate(z, 2, mask=G(3, dtype=torch.uint8)), lambda: muon.gate(z, 2, mask=G(4, dtype=torch.bool)),
        lambda: muon.gate(z, 2, mask=torch.ones(3, dtype=torch.bool)),
        lambda: muon.gate_backward(G(3, 2), z, muon.Gating(G(3, 2), G(3, 2, dtype=torch.int64))),
        lambda: muon.gate_backward(G(3, 3), z, muon.Gating(G(3, 2), ids)),
        lambda: muon.gate_backward(G(3, 2), z, muon.Gating(G(3, 3), ids)),
        lambda: muon.gate_backward(G(3, 2, dtype=BF), z, muon.Gating(G(3, 2), ids)),
        lambda: muon.gate_backward(host[:, :2], z, muon.Gating(G(3, 2), ids)),
        lambda: muon.balance_loss(host, ids), lambda: muon.balance_loss(z, G(4, 2, dtype=I32)),
        lambda: muon.balance_loss(z, G(3, 2)), lambda: muon.balance_loss(z, G(6, dtype=I32)),
        lambda: muon.balance_loss(z, torch.zeros(3, 2, dtype=I32)), lambda: muon.balance_loss(z, G(3, 0, dtype=I32)),
        lambda: muon.balance_loss(z, ids, mask=G(2, dtype=torch.bool)),
        lambda: muon.balance_backward(G(2), z, ids, G(9)), lambda: muon.balance_backward(G(), z, ids, G(8)),
        lambda: muon.balance_backward(torch.zeros(()), z, ids, G(9)),
        lambda: muon.mx_quantize(host), lambda: muon.mx_quantize(G(8)), lambda: muon.mx_quantize(G(2, 2, 2, 2)),
        lambda: muon.mx_quantize(G(8, 8, dtype=torch.float16)), lambda: muon.mx_quantize(G(0, 8, 8)),
        lambda: muon.mx_quantize(G((1 << 23) + 1, 1)),
    ]
    for i, call in enumerate(bad):
        with pytest.raises((ValueError, TypeError)):
            call()
            print("not refused:", i)


def test_the_binding_refuses_weights_that_do_not_fit(block, mx):
    import muon_newton_schulz_05_amd as muon
    U8, G = torch.uint8, Elsewhere

    def weight(k=40, n=4, lead=(), values=None, scales=None):
        return muon.MxWeight(G(*lead, (k + 127) // 128, n, 64, dtype=U8) if values is None else values,
                             G(*lead, (k + 511) // 512, n, 16, dtype=U8) if scales is None else scales, k)
    x, off = G(3, 40), G(3, dtype=torch.int32)
    for w in (weight(values=G(2, 4, 64, dtype=U8)), weight(values=G(1, 4, 32, dtype=U8)), weight(values=G(1, 4, 64)),
              weight(values=G(4, 64, dtype=U8)), weight(scales=G(2, 4, 16, dtype=U8)), weight(scales=G(1, 4, 16)),
              weight(scales=G(1, 5, 16, dtype=U8)), weight(values=torch.zeros(1, 4, 64, dtype=U8)),
              weight(scales=torch.zeros(1, 4, 16, dtype=U8)), muon.MxWeight(G(0, 4, 64, dtype=U8), G(0, 4, 16, dtype=U8), -1)):
        for call in (lambda: muon.mx_linear(x, w), lambda: muon.mx_dequantize(w)):
            with pytest.raises(ValueError):
                call()
    assert weight(lead=(2,)).shape == (2, 40, 4) and weight().shape == (40, 4)
    for call in (lambda: muon.mx_linear(G(3, 41), weight()), lambda: muon.mx_linear(x, weight(lead=(2,))),
                 lambda: muon.mx_expert_linear(x, weight(), off), lambda: muon.mx_expert_linear(x, weight(lead=(2,)), None),
                 lambda: muon.mx_expert_linear(x, weight(lead=(3,)), off), lambda: muon.mx_linear(x, weight(), G(5)),
                 lambda: muon.mx_linear(x, weight(), residual=G(3, 5)), lambda: muon.mx_linear(x, weight(), activation="tanh"),
                 lambda: muon.mx_linear(torch.zeros(3, 40), weight()), lambda: muon.mx_linear(x, weight(), torch.zeros(4))):
        with pytest.raises(ValueError):
            call()


# ------------------------------------------------------------------ the references' own pins


def test_norm_reference_against_autograd_and_differences():
    g = torch.Generator().manual_seed(1)
    x, r, w, b, dy, ds = (torch.randn(s, generator=g, dtype=torch.float64) for s in
                          ((5, 12), (5, 12), (12,), (12,), (5, 12), (5, 12)))
    for layer in (True, False):
        leaves = [t.clone().requires_grad_() for t in (x, w, b)]
        h = leaves[0] + r
        y = torch.nn.functional.layer_norm(h, (12,), leaves[1], leaves[2], 1e-5) if layer else \
            h * torch.rsqrt(h.square().mean(1, keepdim=True) + 1e-5) * leaves[1] + leaves[2]
        got = torch.autograd.grad((y, h), leaves, (dy, ds))
        want = ref.norm64(x, r, w, b, dy, ds, 1e-5, layer)
        for name, v in zip(("y", "dx", "dw", "db"), (y.detach(), *got)):
            assert torch.allclose(want[name][0], v, rtol=1e-12, atol=1e-12), name
        # one direction by central differences
        e = 1e-6 * torch.randn(5, 12, generator=g, dtype=torch.float64)
        up, down = (ref.norm64(x + q * e, r, w, b, None, None, 1e-5, layer)["y"][0] for q in (1, -1))
        assert torch.allclose(((up - down) / 2 * dy).sum() + (e * ds).sum(), (want["dx"][0] * e).sum(), rtol=1e-6)


def test_gate_and_balance_references_against_autograd():
    g = torch.Generator().manual_seed(2)
    z, dw = torch.randn(6, 9, generator=g, dtype=torch.float64), torch.randn(6, 3, generator=g, dtype=torch.float64)
    mask = torch.tensor([1, 1, 0, 1, 1, 1], dtype=torch.bool)
    for normalize in (True, False):
        leaf = z.clone().requires_grad_()
        p = torch.softmax(leaf, 1)
        w, ids = torch.topk(p, 3, dim=1)
        w = (w / w.sum(1, keepdim=True) if normalize else w) * mask[:, None]
        want = ref.gate64(z, 3, normalize, mask, dw)
        assert torch.equal(want["ids"], torch.where(mask[:, None], ids, -1))
        assert torch.allclose(want["weights"][0], w.detach(), rtol=1e-12)
        assert torch.allclose(want["dz"][0], torch.autograd.grad(w, leaf, dw)[0], rtol=1e-10, atol=1e-15)
    ids = torch.randint(-1, 10, (6, 4), generator=g)
    leaf = z.clone().requires_grad_()
    f = torch.stack([(ids[mask] == e).sum() for e in range(9)]).double() / (5 * 4)
    loss = 9 * (f * torch.softmax(leaf, 1)[mask].mean(0)).sum()
    want = ref.balance64(z, ids, mask, 0.5)
    assert torch.allclose(want["loss"][0], loss.detach()) and torch.equal(want["counts"], (f * 20).round().long())
    assert torch.allclose(want["dz"][0], torch.autograd.grad(loss, leaf)[0] * 0.5, rtol=1e-10, atol=1e-15)


def test_gate_reference_orders_ties_and_what_is_not_finite():
    inf, nan = float("inf"), float("nan")
    z = torch.tensor([[1., 2., 2., -0., 0.], [-inf, -inf, 3., -inf, -inf], [nan, 5., inf, 1., nan], [-inf] * 5])
    assert ref.choose(z, 3, None).tolist() == [[1, 2, 0], [2, -1, -1], [0, 4, 2], [-1, -1, -1]]
    assert ref.choose(z[:1], 5, None).tolist() == [[1, 2, 0, 3, 4]]


def test_four_bit_reference():
    """Every level, the borders between them (to the even code), saturation, and the scale of a small block."""
    row = torch.tensor([[0.0, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 7.9, -0.26, -6.0] + [0.0] * 21])
    values, codes, scales = ref.blocks64(row)
    assert values[0, :11].tolist() == [0.0, 0.0, 1.0, 1.0, 2.0, 2.0, 4.0, 4.0, 6.0, -0.5, -6.0] and scales.tolist() == [[127]]
    assert codes[0, :11].tolist() == [0, 0, 2, 2, 4, 4, 6, 6, 7, 9, 15]
    small = torch.zeros(1, 32, dtype=torch.float64)
    small[0, 0] = 2.0 ** -140
    assert ref.blocks64(small)[2].item() == 0 and ref.blocks64(small)[0][0, 0] == 0
    assert ref.blocks64(torch.full((1, 32), 2.0 ** 127))[2].item() == 127 + 125
    assert ref.blocks64(torch.tensor([[float("inf")] + [1.0] * 31]))[2].item() == 255
    v = torch.randn(7, 75, generator=torch.Generator().manual_seed(1)) * 3
    assert torch.equal(ref.blocks64(v)[0], ref.fast_blocks64(v))


@no_gpu
def test_sizes_past_a_launch_are_refused_before_one(block):
    """What one launch cannot hold is said with the arguments, not by the runtime half way through."""
    lib = block.load_block()
    for kw in (dict(rows=1 << 30, k=1 << 16, n=8, ldx=1 << 16), dict(rows=(1 << 31) - 1024, k=512, n=1 << 20, ldx=512)):
        d = mx_desc(block, **kw)
        assert lib.muon_mx_linear(ctypes.byref(d), None, A, A, A, None, None, A, A, (1 << 63), None) == INVALID
    d = mx_desc(block, k=1 << 23, n=1 << 23, ldw=1 << 23)
    assert lib.muon_mx_quantize(ctypes.byref(d), A, A, A, None) == INVALID
    assert lib.muon_mx_dequantize(ctypes.byref(d), A, A, A, None) == INVALID


def test_missing_nodes_are_said(block, monkeypatch):
    """Without the module that launches there is an error, not another way round."""
    import sys
    monkeypatch.setattr(block, "_module", None)
    monkeypatch.setitem(sys.modules, "muon_newton_schulz_05_amd._nodes", None)
    import muon_newton_schulz_05_amd as pkg
    monkeypatch.delattr(pkg, "_nodes", raising=False)
    with pytest.raises(RuntimeError, match="not built"):
        block._nodes("a norm")
