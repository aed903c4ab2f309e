"""Host-side tests of the layer operators (no GPU): exported symbols, refusals and their codes, workspaces, the
references' own pins."""

from __future__ import annotations

import ctypes
import os
import re
import subprocess
import tempfile

import pytest
import torch

import ops_reference as ref

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "muon_ops.h")
INVALID = 1


@pytest.fixture(scope="module")
def ops():
    import muon_newton_schulz_05_amd as pkg
    if not os.path.exists(pkg.LIB_PATH):
        pytest.skip("libmuon.so not built (run __graft_entry__.build())")
    from muon_newton_schulz_05_amd import ops as o
    o.load_ops()
    return o


def test_exports_every_declared_function(ops):
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    declared = set(re.findall(r"\b(muon_[a-z_]+)\s*\(", text))
    assert declared == set(ops.EXPORTED_OPS)
    for name in declared:
        assert hasattr(ops.load_ops(), name), name


def test_public_names_resolve():
    import muon_newton_schulz_05_amd as pkg
    for name in pkg._OPS:
        assert callable(getattr(pkg, name))


def test_struct_layout_matches_c(ops):
    src = r'''
#include <stddef.h>
#include <stdio.h>
#include "muon_ops.h"
int main(void) {
  printf("%zu %zu %zu %zu\n", sizeof(muon_linear_desc_t), offsetof(muon_linear_desc_t, rows),
         offsetof(muon_linear_desc_t, w_stride), offsetof(muon_linear_desc_t, ldg));
  printf("%zu %zu %zu\n", sizeof(muon_move_desc_t), offsetof(muon_move_desc_t, tokens),
         offsetof(muon_move_desc_t, ldr));
  return 0;
}
'''
    with tempfile.TemporaryDirectory() as d:
        c, exe = os.path.join(d, "t.c"), os.path.join(d, "t")
        open(c, "w").write(src)
        subprocess.run(["gcc", "-std=c99", "-I", os.path.join(ROOT, "include"), c, "-o", exe], check=True)
        vals = [int(x) for x in subprocess.run([exe], capture_output=True, text=True, check=True).stdout.split()]
    L, M = ops.LinearDesc, ops.MoveDesc
    assert vals == [ctypes.sizeof(L), L.rows.offset, L.w_stride.offset, L.ldg.offset,
                    ctypes.sizeof(M), M.tokens.offset, M.ldr.offset]


def _desc(ops, **kw):
    d = dict(dtype=1, act=0, groups=0, w_layout=0, rows=4, k=8, n=8, ldx=8, ldw=8, w_stride=0, ldr=8, ldg=8)
    d.update(kw)
    return ops.LinearDesc(*[d[f[0]] for f in ops.LinearDesc._fields_])


@pytest.mark.parametrize("kw", [dict(dtype=7), dict(act=9), dict(act=-1), dict(groups=-1), dict(groups=70000),
                                dict(w_layout=2), dict(rows=-1), dict(k=1 << 31), dict(n=-5), dict(ldx=-8),
                                dict(w_stride=-1)])
def test_linear_refuses_bad_descriptors(ops, kw):
    lib, d = ops.load_ops(), _desc(ops, **kw)
    need = ctypes.c_uint64(1)
    assert lib.muon_linear_workspace(ctypes.byref(d), 0, ctypes.byref(need)) == INVALID
    q = 4096  # never read: the descriptor is refused first
    assert lib.muon_linear_forward(ctypes.byref(d), None, q, q, None, None, q, None, None, 0, None) == INVALID
    assert lib.muon_linear_grad_act(ctypes.byref(d), None, q, q, q, None, None, 0, None) == INVALID
    assert lib.muon_linear_grad_input(ctypes.byref(d), None, q, q, q, None, 0, None) == INVALID
    assert lib.muon_linear_grad_weight(ctypes.byref(d), None, q, q, q, None, 0, None) == INVALID
    assert ops.muon_last_error()


def test_linear_refuses_bad_pointers(ops):
    lib, q = ops.load_ops(), 4096
    d, g = _desc(ops), _desc(ops, groups=2, w_stride=64)
    f = lib.muon_linear_forward
    assert f(None, None, q, q, None, None, q, None, None, 0, None) == INVALID
    for args in [(None, None, q, None, None, q, None), (None, q, None, None, None, q, None),
                 (None, q, q, None, None, None, None), (None, q + 1, q, None, None, q, None),
                 (None, q, q, q + 1, None, q, None), (None, q, q, None, q + 1, q, None),
                 (q, q, q, None, None, q, None)]:                  # offsets without groups
        assert f(ctypes.byref(d), *args, None, 0, None) == INVALID, args
    assert f(ctypes.byref(g), None, q, q, None, None, q, None, None, 0, None) == INVALID   # groups without offsets
    assert f(ctypes.byref(g), q, q, q, None, q, q, None, None, 0, None) == INVALID         # a grouped residual
    s = _desc(ops, act=2)
    assert lib.muon_linear_grad_act(ctypes.byref(s), None, q, None, q, None, None, 0, None) == INVALID  # no z
    assert lib.muon_linear_grad_act(ctypes.byref(d), None, q, None, None, q, None, 0, None) == INVALID  # no workspace


def test_linear_split_needs_its_workspace(ops):
    lib, q = ops.load_ops(), 4096
    d = _desc(ops, rows=2, k=16384, n=64, ldx=16384, ldw=64)
    need = ctypes.c_uint64(0)
    assert lib.muon_linear_workspace(ctypes.byref(d), 0, ctypes.byref(need)) == 0
    assert need.value >= 2 * 64 * 4
    assert lib.muon_linear_forward(ctypes.byref(d), None, q, q, None, None, q, None, None, 0, None) == INVALID
    assert lib.muon_linear_forward(ctypes.byref(d), None, q, q, None, None, q, None, q, 16, None) == INVALID


def test_linear_copies_need_their_workspace(ops):
    """A large odd product lays out both operands anew; a smaller one, and float32, need nothing."""
    lib, q = ops.load_ops(), 4096
    odd = dict(rows=2001, k=1001, n=2003, ldx=1001, ldw=2003, ldg=2003)
    d, need = _desc(ops, **odd), ctypes.c_uint64(0)
    assert lib.muon_linear_workspace(ctypes.byref(d), 0, ctypes.byref(need)) == 0
    assert need.value >= 2 * (2001 * 1008 + 1001 * 2008)
    f = lib.muon_linear_forward
    assert f(ctypes.byref(d), None, q, q, None, None, q, None, None, 0, None) == INVALID
    assert f(ctypes.byref(d), None, q, q, None, None, q, None, q, need.value - 1, None) == INVALID
    assert f(ctypes.byref(d), None, q, q, None, None, q, None, q + 8, need.value, None) == INVALID
    for other in (dict(odd, dtype=0), dict(odd, rows=65)):
        assert lib.muon_linear_workspace(ctypes.byref(_desc(ops, **other)), 0, ctypes.byref(need)) == 0
        assert need.value < 2 * 1001 * 2008


def test_linear_workspace_covers_one_unaligned_operand(ops):
    """x alone out of reach is copied where both together are not: the larger need is told."""
    lib, need = ops.load_ops(), ctypes.c_uint64(0)
    d = _desc(ops, rows=100, k=4096, n=4096, ldx=4096, ldw=4096)
    assert lib.muon_linear_workspace(ctypes.byref(d), 0, ctypes.byref(need)) == 0
    assert 2 * 100 * 4096 <= need.value


def test_linear_backward_needs_its_workspace(ops):
    """Up to 64 rows: two rows of dz for each, each row of x twice, and dx in float32; more rows keep one."""
    lib, q, need = ops.load_ops(), 4096, ctypes.c_uint64(0)
    d = _desc(ops, act=2, rows=64, k=24, n=72, ldx=24, ldw=72, ldg=72)
    assert lib.muon_linear_workspace(ctypes.byref(d), 4, ctypes.byref(need)) == 0
    assert need.value >= 2 * 64 * (2 * 72 + 2 * 24 + 4 * 24)
    f = lib.muon_linear_backward
    assert f(ctypes.byref(d), None, q, q, q, q, q, q, q, None, 0, None) == INVALID
    assert f(ctypes.byref(d), None, q, q, q, q, q, q, q, q, 64, None) == INVALID
    assert f(ctypes.byref(d), None, q, q, q, q, q, q, q, q + 8, need.value, None) == INVALID
    for other in (dict(rows=65), dict(act=0), dict(dtype=0)):
        o = _desc(ops, **{**dict(act=2, rows=64, k=24, n=72, ldx=24, ldw=72, ldg=72), **other})
        assert lib.muon_linear_workspace(ctypes.byref(o), 4, ctypes.byref(need)) == 0
        assert need.value < 2 * 64 * (2 * 72 + 2 * 24 + 4 * 24)


def test_route_refuses(ops):
    lib, q = ops.load_ops(), 4096
    need = ctypes.c_uint64(0)
    for e in (0, -1, 1025):
        assert lib.muon_route_workspace(8, e, ctypes.byref(need)) == INVALID
    assert lib.muon_route_workspace(-1, 4, ctypes.byref(need)) == INVALID
    f = lib.muon_route
    assert f(q, 2, 4, 2, 4, q, q, q, q, 1 << 20, None) == INVALID
    assert f(q, 8, 4, 0, 4, q, q, q, q, 1 << 20, None) == INVALID
    assert f(None, 8, 4, 2, 4, q, q, q, q, 1 << 20, None) == INVALID
    assert f(q + 4, 8, 4, 2, 4, q, q, q, q, 1 << 20, None) == INVALID
    assert f(q, 8, 4, 2, 4, q, q, q, None, 0, None) == INVALID
    assert f(q, 8, 1 << 30, 4, 4, q, q, q, q, 1 << 40, None) == INVALID


def test_moves_refuse(ops):
    lib, q = ops.load_ops(), 4096
    good = dict(dtype=1, experts=4, top=2, reserved=0, tokens=3, h=8, ldx=8, ldg=8, ldr=8)
    for kw in [dict(dtype=3), dict(top=0), dict(tokens=-1), dict(h=-1), dict(experts=0), dict(experts=2000),
               dict(tokens=1 << 31), dict(ldx=-1)]:
        d = ops.MoveDesc(*{**good, **kw}.values())
        assert lib.muon_dispatch(ctypes.byref(d), q, q, q, q, None) == INVALID, kw
        assert lib.muon_dispatch_grad(ctypes.byref(d), q, q, q, None) == INVALID, kw
        assert lib.muon_combine(ctypes.byref(d), q, q, q, None, q, None) == INVALID, kw
        assert lib.muon_combine_grad(ctypes.byref(d), q, q, q, q, q, q, q, None) == INVALID, kw
    d = ops.MoveDesc(*good.values())
    assert lib.muon_dispatch(ctypes.byref(d), None, q, q, q, None) == INVALID
    assert lib.muon_dispatch(ctypes.byref(d), q, q, q + 1, q, None) == INVALID
    assert lib.muon_combine(ctypes.byref(d), q, q + 2, q, None, q, None) == INVALID


def test_dropout_refuses(ops):
    lib, q = ops.load_ops(), 4096
    for p in (-0.1, 1.0, 1.5, float("nan"), 0.9999999):
        assert lib.muon_dropout(1, 8, q, None, q, p, 0, 0, None, None) == INVALID, p
    assert lib.muon_dropout(5, 8, q, None, q, 0.5, 0, 0, None, None) == INVALID
    assert lib.muon_dropout(1, -1, q, None, q, 0.5, 0, 0, None, None) == INVALID
    assert lib.muon_dropout(1, 8, None, None, q, 0.5, 0, 0, None, None) == INVALID
    assert lib.muon_dropout(0, 8, q + 2, None, q, 0.5, 0, 0, None, None) == INVALID
    assert lib.muon_dropout(1, 8, q, None, q, 0.5, 0, 0, q + 4, None) == INVALID


def test_binding_refuses_cpu_tensors(ops):
    x, w = torch.zeros(2, 4), torch.zeros(4, 4)
    with pytest.raises(ValueError):
        ops.linear(x, w)
    with pytest.raises(ValueError):
        ops.route(torch.zeros(2, 2, dtype=torch.int64), 4)
    with pytest.raises(ValueError):
        ops.dropout(x, 0.5)
    with pytest.raises(ValueError):
        ops.linear(x, w, activation="swish")


def test_philox_known_answers():
    """The generator's published known answers (zero, and all bits set)."""
    assert ref.philox(0, 0, 0) == [0x6627e8d5, 0xe169c58d, 0xbc57ac4c, 0x9b00dbd8]
    ones = (1 << 64) - 1
    assert ref.philox(ones, ones, ones) == [0x408f276d, 0x41c83b0e, 0xa20bc7c6, 0x6d5451fd]


@pytest.mark.parametrize("act", ["relu", "silu", "gelu", "gelu_tanh"])
def test_reference_slopes_match_differences(act):
    z = torch.linspace(-6, 6, 997, dtype=torch.float64) + 1e-3
    h = 1e-6
    diff = (ref.act64(z + h, act)[0] - ref.act64(z - h, act)[0]) / (2 * h)
    # central differences: h^2 / 6 times a third derivative of a few, and 2^-52 / h.
    assert (ref.act64(z, act)[1] - diff).abs().max() < 1e-8
