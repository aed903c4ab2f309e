"""Host-side tests (no GPU) of the operators around a block's products where calls are unusual."""

from __future__ import annotations

import ctypes
import os
import sys

import pytest
import torch

from test_block_host import A, Elsewhere, block, norm_desc, no_gpu  # noqa: F401 (block is a fixture)


@no_gpu
@pytest.mark.parametrize("cols", [8, 8192, 8193, 20000])
def test_a_norm_gradient_of_no_rows_launches_nothing_for_dx(block, cols):  # noqa: F811
    """dx has an address and no elements: a launch of no workgroups is an error of the runtime."""
    lib = block.load_block()
    d = norm_desc(block, rows=0, cols=cols)
    assert lib.muon_norm_backward(ctypes.byref(d), None, None, None, None, None, None, A, None, None, None, 0, None) == 0


def test_entries_that_32_bits_do_not_count_are_refused(block):  # noqa: F811
    """tokens * top at 2^31 and above, a list whose length is small in its low 32 bits among them."""
    import muon_newton_schulz_05_amd as muon
    z, one = Elsewhere(1, 8), Elsewhere(dtype=torch.float32)
    for top in (1 << 31, (1 << 32) + 2, 1 << 33):
        ids = Elsewhere(1, top, dtype=torch.int32)
        for call in (lambda: muon.balance_loss(z, ids), lambda: muon.balance_forward(z, ids),
                     lambda: muon.balance_backward(one, z, ids, Elsewhere(9))):
            with pytest.raises(ValueError, match="entries"):
                call()
    with pytest.raises(ValueError, match="entries"):
        muon.balance_loss(Elsewhere(1 << 28, 8), Elsewhere(1 << 28, 8, dtype=torch.int32))


# ------------------------------------------------------------------ the build


@pytest.fixture
def fake_build(monkeypatch, tmp_path):
    """The build with every command replaced by an empty output, in a folder of its own; an older _nodes.so is there."""
    from muon_newton_schulz_05_amd import build as b
    lib, nodes = str(tmp_path / "libmuon.so"), str(tmp_path / "_nodes.so")
    for name, value in (("LIB", lib), ("NODES", nodes), ("BUILD_DIR", str(tmp_path / "_build")), ("HIPCC", sys.executable)):
        monkeypatch.setattr(b, name, value)
    open(nodes, "w").close()

    def run(what, cmd):
        if b.CXX == "broken" and cmd[0] == b.CXX:
            raise RuntimeError(f"{what} failed")
        open(cmd[cmd.index("-o") + 1], "w").write(what)
    monkeypatch.setattr(b, "_run", run)
    return b, lib, nodes


def test_build_makes_both(fake_build):
    b, lib, nodes = fake_build
    assert b.build() == lib and os.path.exists(lib) and os.path.getsize(nodes)


@pytest.mark.parametrize("missing", ["torch", "ROCm", "compiler"])
def test_the_library_is_built_without_torch(fake_build, monkeypatch, capsys, missing):
    """The C ABI needs hipcc alone; the module that binds it to torch is left out, said to be, and no older one stays."""
    b, lib, nodes = fake_build
    if missing == "torch":
        for name in ("torch", "torch.utils", "torch.utils.cpp_extension"):
            monkeypatch.setitem(sys.modules, name, None)
    elif missing == "ROCm":
        monkeypatch.setattr(torch.version, "hip", None)
    else:
        monkeypatch.setattr(b, "CXX", "/nowhere/g++")
    assert b.build() == lib and os.path.exists(lib) and not os.path.exists(nodes)
    assert "_nodes.so" in capsys.readouterr().err


def test_a_module_that_does_not_compile_is_an_error_after_the_library(fake_build, monkeypatch):
    b, lib, nodes = fake_build
    monkeypatch.setattr(b, "CXX", "broken")
    monkeypatch.setattr(b.shutil, "which", lambda name: name)
    with pytest.raises(RuntimeError, match="failed"):
        b.build()
    assert os.path.exists(lib) and not os.path.exists(nodes)
