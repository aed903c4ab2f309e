"""Build libmuon.so in-tree with hipcc for gfx950, and _nodes.so, which binds part of it to torch.

    python -m muon_newton_schulz_05_amd.build            # compile (always)
"""

from __future__ import annotations

import os
import shutil
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
LIB = os.path.join(PKG, "libmuon.so")
NODES = os.path.join(PKG, "_nodes.so")
BUILD_DIR = os.path.join(PKG, "_build")
SOURCES = ["api.cpp", "planner.cpp", "skinny.hip", "stream.hip", "stream_big.hip", "noalloc.hip",
           "ops_api.cpp", "linear_bf16.hip", "linear_f32.hip", "route.hip", "dropout.hip",
           "block_api.cpp", "norm.hip", "gate.hip", "mx.hip", "linear_mx.hip"]

NODES_SOURCE = "block_nodes.cpp"

CXX = os.environ.get("CXX", "g++")
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
ARCH = "gfx950"
# Packed float32 instructions are switched off for the device code.
DEVICE_FLAGS = ["-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops"]
COMMON = ["-O3", "-std=c++17", "-fPIC", f"--offload-arch={ARCH}", "-I", os.path.join(ROOT, "include"),
          "-Wno-unused-command-line-argument"]


def _run(what: str, cmd: list[str]) -> None:
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{what} failed: {' '.join(cmd)}\n{r.stdout}\n{r.stderr}")


def _compile(src: str) -> str:
    obj = os.path.join(BUILD_DIR, os.path.splitext(src)[0] + ".o")
    if src == NODES_SOURCE:
        import sysconfig

        from torch.utils import cpp_extension
        include = [*cpp_extension.include_paths(), sysconfig.get_paths()["include"], "/opt/rocm/include"]
        flags = ["-O2", "-std=c++17", "-fPIC", "-w", "-D__HIP_PLATFORM_AMD__", "-DTORCH_EXTENSION_NAME=_nodes",
                 "-DUSE_ROCM", *[f"-I{d}" for d in include]]
        _run("compile", [CXX, *flags, "-c", os.path.join(CSRC, src), "-o", obj])
        return obj
    lang = ["-x", "hip"] if src.endswith(".hip") else []
    _run("compile", [HIPCC, *COMMON, *DEVICE_FLAGS, *lang, "-c", os.path.join(CSRC, src), "-o", obj])
    return obj


def _no_nodes() -> str | None:
    """Why _nodes.so cannot be built here, or None.  libmuon.so takes neither torch nor a second compiler."""
    try:
        import torch
        from torch.utils import cpp_extension  # noqa: F401
    except (ImportError, OSError) as e:
        return f"torch is not importable ({e})"
    if torch.version.hip is None:
        return "torch is not built for ROCm"
    return None if shutil.which(CXX) else f"{CXX} is not found"


def _link_nodes(obj: str) -> None:
    from torch.utils import cpp_extension
    libs = [f"-L{d}" for d in cpp_extension.library_paths()]
    tmp = NODES + ".tmp"
    _run("link", [CXX, "-shared", "-o", tmp, obj, *libs, "-lc10", "-lc10_hip", "-ltorch_cpu", "-ltorch_hip", "-ltorch_python",
                  f"-L{os.path.dirname(LIB)}", "-l:libmuon.so", "-Wl,-rpath,$ORIGIN"])
    os.replace(tmp, NODES)


def build(verbose: bool = False) -> str:
    """libmuon.so, and _nodes.so where torch and a C++ compiler are there.  A _nodes.so that is not built raises, where it
    could have been, once libmuon.so is in place; one of an earlier library does not stay beside it either way."""
    if not os.path.exists(HIPCC) and shutil.which("hipcc") is None:
        raise RuntimeError("hipcc not found")
    os.makedirs(BUILD_DIR, exist_ok=True)
    without = _no_nodes()
    with ThreadPoolExecutor(max_workers=min(8, len(SOURCES) + 1)) as ex:
        nodes = None if without else ex.submit(_compile, NODES_SOURCE)
        objs = list(ex.map(_compile, SOURCES))
        tmp = LIB + ".tmp"
        _run("link", [HIPCC, f"--offload-arch={ARCH}", "-shared", "-fPIC", "-o", tmp, *objs])
        os.replace(tmp, LIB)
        built = False
        try:
            if nodes:
                _link_nodes(nodes.result())
                built = True
        finally:
            if not built and os.path.exists(NODES):
                os.remove(NODES)
    if without:
        print(f"_nodes.so is left out: {without}.  The C ABI and the Muon step do not need it; layer_norm, rms_norm, gate, "
              "balance_loss and the layers in four bits do.", file=sys.stderr)
    if verbose:
        print(f"built {LIB}" + ("" if without else f" and {NODES}"))
    return LIB


if __name__ == "__main__":
    build(verbose=True)
    sys.exit(0)
