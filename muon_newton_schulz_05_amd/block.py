"""Operators around a block's products on torch tensors: norms, a router's gate and its balance loss.

Everything runs in the HIP kernels behind the C ABI of ``include/muon_block.h``, in
the manner of the layer operators: float32 or bfloat16 tensors on one GPU, on the current torch stream; rows may be
strided; each call is differentiable backwards, once; forward-mode differentiation
and tracers raise.

* ``layer_norm`` and ``rms_norm``: a norm of rows, with the residual added ahead of it;
* ``gate``: the experts of each token and their weights, for ``route`` and ``combine``;
* ``balance_loss``: the loss that evens the experts' loads, and their counts.

The ``*_forward`` and ``*_backward`` functions are the same passes without
autograd, for code that captures them into a HIP graph.
"""

from __future__ import annotations

import ctypes
import math
from typing import NamedTuple, Optional

import torch
from torch.autograd import forward_ad

from .ops import _dtype, _gpu, _same, _traced, _tracked, load_ops

GATE_MAX_EXPERTS = 1024
BALANCE_MAX_ENTRIES = (1 << 31) - 1024  # counts are held in 32 bits
NORMS = {"layer": 0, "rms": 1}
EXPORTED_BLOCK = ("muon_norm_workspace", "muon_norm_forward", "muon_norm_backward", "muon_gate_forward",
                  "muon_gate_backward", "muon_balance_workspace", "muon_balance_forward", "muon_balance_backward",
                  "muon_mx_sizes", "muon_mx_quantize", "muon_mx_dequantize", "muon_mx_linear_workspace",
                  "muon_mx_linear")


class NormDesc(ctypes.Structure):
    _fields_ = [("dtype", ctypes.c_int32), ("kind", ctypes.c_int32), ("rows", ctypes.c_int64), ("cols", ctypes.c_int64),
                ("ldx", ctypes.c_int64), ("ldr", ctypes.c_int64), ("ldg", ctypes.c_int64), ("ldd", ctypes.c_int64),
                ("eps", ctypes.c_double)]


class GateDesc(ctypes.Structure):
    _fields_ = [("dtype", ctypes.c_int32), ("experts", ctypes.c_int32), ("top", ctypes.c_int32),
                ("normalize", ctypes.c_int32), ("tokens", ctypes.c_int64), ("ldz", ctypes.c_int64)]


class MxDesc(ctypes.Structure):
    _fields_ = [("dtype", ctypes.c_int32), ("act", ctypes.c_int32), ("groups", ctypes.c_int32),
                ("w_layout", ctypes.c_int32), ("rows", ctypes.c_int64), ("k", ctypes.c_int64), ("n", ctypes.c_int64),
                ("ldx", ctypes.c_int64), ("ldw", ctypes.c_int64), ("w_stride", ctypes.c_int64), ("ldr", ctypes.c_int64)]


_lib = None


def load_block():
    """libmuon.so with the signatures of include/muon_block.h; raises if it is not built."""
    global _lib
    if _lib is not None:
        return _lib
    lib = load_ops()
    P, I32, U64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_uint64
    N, G, X, UP = (ctypes.POINTER(t) for t in (NormDesc, GateDesc, MxDesc, U64))
    sig = {
        "muon_norm_workspace": [N, UP],
        "muon_norm_forward": [N] + [P] * 8,
        "muon_norm_backward": [N] + [P] * 10 + [U64, P],
        "muon_gate_forward": [G] + [P] * 5,
        "muon_gate_backward": [G] + [P] * 7,
        "muon_balance_workspace": [G, UP],
        "muon_balance_forward": [G, P, P, I32, P, P, P, P, P, U64, P],
        "muon_balance_backward": [G] + [P] * 6,
        "muon_mx_sizes": [X, UP, UP],
        "muon_mx_quantize": [X] + [P] * 4,
        "muon_mx_dequantize": [X] + [P] * 4,
        "muon_mx_linear_workspace": [X, UP],
        "muon_mx_linear": [X] + [P] * 8 + [U64, P],
    }
    for name, args in sig.items():
        f = getattr(lib, name)
        f.argtypes = args
        f.restype = ctypes.c_int
    _lib = lib
    return lib


_module = None


def _nodes(what):
    """The module that allocates, launches and ties the calls to autograd (csrc/block_nodes.cpp); raises if it is not
    built, or while a tracer records, which would see the outputs' allocation alone."""
    global _module
    if _traced():
        raise RuntimeError(f"{what} cannot be traced: a tracer would record its outputs' allocation alone")
    if _module is None:
        load_block()
        try:
            from . import _nodes as module
        except ImportError as e:
            raise RuntimeError("_nodes.so is not built: run `python -m muon_newton_schulz_05_amd.build`") from e
        _module = module
    return _module


def _refuse_tangents(what, **tensors):
    if getattr(forward_ad, "_current_level", 0) < 0:
        return
    for name, t in tensors.items():
        if t is not None and forward_ad.unpack_dual(t).tangent is not None:
            raise RuntimeError(f"{what} has no forward-mode derivative, and {name} carries a tangent")


# ------------------------------------------------------------------ norms


def _check_norm(x, weight, bias, residual):
    _gpu(x, "x")
    _dtype(x, "x")
    if x.dim() < 1:
        raise ValueError("x must have at least one dimension")
    _same(x, weight=weight, bias=bias, residual=residual)
    cols = x.shape[-1:]
    if weight is not None and weight.shape != cols:
        raise ValueError(f"weight has shape {tuple(weight.shape)}, expected {tuple(cols)}")
    if bias is not None and bias.shape != cols:
        raise ValueError(f"bias has shape {tuple(bias.shape)}, expected {tuple(cols)}")
    if residual is not None and residual.shape != x.shape:
        raise ValueError(f"residual has shape {tuple(residual.shape)}, x {tuple(x.shape)}")


def _eps(eps):
    if not 0.0 <= eps < 1e30:
        raise ValueError(f"eps is {eps}: at least 0, and finite")
    return eps


def _norm_kind(kind):
    if kind not in NORMS:
        raise ValueError(f"norm {kind!r}: one of {', '.join(NORMS)}")
    return NORMS[kind]


def norm_forward(x, weight=None, bias=None, *, eps=1e-5, residual=None, kind="layer"):
    """``layer_norm`` or, with kind "rms", ``rms_norm`` without autograd: (y, s, stats).

    s is x + residual (x itself without one); stats [rows, 2] float32 holds each row's mean and
    1 / sqrt(var + eps) for ``norm_backward``."""
    code = _norm_kind(kind)
    _check_norm(x, weight, bias, residual)
    y, s, stats = _nodes("norm_forward").norm_forward(x, weight, bias, residual, _eps(eps), code)
    return y, x if s is None else s, stats


def norm_backward(dy, x, weight, stats, *, residual=None, kind="layer", ds=None, needs=(True, True, True)):
    """(dx, dweight, dbias) of ``norm_forward`` for the gradients dy and ds; needs: which of them are computed.

    dx is the gradient of x and of the residual alike.  In their place s may be given as x: that keeps one tensor less
    for the gradient, and takes s as it was rounded."""
    code = _norm_kind(kind)
    _check_norm(x, weight, None, residual)
    for name, t in (("dy", dy), ("ds", ds)):
        if t is not None and t.shape != x.shape:
            raise ValueError(f"{name} has shape {tuple(t.shape)}, x {tuple(x.shape)}")
    _same(x, dy=dy, ds=ds)
    rows = math.prod(x.shape[:-1])
    if stats.dtype is not torch.float32 or stats.shape != (rows, 2) or stats.device != x.device \
            or not stats.is_contiguous():
        raise ValueError("stats must be what norm_forward returned")
    return tuple(_nodes("norm_backward").norm_backward(dy, x, residual, weight, stats, ds, code, *needs))


def _norm(x, weight, bias, residual, eps, kind):
    _check_norm(x, weight, bias, residual)
    _refuse_tangents("a norm", x=x, weight=weight, bias=bias, residual=residual)
    out = _nodes("a norm").norm(x, weight, bias, residual, _eps(eps), kind, _tracked(x, weight, bias, residual))
    return out[0] if residual is None else (out[0], out[1])


def layer_norm(x, weight=None, bias=None, *, eps=1e-5, residual=None):
    """(s - mean) / sqrt(var + eps) * weight + bias over the last dimension, s = x + residual.

    x [..., C]; weight and bias [C], ones and zeros where left out; residual like x.  With a residual
    the result is (y, s): the norm, and the sum that the residual stream goes on with.  Differentiable in
    every tensor (once), through both results.

    bfloat16: y and the gradients come from the float32 sum and are rounded once."""
    return _norm(x, weight, bias, residual, eps, 0)


def rms_norm(x, weight=None, *, eps=1e-6, residual=None):
    """s / sqrt(mean(s^2) + eps) * weight over the last dimension, s = x + residual; otherwise as ``layer_norm``."""
    return _norm(x, weight, None, residual, eps, 1)


# ------------------------------------------------------------------ gate


class Gating(NamedTuple):
    """A token's experts, [tokens, top]: weights float32, ids int32 (-1: none, with weight 0)."""
    weights: torch.Tensor
    ids: torch.Tensor


def _check_logits(logits, mask):
    _gpu(logits, "logits")
    _dtype(logits, "logits")
    if logits.dim() != 2 or not 1 <= logits.shape[1] <= GATE_MAX_EXPERTS:
        raise ValueError(f"logits must be [tokens, experts] with 1 to {GATE_MAX_EXPERTS} experts")
    if mask is not None:
        if mask.dtype is not torch.bool or mask.shape != logits.shape[:1]:
            raise ValueError(f"mask must be bool of shape {tuple(logits.shape[:1])}")
        if mask.device != logits.device:
            raise ValueError(f"mask is on {mask.device}, logits on {logits.device}")


def _check_gate(logits, top, mask):
    _check_logits(logits, mask)
    if not 1 <= top <= logits.shape[1]:
        raise ValueError(f"top is {top}: 1 to {logits.shape[1]} of the experts can be chosen")


def gate_forward(logits, top, *, normalize=True, mask=None):
    """``gate`` without autograd."""
    _check_gate(logits, top, mask)
    return Gating(*_nodes("gate_forward").gate(logits, top, int(bool(normalize)), mask, False))


def gate_backward(dweights, logits, gating, *, normalize=True, mask=None):
    """The gradient of ``gate``'s logits for that of its weights; gating and the other arguments are the forward pass's."""
    weights, ids = gating
    _check_logits(logits, mask)
    want = (logits.shape[0], ids.shape[-1])
    if ids.dtype is not torch.int32 or ids.dim() != 2 or ids.shape != want or not ids.is_contiguous() \
            or not 1 <= want[1] <= logits.shape[1] or weights.dtype is not torch.float32 or weights.shape != want \
            or not weights.is_contiguous():
        raise ValueError("gating must be what gate() returned")
    if dweights.dtype is not torch.float32 or dweights.shape != want:
        raise ValueError(f"dweights must be float32 of shape {want}")
    for t, name in ((weights, "weights"), (ids, "ids"), (dweights, "dweights")):
        if t.device != logits.device:
            raise ValueError(f"{name} is on {t.device}, logits on {logits.device}")
    return _nodes("gate_backward").gate_backward(dweights, logits, weights, ids, int(bool(normalize)), mask)


def gate(logits, top, *, normalize=True, mask=None):
    """The `top` experts of each token and their softmax weights, as ``Gating(weights, ids)``.

    logits [tokens, E], E up to 1024; ids in falling order of the logits, ties to the lower index.  The
    weights are the softmax over the chosen experts (they sum to one) or, with
    normalize=False, the chosen experts' part of the softmax over all.  mask: bool [tokens], False for
    a token (padding, say) that is not routed: ids -1, weights 0, no gradient, whatever its logits.  An
    expert whose logit is -inf is never chosen: -1 and 0 stand where too few are left.
    ``route(ids, E)`` and ``combine(..., weights)`` take these as they are.  Differentiable in logits."""
    _check_gate(logits, top, mask)
    _refuse_tangents("gate", logits=logits)
    return Gating(*_nodes("gate").gate(logits, top, int(bool(normalize)), mask, _tracked(logits)))


# ------------------------------------------------------------------ balance loss


class Balance(NamedTuple):
    """loss: float32, no dimensions.  counts [E] int32: the entries routed to each expert."""
    loss: torch.Tensor
    counts: torch.Tensor


def _check_balance(logits, ids, mask):
    _check_logits(logits, mask)
    if ids.dim() != 2 or ids.shape[0] != logits.shape[0] or ids.shape[1] < 1:
        raise ValueError(f"expert_ids has shape {tuple(ids.shape)}, expected ({logits.shape[0]}, top)")
    if max(ids.shape[0], 1) * ids.shape[1] > BALANCE_MAX_ENTRIES:
        raise ValueError(f"expert_ids has shape {tuple(ids.shape)}: up to 2^31 - 1024 entries are supported")
    if ids.dtype not in (torch.int64, torch.int32):
        raise TypeError(f"expert_ids is {ids.dtype}: int64 or int32 is supported")
    if ids.device != logits.device:
        raise ValueError(f"expert_ids is on {ids.device}, logits on {logits.device}")


def balance_forward(logits, expert_ids, *, mask=None):
    """``balance_loss`` without autograd: (loss, counts, shares); shares is for ``balance_backward``."""
    _check_balance(logits, expert_ids, mask)
    return _nodes("balance_forward").balance_forward(logits, expert_ids, mask)


def balance_backward(dloss, logits, expert_ids, shares, *, mask=None):
    """The gradient of ``balance_loss``'s logits for that of the loss (one float32 on the GPU)."""
    _check_balance(logits, expert_ids, mask)
    if dloss.dtype is not torch.float32 or dloss.numel() != 1 or dloss.device != logits.device:
        raise ValueError("dloss must be one float32 value on the logits' device")
    if shares.dtype is not torch.float32 or shares.shape != (logits.shape[1] + 1,) or not shares.is_contiguous() \
            or shares.device != logits.device:
        raise ValueError("shares must be what balance_forward returned")
    return _nodes("balance_backward").balance_backward(dloss, logits, expert_ids.shape[1], shares, mask)


def balance_loss(logits, expert_ids, *, mask: Optional[torch.Tensor] = None):
    """E sum_e f_e P_e as ``Balance(loss, counts)``: one where tokens and probabilities spread evenly over the E experts.

    f_e is the part of all entries of expert_ids [tokens, top] (int64 or int32, as ``gate`` gives them) that
    goes to expert e, P_e the mean over tokens of softmax(logits)_e.  Tokens that mask (bool [tokens]) leaves
    out count nowhere.  An id outside [0, E) (a dropped entry's -1) is not counted, but its place is: f_e is c_e / (T
    top).  Up to 2^31 - 1024 entries.  Differentiable in logits, through P."""
    _check_balance(logits, expert_ids, mask)
    _refuse_tangents("balance_loss", logits=logits)
    return Balance(*_nodes("balance_loss").balance(logits, expert_ids, mask, _tracked(logits)))
