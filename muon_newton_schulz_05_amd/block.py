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
from typing import NamedTuple, Optional

import torch

from .ops import _call, _check, _dtype, _flat, _gpu, _ld, _ptr, _rows, _same, _tracked, load_ops

GATE_MAX_EXPERTS = 1024
NORMS = {"layer": 0, "rms": 1}
EXPORTED_BLOCK = ("muon_norm_workspace", "muon_norm_forward", "muon_norm_backward", "muon_gate_forward",
                  "muon_gate_backward", "muon_balance_workspace", "muon_balance_forward", "muon_balance_backward",
                  "muon_mx_sizes", "muon_mx_quantize", "muon_mx_dequantize", "muon_mx_linear_workspace",
                  "muon_mx_linear")


class NormDesc(ctypes.Structure):
    _fields_ = [("dtype", ctypes.c_int32), ("kind", ctypes.c_int32), ("rows", ctypes.c_int64), ("cols", ctypes.c_int64),
                ("ldx", ctypes.c_int64), ("ldr", ctypes.c_int64), ("ldg", ctypes.c_int64), ("eps", ctypes.c_double)]


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
        "muon_norm_backward": [N] + [P] * 9 + [U64, P],
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


_plans = {}


def _plan(desc_type, size_call, *args):
    """(descriptor, workspace bytes) of a call, by what its descriptor holds."""
    key = (desc_type, size_call, args)
    got = _plans.get(key)
    if got is None:
        lib = load_block()
        d = desc_type(*args)
        need = ctypes.c_uint64(0)
        if size_call:
            _check(getattr(lib, size_call)(ctypes.byref(d), ctypes.byref(need)), size_call)
        if len(_plans) >= 4096:
            _plans.clear()
        got = _plans[key] = (ctypes.byref(d), need.value)
    return got


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


def _whole(t):
    return t if t is None or t.is_contiguous() else t.contiguous()


def _norm_forward(x, weight, bias, residual, eps, kind, keep):
    """y, s, stats and the rows that the gradient reads, of checked arguments."""
    cols = x.shape[-1]
    x2, r2 = _flat(x, cols), _flat(residual, cols)
    w, b = _whole(weight), _whole(bias)
    rows = x2.shape[0]
    d, _ = _plan(NormDesc, None, _dtype(x, "x"), kind, rows, cols, _ld(x2), 0 if r2 is None else _ld(r2), 0, eps)
    y = torch.empty(x.shape, dtype=x.dtype, device=x.device)
    s = None if r2 is None else torch.empty(x.shape, dtype=x.dtype, device=x.device)
    stats = torch.empty((rows, 2), dtype=torch.float32, device=x.device) if keep else None
    _call("muon_norm_forward", x, d, x2.data_ptr(), _ptr(r2), _ptr(w), _ptr(b), y.data_ptr(), _ptr(s), _ptr(stats))
    return y, s, stats, x2 if s is None else s.view(rows, cols), w


def _norm_backward(dy, s, weight, stats, ds, kind, need_x, need_w, need_b):
    rows, cols = s.shape
    dtype, dev = s.dtype, s.device
    g, d2 = _flat(dy, cols), _flat(ds, cols)
    d, size = _plan(NormDesc, "muon_norm_workspace", _dtype(s, "s"), kind, rows, cols, _ld(s),
                    0 if d2 is None else _ld(d2), _ld(g), 0.0)
    dx = torch.empty((rows, cols), dtype=dtype, device=dev) if need_x else None
    dw = torch.empty((cols,), dtype=dtype, device=dev) if need_w else None
    db = torch.empty((cols,), dtype=dtype, device=dev) if need_b else None
    if not (need_w or need_b):
        size = 0
    ws = torch.empty(size, dtype=torch.uint8, device=dev) if size else None
    _call("muon_norm_backward", s, d, g.data_ptr(), s.data_ptr(), _ptr(weight), stats.data_ptr(), _ptr(d2), _ptr(dx),
          _ptr(dw), _ptr(db), _ptr(ws), size)
    return dx, dw, db


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
    y, s, stats, *_ = _norm_forward(x, weight, bias, residual, eps, code, True)
    return y, x if s is None else s, stats


def norm_backward(dy, s, weight, stats, *, kind="layer", ds=None, needs=(True, True, True)):
    """(dx, dweight, dbias) of ``norm_forward`` for the gradients dy and ds; needs: which of them are computed.

    dx is the gradient of x and of the residual alike."""
    code = _norm_kind(kind)
    _check_norm(s, weight, None, dy)
    _same(s, ds=ds)
    if ds is not None and ds.shape != s.shape:
        raise ValueError(f"ds has shape {tuple(ds.shape)}, s {tuple(s.shape)}")
    s2 = _flat(s, s.shape[-1])
    if stats.dtype is not torch.float32 or stats.shape != (s2.shape[0], 2) or stats.device != s.device \
            or not stats.is_contiguous():
        raise ValueError("stats must be what norm_forward returned")
    dx, dw, db = _norm_backward(dy, s2, _whole(weight), stats, ds, code, *needs)
    return None if dx is None else dx.view(s.shape), dw, db


class _Norm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias, residual, eps, kind):
        y, s, stats, rows, w = _norm_forward(x, weight, bias, residual, eps, kind, True)
        ctx.save_for_backward(rows, w, stats)
        ctx.kind, ctx.x_shape = kind, x.shape
        ctx.set_materialize_grads(False)
        return y if s is None else (y, s)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dy, ds=None):
        need_x, need_w, need_b, need_r = ctx.needs_input_grad[:4]
        if dy is None:  # only s was used
            return ds if need_x else None, None, None, ds if need_r else None, None, None
        rows, w, stats = ctx.saved_tensors
        dx, dw, db = _norm_backward(dy, rows, w, stats, ds, ctx.kind, need_x or need_r, need_w, need_b)
        if dx is not None:
            dx = dx.view(ctx.x_shape)
        return dx if need_x else None, dw, db, dx if need_r else None, None, None


def _norm(x, weight, bias, residual, eps, kind):
    _check_norm(x, weight, bias, residual)
    if not _tracked(x, weight, bias, residual):
        y, s, *_ = _norm_forward(x, weight, bias, residual, eps, kind, False)
        return y if s is None else (y, s)
    return _Norm.apply(x, weight, bias, residual, eps, kind)


def layer_norm(x, weight=None, bias=None, *, eps=1e-5, residual=None):
    """(s - mean) / sqrt(var + eps) * weight + bias over the last dimension, s = x + residual.

    x [..., C]; weight and bias [C], ones and zeros where left out; residual like x.  With a residual
    the result is (y, s): the norm, and the sum that the residual stream goes on with.  Differentiable in
    every tensor (once), through both results.

    bfloat16: y comes from the float32 sum and is rounded once.  The gradient takes the normalised value from
    s as returned, so with a residual it is off by half a step of s over the row's standard deviation."""
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


def _gate_plan(logits, top, normalize):
    return _plan(GateDesc, None, _dtype(logits, "logits"), logits.shape[1], top, normalize, logits.shape[0],
                 _ld(logits))[0]


def _gate_forward(logits, top, normalize, mask):
    z, m = _rows(logits), _whole(mask)
    shape = (z.shape[0], top)
    weights = torch.empty(shape, dtype=torch.float32, device=z.device)
    ids = torch.empty(shape, dtype=torch.int32, device=z.device)
    _call("muon_gate_forward", z, _gate_plan(z, top, normalize), z.data_ptr(), _ptr(m), weights.data_ptr(),
          ids.data_ptr())
    return weights, ids, z, m


def _gate_backward(dweights, z, weights, ids, normalize, mask):
    dw = _whole(dweights)
    dz = torch.empty(z.shape, dtype=z.dtype, device=z.device)
    _call("muon_gate_backward", z, _gate_plan(z, ids.shape[1], normalize), z.data_ptr(), _ptr(mask),
          weights.data_ptr(), ids.data_ptr(), dw.data_ptr(), dz.data_ptr())
    return dz


def _check_gate(logits, top, mask):
    _check_logits(logits, mask)
    if not 1 <= top <= logits.shape[1]:
        raise ValueError(f"top is {top}: 1 to {logits.shape[1]} of the experts can be chosen")


def gate_forward(logits, top, *, normalize=True, mask=None):
    """``gate`` without autograd."""
    _check_gate(logits, top, mask)
    return Gating(*_gate_forward(logits, top, int(bool(normalize)), mask)[:2])


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
    return _gate_backward(dweights, _rows(logits), weights, ids, int(bool(normalize)), _whole(mask))


class _Gate(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, top, normalize, mask):
        weights, ids, z, m = _gate_forward(logits, top, normalize, mask)
        ctx.save_for_backward(z, weights, ids, m)
        ctx.normalize = normalize
        ctx.mark_non_differentiable(ids)
        return weights, ids

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dweights, _):
        z, weights, ids, m = ctx.saved_tensors
        return _gate_backward(dweights, z, weights, ids, ctx.normalize, m), None, None, None


def gate(logits, top, *, normalize=True, mask=None):
    """The `top` experts of each token and their softmax weights, as ``Gating(weights, ids)``.

    logits [tokens, E], E up to 1024; ids in falling order of the logits, ties to the lower index.  The
    weights are the softmax over the chosen experts (they sum to one) or, with
    normalize=False, the chosen experts' part of the softmax over all.  mask: bool [tokens], False for
    a token (padding, say) that is not routed: ids -1, weights 0, no gradient, whatever its logits.  An
    expert whose logit is -inf is never chosen: -1 and 0 stand where too few are left.
    ``route(ids, E)`` and ``combine(..., weights)`` take these as they are.  Differentiable in logits."""
    _check_gate(logits, top, mask)
    code = int(bool(normalize))
    if not _tracked(logits):
        return Gating(*_gate_forward(logits, top, code, mask)[:2])
    return Gating(*_Gate.apply(logits, top, code, mask))


# ------------------------------------------------------------------ balance loss


class Balance(NamedTuple):
    """loss: float32, no dimensions.  counts [E] int32: the entries routed to each expert."""
    loss: torch.Tensor
    counts: torch.Tensor


def _check_balance(logits, ids, mask):
    _check_logits(logits, mask)
    if ids.dim() != 2 or ids.shape[0] != logits.shape[0] or ids.shape[1] < 1:
        raise ValueError(f"expert_ids has shape {tuple(ids.shape)}, expected ({logits.shape[0]}, top)")
    if ids.dtype not in (torch.int64, torch.int32):
        raise TypeError(f"expert_ids is {ids.dtype}: int64 or int32 is supported")
    if ids.device != logits.device:
        raise ValueError(f"expert_ids is on {ids.device}, logits on {logits.device}")


def _balance_plan(z, top):
    return _plan(GateDesc, "muon_balance_workspace", _dtype(z, "logits"), z.shape[1], top, 0, z.shape[0], _ld(z))


def _balance_forward(logits, ids, mask):
    z, i, m = _rows(logits), _whole(ids), _whole(mask)
    e, dev = z.shape[1], z.device
    d, size = _balance_plan(z, i.shape[1])
    loss = torch.empty((), dtype=torch.float32, device=dev)
    counts = torch.empty((e,), dtype=torch.int32, device=dev)
    shares = torch.empty((e + 1,), dtype=torch.float32, device=dev)
    ws = torch.empty(size, dtype=torch.uint8, device=dev) if size else None
    _call("muon_balance_forward", z, d, z.data_ptr(), i.data_ptr(), i.element_size(), _ptr(m), loss.data_ptr(),
          counts.data_ptr(), shares.data_ptr(), _ptr(ws), size)
    return loss, counts, shares, z, m


def _balance_backward(dloss, z, top, shares, mask):
    dz = torch.empty(z.shape, dtype=z.dtype, device=z.device)
    _call("muon_balance_backward", z, _balance_plan(z, top)[0], z.data_ptr(), _ptr(mask), shares.data_ptr(),
          dloss.data_ptr(), dz.data_ptr())
    return dz


def balance_forward(logits, expert_ids, *, mask=None):
    """``balance_loss`` without autograd: (loss, counts, shares); shares is for ``balance_backward``."""
    _check_balance(logits, expert_ids, mask)
    return _balance_forward(logits, expert_ids, mask)[:3]


def balance_backward(dloss, logits, expert_ids, shares, *, mask=None):
    """The gradient of ``balance_loss``'s logits for that of the loss (one float32 on the GPU)."""
    _check_balance(logits, expert_ids, mask)
    if dloss.dtype is not torch.float32 or dloss.numel() != 1 or dloss.device != logits.device:
        raise ValueError("dloss must be one float32 value on the logits' device")
    if shares.dtype is not torch.float32 or shares.shape != (logits.shape[1] + 1,) or not shares.is_contiguous() \
            or shares.device != logits.device:
        raise ValueError("shares must be what balance_forward returned")
    return _balance_backward(dloss, _rows(logits), expert_ids.shape[1], shares, _whole(mask))


class _BalanceLoss(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, ids, mask):
        loss, counts, shares, z, m = _balance_forward(logits, ids, mask)
        ctx.save_for_backward(z, shares, m)
        ctx.top = ids.shape[1]
        ctx.mark_non_differentiable(counts)
        return loss, counts

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dloss, _):
        z, shares, m = ctx.saved_tensors
        return _balance_backward(dloss, z, ctx.top, shares, m), None, None


def balance_loss(logits, expert_ids, *, mask: Optional[torch.Tensor] = None):
    """E sum_e f_e P_e as ``Balance(loss, counts)``: one where tokens and probabilities spread evenly over the E experts.

    f_e is the part of all entries of expert_ids [tokens, top] (int64 or int32, as ``gate`` gives them) that
    goes to expert e, P_e the mean over tokens of softmax(logits)_e.  Tokens that mask (bool [tokens]) leaves
    out count nowhere.  An id outside [0, E) (a dropped entry's -1) is not counted, but its place is: f_e is c_e / (T
    top).  Differentiable in logits, through P."""
    _check_balance(logits, expert_ids, mask)
    if not _tracked(logits):
        return Balance(*_balance_forward(logits, expert_ids, mask)[:2])
    return Balance(*_BalanceLoss.apply(logits, expert_ids, mask))
