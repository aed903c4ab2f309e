"""Linear and expert layers whose weights are held in four bits, on torch tensors.

Values are e2m1 (0, 0.5, 1, 1.5, 2, 3, 4, 6 and their negatives) in blocks of 32 along the
contraction that share a power of two (the Open Compute Project's microscaling formats): 4.25
bits a value.  ``mx_linear`` and ``mx_expert_linear`` take x to the same form
and multiply on the matrix instructions made for it.  They are for evaluation and serving and have no gradient.
"""

from __future__ import annotations

from typing import NamedTuple

import torch
from torch.autograd import forward_ad

from .block import MxDesc, _plan, _whole
from .ops import _activation, _call, _check_linear, _dtype, _flat, _gpu, _layout_ok, _ld, _ptr

MX_MAX_SIZE = 1 << 23


class MxWeight(NamedTuple):
    """A weight [K, N] or [E, K, N] in four bits.

    values [..., ceil(K / 128), N, 64] uint8: each column's values by slices of 128 along K, two a byte, the lower half
    first; scales [..., ceil(K / 512), N, 16] uint8: byte 4 g + s is the power of two (+ 127) of the 32 values g of
    slice s of 512; k is K."""
    values: torch.Tensor
    scales: torch.Tensor
    k: int

    @property
    def shape(self):
        return torch.Size((*self.values.shape[:-3], self.k, self.values.shape[-2]))


def _check_weight(q):
    v, s, k = q
    if v.dim() not in (3, 4) or v.dtype is not torch.uint8 or s.dtype is not torch.uint8 or not 0 <= k <= MX_MAX_SIZE \
            or v.shape[-3] != (k + 127) // 128 or v.shape[-1] != 64 \
            or s.shape != (*v.shape[:-3], (k + 511) // 512, v.shape[-2], 16) \
            or not v.is_contiguous() or not s.is_contiguous():
        raise ValueError("the weight must be what mx_quantize() returned")
    _gpu(v, "the weight")
    if v.device != s.device:
        raise ValueError(f"the weight's values are on {v.device}, its scales on {s.device}")
    if v.data_ptr() % 16 or s.data_ptr() % 16:
        raise ValueError("the weight's values and scales must be 16-byte aligned")


def mx_quantize(weight):
    """weight [K, N] or [E, K, N] (its last two dimensions in either order in memory) in four bits along K, as ``MxWeight``.

    A block's scale is 2^(floor(log2 of its largest magnitude) - 2), at least 2^-127; values are rounded
    to nearest, ties to even, and saturate at 6 scales.  A block with an infinity or NaN becomes NaN.  Takes the weight's
    value: a parameter that requires a gradient may be given."""
    _gpu(weight, "weight")
    code = _dtype(weight, "weight")
    if weight.dim() not in (2, 3):
        raise ValueError(f"weight has {weight.dim()} dimensions, expected 2 or 3")
    k, n = weight.shape[-2:]
    if max(k, n) > MX_MAX_SIZE:
        raise ValueError(f"weight is {k} x {n}: sizes up to 2^23 are supported")
    groups = weight.shape[0] if weight.dim() == 3 else 0
    if weight.dim() == 3 and not 1 <= groups <= 65535:
        raise ValueError(f"{groups} experts: 1 to 65535 are supported")
    w = weight.detach()
    w = w if _layout_ok(w) else w.contiguous()
    if w.stride(-1) == 1 and (k <= 1 or w.stride(-2) >= n):
        layout, ld = 0, w.stride(-2) if k > 1 else max(n, 1)
    else:
        layout, ld = 1, w.stride(-1) if n > 1 else max(k, 1)
    d = _plan(MxDesc, None, code, 0, groups, layout, 0, k, n, 0, ld, w.stride(0) if groups else 0, 0)[0]
    lead = weight.shape[:-2]
    values = torch.empty((*lead, (k + 127) // 128, n, 64), dtype=torch.uint8, device=w.device)
    scales = torch.empty((*lead, (k + 511) // 512, n, 16), dtype=torch.uint8, device=w.device)
    _call("muon_mx_quantize", w, d, w.data_ptr(), values.data_ptr(), scales.data_ptr())
    return MxWeight(values, scales, k)


def mx_dequantize(weight, dtype=torch.float32):
    """The values that an ``MxWeight`` stands for, exactly: [K, N] or [E, K, N], contiguous along K."""
    _check_weight(weight)
    values, scales, k = weight
    n, lead = values.shape[-2], values.shape[:-3]
    out = torch.empty((*lead, n, k), dtype=dtype, device=values.device)
    d = _plan(MxDesc, None, _dtype(out, "dtype"), 0, lead[0] if lead else 0, 0, 0, k, n, 0, n, 0, 0)[0]
    _call("muon_mx_dequantize", values, d, values.data_ptr(), scales.data_ptr(), out.data_ptr())
    return out.transpose(-1, -2)


class _Shape:
    """What ``_check_linear`` asks of a weight, in the type of x."""

    def __init__(self, weight, x):
        self.shape, self.dtype, self.device = weight.shape, x.dtype, weight.values.device

    def dim(self):
        return len(self.shape)


def _linear(x, weight, bias, residual, offsets, activation):
    act = _activation(activation)
    _check_weight(weight)
    _check_linear(x, _Shape(weight, x), bias, residual, offsets)
    for name, t in (("x", x), ("bias", bias), ("residual", residual)):
        if t is None:
            continue
        if torch.is_grad_enabled() and t.requires_grad:
            raise RuntimeError(f"layers in four bits have no gradient, and {name} requires one: call them under "
                               "torch.no_grad()")
        if getattr(forward_ad, "_current_level", 0) >= 0 and forward_ad.unpack_dual(t).tangent is not None:
            raise RuntimeError(f"layers in four bits have no forward-mode derivative, and {name} carries a tangent")
    values, scales, k = weight
    n = values.shape[-2]
    x2, r2, b = _flat(x, k), _flat(residual, n), _whole(bias)
    rows = x2.shape[0]
    d, size = _plan(MxDesc, "muon_mx_linear_workspace", _dtype(x, "x"), act, 0 if offsets is None else values.shape[0], 0,
                    rows, k, n, _ld(x2), 0, 0, 0 if r2 is None else _ld(r2))
    y = torch.empty((*x.shape[:-1], n), dtype=x.dtype, device=x.device)
    ws = torch.empty(size, dtype=torch.uint8, device=x.device) if size else None
    _call("muon_mx_linear", x, d, _ptr(offsets), x2.data_ptr(), values.data_ptr(), scales.data_ptr(), _ptr(b), _ptr(r2),
          y.data_ptr(), _ptr(ws), size)
    return y


def mx_linear(x, weight, bias=None, *, activation="none", residual=None):
    """act(Q(x) W + b) + residual for an ``MxWeight`` of [K, N]; Q takes each row of x to four bits along K.

    x [..., K], bias [N] and residual [..., N] float32 or bfloat16, as y.  Sums are float32, and y is rounded once.
    A block of x that holds an infinity or NaN makes its row NaN.  No gradient: raises where one is asked for."""
    return _linear(x, weight, bias, residual, None, activation)


def mx_expert_linear(x, weight, offsets, bias=None, *, activation="none"):
    """``mx_linear`` of the rows offsets[e] .. offsets[e + 1] with weight e of an ``MxWeight`` of [E, K, N].

    offsets as ``route`` gives them; rows past offsets[E] give zero."""
    if offsets is None:
        raise ValueError("offsets is missing")
    return _linear(x, weight, bias, None, offsets, activation)
