"""Linear and expert layers whose weights are held in four bits, on torch tensors.

Values are e2m1 (0, 0.5, 1, 1.5, 2, 3, 4, 6 and their negatives) in blocks of 32 along the
contraction that share a power of two (the Open Compute Project's microscaling formats): 4.25
bits a value.  ``mx_linear`` and ``mx_expert_linear`` take x to the same form
and multiply on the matrix instructions made for it.  They are for evaluation and serving and have no gradient.
"""

from __future__ import annotations

from typing import NamedTuple

import torch

from .block import _nodes, _refuse_tangents
from .ops import _activation, _check_linear, _dtype, _gpu

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
    value: a parameter that requires a gradient may be given.  K and N up to 2^23, fewer than 2^35 values in all."""
    _gpu(weight, "weight")
    _dtype(weight, "weight")
    if weight.dim() not in (2, 3):
        raise ValueError(f"weight has {weight.dim()} dimensions, expected 2 or 3")
    k, n = weight.shape[-2:]
    if max(k, n) > MX_MAX_SIZE:
        raise ValueError(f"weight is {k} x {n}: sizes up to 2^23 are supported")
    groups = weight.shape[0] if weight.dim() == 3 else 0
    if weight.dim() == 3 and not 1 <= groups <= 65535:
        raise ValueError(f"{groups} experts: 1 to 65535 are supported")
    return MxWeight(*_nodes("mx_quantize").mx_quantize(weight), k)


def mx_dequantize(weight, dtype=torch.float32):
    """The values that an ``MxWeight`` stands for, exactly: [K, N] or [E, K, N], contiguous along K."""
    _check_weight(weight)
    if dtype not in (torch.float32, torch.bfloat16):
        raise TypeError(f"dtype is {dtype}: float32 or bfloat16 is supported")
    return _nodes("mx_dequantize").mx_dequantize(*weight, dtype is torch.bfloat16)


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
    if torch.is_grad_enabled():
        for name, t in (("x", x), ("bias", bias), ("residual", residual)):
            if t is not None and t.requires_grad:
                raise RuntimeError(f"layers in four bits have no gradient, and {name} requires one: call them under "
                                   "torch.no_grad()")
    _refuse_tangents("a layer in four bits", x=x, bias=bias, residual=residual)
    return _nodes("mx_linear").mx_linear(x, *weight, bias, residual, offsets, act)


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
