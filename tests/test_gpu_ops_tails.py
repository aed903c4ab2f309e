"""GPU tests of the activations where they fall towards zero: relative accuracy against float64 forms that cancel
nothing."""

from __future__ import annotations

import math

import pytest
import torch

import ops_reference as ref

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def muon():
    import muon_newton_schulz_05_amd as pkg
    return pkg


def tail64(z, act):
    """act(z) and its slope at z < 0 in forms that cancel nothing."""
    if act == "silu":
        e = torch.exp(z)
        q = e / (1 + e)
        return z * q, q + z * q / (1 + e)
    if act == "gelu":
        cdf = torch.special.log_ndtr(z).exp()
        return z * cdf, cdf + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    c = math.sqrt(2 / math.pi)
    e = torch.exp(2 * c * (z + 0.044715 * z ** 3))
    q = e / (1 + e)
    return z * q, q + z * q / (1 + e) * 2 * c * (1 + 3 * 0.044715 * z * z)


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
def test_activations_keep_their_tails(muon, act, dtype):
    """z from -12 to 0, where act(z) falls to 1e-32: right to a relative tolerance, and so are the slopes."""
    z = -torch.logspace(-4, math.log2(12), 2000, base=2.0).to(dtype)
    if act == "gelu_tanh":
        z = z[z > -9]                                        # beyond, both factors are past float32's range
    x = z[:, None].cuda().requires_grad_()
    y = muon.linear(x, torch.ones(1, 8, device="cuda", dtype=dtype), activation=act)
    (dx,) = torch.autograd.grad(y, x, torch.full_like(y, 0.125))
    want, slope = tail64(z.double(), act)
    # The exponent (-z, z^2 / 2, or 2 u of gelu_tanh) is rounded three times at most, relative to itself; a polynomial
    # of eight steps, a reciprocal, the exponential and the products make ten more roundings; then the store.
    expo = {"silu": -z, "gelu": z * z / 2, "gelu_tanh": 1.6 * (-z - 0.044715 * z ** 3)}[act].double()
    rel = (3 * expo + 10) * ref.U32
    u = ref.unit(dtype)
    ref.check("y", y[:, 0], (want, (rel + u) * want.abs() + 1e-37))
    # The slope is a difference of two such terms; dz is stored once more, and dx sums eight equal values.
    cdf = want / z.double()
    terms = cdf.abs() + (slope - cdf).abs()
    ref.check("dx", dx[:, 0], (slope, 2 * (rel + 4 * ref.U32) * terms + (2 * u + 8 * ref.U32) * slope.abs() + 1e-37))


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
def test_slopes_keep_what_they_add_to_one(muon, act, dtype):
    """z from 0 to 12: act'(z) = 1 - act'(-z), whose small part is made of factors that grow with z^3 and must not be
    multiplied by the error of a difference from one."""
    z = torch.logspace(-4, math.log2(12), 2000, base=2.0).to(dtype)
    if act == "gelu_tanh":
        z = z[z < 9]
    dy = torch.full((z.numel(), 8), 0.125, dtype=dtype, device="cuda")
    x = z[:, None].cuda()
    w = torch.ones(1, 8, device="cuda", dtype=dtype)
    dx, _, _ = muon.linear_backward(dy, x, w, x.expand(-1, 8).contiguous(), act)
    value, slope = tail64(-z.double(), act)
    expo = {"silu": z, "gelu": z * z / 2, "gelu_tanh": 1.6 * (z + 0.044715 * z ** 3)}[act].double()
    cdf = value / -z.double()
    small = cdf.abs() + (slope - cdf).abs()
    want = 1 - slope
    # The small part relative to itself, as for negative z; one more rounding or two of what is near one.
    err = 2 * ((3 * expo + 10) * ref.U32 + 4 * ref.U32) * small + 4 * ref.U32
    u = ref.unit(dtype)
    ref.check("dx", dx[:, 0], (want, err + (2 * u + 8 * ref.U32) * want.abs()))
