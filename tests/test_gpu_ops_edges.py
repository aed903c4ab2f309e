"""GPU tests of the layer operators' edges: non-finite operands, the tails of the activations, paths that only
unusual shapes reach, several streams and threads, against the plain float64 forms of tests/ops_reference.py."""

from __future__ import annotations

import itertools

import pytest
import torch

import ops_reference as ref

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
ACTS = ["none", "relu", "silu", "gelu", "gelu_tanh"]


@pytest.fixture(scope="module")
def muon():
    import muon_newton_schulz_05_amd as pkg
    return pkg


def normal(shape, dtype, seed, std=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * std).to(dtype)


def same_non_finite(got, want):
    """Infinities and NaN in the same places, of the same sign."""
    got, want = got.double().cpu(), want.to(got.dtype).double()
    assert torch.equal(got.isnan(), want.isnan())
    bad = want.isinf()
    assert torch.equal(got.isinf(), bad) and torch.equal(got[bad], want[bad])


# ------------------------------------------------------------------ infinite operands of a gradient


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("rows", [1, 5, 64, 65, 200])
def test_linear_gradients_of_infinite_operands(muon, rows, act):
    """x and W that hold infinities and NaN give the dx and dW that the formula gives, for any number of rows."""
    k, n = 24, 40
    x, w, dy = normal((rows, k), BF16, 1), normal((k, n), BF16, 2), normal((rows, n), BF16, 3)
    z = normal((rows, n), BF16, 4).abs() + 0.25             # a slope that is not zero
    dz = dy.double() * ref.act64(z.double(), act)[1]
    x[0, 3], x[0, 7], x[rows - 1, 20] = float("inf"), float("nan"), -float("inf")
    w[2, 1], w[9, 30], w[9, 31], w[20, 5] = float("inf"), -float("inf"), float("inf"), float("nan")
    dx, dw, _ = muon.linear_backward(dy.cuda(), x.cuda(), w.cuda(), z.cuda(), act)
    same_non_finite(dx, dz @ w.double().t())
    same_non_finite(dw, x.double().t() @ dz)


@pytest.mark.parametrize("act", ["relu", "silu"])
@pytest.mark.parametrize("counts", [[3, 0, 5, 1], [30, 2, 30, 2]], ids=["few", "all"])
def test_experts_gradients_of_infinite_operands(muon, counts, act):
    e, k, n, rows = len(counts), 24, 40, sum(counts)
    offsets = torch.tensor([0, *itertools.accumulate(counts)], dtype=torch.int32)
    x, w, dy = normal((rows, k), BF16, 1), normal((e, k, n), BF16, 2), normal((rows, n), BF16, 3)
    z = normal((rows, n), BF16, 4).abs() + 0.25
    x[0, 3], x[rows - 1, 20], w[2, 2, 1], w[0, 9, 30] = float("inf"), -float("inf"), float("inf"), -float("inf")
    dx, dw, _ = muon.linear_backward(dy.cuda(), x.cuda(), w.cuda(), z.cuda(), act, offsets=offsets.cuda())
    dz = dy.double() * ref.act64(z.double(), act)[1]
    for i in range(e):
        lo, hi = offsets[i], offsets[i + 1]
        same_non_finite(dx[lo:hi], dz[lo:hi] @ w[i].double().t())
        same_non_finite(dw[i], x[lo:hi].double().t() @ dz[lo:hi])


# ------------------------------------------------------------------ offsets that do not ascend


def test_experts_with_overlapping_offsets_stay_inside(muon):
    """Half of 65535 experts claim every row, more blocks than 32 bits count: values are unspecified, what follows
    is not touched."""
    e, rows, k, n = 65535, (1 << 22) + 64, 8, 8
    x, w, b = (normal(s, BF16, i).cuda() for i, s in enumerate(((rows, k), (e, k, n), (e, n))))
    bad = torch.zeros(e + 1, dtype=torch.int32)
    bad[1::2] = rows
    y, z = muon.linear_forward(x, w, b, "silu", offsets=bad.cuda(), keep_z=True)
    dx, _, db = muon.linear_backward(y, x, w, z, "silu", offsets=bad.cuda(), needs=(True, False, True))
    assert y.shape == (rows, n) and dx.shape == x.shape and db.shape == (e, n)
    torch.cuda.synchronize()
    good = torch.full((e + 1,), 64, dtype=torch.int32)
    good[0] = 0
    y = muon.linear_forward(x[:64], w, b, "silu", offsets=good.cuda())[0].cpu()
    ref.check("y", y, ref.linear64(x[:64].cpu(), w[0].cpu(), b[0].cpu(), None, None, "silu")["y"])


# ------------------------------------------------------------------ the accuracy of an expert's gradient


def experts_backward(muon, counts, k, n, act):
    e, rows = len(counts), sum(counts)
    offsets = torch.tensor([0, *itertools.accumulate(counts)], dtype=torch.int32)
    x, w, dy = normal((rows, k), BF16, 1), normal((e, k, n), BF16, 2, k ** -0.5), normal((rows, n), BF16, 3)
    z = muon.linear_forward(x.cuda(), w.cuda(), activation=act, offsets=offsets.cuda(), keep_z=True)[1]
    dx, dw, _ = muon.linear_backward(dy.cuda(), x.cuda(), w.cuda(), z, act, offsets=offsets.cuda())
    dz = dy.double() * ref.act64(z.cpu().double(), act)[1]
    for i in range(e):
        lo, hi = offsets[i], offsets[i + 1]
        yield counts[i], ((dx[lo:hi], dz[lo:hi], w[i].double().t()), (dw[i], x[lo:hi].double().t(), dz[lo:hi]))


@pytest.mark.parametrize("counts", [[3] * 64, [1, 40, 0, 7, 30, 2, 16, 32], [200] + [0, 1, 4] * 9], ids=["even", "uneven", "one"])
@pytest.mark.parametrize("k,n", [(64, 72), (200, 1000), (37, 21)])
def test_experts_of_few_rows_keep_what_dz_loses(muon, counts, k, n):
    """Up to 16 rows an expert dx and dW are one rounding off, whatever the number of experts."""
    u, terms = ref.unit(BF16), 2 * max(n, max(counts)) + 4
    for _, parts in experts_backward(muon, counts, k, n, "silu"):
        for got, a, b in parts:
            want, size = a @ b, a.abs() @ b.abs()
            err = (terms + 32) * ref.U32 * size + u * u * size   # float32 sums and slopes; dz after two roundings
            ref.check("", got, (want, err + u * (want.abs() + err) + 1e-37))


def test_an_expert_of_few_rows_among_many_is_two_roundings_off(muon):
    """With more rows an expert on average, dz is rounded once for all: dx and dW stay within two roundings' norm."""
    for rows, parts in experts_backward(muon, [400, 3, 1, 300, 2], 200, 264, "silu"):
        for got, a, b in parts:
            want = a @ b
            # The first rounding moves each product by u of itself at most, in a norm of u |a| |b|; on average
            # over many products it is u / sqrt 3 of the result, as is the second.
            assert (got.double().cpu() - want).norm() <= 2 * ref.unit(BF16) * want.norm(), rows


# ------------------------------------------------------------------ paths that only some shapes reach


@pytest.mark.parametrize("w_t", [False, True], ids=["kn", "nk"])
def test_linear_large_tiles_split_in_two(muon, w_t):
    """70 ragged 256-wide tiles over 12296 of contraction, forward and dW."""
    m, k, n = 1100, 12296, 3400
    x, w = normal((m, k), BF16, 1), normal((n, k) if w_t else (k, n), BF16, 2, k ** -0.5)
    gw = w.cuda().t() if w_t else w.cuda()
    y = muon.linear(x.cuda(), gw, activation="silu")
    rows = torch.tensor([0, 255, 256, 1023, 1024, 1099])
    want = ref.linear64(x[rows], w.t() if w_t else w, None, None, None, "silu")
    ref.check("y", y[rows.cuda()], want["y"], 2 * ref.unit(BF16))
    a, dy = normal((k, m), BF16, 3), normal((k, n), BF16, 4)
    v = normal((n, m) if w_t else (m, n), BF16, 5).cuda()
    _, dw, _ = muon.linear_backward(dy.cuda(), a.cuda(), v.t() if w_t else v, needs=(False, True, False))
    want, size = a[:, rows].double().t() @ dy.double(), a[:, rows].double().abs().t() @ dy.double().abs()
    err = (k + 2) * ref.U32 * size
    ref.check("dw", dw[rows.cuda()], (want, err + ref.unit(BF16) * (want.abs() + err)), 2 * ref.unit(BF16))
