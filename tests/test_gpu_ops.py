"""GPU tests of the layer operators against plain float64 forms (tests/ops_reference.py)."""

from __future__ import annotations

import itertools

import pytest
import torch

import ops_reference as ref

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def muon():
    import muon_newton_schulz_05_amd as pkg
    return pkg


def normal(shape, dtype, seed, std=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * std).to(dtype)


# Norm bounds.  A value rounded to its type is off by at most u of itself, u / sqrt(3) on average of a uniform error.
# Gradients add the roundings of z and dz, of the same size and independent: three of them stay below 2 u.
def norm_bound(dtype, k):
    return 2 * ref.unit(dtype) if dtype is BF16 else (k + 16) * ref.U32


# ------------------------------------------------------------------ linear

SHAPES = [(1, 1, 1), (1, 8, 8), (3, 7, 5), (31, 64, 32), (33, 65, 129), (64, 24, 640), (128, 256, 128), (257, 129, 260),
          (300, 520, 264), (1, 4096, 520), (5, 2048, 96), (2, 4100, 33)]


def run_linear(muon, m, k, n, dtype, act, w_t, bias, residual, seed=0):
    x, w = normal((m, k), dtype, seed), normal((n, k) if w_t else (k, n), dtype, seed + 1, k ** -0.5)
    w = w.t() if w_t else w
    b = normal((n,), dtype, seed + 2) if bias else None
    r = normal((m, n), dtype, seed + 3) if residual else None
    dy = normal((m, n), dtype, seed + 4)
    want = ref.linear64(x, w, b, r, dy, act)
    gx = x.cuda().requires_grad_()
    gw = (w.t().contiguous().cuda().t() if w_t else w.cuda()).requires_grad_()
    gb = None if b is None else b.cuda().requires_grad_()
    gr = None if r is None else r.cuda().requires_grad_()
    y = muon.linear(gx, gw, gb, activation=act, residual=gr)
    leaves = {"dx": gx, "dw": gw, "db": gb, "dr": gr}
    leaves = {a: v for a, v in leaves.items() if v is not None}
    got = dict(zip(leaves, torch.autograd.grad(y, tuple(leaves.values()), dy.cuda())))
    ref.check("y", y, want["y"], norm_bound(dtype, k))
    ref.check("dx", got["dx"], want["dx"], norm_bound(dtype, n))
    ref.check("dw", got["dw"], want["dw"], norm_bound(dtype, m))
    if bias:
        ref.check("db", got["db"], want["db"])
    if residual:
        assert torch.equal(got["dr"].cpu(), dy)
    with torch.no_grad():
        assert torch.equal(muon.linear(gx, gw, gb, activation=act, residual=gr), y)


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("m,k,n", SHAPES)
def test_linear_shapes(muon, m, k, n, dtype):
    run_linear(muon, m, k, n, dtype, "none", False, True, False, seed=m + n)
    run_linear(muon, m, k, n, dtype, "gelu", True, False, True, seed=m + n + 10)


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("act", ["none", "relu", "silu", "gelu", "gelu_tanh"])
@pytest.mark.parametrize("w_t", [False, True], ids=["kn", "nk"])
def test_linear_activations(muon, act, w_t, dtype):
    run_linear(muon, 136, 192, 328, dtype, act, w_t, True, True)


@pytest.mark.parametrize("w_t", [False, True], ids=["kn", "nk"])
@pytest.mark.parametrize("m,k,n", [(4096, 72, 4096), (4100, 200, 4104), (300, 4096, 4096), (2040, 256, 4096)])
def test_linear_large_tiles(muon, m, k, n, w_t):
    """Shapes whose products fill the card with 256-wide tiles, whole and ragged ones."""
    run_linear(muon, m, k, n, BF16, "silu", w_t, True, True)


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
def test_linear_strided_rows_and_leading_dims(muon, dtype):
    big = normal((6, 10, 80), dtype, 1)
    x = big[:, ::2, 8:72]                                   # [6, 5, 64], not flattenable
    w = normal((96, 100), dtype, 2, 0.1)[8:72, 4:52]        # [64, 48], row stride 100
    r = normal((6, 5, 64), dtype, 3)[..., 8:56]
    dy = normal((6, 5, 48), dtype, 4)
    want = ref.linear64(x.reshape(30, 64), w, None, r.reshape(30, 48), dy.reshape(30, 48), "silu")
    gx = big.cuda()[:, ::2, 8:72].requires_grad_()
    gw = normal((96, 100), dtype, 2, 0.1).cuda()[8:72, 4:52].requires_grad_()
    y = muon.linear(gx, gw, activation="silu", residual=normal((6, 5, 64), dtype, 3).cuda()[..., 8:56])
    assert y.shape == (6, 5, 48)
    dx, dw = torch.autograd.grad(y, (gx, gw), dy.cuda())
    assert dx.shape == gx.shape and dw.shape == gw.shape
    ref.check("y", y.reshape(30, 48), want["y"])
    ref.check("dx", dx.reshape(30, 64), want["dx"])
    ref.check("dw", dw, want["dw"])


def test_linear_broadcast_gradients_and_bias(muon):
    """A gradient with strides of zero (that of a sum), and a weight that is a broadcast view."""
    x, w = normal((40, 64), F32, 1), normal((64, 24), F32, 2)
    gx, gw = x.cuda().requires_grad_(), w.cuda().requires_grad_()
    muon.linear(gx, gw).sum().backward()
    want = ref.linear64(x, w, None, None, torch.ones(40, 24), "none")
    ref.check("dx", gx.grad, want["dx"])
    ref.check("dw", gw.grad, want["dw"])
    row = normal((1, 24), F32, 3)
    gr = row.cuda().requires_grad_()
    y = muon.linear(x.cuda(), gr.expand(64, 24))
    ref.check("y", y, ref.linear64(x, row.expand(64, 24), None, None, None, "none")["y"])
    (d,) = torch.autograd.grad(y, gr, torch.ones_like(y))
    assert d.shape == (1, 24)


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
def test_linear_empty(muon, dtype):
    w = normal((16, 8), dtype, 1).cuda().requires_grad_()
    b = normal((8,), dtype, 2).cuda().requires_grad_()
    x = torch.empty((0, 16), dtype=dtype, device="cuda", requires_grad=True)
    y = muon.linear(x, w, b, activation="gelu")
    assert y.shape == (0, 8)
    dx, dw, db = torch.autograd.grad(y, (x, w, b), torch.empty_like(y))
    assert dx.shape == (0, 16) and not dw.any() and not db.any()
    # A contraction of length zero: the bias alone.
    y = muon.linear(torch.empty((3, 0), dtype=dtype, device="cuda"), torch.empty((0, 8), dtype=dtype, device="cuda"), b)
    assert torch.equal(y, b.detach().expand(3, 8))


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
def test_linear_keeps_infinities_in_their_rows(muon, dtype):
    x = normal((70, 72), dtype, 1)
    x[3, 5], x[69, 71] = float("inf"), float("nan")
    w = normal((72, 40), dtype, 2)
    y = muon.linear(x.cuda(), w.cuda()).cpu()
    rows = torch.ones(70, dtype=torch.bool)
    rows[[3, 69]] = False
    assert torch.isfinite(y[rows].float()).all() and not torch.isfinite(y[~rows].float()).any()


def test_linear_gradient_matches_differences(muon):
    """float32 against central differences of the kernel's own forward pass."""
    x, w, b = normal((9, 20), F32, 1), normal((20, 12), F32, 2, 0.3), normal((12,), F32, 3)
    dy = normal((9, 12), F32, 4)
    for act in ("silu", "gelu", "gelu_tanh"):
        g = [t.cuda().requires_grad_() for t in (x, w, b)]
        grads = torch.autograd.grad(muon.linear(*g, activation=act), g, dy.cuda())
        for t, grad in zip(g, grads):
            d = normal(t.shape, F32, 7).cuda()
            h = 2.0 ** -7
            f = lambda s: (muon.linear(*[(v + s * d if v is t else v).detach() for v in g], activation=act)  # noqa: E731
                           .double() * dy.cuda().double()).sum()
            slope = float(f(h) - f(-h)) / (2 * h)
            # h^2 / 6 of a third derivative of order |d|^3 |dy| and float32 noise over 2 h.
            assert abs(slope - float((grad.double() * d.double()).sum())) < 2e-2 * (1 + abs(slope))


def test_linear_is_deterministic_and_split_joins(muon):
    x, w = normal((2, 16384), BF16, 1).cuda(), normal((16384, 64), BF16, 2, 0.01).cuda()
    y = muon.linear(x, w)
    for _ in range(3):
        assert torch.equal(muon.linear(x, w), y)


def test_linear_on_a_side_stream(muon):
    x, w = normal((256, 256), BF16, 1).cuda(), normal((256, 256), BF16, 2, 0.1).cuda()
    want = muon.linear(x, w, activation="relu")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        y = muon.linear(x, w, activation="relu")
    s.synchronize()
    assert torch.equal(y, want)


def test_linear_refusals(muon):
    x, w = torch.zeros(4, 8, device="cuda"), torch.zeros(8, 6, device="cuda")
    for call in [lambda: muon.linear(x, w.t()), lambda: muon.linear(x, w[None]), lambda: muon.linear(x, w, w[0, :5]),
                 lambda: muon.linear(x, w, residual=x), lambda: muon.linear(x, w.cpu()),
                 lambda: muon.linear(x, w, activation="tanh"),
                 lambda: muon.expert_linear(x, w[None], torch.zeros(3, dtype=torch.int32, device="cuda")),
                 lambda: muon.expert_linear(x, w[None], torch.zeros(2, dtype=torch.int64, device="cuda")),
                 lambda: muon.expert_linear(x, w[None], torch.zeros(2, dtype=torch.int32))]:
        with pytest.raises(ValueError):
            call()
    for call in [lambda: muon.linear(x, w.bfloat16()), lambda: muon.linear(x.half(), w.half()),
                 lambda: muon.linear(x.double(), w.double())]:
        with pytest.raises(TypeError):
            call()


@pytest.mark.parametrize("w_t", [False, True], ids=["kn", "nk"])
def test_linear_large_tiles_split_in_two(muon, w_t):
    """256-wide tiles that fill half the card, over a contraction long enough to be split."""
    m, k, n = 2000, 16392, 4000
    x, w = normal((m, k), BF16, 1), normal((n, k) if w_t else (k, n), BF16, 2, k ** -0.5)
    r, b = normal((m, n), BF16, 3), normal((n,), BF16, 4)
    gw = w.cuda().t() if w_t else w.cuda()
    y = muon.linear(x.cuda(), gw, b.cuda(), activation="silu", residual=r.cuda())
    rows = torch.tensor([0, 1, 255, 256, 1023, 1024, 1791, 1792, 1999])
    want = ref.linear64(x[rows], w.t() if w_t else w, b, r[rows], None, "silu")
    ref.check("y", y[rows.cuda()], want["y"], norm_bound(BF16, k))


@pytest.mark.parametrize("w_t", [False, True], ids=["kn", "nk"])
@pytest.mark.parametrize("m,k,n", [(1031, 1001, 1003), (2001, 1001, 2003), (1201, 1000, 1003), (1537, 1023, 1336)])
def test_linear_large_and_odd(muon, m, k, n, w_t):
    """Products over 2 and over 8 GFLOP with one operand, or both, out of reach of 16-byte loads."""
    run_linear(muon, m, k, n, BF16, "silu", w_t, True, True)


@pytest.mark.parametrize("off_x,off_w", [(1, 0), (0, 1), (2, 1), (1, 1)])
@pytest.mark.parametrize("m,k,n", [(100, 4096, 4096), (1100, 1024, 1024), (2100, 1024, 2048)])
def test_linear_large_with_unaligned_storage(muon, m, k, n, off_x, off_w):
    """Rows that are whole 16-byte pieces apart, but begin between them, of either operand or of both."""
    x, w, dy = normal((m, k), BF16, 1), normal((k, n), BF16, 2, k ** -0.5), normal((m, n), BF16, 3)
    want = ref.linear64(x, w, None, None, dy, "none")

    def shifted(t, by):
        s = torch.full((t.numel() + by,), float("nan"), dtype=BF16, device="cuda")
        s[by:] = t.flatten().cuda()
        return s[by:].view(t.shape).requires_grad_()
    gx, gw = shifted(x, off_x), shifted(w, off_w)
    y = muon.linear(gx, gw)
    dx, dw = torch.autograd.grad(y, (gx, gw), shifted(dy, off_x).detach())
    ref.check("y", y, want["y"], norm_bound(BF16, k))
    ref.check("dx", dx, want["dx"], norm_bound(BF16, n))
    ref.check("dw", dw, want["dw"], norm_bound(BF16, m))


def test_linear_large_and_odd_keeps_infinities_in_their_rows(muon):
    """The zeros behind a copied row meet no infinity of the other operand."""
    x, w = normal((1031, 1001), BF16, 1), normal((1001, 1003), BF16, 2)
    rest = [i for i in range(1031) if i not in (7, 1030)]
    want = ref.linear64(x[rest], w, None, None, None, "none")
    x[7], x[1030, 1000] = float("inf"), float("nan")
    y = muon.linear(x.cuda(), w.cuda()).cpu()
    assert not y[7].isfinite().any() and y[1030].isnan().all()
    ref.check("y", y[rest], want["y"])


def few_rows_bounds(x, w, z, dy, act):
    """dx and dw of a layer whose z is given, and their tolerances where dz is carried to twice bf16's digits."""
    u, x, w, z, dy = ref.unit(BF16), *(t.double() for t in (x, w, z, dy))
    dz = dy * ref.act64(z, act)[1]
    # dz: the slope in float32, the rest after two roundings; float32 sums of 2 (rows or columns) products; one rounding.
    edz = 16 * ref.U32 * dy.abs() + u * u * dz.abs()
    out = {}
    for name, v, far, size, terms in (("dx", dz @ w.t(), edz @ w.abs().t(), dz.abs() @ w.abs().t(), w.shape[1]),
                                      ("dw", x.t() @ dz, x.abs().t() @ edz, x.abs().t() @ dz.abs(), x.shape[0])):
        err = far + (2 * terms + 4) * ref.U32 * size
        out[name] = v, err + u * (v.abs() + err) + 1e-37
    return out


@pytest.mark.parametrize("act", ["relu", "silu", "gelu", "gelu_tanh"])
@pytest.mark.parametrize("m,k,n,w_t", [(1, 1656, 64, True), (1, 24, 4096, False), (3, 37, 21, False), (17, 520, 264, True),
                                       (64, 2048, 24, False), (63, 65, 1001, True), (64, 512, 1024, False)])
def test_linear_gradients_of_few_rows(muon, m, k, n, w_t, act):
    """Up to 64 rows the gradient of the activation loses nothing that dx and dw keep."""
    x, w, dy = normal((m, k), BF16, 1), normal((n, k) if w_t else (k, n), BF16, 2, k ** -0.5), normal((m, n), BF16, 3)
    gx, gw = x.cuda(), w.cuda().t() if w_t else w.cuda()
    w = w.t() if w_t else w
    z = muon.linear_forward(gx, gw, activation=act, keep_z=True)[1]
    dx, dw, db = muon.linear_backward(dy.cuda(), gx, gw, z, act)
    want = few_rows_bounds(x, w, z.cpu(), dy, act)
    ref.check("dx", dx, want["dx"])
    ref.check("dw", dw, want["dw"])
    for needs in ((True, False, False), (False, True, False)):
        one = muon.linear_backward(dy.cuda(), gx, gw, z, act, needs=needs)
        assert all(torch.equal(a, b) for a, b, need in zip(one, (dx, dw, db), needs) if need)


@pytest.mark.parametrize("bad", [float("inf"), float("nan"), 3.3895e38])
def test_linear_gradients_of_few_rows_keep_infinities(muon, bad):
    """What a rounding lost is nothing where the value is not finite: an infinite gradient stays one."""
    x, w, dy = normal((5, 16), BF16, 1).abs() + 1, normal((16, 8), BF16, 2).abs() + 1, normal((5, 8), BF16, 3)
    dy[2, 4] = bad
    gx, gw = x.cuda(), w.cuda()
    z = torch.full((5, 8), 0.75, dtype=BF16, device="cuda")
    dx, dw, db = (t.cpu() for t in muon.linear_backward(dy.cuda(), gx, gw, z, "silu"))
    dz = dy.double() * ref.act64(z.cpu().double(), "silu")[1]
    assert dx[[0, 1, 3, 4]].isfinite().all() and dw[:, [0, 1, 2, 3, 5, 6, 7]].isfinite().all()
    for got, want in ((dx[2], (dz @ w.double().t())[2]), (dw[:, 4], (x.double().t() @ dz)[:, 4])):
        want = want.to(BF16)                                # past the type's range where dz is that large
        assert torch.equal(got.isnan(), want.isnan()) and torch.equal(got[got.isinf()], want[got.isinf()])
        assert torch.equal(got.isinf(), want.isinf())


# ------------------------------------------------------------------ experts

LOADS = {"even": [40, 40, 40], "empty": [0, 130, 0, 0, 7, 0], "one": [300], "single": [1, 0, 1, 1, 257, 2],
         "none": [0, 0, 0], "many": [3, 0, 5, 1] * 25}


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("load", LOADS)
@pytest.mark.parametrize("k,n,w_t,tail", [(64, 72, False, 0), (64, 72, True, 5), (24, 264, False, 130), (37, 21, False, 3),
                                          (21, 50, True, 0)])
def test_experts(muon, load, k, n, w_t, tail, dtype):
    counts = LOADS[load]
    e, used = len(counts), sum(counts)
    rows = used + tail
    offsets = torch.tensor([0, *itertools.accumulate(counts)], dtype=torch.int32)
    x, dy = normal((rows, k), dtype, 1), normal((rows, n), dtype, 2)
    x[used:], dy[used:] = float("nan"), float("inf")        # rows past the last expert reach nothing
    w, b = normal((e, n, k) if w_t else (e, k, n), dtype, 3, k ** -0.5), normal((e, n), dtype, 4)
    g = [t.cuda().requires_grad_() for t in (x, w, b)]
    y = muon.expert_linear(g[0], g[1].transpose(1, 2) if w_t else g[1], offsets.cuda(), g[2], activation="silu")
    dx, dw, db = (t.cpu() for t in torch.autograd.grad(y, g, dy.cuda()))
    y = y.detach().cpu()
    dw = dw.transpose(1, 2) if w_t else dw
    assert not y[used:].any() and not dx[used:].any()
    for i in range(e):
        lo, hi = offsets[i], offsets[i + 1]
        want = ref.linear64(x[lo:hi], w[i].t() if w_t else w[i], b[i], None, dy[lo:hi], "silu")
        for name, got in (("y", y[lo:hi]), ("dx", dx[lo:hi]), ("dw", dw[i]), ("db", db[i])):
            ref.check((name, i), got, want[name])


@pytest.mark.parametrize("counts,tail", [([1], 0), ([0, 3, 0, 1, 50], 5), ([0, 0], 7), ([1] * 60, 0), ([20, 40, 4], 0)],
                         ids=["one", "uneven", "none", "many", "all"])
@pytest.mark.parametrize("k,n,w_t", [(64, 72, False), (37, 21, True), (640, 552, False)])
def test_experts_gradients_of_few_rows(muon, counts, tail, k, n, w_t):
    e, used = len(counts), sum(counts)
    offsets = torch.tensor([0, *itertools.accumulate(counts)], dtype=torch.int32)
    x, dy = normal((used + tail, k), BF16, 1), normal((used + tail, n), BF16, 2)
    x[used:], dy[used:] = float("nan"), float("inf")
    w = normal((e, n, k) if w_t else (e, k, n), BF16, 3, k ** -0.5)
    gx, gw, off = x.cuda(), w.cuda().transpose(1, 2) if w_t else w.cuda(), offsets.cuda()
    w = w.transpose(1, 2) if w_t else w
    z = muon.linear_forward(gx, gw, activation="gelu", offsets=off, keep_z=True)[1]
    dx, dw, _ = muon.linear_backward(dy.cuda(), gx, gw, z, "gelu", offsets=off)
    assert not dx[used:].any()
    for i in range(e):
        lo, hi = offsets[i], offsets[i + 1]
        want = few_rows_bounds(x[lo:hi], w[i], z[lo:hi].cpu(), dy[lo:hi], "gelu")
        ref.check(("dx", i), dx[lo:hi], want["dx"])
        ref.check(("dw", i), dw[i], want["dw"])


@pytest.mark.parametrize("counts", [[700, 0, 513, 256, 900, 2000], [1400, 1400, 1400, 300]], ids=["skewed", "few"])
def test_experts_large_tiles(muon, counts):
    e, k, n = len(counts), 512, 1288
    offsets = torch.tensor([0, *itertools.accumulate(counts)], dtype=torch.int32)
    rows = int(offsets[-1])
    x, dy = normal((rows, k), BF16, 1), normal((rows, n), BF16, 2)
    w, b = normal((e, k, n), BF16, 3, k ** -0.5), normal((e, n), BF16, 4)
    g = [t.cuda().requires_grad_() for t in (x, w, b)]
    y = muon.expert_linear(g[0], g[1], offsets.cuda(), g[2], activation="gelu")
    dx, dw, db = torch.autograd.grad(y, g, dy.cuda())
    for i in range(e):
        lo, hi = offsets[i], offsets[i + 1]
        want = ref.linear64(x[lo:hi], w[i], b[i], None, dy[lo:hi], "gelu")
        for name, got in (("y", y[lo:hi]), ("dx", dx[lo:hi]), ("dw", dw[i]), ("db", db[i])):
            ref.check((name, i), got, want[name], norm_bound(BF16, 1) if hi > lo else None)


@pytest.mark.parametrize("w_t", [False, True], ids=["kn", "nk"])
def test_experts_large_and_odd(muon, w_t):
    """Over 8 GFLOP of odd sizes, experts without rows, and rows past the last one that hold no numbers."""
    counts, tail, k, n = [2100, 0, 1301, 1, 700], 33, 1001, 999
    e, used = len(counts), sum(counts)
    offsets = torch.tensor([0, *itertools.accumulate(counts)], dtype=torch.int32)
    x, dy = normal((used + tail, k), BF16, 1), normal((used + tail, n), BF16, 2)
    x[used:], dy[used:] = float("nan"), float("inf")
    w, b = normal((e, n, k) if w_t else (e, k, n), BF16, 3, k ** -0.5), normal((e, n), BF16, 4)
    g = [t.cuda().requires_grad_() for t in (x, w, b)]
    y = muon.expert_linear(g[0], g[1].transpose(1, 2) if w_t else g[1], offsets.cuda(), g[2], activation="gelu")
    dx, dw, db = torch.autograd.grad(y, g, dy.cuda())
    dw = dw.transpose(1, 2) if w_t else dw
    assert not y[used:].any() and not dx[used:].any()
    for i in range(e):
        lo, hi = offsets[i], offsets[i + 1]
        want = ref.linear64(x[lo:hi], w[i].t() if w_t else w[i], b[i], None, dy[lo:hi], "gelu")
        for name, got in (("y", y[lo:hi]), ("dx", dx[lo:hi]), ("dw", dw[i]), ("db", db[i])):
            ref.check((name, i), got, want[name], norm_bound(BF16, 1) if hi > lo else None)


@pytest.mark.parametrize("e", [32, 35])
def test_experts_weight_gradient_of_many_groups(muon, e):
    """Groups enough to be dealt to sets of XCDs, and a number that does not divide among them."""
    k, n = 200, 136
    counts = [(37 * i) % 1400 for i in range(e)]
    counts[3], counts[-1] = 0, 2500
    offsets = torch.tensor([0, *itertools.accumulate(counts)], dtype=torch.int32)
    rows = int(offsets[-1])
    assert rows >= 512 * e
    x, dy, w = normal((rows, k), BF16, 1), normal((rows, n), BF16, 2), normal((e, k, n), BF16, 3)
    gw = w.cuda().requires_grad_()
    (dw,) = torch.autograd.grad(muon.expert_linear(x.cuda(), gw, offsets.cuda()), gw, dy.cuda())
    for i in range(e):
        lo, hi = offsets[i], offsets[i + 1]
        ref.check(i, dw[i], ref.linear64(x[lo:hi], w[i], None, None, dy[lo:hi], "none")["dw"])


def test_expert_results_do_not_depend_on_the_other_experts(muon):
    """The same rows and weight give the same bits, alone or among others of the same average load."""
    w = normal((4, 64, 128), BF16, 1, 0.1).cuda()
    x = normal((400, 64), BF16, 2).cuda()
    off = torch.tensor([0, 100, 200, 300, 400], dtype=torch.int32).cuda()
    y = muon.expert_linear(x, w, off)
    alone = muon.expert_linear(x[100:200], w[1:2], torch.tensor([0, 100], dtype=torch.int32).cuda())
    assert torch.equal(y[100:200], alone)


# ------------------------------------------------------------------ routing


@pytest.mark.parametrize("dtype", [torch.int64, torch.int32])
@pytest.mark.parametrize("tokens,top,experts", [(0, 2, 4), (1, 1, 1), (1, 8, 64), (63, 3, 5), (700, 6, 1024), (1024, 4, 3),
                                                (2049, 2, 17), (5003, 3, 24), (9000, 8, 64), (6000, 1, 1000)])
def test_route(muon, tokens, top, experts, dtype):
    g = torch.Generator().manual_seed(tokens)
    ids = torch.randint(-1, experts + 1, (tokens, top), generator=g).to(dtype)  # -1 and `experts` are not routed
    r = muon.route(ids.cuda(), experts)
    for got, want in zip(r, ref.route64(ids, experts)):
        assert got.dtype is torch.int32 and torch.equal(got.cpu().long(), want)


def test_route_of_one_expert_and_of_none(muon):
    ids = torch.full((3000, 2), 7, dtype=torch.int64)
    r = muon.route(ids.cuda(), 9)
    assert torch.equal(r.order.cpu(), torch.arange(6000, dtype=torch.int32))
    assert r.offsets.tolist() == [0] * 8 + [6000] * 2
    r = muon.route(torch.full((3000, 2), 1 << 40).cuda(), 9)
    assert r.offsets.tolist() == [0] * 10 and (r.order == -1).all() and (r.position == -1).all()


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("tokens,top,experts,h,drop", [(1, 1, 1, 8, 0), (5, 2, 4, 7, .3), (64, 6, 64, 2048, 0),
                                                       (131, 9, 16, 1000, .2), (600, 3, 24, 513, .1), (9, 2, 4, 520, 1)])
def test_dispatch_and_combine(muon, tokens, top, experts, h, drop, dtype):
    g = torch.Generator().manual_seed(h)
    ids = torch.randint(0, experts, (tokens, top), generator=g)
    ids[torch.rand(tokens, top, generator=g) < drop] = -1
    offsets, order, position = ref.route64(ids, experts)
    used, p = int(offsets[-1]), tokens * top
    x, ys, res = normal((tokens, h), dtype, 1), normal((p, h), dtype, 2), normal((tokens, h), dtype, 3)
    w = torch.rand(tokens, top, generator=g)
    dxs, dy = normal((p, h), dtype, 4), normal((tokens, h), dtype, 5)
    ys[used:], dxs[used:] = float("nan"), float("inf")      # rows of no entry reach nothing
    u = ref.unit(dtype)

    r = muon.route(ids.cuda(), experts)
    gx, gys, gw, gres = (t.cuda().requires_grad_() for t in (x, ys, w, res))
    xs = muon.dispatch(gx, r)
    y = muon.combine(gys, r, gw, gres)
    dx, dys, dw, dres = torch.autograd.grad((xs, y), (gx, gys, gw, gres), (dxs.cuda(), dy.cuda()))

    token = order[:used] // top
    assert torch.equal(xs[:used].cpu(), x[token]) and not xs[used:].any()
    pos, on = position.clamp_min(0), (position >= 0)[..., None]
    zero = torch.zeros((), dtype=torch.float64)
    rows = torch.where(on, ys.double()[pos], zero)
    wd = w.double()[..., None]
    val, size = (wd * rows).sum(1) + res.double(), (wd * rows).abs().sum(1) + res.double().abs()
    ref.check("y", y, (val, u * val.abs() + (top + 2) * ref.U32 * size + 1e-37))
    back = torch.where(on, dxs.double()[pos], zero)
    ref.check("dx", dx, (back.sum(1), u * back.sum(1).abs() + (top + 1) * ref.U32 * back.abs().sum(1) + 1e-37))
    val = w.reshape(-1).double()[order[:used]][:, None] * dy.double()[token]
    ref.check("dys", dys[:used], (val, (u + ref.U32) * val.abs() + 1e-37))
    assert not dys[used:].any()
    prod = rows * dy.double()[:, None]
    ref.check("dw", dw, (prod.sum(2), (h + 1) * ref.U32 * prod.abs().sum(2) + 1e-37))
    assert torch.equal(dres.cpu(), dy)


def test_moves_of_strided_rows(muon):
    ids = torch.tensor([[0, 1], [1, 2], [2, 0]]).cuda()
    r = muon.route(ids, 3)
    x = normal((3, 96), BF16, 1).cuda()
    assert torch.equal(muon.dispatch(x[:, 3:43], r), muon.dispatch(x[:, 3:43].contiguous(), r))
    ys, w = normal((6, 96), BF16, 2).cuda(), torch.rand(3, 2).cuda()
    want = muon.combine(ys[:, 8:48].contiguous(), r, w, x[:, 8:48].contiguous())
    assert torch.equal(muon.combine(ys[:, 8:48], r, w, x[:, 8:48]), want)
    assert torch.equal(muon.combine(ys.t().contiguous().t()[:, 8:48], r, w, x[:, 8:48]), want)


def test_routing_refusals(muon):
    ids = torch.zeros(3, 2, dtype=torch.int64, device="cuda")
    r = muon.route(ids, 4)
    x, ys, w = torch.zeros(3, 8, device="cuda"), torch.zeros(6, 8, device="cuda"), torch.zeros(3, 2, device="cuda")
    for call in [lambda: muon.route(ids[0], 4), lambda: muon.route(ids[:, :0], 4), lambda: muon.dispatch(ys, r),
                 lambda: muon.dispatch(x[0], r), lambda: muon.combine(x, r, w), lambda: muon.combine(ys, r, w[:2]),
                 lambda: muon.combine(ys, r, w, ys), lambda: muon.combine(ys, r, w.double()),
                 lambda: muon.dispatch(x.cpu(), r)]:
        with pytest.raises(ValueError):
            call()
    with pytest.raises(TypeError):
        muon.route(ids.float(), 4)
    with pytest.raises(TypeError):
        muon.dispatch(x.half(), r)
    for e in (0, 1025):
        with pytest.raises(muon.MuonError):
            muon.route(ids, e)


# ------------------------------------------------------------------ dropout


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("shape,p", [((1,), .5), ((7,), .3), ((3, 1001), .1), ((16, 512), .5), ((5, 40, 9), .999),
                                     ((33, 8), 0.0)])
def test_dropout(muon, shape, p, dtype):
    seed, offset = 0x123456789ABCDEF0, (1 << 33) + 5
    x, r, dy = (normal(shape, dtype, i) for i in range(3))
    keep, scale = ref.keep_mask(x.numel(), p, seed, offset)
    keep = keep.view(shape)
    bad = x.clone()
    bad[~keep] = float("nan")                                # what is dropped leaves no trace
    gx, gr = bad.cuda().requires_grad_(), r.cuda().requires_grad_()
    y = muon.dropout(gx, p, seed=seed, offset=offset, residual=gr)
    dx, dr = torch.autograd.grad(y, (gx, gr), dy.cuda())
    u = ref.unit(dtype)
    f = torch.where(keep, torch.tensor(scale, dtype=torch.float64), torch.tensor(0.0, dtype=torch.float64))
    val = x.double() * f + r.double()
    size = (x.double() * f).abs() + r.double().abs()
    ref.check("y", y, (val, u * val.abs() + 3 * ref.U32 * size + 1e-37))
    ref.check("dx", dx, (dy.double() * f, (u + 2 * ref.U32) * (dy.double() * f).abs() + 1e-37))
    assert torch.equal(dr.cpu(), dy)
    assert torch.equal(muon.dropout(gx.detach(), p, seed=seed, offset=offset) == 0, (~keep | (x == 0)).cuda())
    state = torch.tensor([seed, offset]).cuda()
    assert torch.equal(muon.dropout(gx, p, residual=gr, state=state), y)


def test_dropout_unaligned_and_transposed(muon):
    x = normal((65, 33), BF16, 1).cuda()
    want = muon.dropout(x.t().contiguous(), 0.4, seed=3)
    assert torch.equal(muon.dropout(x.t(), 0.4, seed=3), want)
    flat = x.reshape(-1)
    assert torch.equal(muon.dropout(flat[1:], 0.4, seed=3), muon.dropout(flat[1:].clone(), 0.4, seed=3))


def test_dropout_rate(muon):
    """2^22 elements: the kept share within six standard deviations, streams of other seeds and offsets unlike."""
    x = torch.ones(1 << 22, device="cuda")
    masks = [muon.dropout(x, 0.25, seed=s, offset=o) != 0 for s, o in ((1, 0), (2, 0), (1, 1))]
    sd = (0.25 * 0.75 / (1 << 22)) ** 0.5
    for m in masks:
        assert abs(float(m.double().mean()) - 0.75) < 6 * sd
    for a, b in itertools.combinations(masks, 2):
        agree = 0.75 ** 2 + 0.25 ** 2
        assert abs(float((a == b).double().mean()) - agree) < 6 * (agree * (1 - agree) / (1 << 22)) ** 0.5


def test_dropout_refusals(muon):
    x = torch.zeros(8, device="cuda")
    for call in [lambda: muon.dropout(x, 1.0), lambda: muon.dropout(x, -0.1), lambda: muon.dropout(x, 0.5, residual=x[:4]),
                 lambda: muon.dropout(x, 0.5, state=torch.zeros(2, device="cuda")),
                 lambda: muon.dropout(x, 0.5, state=torch.zeros(2, dtype=torch.int64))]:
        with pytest.raises(ValueError):
            call()
    with pytest.raises(TypeError):
        muon.dropout(x.half(), 0.5)


# ------------------------------------------------------------------ graphs


def test_capture_of_forward_and_backward(muon):
    """A captured pass through every operator, replayed between eager work, equals the eager pass each time."""
    t, top, e, h, n = 96, 2, 8, 64, 136
    ids = torch.randint(0, e, (t, top), generator=torch.Generator().manual_seed(1)).cuda()
    x, dy = normal((t, h), BF16, 1).cuda(), normal((t, h), BF16, 2).cuda()
    w1, w2, b1 = normal((e, h, n), BF16, 3, .1).cuda(), normal((e, n, h), BF16, 4, .1).cuda(), normal((e, n), BF16, 5).cuda()
    probs = torch.rand(t, top, generator=torch.Generator().manual_seed(2)).cuda()
    state = torch.tensor([11, 0]).cuda()

    def step():
        r = muon.route(ids, e)
        xs = muon.dispatch_forward(x, r)
        a, z = muon.linear_forward(xs, w1, b1, "gelu", offsets=r.offsets, keep_z=True)
        ys, _ = muon.linear_forward(a, w2, None, "none", offsets=r.offsets)
        y = muon.combine_forward(ys, r, probs, x)
        out = muon.dropout_forward(y, 0.1, state=state)
        g = muon.dropout_forward(dy, 0.1, state=state)
        dys, dp = muon.combine_backward(g, ys, r, probs)
        da, dw2, _ = muon.linear_backward(dys, a, w2, None, "none", r.offsets, (True, True, False))
        dxs, dw1, db1 = muon.linear_backward(da, xs, w1, z, "gelu", r.offsets)
        return out, dp, dw1, dw2, db1, muon.dispatch_backward(dxs, r) + g

    eager = [step() for _ in range(2)][-1]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for replay in range(4):
        state[1] = replay
        x.copy_(normal((t, h), BF16, 10 + replay).cuda())
        eager = step()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(out, eager):
            assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("counts", [[5000, 0, 37, 1300], [64, 4100]], ids=["uneven", "few"])
def test_experts_weight_gradient_over_long_groups(muon, counts, dtype):
    """Few experts with many rows: the contraction is split, with splits of a short or an empty group left empty."""
    e, k, n = len(counts), 72, 40
    offsets = torch.tensor([0, *itertools.accumulate(counts)], dtype=torch.int32)
    rows = int(offsets[-1])
    x, dy, w = normal((rows, k), dtype, 1), normal((rows, n), dtype, 2), normal((e, k, n), dtype, 3)
    gw = w.cuda().requires_grad_()
    (dw,) = torch.autograd.grad(muon.expert_linear(x.cuda(), gw, offsets.cuda()), gw, dy.cuda())
    for i in range(e):
        lo, hi = offsets[i], offsets[i + 1]
        ref.check(i, dw[i], ref.linear64(x[lo:hi], w[i], None, None, dy[lo:hi], "none")["dw"])


@pytest.mark.parametrize("act", ["none", "relu", "silu", "gelu", "gelu_tanh"])
def test_activations_of_large_arguments(muon, act):
    """z over the range where the factors saturate: act(z) is z or nothing, its slope one or nothing."""
    z = torch.tensor([-1e30, -1e10, -200.0, -60.0, -0.0, 0.0, 60.0, 200.0, 1e10, 1e30])
    x = z[:, None].cuda().requires_grad_()
    y = muon.linear(x, torch.ones(1, 8, device="cuda"), activation=act)
    (dx,) = torch.autograd.grad(y, x, torch.ones_like(y))
    want, slope = ref.act64(z.double(), act)
    want, slope = want.nan_to_num(0), slope.nan_to_num(0)   # the reference's own inf * 0 past e^709
    assert torch.allclose(y[:, 0].double().cpu(), want, rtol=1e-5, atol=1e-20)
    ok = z != 0                                              # relu's slope at zero is a convention
    assert torch.allclose(dx[ok, 0].double().cpu() / 8, slope[ok], rtol=1e-5, atol=1e-6)


def test_linear_past_32_bit_offsets(muon):
    """An output of 2^32 elements and more, its gradient read back: sampled rows and columns against float64."""
    m, k, n = 66000, 64, 66048
    x, w = normal((m, k), BF16, 1).cuda(), normal((k, n), BF16, 2, k ** -0.5).cuda()
    y = muon.linear(x, w)
    rows = torch.tensor([0, 1, 32511, 32513, 65023, 65535, m - 1], device="cuda")
    want = x[rows].double() @ w.double()
    ref.check("y", y[rows], (want.cpu(), (ref.unit(BF16) * want.abs()).cpu() + 1e-5))
    dx, dw, db = muon.linear_backward(y, x, w)
    g = y[rows].double()
    want = (g @ w.double().t()).cpu()
    ref.check("dx", dx[rows], (want, ref.unit(BF16) * want.abs() + n * ref.U32 * 8))
    cols = torch.tensor([0, 5, 33024, n - 1], device="cuda")
    g = y[:, cols].double()
    want = (x.double().t() @ g).cpu()
    ref.check("dw", dw[:, cols], (want, ref.unit(BF16) * want.abs() + m * ref.U32 * 8))
    ref.check("db", db[cols], (g.sum(0).cpu(), ref.unit(BF16) * g.sum(0).abs().cpu() + m * ref.U32 * 4))


def test_moves_past_32_bit_offsets(muon):
    """2^31 elements and more of sorted rows."""
    t, top, h = 262144, 8, 1032
    ids = torch.randint(0, 64, (t, top), generator=torch.Generator().manual_seed(1)).cuda()
    r = muon.route(ids, 64)
    x = normal((t, h), BF16, 2).cuda()
    xs = muon.dispatch(x, r)
    at = torch.tensor([0, 1, 1040384, 2080768, 2080769, t * top - 1], device="cuda")
    assert torch.equal(xs[at], x[(r.order[at] // top).long()])
    ones = torch.ones(t, top, device="cuda")
    y = muon.combine(xs, r, ones)
    rows = torch.tensor([0, 77, 131072, t - 1], device="cuda")
    assert torch.equal(y[rows], (x[rows].float() * top).bfloat16())
    dys, dw = muon.combine_backward(x, xs, r, ones)
    assert torch.equal(dys[at], xs[at])
    want = (x[rows].double() ** 2).sum(1, keepdim=True).expand(-1, top).cpu()
    ref.check("dw", dw[rows], (want, h * ref.U32 * want))
    # An order of its rows undoes the sort: every entry comes back to its token.
    assert torch.equal(muon.dispatch_backward(xs, r)[rows], (x[rows].float() * top).bfloat16())
