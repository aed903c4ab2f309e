"""GPU tests of the operators around a block's products where calls are unusual."""

from __future__ import annotations

import ctypes
import itertools

import pytest
import torch

import ops_reference
from ops_reference import U32
from test_gpu_mx import BF16, F32, NAN, both, muon, normal  # noqa: F401 (muon is a fixture)

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------ four bits


@both
def test_quantize_views_whose_strides_do_not_count(muon, dtype):  # noqa: F811
    """Views of one element or of none are contiguous to torch whatever their strides are."""
    big, deep = normal((9, 12), dtype, 1).cuda(), normal((4, 9, 12), dtype, 2).cuda()
    views = [big[::2, ::3][:1, :1], big[1:, 2:].t()[::3, ::2][2:3, 3:4], big[:0, ::2], big[::2, ::3][:, :0], big[:0, :0],
             big[::2, ::3].t()[:0], deep[:, ::2, ::3][:, :1, :1], deep[::3, ::2, ::3][:, 1:2, 2:3], deep[:, :0, ::2],
             deep[:, ::2, ::3][..., :0], big[::2, :1], big[:1, ::3], big.t()[::2, :1], big.t()[:1, ::3], deep[:1, ::2, 4:5]]
    for v in views:
        q, want = muon.mx_quantize(v), muon.mx_quantize(v.clone(memory_format=torch.contiguous_format))
        assert q.shape == v.shape and q.k == want.k
        assert torch.equal(q.values, want.values) and torch.equal(q.scales, want.scales)
        assert muon.mx_dequantize(q).shape == v.shape


def plain_linear(muon, x, q, b, r, act):  # noqa: F811
    """(value, tolerance) in float64 on the GPU; ops_reference's count, with the sums of one contraction."""
    xq = muon.mx_dequantize(muon.mx_quantize(x.t())).t().double()        # the form is checked bit by bit elsewhere
    wq = muon.mx_dequantize(q).double()
    z, size = xq @ wq, xq.abs() @ wq.abs()
    if b is not None:
        z, size = z + b.double(), size + b.double().abs()
    y = ops_reference.act64(z, act)[0]
    e = 1.2 * (x.shape[1] + 2) * U32 * size + 16 * U32 * z.abs()
    if r is not None:
        y = y + r.double()
        e = e + U32 * y.abs()
    return y, e + ops_reference.unit(x.dtype) * y.abs() + 1e-37


# Tiles of 256 x 128 (the first two), of 128 x 128, and of 64 x 64; whole pieces of eight columns, and ragged ones.
TILES = [(4100, 600, 4104), (2050, 200, 4099), (2040, 520, 2104), (2033, 130, 2101), (1000, 520, 2000), (130, 400, 333)]


@both
@pytest.mark.parametrize("act", ["none", "relu", "silu", "gelu", "gelu_tanh"])
@pytest.mark.parametrize("m,k,n", TILES)
def test_every_tile_with_activation_bias_and_residual(muon, m, k, n, act, dtype):  # noqa: F811
    x, w = normal((m, k), dtype, 1, 1.5).cuda(), normal((k, n), dtype, 2, k ** -0.5).cuda()
    b, r = normal((n,), dtype, 3).cuda(), normal((m, n + 8), dtype, 4).cuda()[:, :n]
    q = muon.mx_quantize(w)
    for bias, res in ((b, r), (None, r), (b, None)):
        y = muon.mx_linear(x, q, bias, activation=act, residual=res)
        want, tol = plain_linear(muon, x, q, bias, res, act)
        assert ((y.double() - want).abs() <= tol).all(), (bias is None, res is None)


@both
@pytest.mark.parametrize("act", ["none", "silu", "gelu"])
@pytest.mark.parametrize("n", [2056, 1403])
def test_experts_of_many_rows_with_activation_and_bias(muon, n, act, dtype):  # noqa: F811
    """Groups over both large tiles, ragged and empty ones among them, and rows past the last."""
    counts = [1500, 0, 2100, 900, 3, 1800] if n == 2056 else [300, 500, 0, 129, 700, 450]
    k, offsets = 300, torch.tensor([0, *itertools.accumulate(counts)], dtype=torch.int32)
    rows = int(offsets[-1]) + 40
    x, w, b = normal((rows, k), dtype, 1), normal((len(counts), k, n), dtype, 2, k ** -0.5).cuda(), \
        normal((len(counts), n), dtype, 3).cuda()
    x[int(offsets[-1]):] = NAN
    x = x.cuda()
    q = muon.mx_quantize(w)
    y = muon.mx_expert_linear(x, q, offsets.cuda(), b, activation=act)
    for i in range(len(counts)):
        lo, hi = offsets[i], offsets[i + 1]
        if lo == hi:
            continue
        want, tol = plain_linear(muon, x[lo:hi], muon.MxWeight(q.values[i], q.scales[i], k), b[i], None, act)
        assert ((y[lo:hi].double() - want).abs() <= tol).all(), i
    assert torch.equal(y[int(offsets[-1]):], torch.zeros(40, n, dtype=dtype, device="cuda"))


def inside(t, front, back, fill):
    """A copy of t (1-D bytes) between guards of `fill`: (the whole buffer, the place of t)."""
    whole = torch.full((front + t.numel() + back,), fill, dtype=torch.uint8, device="cuda")
    whole[front:front + t.numel()] = t
    return whole, whole[front:front + t.numel()]


def as_bytes(t):
    return t.contiguous().reshape(-1).view(torch.uint8)


GUARD = 1 << 20


@both
@pytest.mark.parametrize("rows,n", [(8, 72), (40, 72), (700, 72), (1500, 1403), (3000, 2056)])
@pytest.mark.parametrize("share", [None, (0.1, 0.85, 0.14), (0.3, 0.3, 0.3), (-0.01, 1e6, 0.1), (1.0, 1.0, 0.0), (0.0, 0.4, 0.9)], ids=str)
def test_nothing_outside_the_tensors_is_written_or_used(muon, rows, n, share, dtype):  # noqa: F811
    """y and the workspace between guards that must stay, x and the weight between NaN that must not come through, for
    offsets that ascend, that do not, and that leave the tensors.  share: offsets 1 to 3 in rows (None: a plain layer)."""
    from muon_newton_schulz_05_amd import block
    lib, k, e = block.load_block(), 200, 3
    x = normal((rows, k), dtype, 1).cuda()
    lead = () if share is None else (e,)
    q = muon.mx_quantize(normal((*lead, k, n), dtype, 2, 0.1).cuda())
    d = block.MxDesc(muon.MUON_BF16 if dtype is BF16 else muon.MUON_F32, 0, e if lead else 0, 0, rows, k, n, k, 0, 0, 0)
    need = ctypes.c_uint64(0)
    assert lib.muon_mx_linear_workspace(ctypes.byref(d), ctypes.byref(need)) == 0
    offsets = None if share is None else torch.tensor([0, *(max(-2 ** 31, min(2 ** 31 - 1, int(s * rows))) for s in share)],
                                                      dtype=torch.int32).cuda()
    y_size = rows * n * x.element_size()
    # All bits set: NaN as a float, as a bfloat16 and as a scale.
    xw, xv = inside(as_bytes(x), GUARD, GUARD, 255)
    vw, vv = inside(as_bytes(q.values), GUARD, GUARD, 255)
    sw, sv = inside(as_bytes(q.scales), GUARD, GUARD, 255)
    yw, yv = inside(torch.zeros(y_size, dtype=torch.uint8, device="cuda"), GUARD, GUARD, 90)
    ww, wv = inside(torch.full((need.value,), 255, dtype=torch.uint8, device="cuda"), GUARD, GUARD, 90)
    rc = lib.muon_mx_linear(ctypes.byref(d), None if offsets is None else offsets.data_ptr(), xv.data_ptr(), vv.data_ptr(),
                            sv.data_ptr(), None, None, yv.data_ptr(), wv.data_ptr() if need.value else None, need.value,
                            torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    assert rc == 0
    for whole in (yw, ww):
        assert (whole[:GUARD] == 90).all() and (whole[-GUARD:] == 90).all()
    y = yv.view(dtype).view(rows, n)
    assert y.isfinite().all()
    if share is None:
        assert torch.equal(y, muon.mx_linear(x, q))
    elif share == (0.0, 0.4, 0.9):
        assert torch.equal(y, muon.mx_expert_linear(x, q, offsets))


# ------------------------------------------------------------------ norms


@both
@pytest.mark.parametrize("cols", [8, 8192, 9000])
def test_a_norm_gradient_of_no_rows_by_the_c_abi(muon, cols, dtype):  # noqa: F811
    """dw and db are sums of nothing, and dx, which has an address and no elements, is left alone."""
    from muon_newton_schulz_05_amd import block
    lib = block.load_block()
    d = block.NormDesc(muon.MUON_BF16 if dtype is BF16 else muon.MUON_F32, 0, 0, cols, cols, cols, cols, cols, 1e-5)
    need = ctypes.c_uint64(0)
    assert lib.muon_norm_workspace(ctypes.byref(d), ctypes.byref(need)) == 0
    dx, dw, db = (torch.full((cols,), NAN, dtype=dtype, device="cuda") for _ in range(3))
    ws = torch.empty(need.value + 16, dtype=torch.uint8, device="cuda")
    rc = lib.muon_norm_backward(ctypes.byref(d), None, None, None, None, None, None, dx.data_ptr(), dw.data_ptr(),
                                db.data_ptr(), ws.data_ptr(), need.value, torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    assert rc == 0 and dx.isnan().all() and not dw.any() and not db.any()


# ------------------------------------------------------------------ gate


def test_a_normalised_gate_does_not_keep_the_logits(muon):  # noqa: F811
    """Its gradient does not read them: they may be written to, and their memory comes back, ahead of the backward pass."""
    for dtype, e, top, normalised in ((F32, 24, 3, True), (BF16, 200, 8, True), (BF16, 24, 5, False)):
        leaf = normal((500, e), dtype, 1).cuda().requires_grad_()
        dw = normal((500, top), F32, 2).cuda()
        mask = (torch.arange(500) % 7 > 0).cuda()
        want, = torch.autograd.grad(muon.gate(leaf, top, normalize=normalised, mask=mask).weights, leaf, dw)
        logits = leaf * 1
        weights = muon.gate(logits, top, normalize=normalised, mask=mask).weights
        if normalised:
            with torch.no_grad():
                logits.zero_()
        got, = torch.autograd.grad(weights, leaf, dw)
        assert got.dtype is dtype and torch.equal(got, want)
        strided = torch.cat([leaf, leaf], 1)[:, :e]              # and rows that are not dense
        got, = torch.autograd.grad(muon.gate(strided, top, normalize=normalised, mask=mask).weights, leaf, dw)
        assert torch.equal(got, want)
    leaf = normal((1 << 14, 512), F32, 3).cuda().requires_grad_()
    logits = leaf * 1
    weights = muon.gate(logits, 2).weights
    before = torch.cuda.memory_allocated()
    del logits
    assert before - torch.cuda.memory_allocated() >= leaf.numel() * 4
    weights.sum().backward()


# ------------------------------------------------------------------ capture


def test_captured_autograd_over_inputs_that_change(muon):  # noqa: F811
    """Each replay, its outputs spoilt and its inputs renewed beforehand, gives an eager pass's bits on the same values."""
    shapes = {"x": (64, 200), "w": (200,), "b": (200,), "r": (64, 200), "router": (200, 16)}
    leaves = {name: normal(s, F32, i).cuda().requires_grad_() for i, (name, s) in enumerate(shapes.items())}
    dw, dloss, ds = normal((64, 4), F32, 9).cuda(), torch.tensor(0.3, device="cuda"), normal((64, 200), F32, 10).cuda()

    def step(p):
        y, s = muon.layer_norm(p["x"], p["w"], p["b"], residual=p["r"])
        z = muon.linear(muon.rms_norm(y, p["w"]), p["router"])
        dense, ids = muon.gate(z, 4, normalize=False)
        even = muon.gate(z, 4).weights
        loss, counts = muon.balance_loss(z, ids)
        grads = torch.autograd.grad((dense, even, loss, s), tuple(p.values()), (dw, dw, dloss, ds))
        return [*grads, dense.detach(), even.detach(), ids, loss.detach(), counts, s.detach()]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(leaves)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(leaves)
    for replay in range(4):
        with torch.no_grad():
            for i, t in enumerate(leaves.values()):
                t.copy_(normal(t.shape, F32, 100 * replay + i + 20))
            for t in out:
                t.fill_(NAN) if t.dtype.is_floating_point else t.fill_(-7)
        want = step({name: t.detach().clone().requires_grad_() for name, t in leaves.items()})
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for i, (a, b) in enumerate(zip(out, want)):
            assert torch.equal(a, b), (replay, i)
