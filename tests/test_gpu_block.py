"""GPU tests of norms, gate and balance loss against plain float64 forms (tests/block_reference.py)."""

from __future__ import annotations

import itertools

import pytest
import torch

import block_reference as ref
from ops_reference import U32, check

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
INF, NAN = float("inf"), float("nan")
both = pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])


@pytest.fixture(scope="module")
def muon():
    import muon_newton_schulz_05_amd as pkg
    return pkg


def normal(shape, dtype, seed, std=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * std).to(dtype)


# ------------------------------------------------------------------ norms

NORM_SHAPES = [(1, 1), (3, 7), (5, 8), (33, 24), (2, 64), (70, 72), (40, 129), (17, 256), (9, 511), (1100, 512), (5, 513),
               (3, 1000), (6, 1024), (2, 1025), (777, 1001), (4, 2048), (3, 2056), (2, 4096), (5, 4100), (3, 8192),
               (2, 8193), (3, 9000), (2, 16384), (3, 16385), (20, 20000)]


def run_norm(muon, rows, cols, dtype, kind, weight, bias, residual, seed=0):
    layer = kind == "layer"
    x = normal((rows, cols), dtype, seed, 2.0) + 0.25
    r = normal((rows, cols), dtype, seed + 1) if residual else None
    w = normal((cols,), dtype, seed + 2) if weight else None
    b = normal((cols,), dtype, seed + 3) if bias and layer else None
    dy = normal((rows, cols), dtype, seed + 4)
    ds = normal((rows, cols), dtype, seed + 5) if residual else None
    eps = 1e-5 if layer else 1e-6
    want = ref.norm64(x, r, w, b, dy, ds, eps, layer)
    leaves = {n: t.cuda().requires_grad_() for n, t in (("x", x), ("r", r), ("w", w), ("b", b)) if t is not None}

    def forward():
        if layer:
            return muon.layer_norm(leaves["x"], leaves.get("w"), leaves.get("b"), residual=leaves.get("r"))
        return muon.rms_norm(leaves["x"], leaves.get("w"), residual=leaves.get("r"))
    got = forward()
    outs = got if residual else (got,)
    grads = dict(zip(leaves, torch.autograd.grad(outs, tuple(leaves.values()), [dy.cuda()] + ([ds.cuda()] if residual else []))))
    check("y", outs[0], want["y"])
    check("dx", grads["x"], want["dx"])
    if residual:
        check("s", outs[1], want["s"])
        assert torch.equal(grads["r"], grads["x"])
    if weight:
        check("dw", grads["w"], want["dw"])
    if b is not None:
        check("db", grads["b"], want["db"])
    with torch.no_grad():
        again = forward()
        for p, q in zip(again if residual else (again,), outs):
            assert torch.equal(p, q)


@both
@pytest.mark.parametrize("rows,cols", NORM_SHAPES)
def test_norm_shapes(muon, rows, cols, dtype):
    run_norm(muon, rows, cols, dtype, "layer", True, True, True, seed=rows + cols)
    run_norm(muon, rows, cols, dtype, "rms", True, False, False, seed=rows + cols + 10)


@both
@pytest.mark.parametrize("kind,weight,bias,residual", [c for c in itertools.product(
    ("layer", "rms"), (False, True), (False, True), (False, True)) if c[0] == "layer" or not c[2]])
def test_norm_options(muon, kind, weight, bias, residual, dtype):
    run_norm(muon, 130, 328, dtype, kind, weight, bias, residual)
    run_norm(muon, 3, 1100, dtype, kind, weight, bias, residual, 50)
    run_norm(muon, 18, 8200, dtype, kind, weight, bias, residual, 90)


@both
@pytest.mark.parametrize("rows,cols", [(20000, 40), (9000, 300), (3000, 1032), (2000, 9001)])
def test_norm_many_rows(muon, rows, cols, dtype):
    """Every workgroup walks several rows; the weight's gradient comes from many partial sums."""
    run_norm(muon, rows, cols, dtype, "layer", True, True, True, seed=3)


@pytest.mark.parametrize("kind", ["layer", "rms"])
def test_norm_gradient_by_differences(muon, kind):
    """The float32 gradient along a direction against differences of the float64 form."""
    x, w, dy = normal((4, 96), F32, 1).double(), normal((96,), F32, 2).double(), normal((4, 96), F32, 3).double()
    e = normal((4, 96), F32, 4).double()
    up, down = (ref.norm64(x + q * 1e-6 * e, None, w, None, None, None, 1e-5, kind == "layer")["y"][0] for q in (1, -1))
    want = ((up - down) / 2e-6 * dy).sum()
    leaf = x.float().cuda().requires_grad_()
    y, s, stats = muon.norm_forward(leaf, w.float().cuda(), eps=1e-5, kind=kind)
    dx, dw, db = muon.norm_backward(dy.float().cuda(), s, w.float().cuda(), stats, kind=kind)
    got = (dx.double().cpu() * e).sum()
    # 384 products of terms of order one, each a few U32 off; the difference itself to about 1e-9.
    assert abs(got - want) <= 384 * 40 * U32 + 1e-6 * abs(want)


@both
def test_norm_strides_and_broadcasts(muon, dtype):
    big = normal((6, 10, 160), dtype, 1)
    x = big[:, ::2, 8:136]                                      # [6, 5, 128], rows 320 apart and not flattenable
    w = normal((256,), dtype, 2)[::2]                           # a strided weight is copied
    r = normal((128, 6, 5), dtype, 3).permute(1, 2, 0)          # last dimension not contiguous
    want = ref.norm64(x.reshape(30, 128), r.reshape(30, 128), w, None, torch.ones(30, 128, dtype=dtype), None, 1e-5, True)
    gx, gr = big.cuda()[:, ::2, 8:136].requires_grad_(), normal((128, 6, 5), dtype, 3).cuda().permute(1, 2, 0)
    gw = normal((256,), dtype, 2).cuda()[::2].requires_grad_()
    y, s = muon.layer_norm(gx, gw, residual=gr)
    assert y.shape == s.shape == x.shape and y.is_contiguous()
    dx, dw = torch.autograd.grad(y.sum(), (gx, gw))             # a gradient with strides of zero
    check("y", y.reshape(30, 128), want["y"])
    check("s", s.reshape(30, 128), want["s"])
    check("dx", dx.reshape(30, 128), want["dx"])
    check("dw", dw, want["dw"])
    # A row that is given to all: stride 0.
    one = normal((1, 128), dtype, 5)
    y = muon.rms_norm(one.cuda().expand(7, 128))
    check("y", y, ref.norm64(one.expand(7, 128), None, None, None, None, None, 1e-6, False)["y"])


@both
def test_norm_of_unaligned_rows(muon, dtype):
    """Rows that start at any element."""
    buf = normal((40 * 131 + 3,), dtype, 1)
    for start, ld in ((1, 131), (3, 130), (2, 129)):
        x = buf.as_strided((37, 129), (ld, 1), start)
        want = ref.norm64(x, None, None, None, x, None, 1e-5, True)
        g = buf.cuda().as_strided((37, 129), (ld, 1), start)
        y, s, stats = muon.norm_forward(g)
        check("y", y, want["y"])
        check("dx", muon.norm_backward(g, s, None, stats)[0], want["dx"])


def test_norm_partial_gradients(muon):
    """Each gradient alone equals what all of them together give; unused results have none."""
    x, w, b = (normal(s, BF16, i).cuda() for i, s in enumerate(((50, 200), (200,), (200,))))
    dy = normal((50, 200), BF16, 9).cuda()
    y, s, stats = muon.norm_forward(x, w, b, residual=dy)
    whole = muon.norm_backward(dy, x, w, stats, residual=dy, ds=x)
    for i in range(3):
        part = muon.norm_backward(dy, x, w, stats, residual=dy, ds=x, needs=tuple(j == i for j in range(3)))
        assert torch.equal(part[i], whole[i]) and [p is None for p in part] == [j != i for j in range(3)]
    # From the stored sum in their place: xhat is off by half a step of s more, over the standard deviation.
    h = x.double() + dy.double()
    xhat = (h - h.mean(1, keepdim=True)) / h.var(1, correction=0, keepdim=True).sqrt()
    dw, tol = (dy.double() * xhat).sum(0), (dy.double().abs() * h.abs() / h.std(1, keepdim=True)).sum(0) * 2.0 ** -8
    stored = muon.norm_backward(dy, s, w, stats, ds=x)
    assert ((stored[1].double() - dw).abs() <= tol + 2.0 ** -8 * dw.abs() + 1e-3).all()
    assert torch.equal(stored[2], whole[2])
    leaf, res = x.clone().requires_grad_(), dy.clone().requires_grad_()
    y, s = muon.layer_norm(leaf, residual=res)
    g1, g2 = torch.autograd.grad(s, (leaf, res), dy, retain_graph=True)      # y is not used
    assert torch.equal(g1, dy) and torch.equal(g2, dy)
    (only,) = torch.autograd.grad(y, leaf, dy, retain_graph=True)            # s is not used
    want = muon.norm_backward(dy, x, None, muon.norm_forward(x, residual=dy)[2], residual=dy)[0]
    assert torch.equal(only, want)
    (none,) = torch.autograd.grad(muon.layer_norm(x, w.requires_grad_()), w, dy)
    assert none.shape == w.shape


def test_norm_is_differentiable_once(muon):
    x = normal((4, 16), F32, 1).cuda().requires_grad_()
    (g,) = torch.autograd.grad(muon.layer_norm(x).square().sum(), x, create_graph=True)
    with pytest.raises(RuntimeError):
        g.sum().backward()


@both
def test_norm_of_special_rows(muon, dtype):
    """Constant rows, rows of zeros, a large mean, an outlier, infinities and NaN: each touches its own row alone."""
    x = normal((9, 300), dtype, 1)
    x[0], x[1] = 5.0, 0.0
    x[2] += 1000.0
    x[3, 0] = 3e4
    x[4, 7], x[5, 299], x[6] = INF, NAN, -INF
    y = muon.layer_norm(x.cuda()).double().cpu()
    z = muon.rms_norm(x.cuda()).double().cpu()
    assert torch.equal(y[0], torch.zeros(300).double()) and torch.equal(y[1], y[0]) and torch.equal(z[1], y[0])
    assert y[4:7].isnan().all() and z[5].isnan().all()
    fine = [0, 1, 2, 3, 7, 8]
    check("y", y[fine], ref.norm64(x[fine], None, None, None, None, None, 1e-5, True)["y"])
    check("z", z[fine], ref.norm64(x[fine], None, None, None, None, None, 1e-6, False)["y"])
    assert muon.layer_norm(x[:1].cuda(), eps=0.0).isnan().all()              # 0 / 0, as the formula says


def test_norm_without_rows_or_columns(muon):
    w = torch.ones(64, device="cuda", requires_grad=True)
    x = torch.empty(0, 64, device="cuda", requires_grad=True)
    y, s = muon.layer_norm(x, w, w, residual=x)
    dx, dw = torch.autograd.grad((y, s), (x, w), (y, s))
    assert y.shape == dx.shape == (0, 64) and torch.equal(dw, torch.zeros_like(w))
    wide = torch.empty(0, 20000, device="cuda", requires_grad=True)
    ww = torch.ones(20000, device="cuda", requires_grad=True)
    assert torch.equal(torch.autograd.grad(muon.rms_norm(wide, ww).sum(), ww)[0], torch.zeros_like(ww))
    assert muon.layer_norm(torch.empty(5, 0, device="cuda")).shape == (5, 0)


# ------------------------------------------------------------------ gate

GATE_SHAPES = [(1, 1, 1), (1, 8, 2), (5, 7, 7), (64, 64, 6), (300, 24, 3), (33, 9, 9), (70, 16, 16), (257, 33, 8), (100, 128, 4),
               (65, 200, 8), (31, 256, 16), (20, 511, 5), (9, 512, 64), (10, 513, 7), (7, 1000, 100), (3, 1024, 1024)]


def run_gate(muon, t, e, top, dtype, normalize, masked, seed=0, z=None):
    z = normal((t, e), dtype, seed, 2.0) if z is None else z
    mask = torch.rand(t, generator=torch.Generator().manual_seed(seed + 1)) > 0.3 if masked else None
    dw = normal((t, top), F32, seed + 2)
    want = ref.gate64(z, top, normalize, mask, dw)
    leaf = z.cuda().requires_grad_()
    gm = None if mask is None else mask.cuda()
    weights, ids = got = muon.gate(leaf, top, normalize=normalize, mask=gm)
    assert ids.dtype is torch.int32 and weights.dtype is F32
    assert torch.equal(ids.cpu().long(), want["ids"])
    check("weights", weights, want["weights"])
    (dz,) = torch.autograd.grad(weights, leaf, dw.cuda())
    check("dz", dz, want["dz"])
    assert torch.equal(muon.gate_backward(dw.cuda(), leaf, muon.Gating(weights.detach(), ids), normalize=normalize, mask=gm), dz)
    with torch.no_grad():
        again = muon.gate(leaf, top, normalize=normalize, mask=gm)
    assert torch.equal(again.weights, got.weights) and torch.equal(again.ids, ids)


@both
@pytest.mark.parametrize("t,e,top", GATE_SHAPES)
def test_gate_shapes(muon, t, e, top, dtype):
    run_gate(muon, t, e, top, dtype, True, False, t + e)
    run_gate(muon, t, e, top, dtype, False, True, t + e + 7)


@both
@pytest.mark.parametrize("normalize", [True, False])
def test_gate_of_ties_and_of_what_is_left_out(muon, dtype, normalize):
    """Equal logits go to the lower index; experts at -inf are not chosen, also where too few are left."""
    z = torch.randint(-2, 3, (200, 40), generator=torch.Generator().manual_seed(1)).to(dtype)
    z[3] = 0.0
    z[4] = -0.0
    z[5, ::2] = -0.0
    z[10:60][torch.rand(50, 40, generator=torch.Generator().manual_seed(2)) < 0.9] = -INF
    z[7] = -INF
    z[8] = torch.finfo(dtype).min
    z[9, :39] = torch.finfo(dtype).min
    run_gate(muon, 200, 40, 6, dtype, normalize, False, z=z)
    run_gate(muon, 200, 40, 40, dtype, normalize, True, z=z)


@both
def test_gate_of_infinite_and_nan_logits(muon, dtype):
    z = normal((6, 20), dtype, 1)
    z[0, 3], z[1, 5], z[1, 2], z[2] = INF, NAN, NAN, NAN
    z[4] = NAN
    mask = torch.tensor([1, 1, 1, 1, 0, 1], dtype=torch.bool)
    for normalize in (True, False):
        leaf = z.cuda().requires_grad_()
        w, ids = muon.gate(leaf, 4, normalize=normalize, mask=mask.cuda())
        assert torch.equal(ids.cpu().long(), ref.choose(z, 4, mask))
        assert w[0, 0].isnan() and w[1:3].isnan().all()
        assert torch.equal(w[4].cpu(), torch.zeros(4))
        (dz,) = torch.autograd.grad(w, leaf, torch.ones_like(w))
        assert torch.equal(dz[4].cpu(), torch.zeros(20, dtype=dtype))          # masked: NaN does not come through
        want = ref.gate64(z[[3, 5]], 4, normalize, None, torch.ones(2, 4))
        check("weights", w[[3, 5]], want["weights"])
        check("dz", dz[[3, 5]], want["dz"])


@both
def test_gate_of_far_apart_logits(muon, dtype):
    """Probabilities that vanish are zero; a gradient with strides of zero, logits with strides."""
    z = normal((40, 64), dtype, 1, 60.0)
    run_gate(muon, 40, 64, 8, dtype, False, False, z=z)
    big = normal((80, 100), dtype, 2).cuda()
    leaf = big[::2, 3:40].requires_grad_()
    w, ids = muon.gate(leaf, 5, normalize=False)
    want = ref.gate64(leaf.detach().cpu(), 5, False, None, torch.ones(40, 5))
    assert torch.equal(ids.cpu().long(), want["ids"])
    (dz,) = torch.autograd.grad(w.sum(), leaf)
    check("dz", dz, want["dz"])
    t = normal((37, 60), dtype, 3).cuda().t()                                   # columns contiguous: copied
    assert torch.equal(muon.gate(t, 3).ids, muon.gate(t.contiguous(), 3).ids)


def test_gate_without_tokens(muon):
    z = torch.empty(0, 8, device="cuda", requires_grad=True)
    w, ids = muon.gate(z, 2)
    assert w.shape == ids.shape == (0, 2)
    assert torch.autograd.grad(w, z, w)[0].shape == (0, 8)


# ------------------------------------------------------------------ balance loss

BALANCE_SHAPES = [(1, 1, 1), (1, 8, 2), (64, 64, 6), (5003, 24, 3), (300, 7, 9), (1000, 16, 2), (129, 33, 8), (700, 128, 4),
                  (65, 256, 8), (130, 512, 5), (33, 1000, 10), (20000, 8, 2), (70000, 40, 1)]


def run_balance(muon, t, e, top, dtype, masked, wide, seed=0, z=None, ids=None):
    g = torch.Generator().manual_seed(seed + 1)
    z = normal((t, e), dtype, seed, 1.5) if z is None else z
    ids = torch.randint(-1, e + 1, (t, top), generator=g) if ids is None else ids
    mask = torch.rand(t, generator=g) > 0.3 if masked else None
    dloss = 0.37
    want = ref.balance64(z, ids, mask, torch.tensor(dloss, dtype=F32).double())
    leaf, gm = z.cuda().requires_grad_(), None if mask is None else mask.cuda()
    gi = ids.cuda().to(torch.int64 if wide else torch.int32)
    loss, counts = muon.balance_loss(leaf, gi, mask=gm)
    assert loss.dtype is F32 and loss.shape == () and counts.dtype is torch.int32
    assert torch.equal(counts.cpu().long(), want["counts"])
    check("loss", loss, want["loss"])
    (dz,) = torch.autograd.grad(loss, leaf, torch.tensor(dloss, device="cuda"))
    check("dz", dz, want["dz"])
    again = muon.balance_forward(leaf, gi, mask=gm)
    assert torch.equal(again[0], loss) and torch.equal(again[1], counts)
    assert torch.equal(muon.balance_backward(torch.tensor(dloss, device="cuda"), leaf, gi, again[2], mask=gm), dz)


@both
@pytest.mark.parametrize("t,e,top", BALANCE_SHAPES)
def test_balance_shapes(muon, t, e, top, dtype):
    run_balance(muon, t, e, top, dtype, False, False, t + e)
    run_balance(muon, t, e, top, dtype, True, True, t + e + 5)


@both
def test_balance_of_special_rows(muon, dtype):
    """Experts at -inf, a row of nothing else, the lowest values; what a masked token holds reaches nothing."""
    z = normal((60, 20), dtype, 1)
    z[0, ::3], z[1], z[2], z[3, 1:] = -INF, -INF, torch.finfo(dtype).min, torch.finfo(dtype).min
    run_balance(muon, 60, 20, 3, dtype, False, False, z=z)
    z = normal((50, 20), dtype, 2)
    ids = torch.randint(0, 20, (50, 3), generator=torch.Generator().manual_seed(3))
    mask = torch.ones(50, dtype=torch.bool)
    mask[::7] = False
    dirty = z.clone()
    dirty[~mask] = NAN
    a = muon.balance_loss(z.cuda(), ids.cuda(), mask=mask.cuda())
    leaf = dirty.cuda().requires_grad_()
    b = muon.balance_loss(leaf, ids.cuda(), mask=mask.cuda())
    assert torch.equal(a.loss, b.loss) and torch.equal(a.counts, b.counts) and int(a.counts.sum()) == 3 * int(mask.sum())
    (dz,) = torch.autograd.grad(b.loss, leaf)
    assert torch.equal(dz[~mask.cuda()], torch.zeros_like(dz[~mask.cuda()])) and dz.isfinite().all()
    assert muon.balance_loss(dirty.cuda(), ids.cuda()).loss.isnan()


def test_balance_of_nothing(muon):
    """No tokens, and none that the mask leaves: zero, and a zero gradient."""
    for t, mask in ((0, None), (9, torch.zeros(9, dtype=torch.bool, device="cuda"))):
        z = torch.ones(t, 6, device="cuda", requires_grad=True)
        loss, counts = muon.balance_loss(z, torch.zeros(t, 2, dtype=torch.int32, device="cuda"), mask=mask)
        assert loss.item() == 0 and counts.tolist() == [0] * 6
        assert torch.equal(torch.autograd.grad(loss, z)[0], torch.zeros(t, 6, device="cuda"))


def test_balance_of_even_loads_is_one(muon):
    ids = torch.arange(64, device="cuda").view(32, 2) % 8
    loss, counts = muon.balance_loss(torch.zeros(32, 8, device="cuda"), ids)
    assert loss.item() == 1.0 and counts.tolist() == [8] * 8


# ------------------------------------------------------------------ large offsets, streams, graphs, a block


def test_past_32_bit_offsets(muon):
    """Rows more than 2^32 elements into a tensor give what the same rows give alone."""
    rows, cols = 66000, 65600                                                   # 4.3e9 elements, wide rows
    x = torch.zeros(rows, cols, dtype=BF16, device="cuda")
    at = torch.tensor([0, 1, 40000, 65535, rows - 1], device="cuda")
    x[at] = normal((5, cols), BF16, 1).cuda()
    w = normal((cols,), BF16, 2).cuda()
    y, _, stats = muon.norm_forward(x, w)
    few, _, fstats = muon.norm_forward(x[at], w)
    assert torch.equal(y[at], few) and torch.equal(stats[at], fstats)
    del y
    dx, _, _ = muon.norm_backward(x, x, w, stats, needs=(True, False, False))
    assert torch.equal(dx[at], muon.norm_backward(x[at], x[at], w, fstats, needs=(True, False, False))[0])
    del dx
    x = x.view(-1)
    narrow = x.as_strided((4200000, 1000), (1024, 1))
    narrow[-1] = normal((1000,), BF16, 3).cuda()
    y, _, stats = muon.norm_forward(narrow)
    assert torch.equal(y[-1:], muon.norm_forward(narrow[-1:])[0])
    del y
    z = x.as_strided((4096, 200), (1 << 20, 1))                                  # logits far apart
    z[-3:] = normal((3, 200), BF16, 4).cuda()
    a, b = muon.gate_forward(z, 5, normalize=False), muon.gate_forward(z[-3:], 5, normalize=False)
    assert torch.equal(a.ids[-3:], b.ids) and torch.equal(a.weights[-3:], b.weights)
    g = torch.ones(4096, 5, device="cuda")
    assert torch.equal(muon.gate_backward(g, z, a, normalize=False)[-3:], muon.gate_backward(g[:3], z[-3:], b, normalize=False))
    loss, counts, shares = muon.balance_forward(z, a.ids)
    near = muon.balance_forward(z.contiguous(), a.ids)
    assert torch.equal(loss, near[0]) and torch.equal(counts, near[1]) and torch.equal(shares, near[2])
    one = torch.ones((), device="cuda")
    assert torch.equal(muon.balance_backward(one, z, a.ids, shares), muon.balance_backward(one, z.contiguous(), a.ids, shares))


def test_two_streams_at_once(muon):
    """Calls on two streams, with what torch allocates for each, do not meet."""
    x, w = normal((4096, 1024), BF16, 1).cuda(), normal((1024,), BF16, 2).cuda()
    z = normal((4096, 64), F32, 3).cuda()
    y, s, st = muon.norm_forward(x, w)
    want = (muon.norm_backward(x, s, w, st), muon.balance_forward(z, muon.gate_forward(z, 4).ids)[0])
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = []
    for _ in range(10):
        for stream in streams:
            with torch.cuda.stream(stream):
                y, s, st = muon.norm_forward(x, w)
                got.append((muon.norm_backward(x, s, w, st), muon.balance_forward(z, muon.gate_forward(z, 4).ids)[0]))
    torch.cuda.synchronize()
    for grads, loss in got:
        assert all(torch.equal(a, b) for a, b in zip(grads, want[0])) and torch.equal(loss, want[1])


def _block_step(muon, x, p, mask, dy, dloss):
    """A block's forward pass by the calls with autograd: norm, gate, experts, the balance loss."""
    h, s = muon.layer_norm(x, p["g"], p["b"], residual=p["r"])
    logits = muon.linear(h, p["router"])
    w, ids = muon.gate(logits, 2, mask=mask)
    balance = muon.balance_loss(logits, ids, mask=mask)
    r = muon.route(ids, 6)
    u = muon.expert_linear(muon.dispatch(h, r), p["up"], r.offsets, activation="silu")
    y = muon.combine(muon.expert_linear(u, p["down"], r.offsets), r, w, residual=s)
    return y, balance, ids


def test_a_block_and_its_gradients(muon):
    """Norm, gate, routed experts and the balance loss together, against torch's own float64 autograd."""
    t, h, n, e = 90, 48, 72, 6
    shapes = {"g": (h,), "b": (h,), "r": (t, h), "router": (h, e), "up": (e, h, n), "down": (e, n, h)}
    p = {k: normal(v, F32, i, 0.3) for i, (k, v) in enumerate(shapes.items())}
    p["g"] += 1
    x, dy, dloss = normal((t, h), F32, 20), normal((t, h), F32, 21), torch.tensor(0.25)
    mask = torch.rand(t, generator=torch.Generator().manual_seed(5)) > 0.1
    gp = {k: v.cuda().requires_grad_() for k, v in p.items()}
    gx = x.cuda().requires_grad_()
    y, balance, ids = _block_step(muon, gx, gp, mask.cuda(), dy, dloss)
    got = torch.autograd.grad((y, balance.loss), [gx, *gp.values()], (dy.cuda(), dloss.cuda()))

    lp = {k: v.double().requires_grad_() for k, v in p.items()}
    lx = x.double().requires_grad_()
    s = lx + lp["r"]
    hid = torch.nn.functional.layer_norm(s, (h,), lp["g"], lp["b"], 1e-5)
    logits = hid @ lp["router"]
    top, want_ids = torch.topk(logits, 2, dim=1)
    assert torch.equal(torch.where(mask[:, None], want_ids, -1), ids.cpu().long())
    w = torch.softmax(top, 1) * mask[:, None]
    outs = torch.stack([torch.nn.functional.silu(hid @ lp["up"][i]) @ lp["down"][i] for i in range(e)], 1)
    want_y = (w[:, :, None] * outs.gather(1, want_ids[:, :, None].expand(-1, -1, h))).sum(1) + s
    f = torch.stack([(want_ids[mask] == i).sum() for i in range(e)]).double() / (2 * int(mask.sum()))
    loss = e * (f * torch.softmax(logits[mask], 1).mean(0)).sum()
    want = torch.autograd.grad((want_y, loss), [lx, *lp.values()], (dy.double(), dloss.double()))
    # float32 throughout: chains of sums of up to 90 and 72 terms, each product and sum a few U32 off.
    assert float((y.detach().double().cpu() - want_y.detach()).norm() / want_y.detach().norm()) < 200 * U32
    for name, a, b in zip(["x", *p], got, want):
        assert float((a.double().cpu() - b).norm() / b.norm()) < 400 * U32, name


def test_capture_of_forward_and_backward(muon):
    """A captured pass through every operator here, replayed between eager work, equals the eager pass each time."""
    t, h, e, n = 200, 264, 24, 320
    x, dy = normal((t, h), BF16, 1).cuda(), normal((t, h), BF16, 2).cuda()
    g, b, router = normal((h,), BF16, 3).cuda(), normal((h,), BF16, 4).cuda(), normal((h, e), BF16, 5, 0.2).cuda()
    up = muon.mx_quantize(normal((e, h, n), BF16, 6, 0.1).cuda())
    dw, dloss = normal((t, 3), F32, 7).cuda(), torch.tensor(0.1, device="cuda")
    mask = (torch.arange(t) % 5 > 0).cuda()

    def step():
        y, s, stats = muon.norm_forward(x, g, b, residual=dy)
        z, _ = muon.linear_forward(y, router)
        gating = muon.gate_forward(z, 3, normalize=False, mask=mask)
        loss, counts, shares = muon.balance_forward(z, gating.ids, mask=mask)
        r = muon.route(gating.ids, e)
        u = muon.mx_expert_linear(muon.dispatch_forward(y, r), up, r.offsets, activation="gelu")
        dz = muon.gate_backward(dw, z, gating, normalize=False, mask=mask)
        dz = dz + muon.balance_backward(dloss, z, gating.ids, shares, mask=mask)
        return (y, s, loss, counts, u, dz, *muon.norm_backward(dy, x, g, stats, residual=dy, ds=x), gating.weights, gating.ids)

    step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for replay in range(4):
        x.copy_(normal((t, h), BF16, 10 + replay).cuda())
        eager = step()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for a, b_ in zip(out, eager):
            assert torch.equal(a, b_)


def test_captured_autograd(muon):
    """A training pass through autograd, captured with leaves of its own."""
    x, w = normal((64, 200), F32, 1).cuda().requires_grad_(), torch.ones(200, device="cuda", requires_grad=True)
    router = normal((200, 16), F32, 2).cuda().requires_grad_()

    def step():
        z = muon.linear(muon.rms_norm(x, w), router)
        weights, ids = muon.gate(z, 4, normalize=False)
        return torch.autograd.grad((weights.square().sum() + muon.balance_loss(z, ids).loss,), (x, w, router))

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        want = [g.clone() for g in step()]
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for _ in range(3):
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(out, want):
            # torch's own sum of the squares may add in another order under capture
            assert torch.allclose(a, b, rtol=1e-5, atol=1e-7)


# ------------------------------------------------------------------ autograd


def test_what_a_gradient_needs_must_not_change(muon):
    """A tensor kept for the gradient and written to since is refused, as torch's own operators refuse it."""
    x, w = normal((8, 64), F32, 1).cuda().requires_grad_(), torch.ones(64, device="cuda", requires_grad=True)
    r = normal((8, 64), F32, 2).cuda()
    y, s = muon.layer_norm(x, w, residual=r)
    with torch.no_grad():
        r.add_(1)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.sum().backward()
    y, s = muon.layer_norm(x, w, residual=r)
    s.add_(1)                                                   # the sum is the caller's
    (y.sum() + s.sum()).backward()
    z = normal((8, 64), F32, 3).cuda().requires_grad_()
    weights, _ = muon.gate(z, 3, normalize=False)
    loss = muon.balance_loss(z, torch.zeros(8, 2, dtype=torch.int32, device="cuda")).loss
    with torch.no_grad():
        z.mul_(2)
    for out in (weights.sum(), loss):
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            out.backward()


def test_each_operator_is_differentiable_once(muon):
    z = normal((8, 16), F32, 1).cuda().requires_grad_()
    ids = torch.zeros(8, 2, dtype=torch.int32, device="cuda")
    for out in (muon.rms_norm(z).sum(), muon.gate(z, 2, normalize=False).weights.sum(), muon.balance_loss(z, ids).loss):
        (g,) = torch.autograd.grad(out, z, create_graph=True)
        with pytest.raises(RuntimeError, match="differentiable once"):
            g.square().sum().backward()
    with torch.enable_grad():
        assert not muon.gate(z, 2).ids.requires_grad and not muon.balance_loss(z, ids).counts.requires_grad
        assert not muon.layer_norm(z.detach()).requires_grad


def test_a_graph_is_walked_twice_and_from_another_thread(muon):
    """retain_graph gives the same bits again; a backward pass on another thread and stream as well."""
    import threading
    x, w = normal((300, 200), BF16, 1).cuda().requires_grad_(), normal((200,), BF16, 2).cuda().requires_grad_()
    dy = normal((300, 200), BF16, 3).cuda()
    y = muon.layer_norm(x, w)
    want = torch.autograd.grad(y, (x, w), dy, retain_graph=True)
    got = []

    def walk():
        with torch.cuda.stream(torch.cuda.Stream()):
            got.append(torch.autograd.grad(y, (x, w), dy))
    t = threading.Thread(target=walk)
    torch.cuda.synchronize()
    t.start()
    t.join()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got[0]))


def test_the_gradient_of_a_shared_input_is_summed(muon):
    """One tensor as x and as residual, and a weight that two norms share."""
    x, w = normal((20, 96), F32, 1).cuda().requires_grad_(), normal((96,), F32, 2).cuda().requires_grad_()
    y, s = muon.layer_norm(x, w, residual=x)
    z = muon.rms_norm(s, w)
    dx, dw = torch.autograd.grad((y, z), (x, w), (torch.ones_like(y), torch.ones_like(z)))
    xd, wd = x.detach().double().requires_grad_(), w.detach().double().requires_grad_()
    sd = xd + xd
    yd = torch.nn.functional.layer_norm(sd, (96,), wd, None, 1e-5)
    zd = sd * torch.rsqrt(sd.square().mean(1, keepdim=True) + 1e-6) * wd
    ex, ew = torch.autograd.grad((yd, zd), (xd, wd), (torch.ones_like(yd), torch.ones_like(zd)))
    # chains of a few sums of 96 and 20 float32 terms
    assert float((dx - ex).norm() / ex.norm()) < 100 * U32 and float((dw - ew).norm() / ew.norm()) < 100 * U32
