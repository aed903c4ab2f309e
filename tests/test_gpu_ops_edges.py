"""GPU tests of the layer operators' edges: non-finite operands, the tails of the activations, paths that only
unusual shapes reach, several streams and threads, against the plain float64 forms of tests/ops_reference.py."""

from __future__ import annotations

import ctypes
import itertools
import threading

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


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("w_t", [False, True], ids=["kn", "nk"])
@pytest.mark.parametrize("k,n", [(24, 1104), (64, 1024), (8, 2056)])
def test_experts_of_narrow_outputs_and_long_contractions(muon, k, n, w_t, dtype):
    """dx of thin experts, whose contraction four sets of waves share: ragged and empty groups, a tail of no numbers."""
    counts, tail = [70, 0, 33, 1, 130, 0, 64], 9
    e, used = len(counts), sum(counts)
    offsets = torch.tensor([0, *itertools.accumulate(counts)], dtype=torch.int32)
    x, dy = normal((used + tail, k), dtype, 1), normal((used + tail, n), dtype, 2)
    x[used:], dy[used:] = float("nan"), float("inf")
    w = normal((e, n, k) if w_t else (e, k, n), dtype, 3, k ** -0.5)
    gw = w.cuda().transpose(1, 2) if w_t else w.cuda()
    w = w.transpose(1, 2) if w_t else w
    dx, dw, db = muon.linear_backward(dy.cuda(), x.cuda(), gw, offsets=offsets.cuda())
    assert not dx[used:].any()
    for i in range(e):
        lo, hi = offsets[i], offsets[i + 1]
        want = ref.linear64(x[lo:hi], w[i], None, None, dy[lo:hi], "none")
        for name, got in (("dx", dx[lo:hi]), ("dw", dw[i]), ("db", db[i])):
            ref.check((name, i), got, want[name])
    # The same operation forward: a contraction of k = n over weights [E, n, k].
    y = muon.expert_linear(dy.cuda(), gw.transpose(1, 2), offsets.cuda())
    assert torch.equal(y, dx)


def wide(rows, cols, ld, dtype, seed):
    """A tensor of `rows` rows that lie ld elements apart on the GPU, and the same values on the CPU."""
    v = normal((rows, cols), dtype, seed)
    t = torch.empty((rows - 1) * ld + cols, dtype=dtype, device="cuda").as_strided((rows, cols), (ld, 1))
    t.copy_(v)
    return t, v


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("m,k,n,of", [(5, 24, 40, "x"), (9, 72, 70, "w"), (70, 9, 40, "both"), (1500, 16, 1504, "x")])
def test_linear_rows_too_far_apart_for_32_bits(muon, m, k, n, of, dtype):
    """Rows whose offsets inside a tile pass 32 bits take the loads of any alignment."""
    es = torch.finfo(dtype).bits // 8
    far_x, far_w = (1 << 31) // (256 * es) + 8, (1 << 31) // 128 + 8
    x, cx = wide(m, k, far_x if of in ("x", "both") else k, dtype, 1)
    w, cw = wide(k, n, far_w if of in ("w", "both") else n, dtype, 2)
    dy, cdy = normal((m, n), dtype, 3).cuda(), normal((m, n), dtype, 3)
    want = ref.linear64(cx, cw, None, None, cdy, "none")
    y = muon.linear(x, w)
    dx, dw, _ = muon.linear_backward(dy, x, w)
    for name, got in (("y", y), ("dx", dx), ("dw", dw)):
        ref.check(name, got, want[name])


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("w_t", [False, True], ids=["kn", "nk"])
@pytest.mark.parametrize("m,k,n", [(3, 2048, 64), (70, 64, 16384), (130, 72, 264), (37, 21, 19)])
def test_linear_gradient_steps_one_by_one(muon, m, k, n, w_t, dtype):
    """The C calls behind the one-call gradient, each for itself."""
    from muon_newton_schulz_05_amd import ops
    lib, act = ops.load_ops(), "gelu_tanh"
    x, w = normal((m, k), dtype, 1), normal((n, k) if w_t else (k, n), dtype, 2, k ** -0.5)
    dy, z = normal((m, n), dtype, 3), normal((m, n), dtype, 4)
    gx, gw, gdy, gz = (t.cuda() for t in (x, w, dy, z))
    d = ops.LinearDesc(ops._dtype(x, "x"), ops.ACTIVATIONS[act], 0, int(w_t), m, k, n, k, k if w_t else n, 0, n, n)

    def call(op, f, *args):
        need = ctypes.c_uint64(0)
        assert lib.muon_linear_workspace(ctypes.byref(d), op, ctypes.byref(need)) == 0
        ws = torch.empty(need.value, dtype=torch.uint8, device="cuda")
        args = [t if t is None else t.data_ptr() for t in args]
        assert f(ctypes.byref(d), None, *args, ws.data_ptr() if need.value else None, need.value,
                 torch.cuda.current_stream().cuda_stream) == 0
    dz, db = torch.empty_like(gdy), torch.empty(n, dtype=dtype, device="cuda")
    dx, dw = torch.empty_like(gx), torch.empty_like(gw)
    call(1, lib.muon_linear_grad_act, gdy, gz, dz, db)
    call(2, lib.muon_linear_grad_input, dz, gw, dx)
    call(3, lib.muon_linear_grad_weight, gx, dz, dw)
    u = ref.unit(dtype)
    slope = ref.act64(z.double(), act)[1]
    want = dy.double() * slope
    edz = 16 * ref.U32 * dy.double().abs()
    ref.check("dz", dz, (want, edz + u * (want.abs() + edz) + 1e-37))
    err = edz.sum(0) + (m + 2) * ref.U32 * want.abs().sum(0)
    ref.check("db", db, (want.sum(0), err + u * (want.sum(0).abs() + err) + 1e-37))
    exact = ref.linear64(x, w.t() if w_t else w, None, None, dz.cpu(), "none")   # of dz as it was stored
    ref.check("dx", dx, exact["dx"])
    ref.check("dw", dw.t() if w_t else dw, exact["dw"])


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
def test_linear_split_contraction_joins_to_its_value(muon, dtype):
    x, w, b, r = (normal(s, dtype, i, 0.1) for i, s in enumerate(((2, 16384), (16384, 64), (64,), (2, 64))))
    y = muon.linear(x.cuda(), w.cuda(), b.cuda(), activation="gelu", residual=r.cuda())
    ref.check("y", y, ref.linear64(x, w, b, r, None, "gelu")["y"])


# ------------------------------------------------------------------ streams and threads


def block_pass(muon, seed):
    """A routed block with its gradients, on the current stream."""
    t, top, e, h, n = 300, 2, 8, 64, 136
    g = torch.Generator().manual_seed(seed)
    ids = torch.randint(0, e, (t, top), generator=g).cuda()
    x = normal((t, h), BF16, seed).cuda().requires_grad_()
    w1, w2 = (normal(s, BF16, seed + i, 0.1).cuda().requires_grad_() for i, s in ((1, (e, h, n)), (2, (e, n, h))))
    p = torch.rand(t, top, generator=g).cuda().requires_grad_()
    dy = normal((t, h), BF16, seed + 3).cuda()

    def run():
        r = muon.route(ids, e)
        u = muon.expert_linear(muon.dispatch(x, r), w1, r.offsets, activation="silu")
        y = muon.combine(muon.expert_linear(u, w2, r.offsets), r, p, residual=x)
        y = muon.dropout(muon.linear(y, w1[0], activation="gelu") @ w1[0].detach().t(), 0.1, seed=seed)
        return (y, *torch.autograd.grad(y, (x, w1, w2, p), dy))
    return run


def test_two_streams_at_once(muon):
    """Passes on two streams, enqueued in turn without waiting, give what each gives alone."""
    passes = [block_pass(muon, s) for s in (1, 2)]
    want = [p() for p in passes]
    streams = [torch.cuda.Stream() for _ in passes]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(5):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(passes[i]())
    torch.cuda.synchronize()
    for i in range(2):
        for outs in got[i]:
            assert all(torch.equal(a, b) for a, b in zip(outs, want[i]))


def test_two_host_threads(muon):
    """Two threads, each with its own stream: values, and a refusal's message stays with its thread."""
    passes = [block_pass(muon, s) for s in (3, 4)]
    want = [p() for p in passes]
    torch.cuda.synchronize()
    got, failed = [[], []], []

    def work(i):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(5):
                    got[i].append(passes[i]())
                    with pytest.raises(muon.MuonError, match="experts outside" if i else "rounds to 1"):
                        if i:
                            muon.route(torch.zeros(2, 2, dtype=torch.int64, device="cuda"), 2000)
                        else:
                            muon.dropout_forward(torch.zeros(8, device="cuda"), 1 - 2.0 ** -20)
                torch.cuda.current_stream().synchronize()
        except BaseException as err:
            failed.append(err)
    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed, failed
    for i in range(2):
        for outs in got[i]:
            assert all(torch.equal(a, b) for a, b in zip(outs, want[i]))


def test_gradient_through_a_second_stream(muon):
    """The forward pass on a side stream, the gradient asked for from the first one, after it waits."""
    x, w = normal((256, 64), BF16, 1).cuda().requires_grad_(), normal((64, 128), BF16, 2).cuda().requires_grad_()
    dy = normal((256, 128), BF16, 3).cuda()
    want = torch.autograd.grad(muon.dropout(muon.linear(x, w, activation="silu"), 0.2, seed=1), (x, w), dy)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(5):
        with torch.cuda.stream(side):
            y = muon.dropout(muon.linear(x, w, activation="silu"), 0.2, seed=1)
        torch.cuda.current_stream().wait_stream(side)
        got = torch.autograd.grad(y, (x, w), dy)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
