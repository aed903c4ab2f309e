"""GPU tests of the layers in four bits against plain float64 forms (tests/block_reference.py)."""

from __future__ import annotations

import itertools

import pytest
import torch

import block_reference as ref
import ops_reference

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


def held(codes):
    """values [slices, N, 64] from codes [N, padded K], the lower half of a byte first."""
    n = codes.shape[0]
    full = torch.zeros(n, -(-codes.shape[1] // 128) * 128, dtype=torch.int64)
    full[:, :codes.shape[1]] = codes
    return (full[:, ::2] | full[:, 1::2] << 4).to(torch.uint8).view(n, -1, 64).transpose(0, 1)


def placed(scales, k):
    """scales [chunks, N, 16] from [N, blocks]: byte 4 g + s is that of the 32 values g of slice s of 512."""
    n, nb = scales.shape
    out = torch.zeros(-(-k // 512), n, 16, dtype=torch.uint8)
    for b in range(nb):
        out[b // 16, :, 4 * (b % 4) + b // 4 % 4] = scales[:, b].to(torch.uint8)
    return out


SHAPES = [(1, 1), (5, 3), (31, 9), (32, 8), (33, 130), (64, 64), (100, 17), (255, 40), (256, 7), (257, 300), (520, 33),
          (1001, 129)]


@both
@pytest.mark.parametrize("w_t", [False, True], ids=["kn", "nk"])
@pytest.mark.parametrize("k,n", SHAPES)
def test_quantize_bits(muon, k, n, w_t, dtype):
    """Every bit of the form, what pads it included, and the values that come back."""
    w = normal((k, n), dtype, k + n, 2.0) * torch.exp2(torch.randint(-30, 30, (k, 1), generator=torch.Generator().manual_seed(n)))
    w = w.to(dtype)
    values, codes, scales = ref.blocks64(w.t())
    g = w.t().contiguous().cuda().t() if w_t else w.cuda()
    q = muon.mx_quantize(g)
    assert q.k == k and q.shape == (k, n)
    assert torch.equal(q.values.cpu(), held(codes)) and torch.equal(q.scales.cpu(), placed(scales, k))
    for out in (BF16, F32):
        back = muon.mx_dequantize(q, out)
        assert back.dtype is out and back.shape == (k, n) and torch.equal(back.double().cpu(), values.t())
    # and again: what four bits hold, they hold
    assert torch.equal(muon.mx_quantize(muon.mx_dequantize(q)).values, q.values) or not values.ne(0).any()


@both
def test_quantize_borders_and_extremes(muon, dtype):
    """Every border between levels and its neighbours, at scales over the type's whole range, subnormal values,
    saturation, and blocks with infinities or NaN."""
    a = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, 7.0, 7.9])
    near = torch.cat([a, torch.nextafter(a, torch.tensor(0.0)), torch.nextafter(a, torch.tensor(9.0))]).to(dtype).float()
    near[near >= 8] = 7.5
    block = torch.cat([near, torch.tensor([4.0, -0.0])])
    block[::3] *= -1
    exps = list(range(-146, 126, 7)) + [-130, -129, -128, -127, -126, -125, -124, 124, 125]
    rows = [torch.ldexp(block.double(), torch.tensor(e)).float() for e in exps]
    bad = [torch.ones(32), torch.ones(32), torch.ones(32), torch.zeros(32), -torch.zeros(32), torch.full((32,), 2.0 ** -149)]
    bad[0][5], bad[1][31], bad[2][0] = INF, NAN, -INF
    v = torch.stack(rows + bad).to(dtype)
    if dtype is BF16:
        v[-1] = 2.0 ** -133                                     # its least value
    values, codes, scales = ref.blocks64(v)
    for g in (v.cuda().t(), v.cuda().t().contiguous()):
        q = muon.mx_quantize(g)
        assert torch.equal(q.scales.cpu(), placed(scales, 32))
        ok = scales[:, 0] != 255
        assert torch.equal(q.values.cpu()[:, ok], held(codes)[:, ok])
        back = muon.mx_dequantize(q, dtype).double().cpu().t()
        assert torch.equal(back[ok], values[ok]) and back[~ok].isnan().all()


@both
@pytest.mark.parametrize("w_t", [False, True], ids=["kn", "nk"])
def test_quantize_experts_and_strides(muon, w_t, dtype):
    """A 3-D weight and views with their own strides, at any element alignment."""
    big = normal((3, 90, 150), dtype, 1)
    for k0, n0 in ((0, 0), (3, 5)):
        w = big[:, k0:k0 + 70, n0:n0 + 44]
        g = big.transpose(1, 2).contiguous().cuda().transpose(1, 2)[:, k0:k0 + 70, n0:n0 + 44] if w_t else \
            big.cuda()[:, k0:k0 + 70, n0:n0 + 44]
        q = muon.mx_quantize(g)
        back = muon.mx_dequantize(q).double().cpu()
        for i in range(3):
            assert torch.equal(back[i], ref.fast_blocks64(w[i].t()).t())
            alone = muon.mx_quantize(g[i])
            assert torch.equal(alone.values, q.values[i]) and torch.equal(alone.scales, q.scales[i])
    neither = big.cuda()[0, ::2, ::3]                            # no contiguous dimension: copied
    assert torch.equal(muon.mx_dequantize(muon.mx_quantize(neither)).double().cpu(), ref.fast_blocks64(big[0, ::2, ::3].t()).t())


def run_linear(muon, m, k, n, dtype, act, bias, residual, seed=0):
    x, w = normal((m, k), dtype, seed, 1.5), normal((k, n), dtype, seed + 1, k ** -0.5)
    b = normal((n,), dtype, seed + 2) if bias else None
    r = normal((m, n), dtype, seed + 3) if residual else None
    # The values in four bits are exact in either type.
    xq, wq = ref.fast_blocks64(x).to(dtype), ref.fast_blocks64(w.t()).t().to(dtype)
    want = ops_reference.linear64(xq, wq, b, r, None, act)
    q = muon.mx_quantize(w.cuda())
    y = muon.mx_linear(x.cuda(), q, None if b is None else b.cuda(), activation=act, residual=None if r is None else r.cuda())
    ops_reference.check("y", y, want["y"])
    return y


@both
@pytest.mark.parametrize("m,k,n", [(1, 1, 1), (1, 32, 8), (3, 7, 5), (31, 64, 32), (33, 65, 129), (64, 24, 640), (128, 256, 128),
                                   (257, 129, 260), (300, 520, 264), (1, 4096, 520), (5, 2048, 96), (2, 4100, 33),
                                   (1, 16384, 200), (17, 9000, 100), (200, 8192, 130)])
def test_linear_shapes(muon, m, k, n, dtype):
    run_linear(muon, m, k, n, dtype, "none", True, False, m + n)
    run_linear(muon, m, k, n, dtype, "gelu", False, True, m + n + 10)


@both
@pytest.mark.parametrize("act", ["none", "relu", "silu", "gelu", "gelu_tanh"])
def test_linear_activations(muon, act, dtype):
    run_linear(muon, 136, 192, 328, dtype, act, True, True)


@pytest.mark.parametrize("m,k,n", [(4096, 72, 4096), (4100, 600, 4104), (2040, 1030, 4096), (1000, 520, 2000), (4096, 8192, 1030),
                                   (1100, 49152, 2300)])
def test_linear_tiles(muon, m, k, n):
    """Shapes that take each tile, whole and ragged, and split contractions; on the GPU's own float64 products."""
    x, w = normal((m, k), BF16, 1).cuda(), normal((k, n), BF16, 2, k ** -0.5).cuda()
    q = muon.mx_quantize(w)
    xq = muon.mx_dequantize(muon.mx_quantize(x.t())).t().double()        # checked bit by bit above
    wq = muon.mx_dequantize(q).double()
    b = normal((n,), BF16, 3).cuda()
    y = muon.mx_linear(x, q, b)
    z, size = xq @ wq + b.double(), xq.abs() @ wq.abs() + b.double().abs()
    tol = (k + 4) * ops_reference.U32 * size + 2.0 ** -8 * z.abs() + 1e-37
    assert ((y.double() - z).abs() <= tol).all()
    off = (y.double() - z).norm() / z.norm()
    assert off <= 2.0 ** -8


def test_linear_past_the_workspace_of_a_sum(muon):
    """The partial sums of a split contraction are added in order: the same bits every time."""
    x, q = normal((4, 32768), BF16, 1).cuda(), muon.mx_quantize(normal((32768, 96), BF16, 2, 0.01).cuda())
    y = muon.mx_linear(x, q)
    for _ in range(5):
        assert torch.equal(muon.mx_linear(x, q), y)


@both
def test_linear_strided_rows_and_leading_dims(muon, dtype):
    big = normal((6, 10, 80), dtype, 1)
    x = big[:, ::2, 9:73]
    w = normal((64, 48), dtype, 2, 0.1)
    r = normal((6, 5, 64), dtype, 3)[..., 8:56]
    xq, wq = ref.fast_blocks64(x.reshape(30, 64)).to(dtype), ref.fast_blocks64(w.t()).t().to(dtype)
    want = ops_reference.linear64(xq, wq, None, r.reshape(30, 48), None, "silu")
    y = muon.mx_linear(big.cuda()[:, ::2, 9:73], muon.mx_quantize(w.cuda()), activation="silu",
                       residual=normal((6, 5, 64), dtype, 3).cuda()[..., 8:56])
    assert y.shape == (6, 5, 48)
    ops_reference.check("y", y.reshape(30, 48), want["y"])


@both
@pytest.mark.parametrize("counts", [[5], [0, 7, 0], [1, 2, 3, 4], [33, 0, 130, 1, 64], [0, 0], [300, 5], [700, 0, 900, 650]], ids=str)
@pytest.mark.parametrize("tail", [0, 9])
def test_experts(muon, counts, tail, dtype):
    """Empty and ragged groups, rows past the last one (zeros, whatever they hold), bias and activation."""
    e, k, n = len(counts), 200, 264
    offsets = torch.tensor([0, *itertools.accumulate(counts)], dtype=torch.int32)
    rows = int(offsets[-1]) + tail
    x, w, b = normal((rows, k), dtype, 1), normal((e, k, n), dtype, 2, k ** -0.5), normal((e, n), dtype, 3)
    x[int(offsets[-1]):] = NAN
    y = muon.mx_expert_linear(x.cuda(), muon.mx_quantize(w.cuda()), offsets.cuda(), b.cuda(), activation="silu")
    for i in range(e):
        lo, hi = offsets[i], offsets[i + 1]
        xq, wq = ref.fast_blocks64(x[lo:hi]).to(dtype), ref.fast_blocks64(w[i].t()).t().to(dtype)
        ops_reference.check(i, y[lo:hi], ops_reference.linear64(xq, wq, b[i], None, None, "silu")["y"])
    assert torch.equal(y[int(offsets[-1]):].cpu(), torch.zeros(tail, n, dtype=dtype))


def test_experts_of_many_rows(muon):
    """Groups that fill the large tiles, against each expert's rows alone."""
    counts = [1500, 0, 2100, 900, 3, 1800]
    offsets = torch.tensor([0, *itertools.accumulate(counts)], dtype=torch.int32).cuda()
    x, w = normal((int(offsets[-1]), 712), BF16, 1).cuda(), normal((6, 712, 2056), BF16, 2, 0.04).cuda()
    q = muon.mx_quantize(w)
    y = muon.mx_expert_linear(x, q, offsets)
    for i in range(6):
        lo, hi = int(offsets[i]), int(offsets[i + 1])
        alone = muon.mx_linear(x[lo:hi], muon.MxWeight(q.values[i], q.scales[i], q.k)).double()
        off = (y[lo:hi].double() - alone).abs()
        # two float32 sums of 712 products in any order, then one rounding each
        assert (off <= 2.0 ** -7 * alone.abs() + 1e-3).all()


def test_what_is_not_finite_stays_in_its_row_or_column(muon):
    x, w = normal((70, 300), F32, 1), normal((300, 90), F32, 2, 0.06)
    clean = muon.mx_linear(x.cuda(), muon.mx_quantize(w.cuda()))
    x[3, 299], x[40, 0], w[17, 5], w[299, 88] = NAN, INF, NAN, -INF
    y = muon.mx_linear(x.cuda(), muon.mx_quantize(w.cuda()))
    rows, cols = [3, 40], [5, 88]
    assert y[rows].isnan().all() and y[:, cols].isnan().all()
    keep_r, keep_c = [i for i in range(70) if i not in rows], [j for j in range(90) if j not in cols]
    assert torch.equal(y[keep_r][:, keep_c], clean[keep_r][:, keep_c])


@both
def test_sizes_of_zero(muon, dtype):
    q = muon.mx_quantize(normal((64, 48), dtype, 1).cuda())
    assert muon.mx_linear(torch.empty(0, 64, dtype=dtype, device="cuda"), q).shape == (0, 48)
    none = muon.mx_quantize(torch.empty(64, 0, dtype=dtype, device="cuda"))
    assert muon.mx_linear(torch.zeros(3, 64, dtype=dtype, device="cuda"), none).shape == (3, 0)
    empty = muon.mx_quantize(torch.empty(0, 48, dtype=dtype, device="cuda"))
    b = normal((48,), dtype, 2).cuda()
    y = muon.mx_linear(torch.empty(3, 0, dtype=dtype, device="cuda"), empty, b)
    assert torch.equal(y, b.expand(3, 48)) and muon.mx_dequantize(empty).shape == (0, 48)


def test_one_weight_serves_both_types(muon):
    """A weight quantised from float32 takes bfloat16 rows, and the other way round."""
    w = normal((96, 40), BF16, 1)
    a, b = muon.mx_quantize(w.cuda()), muon.mx_quantize(w.float().cuda())
    assert torch.equal(a.values, b.values) and torch.equal(a.scales, b.scales)
    x = normal((9, 96), BF16, 2).cuda()
    y = muon.mx_linear(x, a)
    assert torch.equal(y, muon.mx_linear(x.float(), a).to(BF16))


def test_past_32_bit_offsets(muon):
    """Rows, experts and outputs more than 2^32 elements apart."""
    flat = torch.zeros((1 << 32) + (1 << 23), dtype=BF16, device="cuda")
    x = flat.as_strided((4097, 300), (1 << 20, 1))
    x[-2:] = normal((2, 300), BF16, 1).cuda()
    q = muon.mx_quantize(normal((300, 64), BF16, 2).cuda())
    assert torch.equal(muon.mx_linear(x, q)[-2:], muon.mx_linear(x[-2:].contiguous(), q))
    w = flat.as_strided((3, 300, 70), (1 << 31, 4096, 1))
    w[2] = normal((300, 70), BF16, 3).cuda()
    far, near = muon.mx_quantize(w), muon.mx_quantize(w[2].contiguous())
    assert torch.equal(far.values[2], near.values) and torch.equal(far.scales[2], near.scales)
    w = flat.as_strided((4097, 40), (1 << 20, 1))
    w[-40:] = normal((40, 40), BF16, 4).cuda()
    assert torch.equal(muon.mx_quantize(w).values, muon.mx_quantize(w.contiguous()).values)
    rows, n = 70000, 65600                                        # an output of 4.6e9 elements
    x, q = normal((rows, 64), BF16, 5).cuda(), muon.mx_quantize(normal((64, n), BF16, 6, 0.1).cuda())
    y = muon.mx_linear(x, q)
    at = torch.tensor([0, 65535, 65536, rows - 1], device="cuda")
    want = (muon.mx_dequantize(muon.mx_quantize(x[at].t())).t().double() @ muon.mx_dequantize(q).double())
    assert ((y[at].double() - want).abs() <= 2.0 ** -8 * want.abs() + 1e-4).all()


@both
@pytest.mark.parametrize("k", [70, 2600])
@pytest.mark.parametrize("counts", [[3, 0, 9, 1], [10, 3, 20, 0, 17], [40, 9, 16]], ids=str)
def test_experts_of_few_rows(muon, counts, k, dtype):
    """Rows that are taken to four bits by the product or ahead of it, short and long contractions, columns of each width."""
    e = len(counts)
    offsets = torch.tensor([0, *itertools.accumulate(counts)], dtype=torch.int32)
    for n in (24, 1030):
        x, w = normal((int(offsets[-1]) + 2, k), dtype, 1), normal((e, k, n), dtype, 2, k ** -0.5)
        y = muon.mx_expert_linear(x.cuda(), muon.mx_quantize(w.cuda()), offsets.cuda())
        for i in range(e):
            lo, hi = offsets[i], offsets[i + 1]
            xq, wq = ref.fast_blocks64(x[lo:hi]).to(dtype), ref.fast_blocks64(w[i].t()).t().to(dtype)
            ops_reference.check(i, y[lo:hi], ops_reference.linear64(xq, wq, None, None, None, "none")["y"])
        assert torch.equal(y[-2:].cpu(), torch.zeros(2, n, dtype=dtype))


@both
@pytest.mark.parametrize("m", [4, 5, 16, 17, 32, 33])
def test_rows_at_the_borders_of_the_rules(muon, m, dtype):
    """Neighbouring row counts take different kernels: each row's result is the same sum in another order."""
    x, w = normal((40, 1100), dtype, 1), normal((1100, 96), dtype, 2, 0.03)
    q = muon.mx_quantize(w.cuda())
    xq, wq = ref.fast_blocks64(x[:m]).to(dtype), ref.fast_blocks64(w.t()).t().to(dtype)
    ops_reference.check("y", muon.mx_linear(x[:m].cuda(), q), ops_reference.linear64(xq, wq, None, None, None, "none")["y"])


def test_offsets_that_do_not_ascend_stay_in_bounds(muon):
    """Offsets against the rules give unspecified values, and read and write nothing outside the tensors."""
    x, q = normal((700, 200), BF16, 1).cuda(), muon.mx_quantize(normal((3, 200, 72), BF16, 2).cuda())
    for rows in (8, 40, 700):
        for off in ([0, 600, 100, 700], [5, 5, 5, 5], [0, -9, 1 << 30, 4], [0, 700, 700, 0]):
            y = muon.mx_expert_linear(x[:rows], q, torch.tensor(off, dtype=torch.int32).cuda())
            torch.cuda.synchronize()
            assert y.shape == (rows, 72)
