"""GPU tests of the operators around a block's products where calls are unusual."""

from __future__ import annotations

import ctypes

import pytest
import torch

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
