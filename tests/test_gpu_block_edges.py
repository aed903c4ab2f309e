"""GPU tests of the operators around a block's products where calls are unusual."""

from __future__ import annotations

import pytest
import torch

from test_gpu_mx import both, muon, normal  # noqa: F401 (muon is a fixture)

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
