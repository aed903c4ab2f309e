"""Host-side tests (no GPU) of the operators around a block's products where calls are unusual."""

from __future__ import annotations

import ctypes

import pytest

from test_block_host import A, block, norm_desc, no_gpu  # noqa: F401 (block is a fixture)


@no_gpu
@pytest.mark.parametrize("cols", [8, 8192, 8193, 20000])
def test_a_norm_gradient_of_no_rows_launches_nothing_for_dx(block, cols):  # noqa: F811
    """dx has an address and no elements: a launch of no workgroups is an error of the runtime."""
    lib = block.load_block()
    d = norm_desc(block, rows=0, cols=cols)
    assert lib.muon_norm_backward(ctypes.byref(d), None, None, None, None, None, None, A, None, None, None, 0, None) == 0
