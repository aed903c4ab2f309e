"""Host-side tests (no GPU) of the operators around a block's products where calls are unusual."""

from __future__ import annotations

import ctypes

import pytest
import torch

from test_block_host import A, Elsewhere, block, norm_desc, no_gpu  # noqa: F401 (block is a fixture)


@no_gpu
@pytest.mark.parametrize("cols", [8, 8192, 8193, 20000])
def test_a_norm_gradient_of_no_rows_launches_nothing_for_dx(block, cols):  # noqa: F811
    """dx has an address and no elements: a launch of no workgroups is an error of the runtime."""
    lib = block.load_block()
    d = norm_desc(block, rows=0, cols=cols)
    assert lib.muon_norm_backward(ctypes.byref(d), None, None, None, None, None, None, A, None, None, None, 0, None) == 0


def test_entries_that_32_bits_do_not_count_are_refused(block):  # noqa: F811
    """tokens * top at 2^31 and above, a list whose length is small in its low 32 bits among them."""
    import muon_newton_schulz_05_amd as muon
    z, one = Elsewhere(1, 8), Elsewhere(dtype=torch.float32)
    for top in (1 << 31, (1 << 32) + 2, 1 << 33):
        ids = Elsewhere(1, top, dtype=torch.int32)
        for call in (lambda: muon.balance_loss(z, ids), lambda: muon.balance_forward(z, ids),
                     lambda: muon.balance_backward(one, z, ids, Elsewhere(9))):
            with pytest.raises(ValueError, match="entries"):
                call()
    with pytest.raises(ValueError, match="entries"):
        muon.balance_loss(Elsewhere(1 << 28, 8), Elsewhere(1 << 28, 8, dtype=torch.int32))
