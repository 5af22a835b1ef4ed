"""Workspace of the 4-bit product by the height of its tiles, on the CPU.  Matrices of fewer
than 193 rows take tiles of at most 128 rows of A: a taller tile's loads of B add up to 192
rows to a scalar offset, which may not pass the resource.  One counter per XCD is
needed as soon as there may be more tiles than 256 workgroups."""
import os

import pytest

import fp8_block_scaled_sigmoid_amd as moe


@pytest.fixture(scope="module")
def need():
    if not os.path.exists(moe.LIB_PATH):
        pytest.fail("libmoe_fp8.so is not built (run __graft_entry__.build())")
    return moe.moe_grouped_gemm_mxfp4_workspace_bytes


@pytest.mark.parametrize("n,rows_a_tile", [(1, 128), (64, 128), (192, 128), (193, 256), (256, 256)])
def test_tiles_of_narrow_matrices(need, n, rows_a_tile):
    """One group: rows / height + 1 tiles at most."""
    last = 256 * rows_a_tile - 1
    assert need(1, last, n, 512) == 0
    assert need(1, last + 1, n, 512) > 0


def test_a_large_batch_needs_a_workspace(need):
    """33 groups of together 16384 rows: more tiles than workgroups."""
    import ctypes
    a = moe.GemmMxfp4Args()
    fields = dict(a_q=16, lda=3584, a_e=16, lde=224, a_rows=16384, b_q=16, b_e=16, group_offsets=16, num_groups=33,
                  total_rows=16384, n_out=4096, k_dim=7168, epilogue=0, out=16, ldo=4096)
    for f, v in fields.items():
        setattr(a, f, v)
    size = need(33, 16384, 4096, 7168)
    assert size > 0
    call = moe.lib().moe_grouped_gemm_mxfp4
    assert call(ctypes.byref(a), None, 0, None) == 4
    assert call(ctypes.byref(a), 16, size - 1, None) == 4
    assert call(ctypes.byref(a), 24, size, None) == 3
