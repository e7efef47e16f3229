"""Rows of a product need source rows to come from: none is a shape that every
form of the product refuses, on the host (the addresses below are never
dereferenced)."""
import ctypes

import pytest

A = 1 << 20
MB = 1 << 20


@pytest.fixture(scope="module")
def smoe():
    import __graft_entry__
    __graft_entry__.build_library()
    import moe_expert_ffn_smoe_gb300 as m
    return m


@pytest.mark.parametrize("rows,n_in", [(1, 256), (2, 256), (128, 256), (128, 0)])  # dots, tensor cores, no columns
def test_no_source_rows_are_refused(smoe, rows, n_in):
    L = smoe._lib
    assert L.smoe_experts_matmul_q8_workspace_bytes(0, rows, 8, 96, n_in) == ctypes.c_size_t(-1).value
    for order in (A + 2 * MB, None):
        assert L.smoe_experts_matmul_q8(A, A + MB, 0, order, 8, A + 3 * MB, rows, 8, A + 4 * MB, A + 5 * MB, 96, n_in, A + 6 * MB,
                                        0, A + 7 * MB, MB, None) == smoe.SMOE_ERR_SHAPE
    # no rows need none
    assert L.smoe_experts_matmul_q8_workspace_bytes(0, 0, 8, 96, n_in) == 0
    assert L.smoe_experts_matmul_q8(None, None, 0, None, 8, None, 0, 8, None, None, 96, n_in, None, 0, None, 0,
                                    None) == smoe.SMOE_OK
