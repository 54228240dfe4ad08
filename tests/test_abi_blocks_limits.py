"""Workspaces of the products by group and the optimiser's sizes at the ends of what is declared: host arithmetic,
no GPU."""
import ctypes
import os

import pytest

import tensor_product_convolution_amd as tpc
from tests.test_abi_blocks import BF16, F32, _grouped

pytestmark = pytest.mark.skipif(not os.path.exists(tpc.LIB_PATH),
                                reason="libtpconv.so not built (run __graft_entry__.build())")


def need(want_x, want_w, **kw):
    n = ctypes.c_size_t()
    assert tpc.lib().tp_grouped_linear_workspace(ctypes.byref(_grouped(**kw)), want_x, want_w, ctypes.byref(n)) == 0
    return n.value


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_parts_of_a_source_row_are_float32(dtype):
    assert need(1, 0, dtype=dtype, fan=2) == 4096 * 16 * 4
    assert need(1, 0, dtype=dtype, fan=1) == 0
    assert need(1, 0, dtype=dtype, fan=2, n_slots=6, n_in=3) == 6 * 3 * 4 + 8          # whole 16 bytes


def test_workspace_of_the_most_slots():
    """Two places for each run of a part's length, whatever the slots are divided into."""
    n, row = 2 ** 31 - 5000, (16 * 8 + 8) * 4
    w = need(0, 1, dtype=BF16, n_slots=n, n_groups=1)
    assert w % (2 * row) == 0 and 0 < w < 2 * row * 1000
    assert need(0, 1, dtype=BF16, n_slots=0) == 0
