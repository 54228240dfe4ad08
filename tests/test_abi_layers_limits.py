"""Sizes that one launch cannot cover are refused on the host, before a HIP call, so this
runs without a GPU."""
import ctypes
import os

import pytest

import tensor_product_convolution_amd as tpc

from .test_abi_layers import OVER, A, B, C, D, _desc

pytestmark = pytest.mark.skipif(not os.path.exists(tpc.LIB_PATH),
                                reason="libtpconv.so not built (run __graft_entry__.build())")

# more than 2^32 threads in the grid's first dimension, whichever workgroup is chosen
MANY = [dict(n_nodes=2_000_000_000, n_segments=60_000_000), dict(n_nodes=2_000_000_000, n_segments=66_000_000),
        dict(n_nodes=1_000, n_segments=70_000_000)]


@pytest.mark.parametrize("many", MANY, ids=str)
def test_attention_of_more_structures_than_a_launch_covers(many):
    d = ctypes.byref(_desc(**many))
    f = tpc.lib()
    assert f.tp_attn_forward(d, A, 64, A, 32, A, 32, B, 64, C, None) == OVER
    assert "too many" in f.tp_conv_last_error().decode()
    assert f.tp_attn_backward(d, A, 64, A, 32, A, 32, A, 64, C, A, 64, B, 64, B, 32, B, 32, D, D, 1 << 62, None) == OVER
