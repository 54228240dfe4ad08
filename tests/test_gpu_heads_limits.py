"""Norm and rotation of queries and keys on the GPU at the ends of what is declared, against the float64
reference.  Tolerances (derived): as in test_gpu_heads.py, u = 2^-24, where no other is given."""
import ctypes

import numpy as np
import pytest

from oracle import blocks as ob
from tests._blocks import DT, U, dev, f64, ints, near, same, torch
from tests.test_gpu_heads import check, problem

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def tpc():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import tensor_product_convolution_amd as m
    m.lib()
    return m


@pytest.mark.parametrize("code", [0, 1])
def test_no_rows_and_no_frequencies(tpc, code):
    """Through the C entry point: without rows there is nothing that freq would be read for."""
    from tensor_product_convolution_amd.blocks import _Heads
    gamma, pos = torch.ones(16, device="cuda"), torch.full((3,), 5.0, device="cuda")
    out = torch.full((2, 16), 7.0, device="cuda")
    h = _Heads(code, 4, 2, 16, 0, gamma.data_ptr(), gamma.data_ptr(), 1e-6, 0, 3, None, None, 8, 0)
    rows = [x for s in (64, 32) * 3 for x in (None, s)]
    assert tpc.lib().tp_head_norm_rotate_backward(ctypes.byref(h), *rows, out[0].data_ptr(), out[1].data_ptr(), pos.data_ptr(), None, 0,
                                                  torch.cuda.current_stream().cuda_stream) == 0
    torch.cuda.synchronize()
    assert (out == 0).all() and (pos == 5).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shape", [(1, 1, 1, 16, 8, 3, 0), (33, 4, 2, 16, 8, 3, 0), (130, 3, 5, 40, 12, 2, 0), (700, 5, 1, 24, 0, 0, 0)], ids=str)
def test_eps_zero(tpc, dtype, shape):
    """No head is zero, but the last turn of a workgroup has threads without a head."""
    s = problem(*shape[:6], dtype, True, 0)
    kw = dict(s["kw"], eps=0.0)
    want_pos = shape[4] > 0
    fwd = tpc.head_norm_rotate_forward(s["q"], s["k"], **kw)
    back = tpc.head_norm_rotate_backward(s["gq"], s["gk"], s["q"], s["k"], want_pos=want_pos, **kw)
    check(s, False, 0.0, dtype, fwd, back)
