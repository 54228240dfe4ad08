"""Norm and rotation of queries and keys on the GPU at the ends of what is declared, against the float64
reference.  Tolerances (derived): as in test_gpu_heads.py, u = 2^-24, where no other is given."""
import ctypes

import numpy as np
import pytest

from oracle import blocks as ob
from tests._blocks import U, f64, torch
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


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("bad", [float("inf"), float("nan")])
def test_a_bad_value_that_does_not_turn_stays_alone(tpc, dtype, interleaved, norm, bad):
    """Values behind the turned pairs reach neither each other nor the positions' gradient, but for the
    norm of their head."""
    s = problem(40, 3, 2, 40, 11, 2, dtype, norm, 0)
    kw = dict(s["kw"], interleaved=interleaved)
    run = lambda: tpc.head_norm_rotate_forward(s["q"], s["k"], **kw)
    back = lambda: tpc.head_norm_rotate_backward(s["gq"], s["gk"], s["q"], s["k"], want_pos=True, **kw)
    clean, clean_back = run(), back()
    s["gq"][7, 1, 33], s["gk"][9, 0, 22] = bad, bad
    got = back()
    assert torch.equal(got[4], clean_back[4])
    if norm:
        for g, c, at in ((got[2], clean_back[2], 33), (got[3], clean_back[3], 22)):
            keep = torch.arange(40, device="cuda") != at
            assert torch.equal(g[keep], c[keep]) and not torch.isfinite(g[at])
    else:
        for g, c, at in ((got[0], clean_back[0], (7, 1, 33)), (got[1], clean_back[1], (9, 0, 22))):
            want = c.clone()
            want[at] = bad
            assert torch.equal(g.nan_to_num(nan=5e30, posinf=6e30), want.nan_to_num(nan=5e30, posinf=6e30))
    s["q"][4, 2, 30], s["k"][5, 1, 39] = bad, bad
    for g, c, at in zip(run(), clean, ((4, 2, 30), (5, 1, 39))):
        want = c.clone()
        if norm:                           # 1 / sqrt of infinity is 0
            want[at[:2]] = 0 if bad == float("inf") else float("nan")
            want[at] = float("nan")
        else:
            want[at] = bad
        assert torch.equal(g.nan_to_num(nan=5e30, posinf=6e30), want.nan_to_num(nan=5e30, posinf=6e30))


@pytest.mark.parametrize("interleaved", [False, True])
def test_small_sines_and_cosines(tpc, interleaved):
    """Angles within 1.3e-3 of half and quarter turns, where a sine or cosine is small: an angle rounded to
    float32 behind its whole turns would leave it 1e-7 off.

    Tolerance (derived): sine and cosine of the rounded angle to 4 units in the last place (8 u), the
    correction for its rounding and the sum two more: 16 u of each; the angle in 64 bits is off by 3 2^-53 of the
    turns before it, at most 1,000: 2 pi 1,000 3 2^-53 = 2.1e-12."""
    r = np.random.default_rng(4)
    n = 120
    part = np.repeat([0.5, 0.25, -0.25, 0.0], n // 4) + r.uniform(-2e-4, 2e-4, size=n)
    turns = np.where(np.arange(n) % 2, r.integers(-1000, 1000, size=n), 0) + part
    freq = torch.tensor(2 * np.pi * turns[:, None], device="cuda")
    x = torch.zeros(1, 1, 2 * n, device="cuda")
    a, b = ob.pair_places(n, interleaved)
    x[..., torch.as_tensor(a)] = 1.0
    pos = torch.ones(1, 1, device="cuda")
    out = f64(tpc.head_norm_rotate_forward(x, x.clone(), pos=pos, freq=freq, interleaved=interleaved)[0])[0, 0]
    t = f64(freq)[:, 0]
    for got, want in ((out[a], np.cos(t)), (out[b], np.sin(t))):
        assert (np.abs(got - want) <= 16 * U * np.abs(want) + 2.1e-12).all(), np.abs(got - want).max()
