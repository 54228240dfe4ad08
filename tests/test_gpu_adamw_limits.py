"""The AdamW step on the GPU at the ends of what is declared, against the float64 reference.
Tolerances (derived): as in test_gpu_adamw.py, u = 2^-24, where no other is given."""
import numpy as np
import pytest

from oracle import blocks as ob
from tests._blocks import DT, U, dev, f64, near, same, torch
from tests.test_gpu_adamw import B1, B2, EPS, LR, check_step

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def tpc():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import tensor_product_convolution_amd as m
    m.lib()
    return m


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_bad_gradients_stay_with_their_parameters(tpc, bad, dtype):
    """8-bit states without max_norm: a bad gradient's moments begin anew, the block's other values know nothing of it."""
    r = np.random.default_rng(7)
    at = [3, 255, 256, 511, 512, 700]
    p, q = [dev(np.linspace(-1, 1, 1000)) for _ in range(2)]
    kw = dict(lr=LR, betas=(B1, B2), eps=EPS, weight_decay=0.1, bits=8, seed=3)
    a, b = tpc.AdamW([p], **kw), tpc.AdamW([q], **kw)
    keep = torch.ones(1000, dtype=torch.bool, device="cuda")
    keep[at] = False
    for step in range(4):
        g = dev(r.normal(size=1000), DT[dtype])
        g[512:768] = 0                     # a block of nothing but bad ones
        g[~keep] = 0
        h = g.clone()
        if step in (0, 2):
            g[~keep] = bad
        a.step([g])
        b.step([h])
        assert torch.equal(p[keep], q[keep]) and torch.isfinite(p[keep]).all() and torch.isnan(p[~keep]).all(), step
        assert same(a.state()[1:], b.state()[1:])
        assert all((m[:1000][~keep] == 0).all() for m in a.moments())

