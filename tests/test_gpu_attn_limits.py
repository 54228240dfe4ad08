"""Attention at the ends of what its entry points accept: bucket ranges that pass the
largest float.

Tolerances are those derived in test_gpu_attn.py, whose cases these are.
"""
import numpy as np
import pytest

from .test_gpu_attn import Case, tpc  # noqa: F401  (tpc is the module's fixture)

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("r_min,steps,nb", [(1e10, 1, 64), (6.1e9, 1, 64), (1e15, 1, 64), (1e15, 1, 3), (5e14, 2, 64),
                                            (1e15, 4, 64), (1e15, 8, 20)])
def test_bucket_ranges_that_pass_the_largest_float(tpc, dtype, r_min, steps, nb):
    """Distances below the range, inside it and so large that their squares are infinite."""
    print(f"attn bucket range {dtype} {r_min} {steps} {nb}", flush=True)
    c = Case(dtype, [75, 40], 2, 2, 16, nb=nb, steps=steps, r_min=r_min, masked=0.1)
    r = np.random.default_rng(5)
    far = 10.0 ** r.uniform(0, 20, size=(115, 1)) * r.normal(size=(115, 3))
    c.kw["pos"] = torch.tensor(far.astype(np.float32), device="cuda")
    c.check(tpc)
