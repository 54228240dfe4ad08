"""Helpers of the GPU tests of the operators around the attention block."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
U, W = 2.0 ** -24, 2.0 ** -8          # half a step of float32 and bfloat16, relative
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def dev(a, dt=torch.float32):
    return torch.tensor(np.asarray(a), device="cuda").to(dt)


def ints(a):
    return torch.tensor(np.asarray(a), dtype=torch.int32, device="cuda")


def f64(t):
    return t.double().cpu().numpy()


def near(got, ref, bound, name, dtype="f32"):
    """|got - ref| within bound (float32 arithmetic) and the output's one rounding."""
    got = f64(got)
    assert got.shape == ref.shape, name
    # the rounding is of a value that is itself off by the bound
    over = np.abs(got - ref) - (bound * (1 + 2 * W) + (W if dtype == "bf16" else 2 * U) * np.abs(ref) + 1e-37)
    assert over.size == 0 or not (over.max() > 0 or np.isnan(got).any()), (name, float(over.max()))


def same(a, b):
    return all((x is None and y is None) or torch.equal(x, y) for x, y in zip(a, b))
