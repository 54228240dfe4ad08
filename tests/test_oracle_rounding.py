"""The moments of test_gpu_adamw_limits.py that move by less than half a code a step, in the float64 reference: rounded
at random they arrive, to nearest they stay behind, by far more than that test allows.  No GPU."""
import numpy as np
import pytest

pytest.importorskip("torch")
from oracle import blocks as ob  # noqa: E402
from tests.test_gpu_adamw_limits import SPREAD, mean_of_200_steps, slow_moments  # noqa: E402
from tests.test_gpu_adamw import B1, B2  # noqa: E402


def means(rounding):
    c, start = slow_moments()
    held = list(start)

    def step(i):
        m, v = ob.decode(held[0], held[1], False), ob.decode(held[2], held[3], True)
        a, b = rounding(len(c))
        held[:] = (*ob.encode(B1 * m + (1 - B1) * c, False, a), *ob.encode(B2 * v + (1 - B2) * c * c, True, b))
        return ob.decode(held[0], held[1], False), ob.decode(held[2], held[3], True)

    return np.abs(mean_of_200_steps(c, start, step))


def test_rounded_at_random_they_arrive():
    r = np.random.default_rng(1)
    off = means(lambda n: r.integers(0, 65536, size=(2, n)) / 65536)
    assert off[0] < SPREAD[0] and off[1] < SPREAD[1]


@pytest.mark.parametrize("u", [0.0, 0.5])
def test_rounded_to_nearest_or_down_they_stay_behind(u):
    off = means(lambda n: (u, u))
    assert off[0] > 0.2 > 30 * SPREAD[0] and off[1] > 0.3 > 9 * SPREAD[1]
