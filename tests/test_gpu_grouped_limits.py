"""Products by group on the GPU at the ends of what is declared: groups in front that no slot chooses, no
slots at all, against the float64 reference.

Tolerances (derived): as in test_gpu_grouped.py, u = 2^-24: a float32 sum of K products is off by at
most (K + 16) u of the sum of their absolute values; bfloat16 outputs add one rounding.
"""
import numpy as np
import pytest

from oracle import blocks as ob
from tests._blocks import DT, U, dev, f64, ints, near, same, torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def tpc():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import tensor_product_convolution_amd as m
    m.lib()
    return m


# slots, groups, in, out: weight gradients in tiles of 64, 64 in parts, 128 and (bfloat16) 256, and rows of any alignment
SHAPES = [(300, 5, 64, 72), (3000, 3, 136, 64), (4096, 3, 512, 512), (600, 64, 512, 520), (130, 4, 33, 65),
          (0, 5, 64, 72), (0, 256, 136, 136), (0, 3, 33, 65)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("kind", ["last", "upper", "none"])
def test_groups_in_front_without_slots(tpc, kind, shape, dtype):
    slots, groups, i, o = shape
    r = np.random.default_rng(slots + groups)
    low = {"last": groups - 1, "upper": groups // 2, "none": groups}[kind]
    index = r.integers(low, groups + 1, size=slots) if kind == "none" else r.integers(low, groups, size=slots)
    dt = DT[dtype]
    x, w, gz = dev(r.normal(size=(slots, i)), dt), dev(r.normal(size=(groups, i, o)), dt), dev(r.normal(size=(slots, o)), dt)
    g = tpc.group_rows(ints(index), groups)
    ptr, rows = ob.group_rows(index, groups)
    for x_rows, y_rows in (("source", "source"), ("grouped", "source"), ("source", "grouped")):
        print(f"groups in front {kind} {dtype} {shape} {x_rows} {y_rows}", flush=True)
        order = dict(x_rows=x_rows, y_rows=y_rows)
        back = tpc.grouped_linear_backward(gz, x, w, g, want_bias=True, **order)
        want = ob.grouped_backward(f64(gz), f64(x), f64(w), ptr, rows, 1, x_rows, y_rows)
        size = ob.grouped_backward(np.abs(f64(gz)), np.abs(f64(x)), np.abs(f64(w)), ptr, rows, 1, x_rows, y_rows)
        for got, ref, s, k, name in zip(back, want, size, (o, slots, slots), ("grad_x", "grad_w", "grad_bias")):
            near(got, ref, (k + 16) * U * s, name, dtype)
        assert (back[1][:min(low, groups)] == 0).all() and (back[2][:min(low, groups)] == 0).all()
        assert same(back, tpc.grouped_linear_backward(gz, x, w, g, want_bias=True, **order))


def test_an_infinity_behind_groups_without_slots(tpc):
    """The second pass for infinite operands, next to groups that have nothing to pass over."""
    r = np.random.default_rng(3)
    x, gz = dev(r.normal(size=(200, 64))), dev(r.random(size=(200, 64)) + 0.5)
    g = tpc.group_rows(ints(np.where(np.arange(200) < 150, 2, 3)), 4)
    w = dev(np.zeros((4, 64, 64)))
    clean = tpc.grouped_linear_backward(gz, x, w, g, want_x=False)[1]
    x[7, 5] = float("inf")
    bad = tpc.grouped_linear_backward(gz, x, w, g, want_x=False)[1]
    assert (bad[:2] == 0).all() and torch.equal(bad[3], clean[3]) and (bad[2, 5] == float("inf")).all()
    keep = torch.ones(64, dtype=torch.bool, device="cuda")
    keep[5] = False
    near(bad[2, keep], f64(clean[2, keep]), (200 + 16) * U * 150 * 8, "rows without it")


def test_combine_of_the_longest_rows(tpc):
    """The place behind a row's last chunk passes 2^31.  Only the last columns hold gradients, small whole
    numbers, so that their sum is exact."""
    c = 2 ** 31 - 1
    y = torch.ones(1, c, device="cuda", dtype=torch.bfloat16)
    y[0, -3000:] = torch.arange(3000, device="cuda").remainder(5).bfloat16()
    assert torch.equal(tpc.combine_forward(y, dev([[1.0]])), y)
    go = torch.zeros_like(y)
    go[0, -3000:] = torch.arange(3000, device="cuda").remainder(3).bfloat16()
    gy, gw = tpc.combine_backward(go, y, dev([[2.0]]))
    assert torch.equal(gy[0, -5000:], 2 * go[0, -5000:]) and not gy[0, :5000].any()
    assert float(gw) == float((go[0, -3000:].float() * y[0, -3000:].float()).sum())


def test_weight_gradient_of_the_most_slots(tpc):
    """A group of nearly 2^31 slots, whose parts end past 2^31.  Only the first and last slots hold gradients;
    the sums are whole numbers that bfloat16 holds."""
    n, fan = 2 ** 31 - 5000, 8
    g = tpc.group_rows(torch.zeros(n // fan, fan, dtype=torch.int32, device="cuda"), 1)
    assert g.ptr.tolist() == [0, n] and int(g.rows[-1]) == n - 1
    x, w = torch.ones(n // fan, 8, device="cuda", dtype=torch.bfloat16), torch.ones(1, 8, 8, device="cuda", dtype=torch.bfloat16)
    gz = torch.zeros(n, 8, device="cuda", dtype=torch.bfloat16)
    gz[:64], gz[-4000:] = 1, 1
    x[-500:, 3] = 2
    _, gw, gb = tpc.grouped_linear_backward(gz, x, w, g, want_x=False, want_bias=True)
    want = torch.full((1, 8, 8), 4064.0, device="cuda")
    want[:, 3] = 8064
    assert torch.equal(gw.float(), want) and (gb == 4064).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("case", [(600, 5, 64, 72, 2), (3000, 7, 136, 512, 3), (4096, 4, 33, 65, 16), (64, 32, 128, 256, 4),
                                  (70000, 3, 264, 256, 2), (33000, 2, 2056, 264, 2)], ids=str)
def test_gradient_of_rows_of_several_slots(tpc, case, dtype):
    """The slots' parts are summed in float32 and rounded once.  They come in pairs that all but cancel."""
    slots, groups, i, o, fan = case
    print(f"several slots {dtype} {case}", flush=True)
    r = np.random.default_rng(slots + fan)
    dt = DT[dtype]
    index = r.integers(0, groups, size=(slots // fan, fan))
    index[:, 1] = index[:, 0]
    n = index.size
    g = tpc.group_rows(ints(index), groups)
    ptr, rows = ob.group_rows(index, groups)
    gz = r.normal(size=(n // fan, fan, o))
    gz[:, 1] = -gz[:, 0] + 0.01 * gz[:, 1]
    if fan > 2:
        gz[:, 2:] *= 0.01
    gz, w = dev(gz.reshape(n, o), dt), dev(r.normal(size=(groups, i, o)), dt)
    x = dev(np.zeros((n // fan, i)), dt)
    got = tpc.grouped_linear_backward(gz, x, w, g, want_w=False)[0]
    want = ob.grouped_backward(f64(gz), f64(x), f64(w), ptr, rows, fan, "source", "source")[0]
    size = ob.grouped_backward(np.abs(f64(gz)), f64(x), np.abs(f64(w)), ptr, rows, fan, "source", "source")[0]
    near(got, want, (o + 16 + fan) * U * size, "grad_x", dtype)


@pytest.mark.parametrize("width", [1, 4])
def test_activation_and_its_slope_are_right_relatively(tpc, width):
    """Float32, from z = -87, below which the sigmoid's exponential underflows, to 60.

    Tolerance (derived): exponential and reciprocal to a unit in the last place (2 u) each, the argument's
    remainder, two sums and three products u each: 10 u of the value; the slope s (1 + z (1 - s)) twice
    that of its absolute terms."""
    r = np.random.default_rng(6)
    n = 4000
    z = np.r_[np.linspace(-87, 60, n - 1000), r.uniform(-4, 4, size=999), 0.0]
    x = np.zeros((n, width))
    x[:, 0] = z
    x, w = dev(x), torch.eye(width, device="cuda").view(1, width, width).contiguous()
    g = tpc.group_rows(ints(np.zeros(n)), 1)
    y, pre = tpc.grouped_linear_forward(x, w, g, act="silu", want_pre=True)
    z = f64(x[:, 0])
    assert np.array_equal(f64(pre[:, 0]), z)
    s, rest = 1 / (1 + np.exp(-z)), 1 / (1 + np.exp(z))
    off = np.abs(f64(y[:, 0]) - z * s) / np.maximum(np.abs(z * s), 1e-37)
    assert off.max() < 10 * U, (off.max() / U, z[off.argmax()])
    one = torch.ones(n, width, device="cuda")
    slope = f64(tpc.grouped_linear_backward(one, x, w, g, pre=x, want_w=False)[0][:, 0])
    off = np.abs(slope - s * (1 + z * rest)) / (s * (1 + np.abs(z) * rest))
    assert off.max() < 20 * U, (off.max() / U, z[off.argmax()])
    # what is not finite: infinities of z keep their limit or are no number, as z / (1 + exp(-z)) is
    bad = dev([[float("inf")] + [0.0] * (width - 1), [float("nan")] + [0.0] * (width - 1)])
    if width == 1:
        got = tpc.grouped_linear_forward(bad, w, tpc.group_rows(ints([0, 0]), 1), act="silu")
        assert float(got[0, 0]) == float("inf") and torch.isnan(got[1, 0])
