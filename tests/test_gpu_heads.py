"""Norm and rotation of queries and keys on the GPU against the float64 reference.

Tolerances (derived): u = 2^-24.  A head's sum of d squares in float32 is off by at most (d + 4) u
relative, r by half of that, y by a few roundings more.  A turn's fraction is rounded to float32
(2^-26 turns, 1.6 u of a radian), cos and sin by a few u: a turned value is off by at most
e = (d + 24) u times the sum of its pair's absolute values.  Places of 2^28 lose 3 2^-53 of their
turns in 64 bits, below u.  Backward: the same for the gradient turned back, and each of the sums over
a head adds (d + 4) u of its absolute terms: 4 e of the absolute terms of an output.  Sums over
rows and heads: their number of u more.  bfloat16 outputs add one rounding.
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


def problem(rows, hq, hk, d, pairs, axes, dtype, norm, reach, seed=0):
    """Views of one projected row with values behind them, and the gradients."""
    r = np.random.default_rng(seed + rows * 31 + d)
    row = dev(r.normal(size=(rows, (hq + 2 * hk) * d)), DT[dtype])
    up = dev(r.normal(size=(rows, (hq + hk) * d)), DT[dtype])
    s = dict(q=row[:, :hq * d].view(rows, hq, d), k=row[:, hq * d:(hq + hk) * d].view(rows, hk, d),
             gq=up[:, :hq * d].view(rows, hq, d), gk=up[:, hq * d:].view(rows, hk, d), kw={})
    if norm:
        s["kw"].update(gamma_q=dev(1 + 0.3 * r.normal(size=d)), gamma_k=dev(r.normal(size=d)))
    if pairs:
        if reach:
            s["kw"]["pos"] = ints(r.integers(-reach, reach, size=(rows, axes)))
        else:
            s["kw"]["pos"] = dev(r.uniform(-30, 30, size=(rows, axes)))
        s["kw"]["freq"] = torch.tensor(r.normal(size=(pairs, axes)), device="cuda")
    return s


def pair_sum(x, pairs, interleaved):
    """Each value's pair's sum of absolute values (its own where it is not turned)."""
    s = np.abs(x)
    a, b = ob.pair_places(pairs, interleaved)
    t = s[..., a] + s[..., b]
    s[..., a] = s[..., b] = t
    return s


def check(s, interleaved, eps, dtype, fwd, back):
    kw = {n: f64(t) for n, t in s["kw"].items()}
    pos, freq = kw.get("pos"), kw.get("freq")
    pairs = 0 if freq is None else len(freq)
    d = s["q"].shape[2]
    e = (d + 24) * U
    total = 0
    for name, out, i in (("q", fwd[0], 0), ("k", fwd[1], 1)):
        x, g, gamma = f64(s[name]), f64(s["g" + name]), kw.get("gamma_" + name)
        near(out, ob.head_forward(x, gamma, pos, freq, interleaved, eps),
             e * pair_sum(ob.head_forward(x, gamma, None, None, interleaved, eps), pairs, interleaved), name, dtype)
        gx, gg, gpos = ob.head_backward(g, x, gamma, pos, freq, interleaved, eps)
        habs = pair_sum(g, pairs, interleaved)
        r = np.ones(x.shape[:2] + (1,)) if gamma is None else 1 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
        z = np.abs(x) * r
        size = habs
        if gamma is not None:
            sabs = habs * np.abs(gamma)
            size = r * (sabs + z * (sabs * z).mean(-1, keepdims=True))
            near(back[2 + i], gg, (x.shape[0] * x.shape[1] + 4 * (d + 24)) * U * (habs * z).sum((0, 1)), "gamma_" + name)
        near(back[i], gx, 4 * e * size, "grad_" + name, dtype)
        if back[4] is not None:
            y = z if gamma is None else z * np.abs(gamma)
            a, b = ob.pair_places(pairs, interleaved)
            total = total + np.stack([(habs[..., a] * (y[..., a] + y[..., b])).sum(1) @ np.abs(freq)[:, i] for i in range(freq.shape[1])], 1)
    if back[4] is not None:
        want = sum(ob.head_backward(f64(s["g" + n]), f64(s[n]), kw.get("gamma_" + n), pos, freq, interleaved, eps)[2] for n in "qk")
        near(back[4], want, (4 * (d + 24) + pairs + s["q"].shape[1] + s["k"].shape[1]) * U * total, "grad_pos")


SHAPES = [  # rows, heads, key heads, dim, pairs, axes, reach of whole positions (0: float32)
    (1, 1, 1, 1, 0, 0, 0), (1, 2, 1, 2, 1, 1, 0), (3, 1, 1, 7, 3, 2, 0), (33, 4, 4, 16, 8, 3, 0), (130, 8, 2, 32, 16, 3, 0),
    (7, 5, 5, 40, 12, 1, 1 << 28), (50, 16, 4, 64, 24, 3, 0), (9, 3, 1, 96, 48, 1, 1000), (5, 2, 2, 128, 64, 3, 0),
    (4, 1, 1, 255, 127, 2, 0), (3, 2, 1, 256, 128, 1, 1 << 20), (2, 1, 3, 256, 1, 3, 0), (2000, 2, 2, 24, 5, 3, 0),
    (3, 1024, 1, 8, 4, 1, 50), (6000, 6, 2, 10, 5, 2, 0)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_heads(tpc, dtype, interleaved, norm, shape):
    rows, hq, hk, d, pairs, axes, reach = shape
    print(f"heads {dtype} {shape} interleaved={interleaved} norm={norm}", flush=True)
    s = problem(rows, hq, hk, d, pairs, axes, dtype, norm, reach)
    kw = dict(s["kw"], interleaved=interleaved, eps=1e-5)
    want_pos = pairs > 0 and not reach
    fwd = tpc.head_norm_rotate_forward(s["q"], s["k"], **kw)
    back = tpc.head_norm_rotate_backward(s["gq"], s["gk"], s["q"], s["k"], want_pos=want_pos, **kw)
    torch.cuda.synchronize()
    assert (back[2] is None) == (not norm) and (back[4] is None) == (not want_pos)
    check(s, interleaved, 1e-5, dtype, fwd, back)
    assert same(back, tpc.head_norm_rotate_backward(s["gq"], s["gk"], s["q"], s["k"], want_pos=want_pos, **kw))
    less = tpc.head_norm_rotate_backward(s["gq"], s["gk"], s["q"], s["k"], want_weights=False, **kw)
    assert same(less[:2], back[:2]) and less[2:] == (None, None, None)
    # in place, over views of rows
    tpc.head_norm_rotate_forward(s["q"], s["k"], outs=(s["q"], s["k"]), **kw)
    assert same((s["q"], s["k"]), fwd)


def test_no_rows(tpc):
    s = problem(0, 2, 1, 16, 4, 3, "f32", True, 0)
    q, k = tpc.head_norm_rotate_forward(s["q"], s["k"], **s["kw"])
    back = tpc.head_norm_rotate_backward(s["gq"], s["gk"], s["q"], s["k"], want_pos=True, **s["kw"])
    assert q.shape == (0, 2, 16) and back[4].shape == (0, 3)
    assert (back[2] == 0).all() and (back[3] == 0).all()


def test_a_bad_head_stays_alone(tpc):
    """NaN and infinity in one head reach its own outputs only; a head of zeros is finite."""
    s = problem(20, 3, 2, 32, 16, 3, "f32", True, 0)
    clean = tpc.head_norm_rotate_forward(s["q"], s["k"], **s["kw"])
    s["q"][4, 1, 7] = float("nan")
    s["k"][9, 0, 3] = float("inf")
    s["q"][11, 2] = 0
    q, k = tpc.head_norm_rotate_forward(s["q"], s["k"], **s["kw"])
    assert torch.isnan(q[4, 1]).all() and torch.isnan(k[9, 0]).any() and (q[11, 2] == 0).all()
    q[4, 1] = clean[0][4, 1]
    q[11, 2] = clean[0][11, 2]
    k[9, 0] = clean[1][9, 0]
    assert same((q, k), clean)


def test_scores_know_differences_alone(tpc):
    """The structure moved by whole periods of its wave vectors: the same rotation."""
    s = problem(64, 2, 2, 32, 16, 3, "f32", True, 0)
    n = torch.randint(-3, 4, (16, 3), device="cuda").double()
    kw = dict(s["kw"], freq=n * (2 * np.pi / 8.0))           # reciprocal lattice of a box of 8
    kw["pos"] = torch.rand(64, 3, device="cuda")
    a = tpc.head_norm_rotate_forward(s["q"], s["k"], **kw)
    kw["pos"] = kw["pos"] + 8.0 * 2 ** 10                    # rounds positions by 2^-11
    b = tpc.head_norm_rotate_forward(s["q"], s["k"], **kw)
    for x, y in zip(a, b):
        # angle: |n| 2 pi / 8 2^-11 over three axes, at most 3.5e-3, of a pair of normed values below 8
        assert (x - y).abs().max() < 3 * 3 * 2 * np.pi / 8 * 2.0 ** -11 * 8


def test_stream_and_graph(tpc):
    s = problem(500, 4, 2, 32, 16, 3, "bf16", True, 0)
    call = lambda: (*tpc.head_norm_rotate_forward(s["q"], s["k"], **s["kw"]),
                    *tpc.head_norm_rotate_backward(s["gq"], s["gk"], s["q"], s["k"], want_pos=True, **s["kw"]))
    eager = call()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = call()
    torch.cuda.current_stream().wait_stream(side)
    assert same(eager, other)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = call()
    for i in range(4):
        s["q"].copy_(torch.randn_like(s["q"]))
        s["kw"]["pos"].add_(1.0)
        graph.replay()
        torch.cuda.synchronize()
        assert same(held, call())


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("shape", [(70001, 1, 1, 8, 3, 2, 0), (70001, 2, 1, 20, 7, 1, 0), (20003, 8, 2, 40, 12, 3, 0), (9001, 3, 3, 64, 32, 1, 0)],
                         ids=str)
def test_many_rows(tpc, dtype, interleaved, shape):
    """More rows than the workgroups of the backward hold at once; gradients in place of the upstream ones."""
    print(f"heads {dtype} {shape} interleaved={interleaved}", flush=True)
    s = problem(*shape[:6], dtype, True, 0)
    kw = dict(s["kw"], interleaved=interleaved, eps=1e-5)
    back = tpc.head_norm_rotate_backward(s["gq"], s["gk"], s["q"], s["k"], want_pos=True, **kw)
    check(s, interleaved, 1e-5, dtype, tpc.head_norm_rotate_forward(s["q"], s["k"], **kw), back)
    own = tpc.head_norm_rotate_backward(s["gq"], s["gk"], s["q"], s["k"], want_pos=True, outs=(s["gq"], s["gk"]), **kw)
    assert own[0] is s["gq"] and same(own, back)
