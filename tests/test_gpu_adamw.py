"""The AdamW step on the GPU against the float64 reference.

Tolerances (derived): u = 2^-24.  Moments in float32 take a product each by a rounded rate, and an
addition: 4 u of the sum of absolute terms.  A parameter's step takes about ten operations, a
square root and a reciprocal among them to a unit in the last place, each at most 2 u: 32 u of the
step's size (with the first moment's absolute terms), and the parameter two roundings and the rounded
rate: 4 u of its size.  The scale of the gradients and the choice of an 8-bit code are formed in 64
bits: codes and units are equal, but where a value lies within 1e-15 of a border, which no
input here does.
"""
import numpy as np
import pytest

from oracle import blocks as ob
from tests._blocks import DT, U, W, dev, f64, near, same, torch

pytestmark = pytest.mark.gpu
B1, B2, EPS, LR = 0.9, 0.999, 1e-8, 1e-2


@pytest.fixture(scope="module")
def tpc():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import tensor_product_convolution_amd as m
    m.lib()
    return m


def layout(opt, tensors):
    a = np.zeros(opt.exp_avg.numel())
    for o, t in zip(opt.offsets, tensors):
        a[o:o + t.numel()] = f64(t).reshape(-1)
    return a


def check_step(opt, before, p0, grads, p1, t, decay, max_norm, norm, low):
    """One step against the reference, from the states as they were."""
    if opt.bits == 8:
        m0, v0 = ob.decode(f64(before[1]), f64(before[3]), False), ob.decode(f64(before[2]), f64(before[4]), True)
    else:
        m0, v0 = f64(before[1]), f64(before[2])
    g = layout(opt, grads)
    factor = 1.0
    if max_norm is not None:
        size = np.sqrt((g * g).sum())
        near(norm, np.asarray(size), 0.0, "norm")
        factor = min(1.0, max_norm / size) if size else 1.0
    d = np.concatenate([np.full((n + 255) // 256 * 256, x) for n, x in zip(opt.numels, decay)] or [np.zeros(0)])
    start = layout(opt, p0)
    p, m, v = ob.adamw(start, g, m0, v0, t, LR, B1, B2, EPS, d, factor)
    sm = np.abs(B1 * m0) + np.abs((1 - B1) * g * factor)
    step = LR * (sm / (1 - B1 ** t)) / (np.sqrt(v / (1 - B2 ** t)) + EPS)
    near(dev(layout(opt, p1), torch.float64), p, 32 * U * step + 4 * U * np.abs(start), "p")
    if opt.bits == 8:
        n = len(m)
        um, uv = ob.rounding(n, opt.seed, t)
        for codes, units, x, second, u in ((opt.exp_avg, opt.exp_avg_unit, m, False, um), (opt.exp_avg_sq, opt.exp_avg_sq_unit, v, True, uv)):
            c, s = ob.encode(x, second, u)
            assert np.array_equal(units.cpu().numpy(), s) and np.array_equal(codes.cpu().numpy(), c)
        for got, codes, units, second in zip(opt.moments(), (opt.exp_avg, opt.exp_avg_sq), (opt.exp_avg_unit, opt.exp_avg_sq_unit), (False, True)):
            near(got, ob.decode(codes.cpu().numpy(), f64(units), second), 0.0, "moments")
    else:
        near(opt.exp_avg, m, 4 * U * sm, "m")
        near(opt.exp_avg_sq, v, 6 * U * v, "v")
    for a, b in zip(low, p1):
        if a is not None:
            assert torch.equal(a, b.to(torch.bfloat16))


def run(tpc, sizes, bits, dtype, max_norm, steps=3, scale=1.0, seed=3):
    r = np.random.default_rng(len(sizes) + bits)
    # at any element alignment
    params = [dev(r.normal(size=n + 1))[1:] if i % 2 else dev(r.normal(size=n)) for i, n in enumerate(sizes)]
    low = [torch.zeros(n, dtype=torch.bfloat16, device="cuda") if i % 3 else None for i, n in enumerate(sizes)]
    decay = [0.1 if i % 2 else 0.0 for i in range(len(sizes))]
    opt = tpc.AdamW(params, lr=LR, betas=(B1, B2), eps=EPS, weight_decay=decay, max_norm=max_norm, bits=bits, copies=low, seed=seed)
    for t in range(1, steps + 1):
        grads = [dev(scale * r.normal(size=n) * 10.0 ** r.uniform(-3, 3), DT[dtype]) for n in sizes]
        p0, before = [p.clone() for p in params], opt.state()
        assert before[0] == t - 1
        norm = opt.step(grads)
        assert (norm is None) == (max_norm is None)
        check_step(opt, before, p0, grads, params, t, decay, max_norm, norm, low)
    return opt


SIZES = {"one": [1], "odd": [1, 7, 255, 256, 257, 2047, 2048, 2049, 5000], "empty": [0, 3, 0], "wide": [100003],
         "many": [1 + 37 * i % 500 for i in range(600)]}


@pytest.mark.parametrize("sizes", list(SIZES))
@pytest.mark.parametrize("bits", [8, 32])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("max_norm", [None, 1.0, float("inf")])
def test_adamw(tpc, sizes, bits, dtype, max_norm):
    print(f"adamw {sizes} {bits} {dtype} {max_norm}", flush=True)
    run(tpc, SIZES[sizes], bits, dtype, max_norm, steps=2 if sizes in ("many", "wide") else 4)


def test_zero_gradients_and_states(tpc):
    """Nothing to divide by: only the decay moves a parameter."""
    for bits in (8, 32):
        p = dev(np.linspace(-1, 1, 700))
        keep = p.clone()
        opt = tpc.AdamW([p], lr=LR, weight_decay=0.5, bits=bits, max_norm=1.0)
        norm = opt.step([torch.zeros_like(p)])
        assert float(norm) == 0 and torch.equal(p, keep * (1 - torch.tensor(LR, device="cuda") * 0.5))
        assert all((m == 0).all() for m in opt.moments())


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("bits", [8, 32])
def test_a_norm_that_is_not_finite_changes_nothing(tpc, bad, bits):
    r = np.random.default_rng(1)
    params = [dev(r.normal(size=n)) for n in (300, 5)]
    low = [torch.zeros(n, dtype=torch.bfloat16, device="cuda") for n in (300, 5)]
    opt = tpc.AdamW(params, max_norm=1.0, bits=bits, copies=low)
    grads = [dev(r.normal(size=n)) for n in (300, 5)]
    opt.step(grads)
    keep = [t.clone() for t in (*params, *low)]
    before = opt.state()
    grads[1][2] = bad
    norm = opt.step(grads)
    assert not torch.isfinite(norm)
    after = opt.state()
    assert same(keep, (*params, *low)) and before[0] == after[0] == 1 and same(before[1:], after[1:])


def test_rounding_keeps_the_mean(tpc):
    """A second moment far from its gradients' squares moves by a thousandth of the way a step, far
    below half a code: over 400 steps of 20,000 values the mean follows (5 standard errors of
    400 roundings of at most an eighth of the value, over 20,000 values: 5 / 8 sqrt(400 / 20000))."""
    n = 20480
    p, g = dev(np.zeros(n)), dev(np.full(n, 1.0))
    opt = tpc.AdamW([p], lr=0.0, weight_decay=0.0, bits=8, seed=11)
    for _ in range(400):
        opt.step([g])
    want = 1 - B2 ** 400
    assert abs(float(opt.moments()[1].mean()) - want) < 5 / 8 * (400 / n) ** 0.5 * want
    assert abs(float(opt.moments()[0].mean()) - 1) < 5 / 8 * (10 / n) ** 0.5 + 1e-3


@pytest.mark.parametrize("bits", [8, 32])
def test_graph_rates_and_checkpoint(tpc, bits):
    """Replays against eager steps, the rate changed under the graph, and a restored state."""
    r = np.random.default_rng(2)
    sizes = [400, 3000, 17]
    make = lambda: [dev(np.random.default_rng(4).normal(size=n)) for n in sizes]
    a, b = make(), make()
    grads = [dev(r.normal(size=n)) for n in sizes]
    lr = dev([1e-2])
    kw = dict(betas=(B1, B2), max_norm=2.0, bits=bits, seed=5)
    x, y = tpc.AdamW(a, lr=lr, **kw), tpc.AdamW(b, lr=lr, **kw)
    x.step(grads)
    y.step(grads)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        norm = x.step(grads)
    for i in range(4):
        lr.mul_(0.5)
        for g in grads:
            g.copy_(torch.randn_like(g))
        graph.replay()
        want = y.step(grads)
        torch.cuda.synchronize()
        assert torch.equal(norm, want) and same(a, b)
        sx, sy = x.state(), y.state()
        assert sx[0] == sy[0] == i + 2 and same(sx[1:], sy[1:])
    c = [t.clone() for t in b]
    z = tpc.AdamW(c, lr=1e-2 * 0.5 ** 4, **kw)
    z.load(*y.state())
    y.step(grads, lr=1e-2 * 0.5 ** 4)
    z.step(grads)
    assert same(b, c) and same(y.state()[1:], z.state()[1:])


def test_another_stream(tpc):
    out = []
    for side in (False, True):
        opt_p = [dev(np.random.default_rng(4).normal(size=5000))]
        opt = tpc.AdamW(opt_p, bits=8, max_norm=1.0)
        g = [dev(np.random.default_rng(6).normal(size=5000))]
        s = torch.cuda.Stream() if side else torch.cuda.current_stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            opt.step(g)
            opt.step(g)
        torch.cuda.current_stream().wait_stream(s)
        torch.cuda.synchronize()
        out.append((opt_p[0], *opt.state()[1:]))
    assert same(*out)


def test_a_tensor_twice_is_refused(tpc):
    p, none = torch.zeros(300, device="cuda"), torch.zeros(0, device="cuda")
    tpc.AdamW([p[:100], p[100:], none, none])
    with pytest.raises(ValueError, match="twice"):
        tpc.AdamW([p, torch.zeros(3, device="cuda"), p])
    with pytest.raises(ValueError, match="twice"):
        tpc.AdamW([p[:200], p[100:]])
    low = torch.zeros(300, device="cuda", dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="twice"):
        tpc.AdamW([p[:100], p[100:200]], copies=[low[:100], low[50:150]])
