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


@pytest.mark.parametrize("bits", [8, 32])
def test_huge_gradients(tpc, bits):
    """Squares past the largest float32: an 8-bit block's unit ends there, and its other values stay numbers."""
    r = np.random.default_rng(8)
    p = [dev(r.normal(size=600))]
    opt = tpc.AdamW(p, lr=LR, betas=(B1, B2), eps=EPS, weight_decay=0.1, bits=bits, seed=5)
    for t in range(1, 4):
        g = r.normal(size=600)
        g[[5, 300]] = 3e38, -1e25
        g = [dev(g)]
        p0, before = [x.clone() for x in p], opt.state()
        opt.step(g)
        assert torch.isfinite(p[0]).all()
        if bits == 8:
            check_step(opt, before, p0, g, p, t, [0.1], None, None, [None])


@pytest.mark.parametrize("eps", [0.0, 1e-40, 1e-30, 1e-8])
@pytest.mark.parametrize("bits", [8, 32])
def test_tiny_gradients_and_eps(tpc, bits, eps):
    """Second moments that are subnormal in float32, or below it: the step is the formula's on the moments that the
    step has (float32 ones with 32 bits), and zeros over a small eps are zeros.  An eps below 2^-126 counts as that.
    In float32 (1 - beta2) g^2 ends at 0 where g^2 is below 2^-150 / (1 - beta2) and its own rounding, half of
    2^-149: g below 8.7e-22; with eps 0 such a gradient is divided by nothing."""
    r = np.random.default_rng(9)
    n = 900
    g = r.choice([-1.0, 1.0], size=n) * 10.0 ** r.uniform(-21.5 if bits == 32 else -30, -17, size=n)
    g[:300] = 10.0 ** r.uniform(-12, 0, size=300)
    if eps:
        g[100:140] = 0
    g, p = dev(g), dev(r.normal(size=n))
    start = f64(p)
    opt = tpc.AdamW([p], lr=LR, betas=(B1, B2), eps=eps, weight_decay=0.1, bits=bits)
    opt.step([g])
    G = f64(g)
    if bits == 32:
        m, v = f64(opt.exp_avg)[:n], f64(opt.exp_avg_sq)[:n]
        assert (v[np.abs(G) > 8.7e-22] > 0).all()
    else:
        m, v = (1 - B1) * G, (1 - B2) * G * G
    e = max(eps, 2.0 ** -126) if eps else 0.0
    some = (v > 0) | (e > 0)
    with np.errstate(divide="ignore"):
        step = LR * (m / (1 - B1)) / (np.sqrt(v / (1 - B2)) + e)
    assert not torch.isfinite(p[torch.tensor(~some, device="cuda")]).any()
    near(p[torch.tensor(some, device="cuda")], (start * (1 - LR * 0.1) - step)[some], (32 * U * np.abs(step) + 4 * U * np.abs(start))[some], "p")


def test_a_parameter_that_has_moved_is_refused(tpc):
    """The addresses are the optimiser's from its start: it writes nothing where a parameter was before."""
    p, low = [torch.nn.Parameter(torch.ones(300, device="cuda")) for _ in range(2)], torch.zeros(300, device="cuda", dtype=torch.bfloat16)
    opt = tpc.AdamW(p, copies=[None, low])
    g = [torch.ones(300, device="cuda") for _ in p]
    opt.step(g)
    p[0].data.copy_(torch.zeros(300))      # other values in the same place are what it goes on from
    opt.step(g)
    assert float(p[0][0]) < 0 < float(p[1][0]) < 1
    was, t = p[1].data, opt.state()[0]
    p[1].data = was.clone()
    keep = was.clone()
    with pytest.raises(ValueError, match="moved"):
        opt.step(g)
    assert torch.equal(was, keep) and torch.equal(p[1], keep) and opt.state()[0] == t == 2
    p[1].data = was
    opt.step(g)
    assert float(p[1][0]) < float(keep[0])
    low.data = low.clone()
    with pytest.raises(ValueError, match="moved"):
        opt.step(g)


def test_autograd_knows_of_a_step(tpc):
    """A graph that saved a parameter before the step is refused its backward, as after any other write in place."""
    p, low = torch.nn.Parameter(torch.ones(30, device="cuda")), torch.zeros(30, device="cuda", dtype=torch.bfloat16)
    opt = tpc.AdamW([p], copies=[low])
    (p * p).sum().backward()
    loss, versions = (p * p).sum(), (p._version, low._version)
    opt.step([p.grad])
    assert p._version > versions[0] and low._version > versions[1]
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()
    (p * p).sum().backward()


def mean_of_200_steps(c, start, step):
    """Of the moments over where they belong, less 1, of values that are not the largest of their blocks."""
    n, t = len(c), 200
    others = np.arange(n) % 256 != 0
    held = ob.decode(*start[:2], False), ob.decode(*start[2:], True)
    want = c + (held[0] - c) * B1 ** t, c * c + (held[1] - c * c) * B2 ** t
    for i in range(t):
        got = step(i)
    return [float((g / w)[others].mean()) - 1 for g, w in zip(got, want)]


def slow_moments():
    """A value in each block that stays where it is and holds the unit, and others whose moments start at half and a
    quarter of where they go."""
    n = 256 * 80
    c = (10.0 ** np.random.default_rng(2).uniform(-1.5, -0.2, size=n)).astype(np.float32).astype(np.float64)
    c[::256] = 1.0
    part = np.where(np.arange(n) % 256 != 0, 0.5, 1.0)
    return c, (*ob.encode(part * c, False, 0.5), *ob.encode((part * c) ** 2, True, 0.5))


# Derived: a rounding's standard deviation is at most half a code's distance, a sixteenth of the value.  Second moments keep
# each of the 200, 200^(1/2) / 16 in all, first moments 1 / (1 - 0.9^2)^(1/2) / 16; five times that over 20,400 values.
SPREAD = 5 / 16 / 20400 ** 0.5 / (1 - B1 ** 2) ** 0.5, 5 / 16 * (200 / 20400) ** 0.5


def test_moments_move_by_less_than_half_a_code(tpc):
    c, start = slow_moments()
    opt = tpc.AdamW([dev(np.zeros(len(c)))], lr=0.0, betas=(B1, B2), weight_decay=0.0, bits=8, seed=11)
    opt.load(1000, *[torch.tensor(t, device="cuda") for t in (start[0], start[2], start[1], start[3])])
    g = [dev(c)]

    def step(i):
        opt.step(g)
        return [f64(m) for m in opt.moments()] if i == 199 else None

    off = mean_of_200_steps(c, start, step)
    print(off, SPREAD)
    assert abs(off[0]) < SPREAD[0] and abs(off[1]) < SPREAD[1]
