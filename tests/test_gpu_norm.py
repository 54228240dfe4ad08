"""Layer norm and dropout on the GPU against the float64 reference.

Tolerances (derived): with u = 2^-24, a row's mean and variance are sums of C values in
float32 (error at most (C + 4) u of the sum of absolute terms; pairwise in the kernel,
so far less), rstd inherits half of the variance's relative error, and each output takes
a few more roundings: e = (C + 16) u relative to the sum of the absolute terms of an
output.  bfloat16 outputs add their one rounding, 2^-8 |reference|.  Weight gradients
sum R rows: (R + C + 16) u of the sum of absolute terms.  Dropout is exact: one float32
multiplication and addition, then the type's rounding, reproduced bit for bit.
"""
import numpy as np
import pytest

from oracle import layers as ol

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
U, W = 2.0 ** -24, 2.0 ** -8
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(scope="module")
def tpc():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import tensor_product_convolution_amd as m
    m.lib()
    return m


def dev(a, dt=torch.float32):
    return torch.tensor(np.asarray(a), device="cuda").to(dt)


def f64(t):
    return t.double().cpu().numpy()


def near(got, ref, bound, name, low):
    over = np.abs(f64(got) - ref) - (bound + (W if low else 2 * U) * np.abs(ref) + 1e-37)
    assert over.size == 0 or over.max() <= 0, (name, float(over.max()))


def check_norm(y, mean, rstd, h, gamma, beta, eps, low):
    C = h.shape[1]
    ry, rm, rr = ol.layer_norm_forward(h, gamma, beta, eps)
    e = (C + 16) * U
    spread = np.abs(h).mean(axis=1)
    near(mean, rm, e * spread, "mean", False)
    # a shift of the mean by e spread changes the variance to second order only
    var = 1 / rr ** 2
    near(rstd, rr, rr * (e + (e * spread) ** 2 / var), "rstd", False)
    z = np.abs(h - rm[:, None]) * rr[:, None]
    near(y, ry, np.abs(gamma) * (2 * e * z + (e * spread * rr)[:, None]) + 4 * U * np.abs(beta), "y", low)


def check_norm_back(got, gy, h, gamma, eps, low, add=0.0):
    gh, gg, gb = got
    R, C = h.shape
    rh, rg, rb = ol.layer_norm_backward(gy, h, gamma, eps)
    _, mean, rstd = ol.layer_norm_forward(h, gamma, gamma, eps)
    z = np.abs(h - mean[:, None]) * rstd[:, None]
    t = np.abs(gy * gamma)
    e = (C + 16) * U
    ze = z + (np.abs(h).mean(axis=1) * rstd)[:, None]          # z with the mean's error
    size = rstd[:, None] * (t + t.mean(axis=1, keepdims=True) + ze * (t * ze).mean(axis=1, keepdims=True))
    near(gh, rh + add, 3 * e * size + 2 * U * np.abs(add), "grad_h", low)
    near(gg, rg, (R + C + 16) * U * (np.abs(gy) * ze).sum(axis=0), "grad_gamma", False)
    near(gb, rb, (R + 16) * U * np.abs(gy).sum(axis=0), "grad_beta", False)


SHAPES = [(1, 1), (3, 2), (5, 7), (64, 8), (33, 15), (1000, 16), (130, 31), (77, 32), (65, 33), (9, 64), (300, 100), (17, 128),
          (6, 129), (1500, 256), (4, 257), (70, 500), (3, 513), (40, 1000), (2, 1025), (30, 1152), (5, 2049), (7, 3001),
          (2, 4097), (3, 8192), (5000, 24)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("pad", [0, 1, 24])
def test_norm(tpc, dtype, shape, pad):
    R, C = shape
    print(f"norm {dtype} {shape} +{pad}", flush=True)
    r = np.random.default_rng(R * 10007 + C)
    x = dev(r.normal(size=(R, C + pad)) * r.uniform(0.2, 3, size=(R, 1)) + r.normal(size=(R, 1)), DT[dtype])[:, pad:]
    gy = dev(r.normal(size=(R, C + pad)), DT[dtype])[:, :C]
    gamma, beta = dev(1 + 0.3 * r.normal(size=C)), dev(r.normal(size=C))
    y, mean, rstd = tpc.layer_norm_forward(x, gamma, beta, eps=1e-5)
    got = tpc.layer_norm_backward(gy, x, gamma, mean, rstd)
    torch.cuda.synchronize()
    low = dtype == "bf16"
    check_norm(y, mean, rstd, f64(x), f64(gamma), f64(beta), 1e-5, low)
    check_norm_back(got, f64(gy), f64(x), f64(gamma), 1e-5, low)
    only, g, b = tpc.layer_norm_backward(gy, x, gamma, mean, rstd, want_weights=False)
    assert g is None and b is None and torch.equal(only, got[0])
    again = tpc.layer_norm_backward(gy, x, gamma, mean, rstd)
    assert all(torch.equal(a, b) for a, b in zip(got, again))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shape", [(1, 1), (5, 7), (40, 8), (33, 30), (100, 64), (11, 130), (7, 1001), (3, 1152), (2, 4099)],
                         ids=str)
@pytest.mark.parametrize("p", [None, 0.0, 0.1, 0.7])
def test_residual_norm(tpc, dtype, shape, p):
    R, C = shape
    print(f"residual norm {dtype} {shape} p={p}", flush=True)
    r = np.random.default_rng(R + C)
    dt = DT[dtype]
    x, res = dev(r.normal(size=(R, C + 3)), dt)[:, :C], dev(r.normal(size=(R, C)), dt)
    gy, gres = dev(r.normal(size=(R, C)), dt), dev(r.normal(size=(R, C)), dt)
    gamma, beta = dev(1 + 0.3 * r.normal(size=C)), dev(r.normal(size=C))
    drop = None if p is None else tpc.Dropout(p, 2 ** 63 + 5, 2 ** 33 + 1)
    y, mean, rstd, h = tpc.layer_norm_residual_forward(x, res, gamma, beta, drop)
    gx, gr, gg, gb = tpc.layer_norm_residual_backward(gy, h, gamma, mean, rstd, drop, grad_h=gres)
    torch.cuda.synchronize()
    f = np.ones((R, C)) if p is None else ol.dropout_factor((R, C), p, 2 ** 63 + 5, 2 ** 33 + 1)
    want = (x.cpu().float() * torch.tensor(f, dtype=torch.float32) + res.cpu().float()).to(dt)
    assert torch.equal(h.cpu(), want)                          # the stored stream is exact
    low = dtype == "bf16"
    check_norm(y, mean, rstd, f64(h), f64(gamma), f64(beta), 1e-5, low)
    check_norm_back((gr, gg, gb), f64(gy), f64(h), f64(gamma), 1e-5, low, add=f64(gres))
    if drop is None:
        assert gx is gr
    else:
        kept = f != 0
        assert not f64(gx)[~kept].any()
        # both are roundings of one float32 value and its multiple
        near(gx, f64(gr) * f, (W if low else 2 * U) * np.abs(f64(gr)) * f, "grad_x", low)
    g0 = tpc.layer_norm_residual_backward(gy, h, gamma, mean, rstd, drop)
    check_norm_back(g0[1:], f64(gy), f64(h), f64(gamma), 1e-5, low)


def test_norm_by_differences(tpc):
    """Step 2^-7 along random directions: truncation and rounding stay below 1e-2 of the
    sum of absolute terms."""
    r = np.random.default_rng(3)
    x, go = dev(r.normal(size=(9, 40))), dev(r.normal(size=(9, 40)))
    gamma, beta = dev(1 + 0.3 * r.normal(size=40)), dev(r.normal(size=40))
    _, mean, rstd = tpc.layer_norm_forward(x, gamma, beta)
    grads = tpc.layer_norm_backward(go, x, gamma, mean, rstd)
    loss = lambda: float((tpc.layer_norm_forward(x, gamma, beta)[0].double() * go.double()).sum())
    for t, g in zip((x, gamma, beta), grads):
        keep, d, h = t.clone(), dev(r.normal(size=tuple(t.shape))), 2.0 ** -7
        t.copy_(keep + h * d)
        up = loss()
        t.copy_(keep - h * d)
        down = loss()
        t.copy_(keep)
        want = float((g.double() * d.double()).sum())
        assert abs((up - down) / (2 * h) - want) < 1e-2 * float((g * d).abs().double().sum())


def test_norm_extremes(tpc):
    """A constant row (variance 0), a large offset, rows of zeros, NaN in one row only."""
    C = 96
    gamma, beta = torch.ones(C, device="cuda"), torch.full((C,), 0.5, device="cuda")
    x = torch.zeros(6, C, device="cuda")
    x[1] = 3.0
    x[2] = 1e4 + torch.arange(C, device="cuda") / 64.0
    x[3, 5] = float("nan")
    x[4] = torch.linspace(-1e18, 1e18, C, device="cuda")
    y, mean, rstd = tpc.layer_norm_forward(x, gamma, beta)
    assert torch.all(y[0] == 0.5) and torch.all(y[1] == 0.5) and torch.all(y[5] == 0.5)
    assert torch.isnan(y[3]).all() and torch.isfinite(y[[0, 1, 2, 4, 5]]).all()
    ref = ol.layer_norm_forward(f64(x[2:3]), np.ones(C), np.full(C, 0.5), 1e-5)[0]
    # the mean of values near 1e4 is off by at most their rounding times a few: 1e4 (log2 C + 2) u over the spread
    assert np.abs(f64(y[2:3]) - ref).max() < 1e4 * 16 * U * float(rstd[2])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("n", [1, 2, 3, 4, 5, 7, 8, 9, 1000, 1023, 4097])
@pytest.mark.parametrize("p", [0.0, 0.1, 0.999])
def test_dropout(tpc, dtype, n, p):
    r = np.random.default_rng(n)
    dt = DT[dtype]
    x, res = dev(r.normal(size=n + 1), dt)[1:], dev(r.normal(size=n), dt)      # x at element alignment
    d = tpc.Dropout(p, 77, 2 ** 40)
    f = torch.tensor(ol.dropout_factor((n,), p, 77, 2 ** 40), dtype=torch.float32)
    out = tpc.dropout_forward(x, d, residual=res)
    assert torch.equal(out.cpu(), (x.cpu().float() * f + res.cpu().float()).to(dt))
    assert torch.equal(tpc.dropout_backward(x, d).cpu(), (x.cpu().float() * f).to(dt))
    keep = x.clone()
    tpc.dropout_forward(x, d, residual=res, out=x)                              # in place
    assert torch.equal(x, tpc.dropout_forward(keep, d, residual=res))


def test_dropped_values_vanish_whatever_they_hold(tpc):
    d = tpc.Dropout(0.5, 3)
    f = ol.dropout_factor((64,), 0.5, 3, 0)
    x = torch.ones(64, device="cuda")
    x[torch.tensor(f == 0)] = float("nan")
    assert torch.isfinite(tpc.dropout_forward(x, d)).all()


def test_element_numbers_beyond_32_bits(tpc):
    """Blocks of four words are counted in 64 bits: a row of a long array draws the
    words of its own element numbers."""
    n = (1 << 32) + 24
    x = torch.ones(n, dtype=torch.bfloat16, device="cuda")
    out = tpc.dropout_forward(x, tpc.Dropout(0.5, 9, 1), out=x)
    torch.cuda.synchronize()
    for at in ((1 << 32) - 8, 1 << 32, (1 << 32) + 16):
        words = ol.philox_block(at // 4, 9, 1) + ol.philox_block(at // 4 + 1, 9, 1)
        want = [2.0 if w >= 2 ** 31 else 0.0 for w in words]
        assert out[at:at + 8].float().cpu().tolist() == want, at


def test_strides_beyond_32_bits(tpc):
    """Rows far apart: element offsets pass 2^31.  Bit for bit the results of dense rows."""
    n, wide, c = 36000, 1 << 16, 40
    x = torch.empty(n, wide, device="cuda", dtype=torch.bfloat16)[:, -c:]
    gy = torch.empty(n, wide, device="cuda", dtype=torch.bfloat16)[:, :c]
    g = torch.Generator(device="cuda").manual_seed(1)
    x[:], gy[:] = (torch.randn(n, c, device="cuda", generator=g) for _ in range(2))
    w, b = torch.rand(c, device="cuda", generator=g), torch.rand(c, device="cuda", generator=g)
    res = []
    for a, d in ((x, gy), (x.contiguous(), gy.contiguous())):
        y, mean, rstd = tpc.layer_norm_forward(a, w, b)
        res.append([y, mean, rstd, *tpc.layer_norm_backward(d, a, w, mean, rstd)])
    assert all(torch.equal(p, q) for p, q in zip(*res))


def test_no_rows_and_refusals(tpc):
    e = torch.empty(0, 16, device="cuda")
    g = torch.ones(16, device="cuda")
    y, mean, rstd = tpc.layer_norm_forward(e, g, g)
    assert y.shape == (0, 16) and mean.shape == (0,)
    gx, gg, gb = tpc.layer_norm_backward(e, e, g, mean, rstd)
    assert gx.shape == (0, 16) and not gg.any() and not gb.any()
    assert tpc.dropout_forward(torch.empty(0, device="cuda"), tpc.Dropout(0.1, 1)).shape == (0,)
    x = torch.ones(4, 16, device="cuda")
    with pytest.raises(ValueError):
        tpc.layer_norm_forward(x.t(), g, g)
    with pytest.raises(ValueError):
        tpc.layer_norm_forward(x, g[:8], g)
    with pytest.raises(TypeError):
        tpc.layer_norm_forward(x.double(), g, g)
    with pytest.raises(TypeError):
        tpc.layer_norm_forward(x, g.bfloat16(), g)
    with pytest.raises(ValueError):
        tpc.layer_norm_forward(x.cpu(), g, g)
    with pytest.raises(tpc.TPError):
        tpc.layer_norm_forward(torch.ones(2, 9000, device="cuda"), torch.ones(9000, device="cuda"),
                               torch.ones(9000, device="cuda"))
    with pytest.raises(tpc.TPError):
        tpc.dropout_forward(x, tpc.Dropout(1.0, 1))
    with pytest.raises(TypeError):
        tpc.dropout_forward(x, tpc.Dropout(0.1, 1), residual=x.bfloat16())


def test_graph_replay(tpc):
    r = np.random.default_rng(1)
    x, res, gy = (dev(r.normal(size=(3000, 96))) for _ in range(3))
    g, b = dev(r.normal(size=96)), dev(r.normal(size=96))
    d = tpc.Dropout(0.2, 5, 6)

    def step():
        y, mean, rstd, h = tpc.layer_norm_residual_forward(x, res, g, b, d)
        return [y, h, *tpc.layer_norm_residual_backward(gy, h, g, mean, rstd, d)]
    want = [t.clone() for t in step()]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for _ in range(3):
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, got))
        step()


# rows that end inside a chunk, on either side of every change of layout, and so many rows that
# a workgroup takes several
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shape", [(50, 3), (50, 5), (50, 9), (40, 19), (40, 43), (33, 61), (33, 86), (30, 125), (30, 135),
                                   (30, 189), (20, 195), (20, 251), (20, 393), (20, 514), (9, 1018), (9, 1029), (9, 2046),
                                   (5, 2051), (5, 4093), (70000, 6), (20000, 131), (3000, 270), (4500, 1101), (600, 2101)], ids=str)
def test_rows_of_odd_length(tpc, dtype, shape):
    test_residual_norm(tpc, dtype, shape, 0.3)
