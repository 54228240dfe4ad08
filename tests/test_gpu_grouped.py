"""Routing, order by group, products by group and sums over choices on the GPU against the
float64 reference.

Tolerances (derived): u = 2^-24.  A sum of K products in float32 is off by at most (K + 8) u of the sum
of their absolute values; of each float32 product up to 2^-21 = 8 u is left out: (K + 16) u in all.
bfloat16 operands multiply exactly.  silu and its slope are off by a few u of |z| + 1; the activation
is that of the stored z, so y is compared with silu of the pre that came back.  Where several slots
share a source row, each part is rounded to the type first.  Softmax: exp of a difference of up to D is
off by (D + 4) u relative, the sum of k or E terms by as many u.  Orders are exact.
"""
import numpy as np
import pytest

from oracle import blocks as ob
from tests._blocks import DT, U, W, dev, f64, ints, near, same, torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def tpc():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import tensor_product_convolution_amd as m
    m.lib()
    return m


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("over_all", [False, True])
@pytest.mark.parametrize("rows,groups,k", [(1, 1, 1), (5, 2, 2), (300, 8, 2), (67, 16, 16), (129, 64, 6), (40, 100, 1), (33, 256, 8),
                                           (20, 257, 3), (9, 1024, 16)])
def test_route(tpc, dtype, over_all, rows, groups, k):
    print(f"route {dtype} {rows} x {groups}, {k} over_all={over_all}", flush=True)
    r = np.random.default_rng(groups * 17 + k)
    wide = dev(2 * r.normal(size=(rows, groups + 3)), DT[dtype])
    wide[:, ::2] = wide[:, ::2].round()                       # ties, zeros of either sign
    l = wide[:, 1:groups + 1]
    if rows > 8:
        l[1] = -float("inf")
        l[2, :-1] = -float("inf")
        l[3, groups // 2] = float("nan")
        l[4] = 0.5
        l[5] = torch.finfo(DT[dtype]).min
        l[6, 0], l[6, 1:] = 60, -40
    weight, index = tpc.route_forward(l, k, over_all)
    x = f64(l)
    rw, ri = ob.route(x, k, over_all)
    assert np.array_equal(index.cpu().numpy(), ri)
    live = np.where(x > -np.inf, x, np.nan)
    spread = np.nan_to_num(np.nanmax(np.where(np.isnan(live), -1e30, live), 1) - np.nanmin(np.where(np.isnan(live), 1e30, live), 1))
    spread = np.clip(spread, 0, 110)[:, None]                 # exp(-110) is below float32
    e = (spread + 8 + (groups if over_all else k)) * U
    near(weight, rw, 2 * e * rw, "weight")
    g = dev(r.normal(size=(rows, k)))
    got = tpc.route_backward(g, l, weight, index, over_all)
    want = ob.route_backward(f64(g), x, rw, ri, over_all)
    size = np.zeros(x.shape)                                  # absolute terms of an output
    ga = (rw * np.abs(f64(g))).sum(1, keepdims=True)
    for i in range(rows):
        at = ri[i] >= 0
        size[i, ri[i][at]] = rw[i][at] * (np.abs(f64(g))[i][at] + ga[i])
    if over_all:
        p = np.exp(np.where(x > -np.inf, x, -np.inf) - np.nanmax(np.where(x > -np.inf, x, -1e300), 1, keepdims=True))
        p = np.nan_to_num(p)
        size += p / np.maximum(p.sum(1, keepdims=True), 1e-300) * ga
    near(got, want, 6 * (e + 20 * U) * size, "grad_logits", dtype)


@pytest.mark.parametrize("n", [0, 1, 63, 64, 65, 1000, 8191, 8192, 8193, 20001, 300000])
@pytest.mark.parametrize("groups", [1, 7, 64, 1024])
def test_group_rows(tpc, n, groups):
    r = np.random.default_rng(n + groups)
    for lo, hi in ((0, groups), (-2, groups + 2), (groups - 1, groups), (-5, 0)):
        index = r.integers(lo, hi, size=n)
        g = tpc.group_rows(ints(index), groups)
        ptr, rows = ob.group_rows(index, groups)
        assert np.array_equal(g.ptr.cpu().numpy(), ptr) and np.array_equal(g.rows.cpu().numpy(), rows), (n, groups, lo)
        assert g.fan == 1
    if n % 2 == 0 and n:
        two = tpc.group_rows(ints(index).view(-1, 2), groups)
        assert two.fan == 2 and torch.equal(two.rows, g.rows)
    extreme = ints(np.full(n, -2 ** 31))
    assert (tpc.group_rows(extreme, groups).ptr == 0).all()


def index_of(kind, slots, groups, r):
    if kind == "even":
        return r.integers(0, groups, size=slots)
    if kind == "one":                                         # all in the last group, the others empty
        return np.full(slots, groups - 1)
    if kind == "none":
        return np.full(slots, -1)
    skew = np.minimum(r.zipf(1.5, size=slots) - 1, groups - 1)
    return np.where(r.random(slots) < 0.1, -1, skew)          # and some without a group


def abs_parts(gz, x, w, ptr, rows, fan, x_rows, y_rows):
    a = np.abs
    return ob.grouped_backward(a(gz), a(x), a(w), ptr, rows, fan, x_rows, y_rows)


CASES = [  # slots, groups, in, out, kind, fan, x rows, y rows
    (1, 1, 1, 1, "even", 1, "source", "source"), (1, 3, 8, 8, "none", 1, "source", "source"),
    (5, 4, 7, 3, "even", 1, "source", "grouped"), (64, 2, 16, 24, "one", 1, "grouped", "source"),
    (100, 5, 33, 65, "skew", 1, "source", "source"), (256, 8, 64, 64, "skew", 2, "source", "grouped"),
    (300, 3, 128, 128, "skew", 3, "source", "source"), (1000, 7, 136, 75, "even", 1, "source", "source"),
    (1024, 2, 200, 130, "skew", 4, "grouped", "source"), (2000, 89, 40, 72, "skew", 1, "source", "source"),
    (77, 118, 9, 300, "even", 1, "grouped", "grouped"), (4096, 4, 256, 136, "skew", 2, "grouped", "source"),
    (6000, 1, 32, 512, "even", 2, "source", "source"), (512, 1024, 16, 16, "even", 1, "source", "source"),
    (700, 2, 1030, 40, "even", 1, "source", "grouped"), (129, 1, 8, 8, "one", 1, "source", "source")]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("case", CASES, ids=str)
def test_grouped(tpc, dtype, case):
    slots, groups, i, o, kind, fan, x_rows, y_rows = case
    print(f"grouped {dtype} {case}", flush=True)
    r = np.random.default_rng(slots + i)
    dt = DT[dtype]
    index = index_of(kind, slots, groups, r)
    g = tpc.group_rows(ints(index).view(-1, fan) if fan > 1 else ints(index), groups)
    ptr, rows = ob.group_rows(index, groups)
    nx = slots // fan if x_rows == "source" else slots
    x = dev(r.normal(size=(nx, i + 5)), dt)[:, 2:2 + i]       # strided, at any alignment
    w, b = dev(r.normal(size=(groups, i, o)), dt), dev(r.normal(size=(groups, o)), dt)
    gz = dev(r.normal(size=(slots, o + 3)), dt)[:, 3:]
    X, Wt, B, G = f64(x), f64(w), f64(b), f64(gz)
    z = ob.grouped_forward(X, Wt, ptr, rows, fan, B, x_rows, y_rows)
    bound = (i + 16) * U * ob.grouped_forward(np.abs(X), np.abs(Wt), ptr, rows, fan, np.abs(B), x_rows, y_rows)
    near(tpc.grouped_linear_forward(x, w, g, bias=b, x_rows=x_rows, y_rows=y_rows), z, bound, "z", dtype)
    y, pre = tpc.grouped_linear_forward(x, w, g, bias=b, act="silu", x_rows=x_rows, y_rows=y_rows, want_pre=True)
    near(pre, z, bound, "pre", dtype)
    near(y, ob.silu(f64(pre)), 8 * U * (np.abs(f64(pre)) + 1), "y", dtype)
    assert torch.equal(y, tpc.grouped_linear_forward(x, w, g, bias=b, act="silu", x_rows=x_rows, y_rows=y_rows))
    near(tpc.grouped_linear_forward(x, w, g, x_rows=x_rows, y_rows=y_rows),
         ob.grouped_forward(X, Wt, ptr, rows, fan, None, x_rows, y_rows), bound, "no bias", dtype)
    back = tpc.grouped_linear_backward(gz, x, w, g, x_rows=x_rows, y_rows=y_rows, want_bias=True)
    want = ob.grouped_backward(G, X, Wt, ptr, rows, fan, x_rows, y_rows)
    size = abs_parts(G, X, Wt, ptr, rows, fan, x_rows, y_rows)
    parts = (W if dtype == "bf16" else U) if fan > 1 and x_rows == "source" else 0.0
    near(back[0], want[0], ((o + 16 + fan) * U + parts) * size[0], "grad_x", dtype)
    near(back[1], want[1], (slots + 16) * U * size[1], "grad_w", dtype)
    near(back[2], want[2], (slots + 16) * U * size[2], "grad_bias", dtype)
    again = tpc.grouped_linear_backward(gz, x, w, g, x_rows=x_rows, y_rows=y_rows, want_bias=True)
    assert same(back, again)
    assert same(tpc.grouped_linear_backward(gz, x, w, g, x_rows=x_rows, y_rows=y_rows, want_w=False), (back[0], None, None))
    assert same(tpc.grouped_linear_backward(gz, x, w, g, x_rows=x_rows, y_rows=y_rows, want_x=False), (None, back[1], None))
    if fan == 1 or x_rows == "grouped":
        p = dev(3 * r.normal(size=(nx, i + 1)), dt)[:, :i]
        got = tpc.grouped_linear_backward(gz, x, w, g, x_rows=x_rows, y_rows=y_rows, pre=p, want_w=False)[0]
        near(got, want[0] * ob.silu_slope(f64(p)), (o + 40) * U * 1.2 * size[0], "grad_pre", dtype)


def test_no_slots(tpc):
    g = tpc.group_rows(ints(np.zeros(0)), 3)
    x, w = dev(np.zeros((0, 5))), dev(np.ones((3, 5, 4)))
    assert tpc.grouped_linear_forward(x, w, g).shape == (0, 4)
    gx, gw, gb = tpc.grouped_linear_backward(dev(np.zeros((0, 4))), x, w, g, want_bias=True)
    assert gx.shape == (0, 5) and (gw == 0).all() and (gb == 0).all()
    assert tpc.combine_forward(dev(np.zeros((0, 4))), dev(np.zeros((0, 2)))).shape == (0, 4)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_bad_rows_stay_alone(tpc, dtype):
    """A row of NaN or infinities reaches its own outputs only, and the weights' gradients of its own
    group; what weights of a group without slots hold reaches nothing."""
    r = np.random.default_rng(5)
    index = np.r_[r.integers(0, 3, size=200)]
    g = tpc.group_rows(ints(index), 5)
    dt = DT[dtype]
    x, w, gz = dev(r.normal(size=(200, 48)), dt), dev(r.normal(size=(5, 48, 40)), dt), dev(r.normal(size=(200, 40)), dt)
    clean = tpc.grouped_linear_forward(x, w, g)
    back = tpc.grouped_linear_backward(gz, x, w, g)
    w[3:] = float("nan")
    x[17], x[50, 3] = float("nan"), float("inf")
    y = tpc.grouped_linear_forward(x, w, g)
    keep = torch.ones(200, dtype=torch.bool, device="cuda")
    keep[17] = keep[50] = False
    assert torch.equal(y[keep], clean[keep]) and torch.isnan(y[17]).all()
    # an infinite value gives infinities of the weight's sign
    assert torch.equal(y[50], torch.copysign(torch.full_like(y[50], float("inf")), w[index[50], 3]))
    bad = tpc.grouped_linear_backward(gz, x, w, g)
    assert torch.equal(bad[0], back[0])
    for e in range(3):
        if e not in (index[17], index[50]):
            assert torch.equal(bad[1][e], back[1][e])
    assert (bad[1][3:] == 0).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,k,cols", [(1, 1, 1), (5, 2, 7), (100, 2, 64), (33, 16, 130), (7, 3, 1001), (2, 4, 5000), (3000, 1, 8)])
def test_combine(tpc, dtype, rows, k, cols):
    r = np.random.default_rng(rows + cols)
    y, go = dev(r.normal(size=(rows * k, cols)), DT[dtype]), dev(r.normal(size=(rows, cols)), DT[dtype])
    w = dev(r.random(size=(rows, k)))
    Y, G, Wt = f64(y).reshape(rows, k, cols), f64(go), f64(w)
    near(tpc.combine_forward(y, w), (Wt[..., None] * Y).sum(1), (k + 2) * U * (Wt[..., None] * np.abs(Y)).sum(1), "out", dtype)
    gy, gw = tpc.combine_backward(go, y, w)
    near(gy, (Wt[..., None] * G[:, None]).reshape(-1, cols), 0.0, "grad_y", dtype)
    near(gw, (G[:, None] * Y).sum(2), (cols + 2) * U * np.abs(G[:, None] * Y).sum(2), "grad_weight")


def test_stream_and_graph(tpc):
    """The run of an expert layer, captured and replayed with other inputs, routes among them."""
    r = np.random.default_rng(9)
    x, l, go = dev(r.normal(size=(900, 64))), dev(r.normal(size=(900, 6))), dev(r.normal(size=(900, 64)))
    w1, b1, w2 = dev(r.normal(size=(6, 64, 96))), dev(r.normal(size=(6, 96))), dev(r.normal(size=(6, 96, 64)))

    def call():
        weight, index = tpc.route_forward(l, 2)
        g = tpc.group_rows(index, 6)
        h, z = tpc.grouped_linear_forward(x, w1, g, bias=b1, act="silu", y_rows="grouped", want_pre=True)
        y = tpc.grouped_linear_forward(h, w2, g, x_rows="grouped")
        gy, gweight = tpc.combine_backward(go, y, weight)
        gz, gw2, _ = tpc.grouped_linear_backward(gy, h, w2, g, x_rows="grouped", pre=z)
        return (weight, index, *g[:2], tpc.combine_forward(y, weight), gz, gw2,
                *tpc.grouped_linear_backward(gz, x, w1, g, y_rows="grouped", want_bias=True),
                tpc.route_backward(gweight, l, weight, index))

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
        l.copy_(torch.randn_like(l) * (i + 1))
        x.copy_(torch.randn_like(x))
        graph.replay()
        torch.cuda.synchronize()
        assert same(held, call())


WIDE = [  # slots, groups, in, out, kind, fan, x rows, y rows, spare values of a row: sizes that take other tiles
    (700, 40, 72, 136, "even", 1, "source", "source", 0), (700, 40, 136, 72, "skew", 2, "source", "grouped", 8),
    (1000, 118, 256, 128, "skew", 1, "source", "source", 0), (900, 3, 40, 264, "skew", 1, "source", "source", 8),
    (2000, 7, 264, 200, "skew", 2, "source", "grouped", 0), (4098, 3, 512, 520, "skew", 3, "grouped", "source", 0),
    (5000, 5, 1032, 512, "even", 1, "source", "source", 8), (16500, 3, 72, 2056, "even", 2, "source", "grouped", 0),
    (16500, 3, 2056, 72, "skew", 1, "grouped", "source", 0), (4000, 16, 1016, 1032, "skew", 1, "source", "source", 0),
    (16500, 2, 33, 2047, "skew", 1, "source", "source", 0), (16500, 2, 2047, 33, "skew", 2, "source", "grouped", 1),
    (16500, 3, 1023, 2047, "skew", 1, "source", "source", 0),
    (9, 2, 1032, 64, "skew", 1, "source", "source", 0), (130, 3, 264, 1000, "skew", 2, "source", "grouped", 8),
    (17000, 3, 512, 1032, "skew", 1, "source", "source", 0), (3000, 8, 200, 512, "skew", 1, "grouped", "source", 0)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("case", WIDE, ids=str)
def test_grouped_tiles(tpc, dtype, case):
    """Rows of whole 16-byte chunks, and sizes from a few rows a group to many tiles."""
    slots, groups, i, o, kind, fan, x_rows, y_rows, spare = case
    print(f"grouped tiles {dtype} {case}", flush=True)
    r = np.random.default_rng(slots + i + o)
    dt = DT[dtype]
    index = index_of(kind, slots, groups, r)
    g = tpc.group_rows(ints(index).view(-1, fan) if fan > 1 else ints(index), groups)
    ptr, rows = ob.group_rows(index, groups)
    nx = slots // fan if x_rows == "source" else slots
    x = dev(r.normal(size=(nx, i + spare)), dt)[:, spare:]
    w, b = dev(r.normal(size=(groups, i, o)), dt), dev(r.normal(size=(groups, o)), dt)
    gz = dev(r.normal(size=(slots, o + spare)), dt)[:, :o]
    X, Wt, B, G = f64(x), f64(w), f64(b), f64(gz)
    z = ob.grouped_forward(X, Wt, ptr, rows, fan, B, x_rows, y_rows)
    bound = (i + 16) * U * ob.grouped_forward(np.abs(X), np.abs(Wt), ptr, rows, fan, np.abs(B), x_rows, y_rows)
    y, pre = tpc.grouped_linear_forward(x, w, g, bias=b, act="silu", x_rows=x_rows, y_rows=y_rows, want_pre=True)
    near(pre, z, bound, "pre", dtype)
    near(y, ob.silu(f64(pre)), 8 * U * (np.abs(f64(pre)) + 1), "y", dtype)
    assert torch.equal(pre, tpc.grouped_linear_forward(x, w, g, bias=b, x_rows=x_rows, y_rows=y_rows))
    back = tpc.grouped_linear_backward(gz, x, w, g, x_rows=x_rows, y_rows=y_rows, want_bias=True)
    want = ob.grouped_backward(G, X, Wt, ptr, rows, fan, x_rows, y_rows)
    size = abs_parts(G, X, Wt, ptr, rows, fan, x_rows, y_rows)
    parts = (W if dtype == "bf16" else U) if fan > 1 and x_rows == "source" else 0.0
    near(back[0], want[0], ((o + 16 + fan) * U + parts) * size[0], "grad_x", dtype)
    near(back[1], want[1], (slots + 16) * U * size[1], "grad_w", dtype)
    near(back[2], want[2], (slots + 16) * U * size[2], "grad_bias", dtype)
    assert same(back, tpc.grouped_linear_backward(gz, x, w, g, x_rows=x_rows, y_rows=y_rows, want_bias=True))
