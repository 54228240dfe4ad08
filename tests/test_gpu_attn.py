"""Attention on the GPU against the float64 reference, element by element.

Tolerances (derived, per element): with u = 2^-24, a score's error is at most
(2 D + 8) u times the sum of its absolute products plus 4 u |s| (rounded bias and
statistics), which multiplies each probability's relative error; sums over n rows in
float32 add n u of the sum of absolute terms.  So float32 outputs may differ by
    e32 = u (n + 2 D + 32 + 4 smax)   (smax: the largest sum of absolute products of a score, plus |bias|, lse)
times the output formed from absolute values.  In bfloat16 (8 significand bits: unit roundoff w = 2^-8)
probabilities and score gradients are rounded once before their products, out is
rounded before grad_out . out, and every output once: 4 w times the absolute-value
output on top, plus w |reference|.  Probabilities below 2^-126 are flushed to 0, so a
sum of n of them times factors up to F may be off by n F 2^-126 besides; FLUSH = 1e-30
covers n F up to 8e7.
"""
import numpy as np
import pytest

from oracle import layers as ol

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
U, W, FLUSH = 2.0 ** -24, 2.0 ** -8, 1e-30


@pytest.fixture(scope="module")
def tpc():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import tensor_product_convolution_amd as m
    m.lib()
    return m


DT = {"f32": torch.float32, "bf16": torch.bfloat16}


class Case:
    def __init__(self, dtype, lens, hq, hk, d, nb=0, masked=0.0, seed=0, steps=4, box=None, packed=True, r_min=0.5):
        r = np.random.default_rng(seed)
        n = sum(lens)
        dt = DT[dtype]
        dev = lambda a, t: torch.tensor(np.asarray(a), device="cuda").to(t)
        self.lens, self.dtype, self.d = lens, dtype, d
        self.seg = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
        # queries, keys and values as views of one row (strides) or on their own
        row = dev(r.normal(size=(n, (hq + 2 * hk) * d)), dt)
        q, k, v = (t.view(n, -1, d) for t in row.split([hq * d, hk * d, hk * d], dim=1))
        if not packed:
            q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
        self.q, self.k, self.v = q, k, v
        self.go = dev(r.normal(size=(n, hq, d)), dt)
        self.kw = dict(r_min=r_min, steps=steps)
        if nb:
            box = box or (max(max(lens), 1) / 0.05) ** (1 / 3)
            self.kw.update(pos=dev(r.uniform(0, box, size=(n, 3)), torch.float32), bias=dev(r.normal(size=(hq, nb)), dt))
        if masked:
            self.kw["key_mask"] = torch.tensor((r.uniform(size=n) >= masked).astype(np.uint8), device="cuda")
        self.segt = torch.tensor(self.seg, device="cuda")

    def run(self, tpc):
        self.out, self.lse = tpc.attn_forward(self.q, self.k, self.v, self.segt, **self.kw)
        self.grads = tpc.attn_backward(self.q, self.k, self.v, self.segt, self.out, self.lse, self.go, **self.kw)
        torch.cuda.synchronize()
        return self

    def host(self):
        f = lambda t: t.double().cpu().numpy() if t.is_floating_point() else t.cpu().numpy()
        kw = {n: f(t) if isinstance(t, torch.Tensor) else t for n, t in self.kw.items()}
        if "pos" in kw:
            kw["pos"] = kw["pos"].astype(np.float32)
        return dict(q=f(self.q), k=f(self.k), v=f(self.v), seg_ptr=self.seg), kw, f(self.go)

    def bounds(self):
        """Elementwise bounds of (out, lse, grad_q, grad_k, grad_v, grad_bias)."""
        c, kw, go = self.host()
        b = [np.zeros(c["q"].shape), np.zeros((c["q"].shape[1], c["q"].shape[0])), np.zeros(c["q"].shape),
             np.zeros(c["k"].shape), np.zeros(c["v"].shape), np.zeros(kw["bias"].shape) if "bias" in kw else None]
        low = self.dtype == "bf16"
        full = dict(pos=None, bias=None, key_mask=None, scale=None)
        full.update(kw)
        for sl, h, g, bk, live, q, k, v, p, lse, sc in ol._each(**c, **full):
            (n, d), sc = q.shape, abs(sc)
            smax = float((np.abs(q) @ np.abs(k).T).max() * sc) + np.abs(lse[np.isfinite(lse)]).max(initial=0.0)
            if bk is not None:
                smax += np.abs(kw["bias"][h][np.isfinite(kw["bias"][h])]).max(initial=0.0)
            e = U * (n + 2 * d + 32 + 4 * smax + (2 * d + 8) * smax)
            a = np.abs(go[sl, h]) @ np.abs(v).T
            A = p * (a + (p * a).sum(axis=1, keepdims=True))
            f, w = (e + 4 * W if low else e), (W if low else 2 * U)
            b[0][sl, h] = f * (p @ np.abs(v))
            b[1][h, sl] = e + 4 * U * np.abs(np.where(np.isfinite(lse), lse, 0))
            b[2][sl, h] = sc * f * (A @ np.abs(k))
            b[3][sl, g] += sc * f * (A.T @ np.abs(q))
            b[4][sl, g] += f * (p.T @ np.abs(go[sl, h]))
            if b[5] is not None:
                np.add.at(b[5][h], bk, f * A)
        return b

    def check(self, tpc):
        self.run(tpc)
        c, kw, go = self.host()
        ref = [*ol.attn_forward(**c, **kw), *ol.attn_backward(**c, **kw, grad_out=go)]
        got = [self.out, self.lse, *self.grads]
        names = ("out", "lse", "grad_q", "grad_k", "grad_v", "grad_bias")
        w = W if self.dtype == "bf16" else 2 * U
        for name, g, r, b in zip(names, got, ref, self.bounds()):
            if r is None:
                assert g is None
                continue
            g = g.double().cpu().numpy()
            fin = np.isfinite(r)
            assert np.array_equal(fin, np.isfinite(g)) and np.array_equal(g[~fin], r[~fin]), name
            extra = 2 * U if name == "lse" else w
            over = np.abs(g - r)[fin] - (b[fin] + extra * np.abs(r[fin]) + FLUSH)
            assert over.size == 0 or over.max() <= 0, (name, float(over.max()), float(np.abs(g - r)[fin].max()))
        return self


# one, two, tile edges and long rows; empty structures; both sides of each variant's rule
LENS = [[1], [2, 0, 1], [31, 32, 33], [64, 65, 5, 0, 0, 63], [200], [129, 1, 260], [3] * 70]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("lens", LENS, ids=str)
def test_lengths(tpc, dtype, lens):
    print(f"attn lengths {dtype} {lens}", flush=True)
    Case(dtype, lens, 4, 4, 16, nb=32).check(tpc)
    Case(dtype, lens, 4, 2, 32, nb=20, masked=0.2, seed=1).check(tpc)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("d", [8, 16, 24, 32, 40, 48, 56, 64, 72, 80, 88, 96, 104, 112, 120, 128])
def test_head_widths(tpc, dtype, d):
    print(f"attn width {dtype} {d}", flush=True)
    Case(dtype, [70, 9], 2, 2, d, nb=8).check(tpc)
    Case(dtype, [40], 2, 1, d, nb=64, masked=0.1).check(tpc)
    Case(dtype, [150], 1, 1, d).check(tpc)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("heads", [(1, 1), (3, 3), (5, 1), (8, 2), (6, 2), (6, 3), (12, 4), (16, 16), (7, 7)])
def test_head_layouts(tpc, dtype, heads):
    print(f"attn heads {dtype} {heads}", flush=True)
    Case(dtype, [37, 80], *heads, 16, nb=33, masked=0.1).check(tpc)
    Case(dtype, [37, 80], *heads, 64, nb=9, packed=False).check(tpc)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("width", [16, 40, 64, 128])
def test_many_tiles(tpc, dtype, width):
    """Enough query tiles for the variants that share staged keys between waves."""
    print(f"attn many tiles {dtype} {width}", flush=True)
    Case(dtype, [90] * 60 + [1, 0, 200], 16, 8, width, nb=16, masked=0.05).check(tpc)


@pytest.mark.parametrize("nb,steps,box,r_min", [(1, 4, 5.0, 0.5), (64, 1, 300.0, 1e-3), (64, 8, 3.0, 0.5), (2, 2, 10.0, 4.0),
                                                (63, 4, 0.0, 0.5), (32, 4, 1e6, 0.5)])
def test_bucket_ranges(tpc, nb, steps, box, r_min):
    print(f"attn buckets {nb} {steps} {box}", flush=True)
    Case("f32", [70], 2, 2, 16, nb=nb, steps=steps, box=box or 1e-30, r_min=r_min).check(tpc)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_rows_without_keys(tpc, dtype):
    """Structures whose mask leaves nothing, beside ones that it does not touch."""
    c = Case(dtype, [40, 33, 1, 64], 4, 2, 32, nb=16, masked=0.5)
    c.kw["key_mask"][:40] = 0
    c.kw["key_mask"][73] = 0
    c.check(tpc)
    assert not c.out[:40].any() and torch.all(c.lse[:, :40] == -np.inf)
    for g in c.grads[:3]:
        assert not g[:40].any() and not g[73].any()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("low", [-np.inf, "lowest"])
def test_bias_that_masks(tpc, dtype, low):
    """Buckets masked by -inf or by the type's lowest value: pairs beyond a cutoff; then
    every bucket, which leaves every row empty."""
    low = torch.finfo(DT[dtype]).min if low == "lowest" else low
    c = Case(dtype, [70, 34], 2, 2, 16, nb=16, box=4.0)
    c.kw["bias"][:, 9:] = low
    c.check(tpc)
    c.kw["bias"][:] = low
    c.check(tpc)
    assert not c.out.any() and not any(g.any() for g in c.grads)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("bad", [np.nan, np.inf, -np.inf])
def test_masked_rows_may_hold_anything(tpc, dtype, bad):
    c = Case(dtype, [70, 20], 4, 2, 32, nb=16, masked=0.3, packed=False).run(tpc)
    dead = c.kw["key_mask"] == 0
    want = [c.out.clone(), c.lse.clone(), *(g.clone() for g in c.grads)]
    c.k[dead], c.v[dead] = bad, bad
    c.run(tpc)
    for g, w in zip([c.out, c.lse, *c.grads], want):
        assert torch.equal(g, w)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_nan_in_a_live_row_shows(tpc, dtype):
    c = Case(dtype, [40, 40], 2, 2, 16, nb=8, packed=False)
    c.k[3, 0, 0] = np.nan
    c.run(tpc)
    assert torch.isnan(c.out[:40, 0]).all() and not torch.isnan(c.out[40:]).any() and not torch.isnan(c.out[:, 1]).any()


@pytest.mark.parametrize("scale", [0.0, -0.5, 3.0])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_scales(tpc, dtype, scale):
    """A scale of zero (bias alone), a negative one, a large one."""
    c = Case(dtype, [50, 70], 4, 2, 16, nb=16, masked=0.1)
    c.kw["scale"] = scale
    c.check(tpc)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_bias_gradient_of_one_crowded_bucket(tpc, dtype):
    """Nearly all pairs in the last bucket: its gradient is a sum of cancelling terms.  The
    tolerance is that of the smaller buckets' own bound, far below n u of the terms."""
    c = Case(dtype, [600, 500], 4, 2, 32, nb=8, seed=7).run(tpc)
    h, kw, go = c.host()
    ref = ol.attn_backward(**h, **kw, grad_out=go)[3]
    got = c.grads[3].double().cpu().numpy()
    # bfloat16: rounded once; float32: 2^-16 of the head's largest bucket
    tol = (W if dtype == "bf16" else 2.0 ** -16) * np.abs(ref).max(axis=1, keepdims=True)
    assert (np.abs(got - ref) <= tol).all(), np.abs(got - ref).max()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_large_scores(tpc, dtype):
    """Scores that overflow exp without the running maximum, growing along the keys."""
    c = Case(dtype, [150], 2, 2, 16, packed=False)
    # one direction dominates: scores rise in steps of 4 to 600
    c.q[:] = 0
    c.q[:, :, 0] = 4
    c.k[:, :, 0] = (torch.arange(150, device="cuda") * 4)[:, None].to(c.k.dtype)
    c.check(tpc)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_repeated_calls_are_bitwise_equal_and_strided_outputs_match(tpc, dtype):
    c = Case(dtype, [150, 33, 90], 4, 2, 24, nb=40, masked=0.1).run(tpc)
    first = [c.out.clone(), c.lse.clone(), *(g.clone() for g in c.grads)]
    c.run(tpc)
    assert all(torch.equal(a, b) for a, b in zip(first, [c.out, c.lse, *c.grads]))
    n = c.q.shape[0]
    row = torch.full((n, 9 * 24), 7.0, device="cuda", dtype=DT[dtype])
    views = [t.view(n, -1, 24) for t in row[:, :8 * 24].split([96, 48, 48], dim=1)]
    tpc.attn_backward(c.q, c.k, c.v, c.segt, c.out, c.lse, c.go, **c.kw, outs=views)
    out = row[:, 24:120].view(n, 4, 24).clone()
    assert all(torch.equal(a, b) for a, b in zip(views, first[2:5]))
    assert torch.all(row[:, 8 * 24:] == 7.0)
    del out
    wide = torch.full((n, 5 * 24), 7.0, device="cuda", dtype=DT[dtype])
    tpc.attn_forward(c.q, c.k, c.v, c.segt, **c.kw, out=wide[:, :96].view(n, 4, 24))
    assert torch.equal(wide[:, :96].reshape(n, 4, 24), first[0]) and torch.all(wide[:, 96:] == 7.0)


def test_gradients_by_differences(tpc):
    """grad_* of the kernels against differences of the kernels' own forward.  Step h =
    2^-6 along a random direction: truncation h^2 |f'''| / 6 and rounding of the
    loss, about 2^-22 |loss| / h, both below 1e-2 of the derivative's scale."""
    c = Case("f32", [40, 21], 4, 2, 16, nb=12, masked=0.2, packed=False).run(tpc)
    r = np.random.default_rng(9)
    loss = lambda: float((tpc.attn_forward(c.q, c.k, c.v, c.segt, **c.kw)[0].double() * c.go.double()).sum())
    for t, g in zip((c.q, c.k, c.v, c.kw["bias"]), c.grads):
        keep = t.clone()
        d = torch.tensor(r.normal(size=tuple(t.shape)), device="cuda", dtype=torch.float32)
        h = 2.0 ** -6
        t.copy_(keep + h * d)
        up = loss()
        t.copy_(keep - h * d)
        down = loss()
        t.copy_(keep)
        want = float((g.double() * d.double()).sum())
        assert abs((up - down) / (2 * h) - want) < 1e-2 * float((g.double().abs() * d.double().abs()).sum()) ** 1.0


def test_other_stream_and_graph_replay(tpc):
    """On a side stream, and captured in a HIP graph that is replayed between eager work."""
    c = Case("bf16", [100, 60], 4, 4, 32, nb=16, masked=0.1).run(tpc)
    want = [c.out.clone(), *(g.clone() for g in c.grads)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        c.run(tpc)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, [c.out, *c.grads]))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out, lse = tpc.attn_forward(c.q, c.k, c.v, c.segt, **c.kw)
        grads = tpc.attn_backward(c.q, c.k, c.v, c.segt, out, lse, c.go, **c.kw)
    for _ in range(3):
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, [out, *grads]))
        c.run(tpc)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_offsets_beyond_32_bits(tpc, dtype):
    """Rows far apart: element offsets pass 2^31.  Bit for bit the results of dense rows."""
    n, wide = 36000, 1 << 16
    dt = DT[dtype]
    big = torch.empty(n, wide, device="cuda", dtype=dt)
    g = torch.Generator(device="cuda").manual_seed(1)
    big[:, -96:] = torch.randn(n, 96, device="cuda", generator=g).to(dt)
    q, k, v = (big[:, -96 + 32 * i:wide - 64 + 32 * i].view(n, 2, 16) for i in range(3))
    seg = torch.arange(0, n + 1, 60, device="cuda", dtype=torch.int32)
    pos = 4 * torch.rand(n, 3, device="cuda", generator=g)
    bias = torch.randn(2, 8, device="cuda", generator=g).to(dt)
    go = torch.randn(n, 2, 16, device="cuda", generator=g).to(dt)
    res = []
    for a in ((q, k, v), tuple(t.contiguous() for t in (q, k, v))):
        out, lse = tpc.attn_forward(*a, seg, pos=pos, bias=bias)
        outs = [torch.empty(n, wide, device="cuda", dtype=dt)[:, -32:].view(n, 2, 16) for _ in range(3)] if a[0] is q else None
        res.append([out, lse, *tpc.attn_backward(*a, seg, out, lse, go, pos=pos, bias=bias, outs=outs)])
    assert all(torch.equal(x, y) for x, y in zip(*res))


def test_empty_batches(tpc):
    e = lambda *s: torch.empty(*s, device="cuda")
    seg = torch.zeros(1, dtype=torch.int32, device="cuda")
    bias = torch.zeros(4, 8, device="cuda")
    for s in (seg, torch.zeros(4, dtype=torch.int32, device="cuda")):
        out, lse = tpc.attn_forward(e(0, 4, 16), e(0, 2, 16), e(0, 2, 16), s, pos=e(0, 3), bias=bias)
        g = tpc.attn_backward(e(0, 4, 16), e(0, 2, 16), e(0, 2, 16), s, out, lse, e(0, 4, 16), pos=e(0, 3), bias=bias)
        assert out.shape == (0, 4, 16) and lse.shape == (4, 0) and torch.equal(g[3], torch.zeros_like(bias))


def test_binding_refusals(tpc):
    c = Case("f32", [20], 4, 2, 16, nb=8)
    f = lambda **kw: tpc.attn_forward(**{**dict(q=c.q, k=c.k, v=c.v, seg_ptr=c.segt), **c.kw, **kw})
    with pytest.raises(TypeError):
        f(k=c.k.bfloat16())
    with pytest.raises(TypeError):
        f(q=c.q.double(), k=c.k.double(), v=c.v.double())
    with pytest.raises(TypeError):
        f(seg_ptr=c.segt.long())
    with pytest.raises(ValueError):
        f(v=c.v[:, :1])
    with pytest.raises(ValueError):
        f(q=c.q.transpose(0, 1))
    with pytest.raises(ValueError):
        f(pos=None)
    with pytest.raises(ValueError):
        f(k=c.k.cpu())
    with pytest.raises(ValueError):
        f(bias=c.kw["bias"][:3])
    with pytest.raises(tpc.TPError):
        f(steps=3)
    with pytest.raises(tpc.TPError):
        f(q=torch.zeros(20, 4, 12, device="cuda"), k=torch.zeros(20, 2, 12, device="cuda"),
          v=torch.zeros(20, 2, 12, device="cuda"))
    with pytest.raises(ValueError):
        f(key_mask=torch.ones(19, dtype=torch.uint8, device="cuda"))


def test_wrong_offsets_stay_in_bounds(tpc):
    """Offsets outside [0, n_nodes] or out of order: results are unspecified, accesses are not."""
    c = Case("f32", [40, 40], 2, 2, 16, nb=8)
    for bad in ([0, 5000, 80], [0, -7, 80], [60, 20, 80], [0, 40, 2 ** 31 - 1]):
        c.segt = torch.tensor(bad, dtype=torch.int32, device="cuda")
        c.run(tpc)
