"""Operators around the attention block where an element's place does not fit 32 bits: the last rows of
large tensors against the same rows in tensors of their own.  Values are small integers or the formulas
are by element, so that every result is exact and the comparison is for equality."""
import pytest

from tests._blocks import same, torch

pytestmark = pytest.mark.gpu
FAR = 2 ** 31


@pytest.fixture(scope="module")
def tpc():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import tensor_product_convolution_amd as m
    m.lib()
    return m


def whole(*shape, dt=torch.bfloat16, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randint(-3, 4, shape, generator=g, device="cuda", dtype=torch.int8).to(dt)


def strided(rows, cols, stride, **kw):
    """[rows, cols] whose rows lie `stride` apart, the last ones past 2^31 values"""
    assert rows * stride > FAR + 100 * stride
    held = torch.empty(rows, stride, device="cuda", dtype=torch.bfloat16)
    held[:, :cols] = whole(rows, cols, **kw)
    return held[:, :cols]


def test_heads(tpc):
    n, stride = 40000, 60000
    q, gq = strided(n, 128, stride).view(n, 4, 32), strided(n, 128, stride, seed=1).view(n, 4, 32)
    k, gk = whole(n, 2, 32, seed=2), whole(n, 2, 32, seed=3)
    gamma = torch.rand(32, device="cuda") + 0.5
    pos, freq = torch.rand(n, 3, device="cuda") * 20, torch.rand(16, 3, device="cuda", dtype=torch.float64)
    kw = dict(gamma_q=gamma, gamma_k=gamma, freq=freq)
    outs = tuple(torch.empty_strided(t.shape, t.stride(), dtype=t.dtype, device="cuda") for t in (q, k))
    full = tpc.head_norm_rotate_forward(q, k, pos=pos, outs=outs, **kw)
    back = tpc.head_norm_rotate_backward(gq, gk, q, k, pos=pos, want_pos=True, **kw)
    last = slice(n - 50, n)
    tail = [t[last].clone() for t in (gq, gk, q, k, pos)]
    assert same([t[last] for t in full], tpc.head_norm_rotate_forward(*tail[2:4], pos=tail[4], **kw))
    few = tpc.head_norm_rotate_backward(*tail[:4], pos=tail[4], want_pos=True, **kw)
    assert same([back[0][last], back[1][last], back[4][last]], [few[0], few[1], few[4]])


def test_route_and_combine(tpc):
    n, e = 2200000, 1000
    logits = whole(n, e)
    weight, index = tpc.route_forward(logits, 2)
    last = slice(n - 70, n)
    few = tpc.route_forward(logits[last].clone(), 2)
    assert same([weight[last], index[last]], few)
    grad = torch.rand(n, 2, device="cuda")
    assert torch.equal(tpc.route_backward(grad, logits, weight, index)[last],
                       tpc.route_backward(grad[last].clone(), logits[last].clone(), *few))
    y, go = whole(n, e, seed=4), whole(n // 2, e, seed=5)
    w = whole(n // 2, 2, dt=torch.float32, seed=6)
    last = slice(n // 2 - 35, n // 2)
    slots = slice(n - 70, n)
    tail = y[slots].clone(), w[last].clone()
    assert torch.equal(tpc.combine_forward(y, w)[last], tpc.combine_forward(*tail))
    gy, gw = tpc.combine_backward(go, y, w)
    assert same([gy[slots], gw[last]], tpc.combine_backward(go[last].clone(), *tail))


def test_grouped_rows(tpc):
    """Rows far behind the first, of any alignment and of whole chunks."""
    n, stride, last = 40000, 60000, slice(40000 - 300, 40000)
    index = torch.randint(-1, 5, (n,), device="cuda", dtype=torch.int32)
    few = tpc.group_rows(index[last].clone(), 5)
    many = tpc.group_rows(index, 5)
    for i, o in ((40, 64), (33, 21)):
        x, gz, p = strided(n, i, stride), strided(n, o, stride, seed=7), strided(n, i, stride, seed=8)
        w, b = whole(5, i, o, seed=9), whole(5, o, seed=10)
        tail = [t[last].clone() for t in (x, gz, p)]
        assert torch.equal(tpc.grouped_linear_forward(x, w, many, bias=b)[last], tpc.grouped_linear_forward(tail[0], w, few, bias=b))
        gx, gw, _ = tpc.grouped_linear_backward(gz, x, w, many, pre=p)
        assert torch.equal(gx[last], tpc.grouped_linear_backward(tail[1], tail[0], w, few, pre=tail[2])[0])
        want = torch.stack([x[index == e].float().T @ gz[index == e].float() for e in range(5)])
        assert torch.equal(gw, want.bfloat16())


def test_grouped_weights(tpc):
    """Weights of the last group lie past 2^31 values."""
    e, i, o = 70, 4096, 8192
    w = torch.empty(e, i, o, device="cuda", dtype=torch.bfloat16)
    w[:2], w[-2:] = whole(2, i, o), whole(2, i, o, seed=1)
    index = torch.tensor([0, 69, 68, 69, -1, 1, 69], device="cuda", dtype=torch.int32)
    x, gz = whole(7, i, seed=2), whole(7, o, seed=3)
    near, far = torch.tensor([0, 5], device="cuda"), torch.tensor([1, 2, 3, 6], device="cuda")
    g = tpc.group_rows(index, e)
    y = tpc.grouped_linear_forward(x, w, g)
    gx, gw, _ = tpc.grouped_linear_backward(gz, x, w, g)
    for rows, part in ((near, slice(0, 2)), (far, slice(e - 2, e))):
        own = tpc.group_rows((index[rows] - part.start).contiguous(), 2)
        a = [x[rows].clone(), w[part].clone(), own]
        assert torch.equal(y[rows], tpc.grouped_linear_forward(*a))
        few = tpc.grouped_linear_backward(gz[rows].clone(), *a)
        assert torch.equal(gx[rows], few[0]) and torch.equal(gw[part], few[1])
    assert (gw[2:-2] == 0).all() and (y[4] == 0).all()


@pytest.mark.parametrize("bits", [32, 8])
def test_adamw(tpc, bits):
    n, last = FAR + 5000, 3000
    p, g = torch.ones(n, device="cuda"), torch.ones(n, device="cuda", dtype=torch.bfloat16)
    p[-last:], g[-last:] = torch.rand(last, device="cuda"), whole(last)
    few_p, few_g = p[-last:].clone(), g[-last:].clone()
    many, few = tpc.AdamW([p], bits=bits), tpc.AdamW([few_p], bits=32)
    many.step([g])
    few.step([few_g])
    # states of 8 bits begin with the first step's exact value times their blocks' unit: the step itself is exact
    assert torch.equal(p[-last:], few_p)
    assert bool((p[:1000] == p[0]).all()) and float(p[0]) < 1
    many.step([g])
    few.step([few_g])
    if bits == 32:
        assert torch.equal(p[-last:], few_p)
    else:
        assert torch.isfinite(p[-last:]).all()
