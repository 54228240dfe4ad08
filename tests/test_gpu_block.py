"""The operators around the attention block in a run, as a program uses them: norm and
rotation, attention, residual norm, elements, router, experts, AdamW, against the float64
references and, in the example, against differences."""
import importlib.util
import os

import numpy as np
import pytest

from oracle import blocks as ob
from oracle import layers as ol
from tests._blocks import dev, f64, ints, torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def tpc():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import tensor_product_convolution_amd as m
    m.lib()
    return m


@pytest.fixture(scope="module")
def example(tpc):
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "atom_attention.py")
    spec = importlib.util.spec_from_file_location("atom_attention", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_a_training_step(tpc):
    """Two sequences of the run: forward, backward and the step of all weights.

    Tolerance (derived): each operator's outputs are off by at most (K + 40) u of their absolute terms, K
    at most 256 here: 2e-5; absolute terms are at most sqrt(K) = 16 times the values in the 2-norm
    (sums of terms of random sign), and ten operators follow each other, whose gradients pass on
    errors about as large as themselves: 10 16 2e-5 = 3e-3 of each result's 2-norm."""
    r = np.random.default_rng(8)
    n, hq, hk, d, u, e, k, hidden, kinds = 150, 4, 2, 16, 64, 5, 2, 96, 3
    sizes = [60, 1, 89]
    seg = np.concatenate([[0], np.cumsum(sizes)])
    pos, freq = r.uniform(0, 12, size=(n, 3)).astype(np.float32), r.normal(size=(6, 3))
    W = {m: r.normal(size=s) * t for m, s, t in (
        ("qkv", (u, (hq + 2 * hk) * d), u ** -0.5), ("out", (hq * d, u), (hq * d) ** -0.5), ("bias", (hq, 20), 0.3),
        ("element", (kinds, u, u), u ** -0.5), ("router", (u, e), u ** -0.5), ("up", (e, u, hidden), u ** -0.5),
        ("b", (e, hidden), 0.1), ("down", (e, hidden, u), hidden ** -0.5))}
    W.update(gq=1 + 0.2 * r.normal(size=d), gk=1 + 0.2 * r.normal(size=d), gamma=1 + 0.2 * r.normal(size=u), beta=0.1 * r.normal(size=u))
    P = {m: dev(t) for m, t in W.items()}
    W = {m: f64(t) for m, t in P.items()}
    x, go, kind = dev(r.normal(size=(n, u))), dev(r.normal(size=(n, u))), r.integers(-1, kinds, size=n)
    # on the GPU
    turn = dict(gamma_q=P["gq"], gamma_k=P["gk"], pos=dev(pos), freq=torch.tensor(freq, device="cuda"))
    attn = dict(pos=dev(pos), bias=P["bias"], r_min=0.5, steps=4)
    qkv = x @ P["qkv"]
    q, kk, v = [t.view(n, -1, d) for t in qkv.split([hq * d, hk * d, hk * d], 1)]
    qr, kr = tpc.head_norm_rotate_forward(q, kk, **turn)
    o, lse = tpc.attn_forward(qr, kr, v, ints(seg), **attn)
    z, mean, rstd, h = tpc.layer_norm_residual_forward(o.view(n, -1) @ P["out"], x, P["gamma"], P["beta"])
    el = tpc.group_rows(ints(kind), kinds)
    s = z + tpc.grouped_linear_forward(z, P["element"], el)
    logits = s @ P["router"]
    weight, index = tpc.route_forward(logits, k)
    ex = tpc.group_rows(index, e)
    a, pre = tpc.grouped_linear_forward(s, P["up"], ex, bias=P["b"], act="silu", y_rows="grouped", want_pre=True)
    y = tpc.grouped_linear_forward(a, P["down"], ex, x_rows="grouped")
    out = s + tpc.combine_forward(y, weight)
    gy, gweight = tpc.combine_backward(go, y, weight)
    gz, g_down, _ = tpc.grouped_linear_backward(gy, a, P["down"], ex, x_rows="grouped", pre=pre)
    gs, g_up, g_b = tpc.grouped_linear_backward(gz, s, P["up"], ex, y_rows="grouped", want_bias=True)
    gl = tpc.route_backward(gweight, logits, weight, index)
    gs = go + gs + gl @ P["router"].t()
    ge, g_el, _ = tpc.grouped_linear_backward(gs, z, P["element"], el)
    gh, gx, g_gamma, g_beta = tpc.layer_norm_residual_backward(gs + ge, h, P["gamma"], mean, rstd)
    gqr, gkr, gv, g_bias = tpc.attn_backward(qr, kr, v, ints(seg), o, lse, (gh @ P["out"].t()).view(n, hq, d), **attn)
    gq, gk, g_gq, g_gk, gpos = tpc.head_norm_rotate_backward(gqr, gkr, q, kk, want_pos=True, **turn)
    grads = dict(qkv=x.t() @ torch.cat([t.reshape(n, -1) for t in (gq, gk, gv)], 1), out=o.view(n, -1).t() @ gh, bias=g_bias,
                 element=g_el, router=s.t() @ gl, up=g_up, b=g_b, down=g_down, gq=g_gq, gk=g_gk, gamma=g_gamma, beta=g_beta)
    # in float64
    X = f64(x)
    Q, K, V = [t.reshape(n, -1, d) for t in np.split(X @ W["qkv"], [hq * d, (hq + hk) * d], 1)]
    side = (pos, freq, False, 1e-6)
    QR, KR = ob.head_forward(Q, W["gq"], *side), ob.head_forward(K, W["gk"], *side)
    O, _ = ol.attn_forward(QR, KR, V, seg, pos=pos, bias=W["bias"], r_min=0.5, steps=4)
    H = O.reshape(n, -1) @ W["out"] + X
    Z, _, _ = ol.layer_norm_forward(H, W["gamma"], W["beta"], 1e-5)
    ep, er = ob.group_rows(kind, kinds)
    S = Z + ob.grouped_forward(Z, W["element"], ep, er, 1, None, "source", "source")
    L = S @ W["router"]
    RW, RI = ob.route(L, k)
    assert np.array_equal(index.cpu().numpy(), RI)             # no choice is within rounding of another here
    xp, xr = ob.group_rows(RI, e)
    PRE = ob.grouped_forward(S, W["up"], xp, xr, k, W["b"], "source", "grouped")
    Y = ob.grouped_forward(ob.silu(PRE), W["down"], xp, xr, k, None, "grouped", "source")
    G = f64(go)
    OUT = S + (RW[..., None] * Y.reshape(n, k, u)).sum(1)
    GY, GW = (RW[..., None] * G[:, None]).reshape(-1, u), (G[:, None] * Y.reshape(n, k, u)).sum(2)
    GZ, D_DOWN, _ = ob.grouped_backward(GY, ob.silu(PRE), W["down"], xp, xr, k, "grouped", "source", pre=PRE)
    GS, D_UP, D_B = ob.grouped_backward(GZ, S, W["up"], xp, xr, k, "source", "grouped")
    GL = ob.route_backward(GW, L, RW, RI)
    GS = G + GS + GL @ W["router"].T
    GE, D_EL, _ = ob.grouped_backward(GS, Z, W["element"], ep, er, 1, "source", "source")
    GH, D_GAMMA, D_BETA = ol.layer_norm_backward(GS + GE, H, W["gamma"], 1e-5)
    GQR, GKR, GV, D_BIAS = ol.attn_backward(QR, KR, V, seg, (GH @ W["out"].T).reshape(n, hq, d), pos=pos, bias=W["bias"], r_min=0.5, steps=4)
    (GQ, D_GQ, p1), (GK, D_GK, p2) = ob.head_backward(GQR, Q, W["gq"], *side), ob.head_backward(GKR, K, W["gk"], *side)
    want = dict(qkv=X.T @ np.concatenate([t.reshape(n, -1) for t in (GQ, GK, GV)], 1), out=O.reshape(n, -1).T @ GH, bias=D_BIAS,
                element=D_EL, router=S.T @ GL, up=D_UP, b=D_B, down=D_DOWN, gq=D_GQ, gk=D_GK, gamma=D_GAMMA, beta=D_BETA)
    off = lambda got, ref: np.linalg.norm(f64(got) - ref) / np.linalg.norm(ref)
    assert off(out, OUT) < 3e-3 and off(gpos, p1 + p2) < 3e-3
    for name in want:
        assert off(grads[name], want[name]) < 3e-3, name
    # the step: where a gradient is far from zero its sign alone decides the first step's size
    names = sorted(P)
    before = {m: P[m].clone() for m in names}
    opt = tpc.AdamW([P[m] for m in names], lr=1e-2, weight_decay=0.1, max_norm=1.0)
    norm = opt.step([grads[m] for m in names])
    total = np.sqrt(sum((want[m] ** 2).sum() for m in names))
    assert abs(float(norm) - total) < 3e-3 * total
    for m in names:
        g = f64(grads[m])
        p, _, _ = ob.adamw(f64(before[m]), g, 0 * g, 0 * g, 1, 1e-2, 0.9, 0.999, 1e-8, 0.1, min(1.0, 1.0 / float(norm)))
        assert np.abs(f64(P[m]) - p).max() < 1e-2 * 64 * 2.0 ** -24 + 4 * 2.0 ** -24 * np.abs(p).max(), m


def test_example_runs(example):
    losses = example.train(steps=5, report=lambda s: None, full=True)
    assert len(losses) == 5 and all(np.isfinite(losses))


def test_example_gradients_by_differences(example):
    """Directional differences of sum(out * c) in every weight and in f, with all experts chosen, so that
    no choice changes.  Step 2^-8: the truncation and the rounding of the loss stay below 2e-2 of the
    sum of absolute terms."""
    gen = torch.Generator(device="cuda").manual_seed(3)
    sizes = (20, 1, 33)
    pos, _, _, seg, _ = example.batch(sizes, 4, 3)
    n = sum(sizes)
    layer = example.FullLayer(32, 0.2, gen, experts=2, chosen=2)
    kind = torch.randint(0, layer.kinds, (n,), device="cuda", generator=gen, dtype=torch.int32)
    rows = torch.randn(n, 96, device="cuda", generator=gen)
    f = rows[:, :32]
    c = torch.randn(n, 32, device="cuda", generator=gen)
    loss = lambda: float((layer.forward(f, seg, pos, 5, kind)[0].double() * c.double()).sum())
    out, saved = layer.forward(f, seg, pos, 5, kind)
    grad_f, grads = layer.backward(c, saved)
    assert set(grads) == set(layer.w) - {"readout"}
    for name, g in [("f", grad_f), *grads.items()]:
        t = f if name == "f" else layer.w[name]
        keep, way, h = t.clone(), torch.randn(t.shape, device="cuda", generator=gen), 2.0 ** -8
        t.copy_(keep + h * way)
        up = loss()
        t.copy_(keep - h * way)
        down = loss()
        t.copy_(keep)
        want = float((g.double() * way.double()).sum())
        assert abs((up - down) / (2 * h) - want) < 2e-2 * float((g * way).abs().double().sum()), name
