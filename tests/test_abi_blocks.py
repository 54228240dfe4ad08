"""Refusals of the entry points around the attention block (norm and rotation, routing, products
by group, the AdamW step): every case is caught on the host before a HIP call, so these run
without a GPU; and sizes that the C entry points do not hold are refused by the binding."""
import ctypes
import os

import pytest

import tensor_product_convolution_amd as tpc
from tensor_product_convolution_amd import blocks

pytestmark = pytest.mark.skipif(not os.path.exists(tpc.LIB_PATH),
                                reason="libtpconv.so not built (run __graft_entry__.build())")

A, B, C, D, ODD = (ctypes.c_void_p(x) for x in (0x10000, 0x20000, 0x30000, 0x40000, 0x10001))
F32, BF16 = 0, 1
ARG, UNSUP, OVER, WS = -1, -3, -4, -5
NAN, INF = float("nan"), float("inf")


def err():
    return tpc.lib().tp_conv_last_error().decode()


# ---- norm and rotation ----------------------------------------------------------------
def _heads(**kw):
    v = dict(dtype=F32, n_heads=4, n_kv_heads=2, head_dim=16, n_rows=8000, gamma_q=A.value, gamma_k=A.value, eps=1e-6, pos_type=0,
             axes=3, pos=A.value, freq=A.value, n_pairs=8, interleaved=0)
    v.update(kw)
    return blocks._Heads(*v.values())


def _fwd(q=A, qs=64, k=A, ks=32, qo=B, qos=64, ko=C, kos=32, **kw):
    return tpc.lib().tp_head_norm_rotate_forward(ctypes.byref(_heads(**kw)), q, qs, k, ks, qo, qos, ko, kos, None)


def _bwd(gqo=A, gko=A, q=A, k=A, gq=B, gk=C, ggq=D, ggk=D, gpos=D, ws=D, nws=1 << 30, s=64, t=32, **kw):
    return tpc.lib().tp_head_norm_rotate_backward(ctypes.byref(_heads(**kw)), gqo, s, gko, t, q, s, k, t, gq, s, gk, t, ggq, ggk,
                                                  gpos, ws, nws, None)


BAD_HEADS = [dict(dtype=2), dict(n_rows=-1), dict(n_heads=0), dict(n_kv_heads=0), dict(gamma_q=None), dict(gamma_k=None),
             dict(eps=-1e-6), dict(eps=NAN), dict(eps=INF), dict(n_pairs=9), dict(n_pairs=-1), dict(interleaved=2), dict(pos_type=2),
             dict(pos=None), dict(freq=None), dict(pos=0x10001), dict(freq=0x10004), dict(gamma_q=0x10002)]


@pytest.mark.parametrize("bad", BAD_HEADS, ids=str)
def test_heads_descriptions(bad):
    assert _fwd(**bad) == ARG and _bwd(**bad) == ARG


def test_heads():
    for kw in (dict(head_dim=0), dict(head_dim=257, n_pairs=0), dict(n_heads=1025), dict(n_kv_heads=1025), dict(axes=0), dict(axes=4)):
        big = dict(qs=1 << 20, ks=1 << 20, qos=1 << 20, kos=1 << 20)
        assert _fwd(**kw, **big) == UNSUP and _bwd(**kw, s=1 << 20, t=1 << 20) == UNSUP, kw
    assert _fwd(n_rows=1 << 50) == OVER
    for name in ("q", "k", "qo", "ko"):
        assert _fwd(**{name: None}) == ARG and _fwd(**{name: ODD}) == ARG, name
    for name in ("qs", "ks", "qos", "kos"):
        assert _fwd(**{name: 31}) == ARG and "stride" in err()
        assert _fwd(**{name: 1 << 60}) == ARG
    for name in ("gqo", "gko", "q", "k", "gq", "gk"):
        assert _bwd(**{name: None}) == ARG and _bwd(**{name: ODD}) == ARG, name
    assert _bwd(ggq=None) == ARG and _bwd(ggk=None) == ARG     # both or none
    assert _bwd(gamma_q=None, gamma_k=None) == ARG and "without a norm" in err()
    assert _bwd(pos_type=1) == ARG and "float32 positions" in err()
    assert _bwd(n_pairs=0, pos=None, freq=None) == ARG
    assert _bwd(nws=16) == WS and _bwd(ws=None) == WS
    assert _fwd(n_rows=0, q=None, k=None, qo=None, ko=None, pos=None, freq=None) == 0
    f, need = tpc.lib().tp_head_norm_rotate_workspace, ctypes.c_size_t()
    assert f(None, ctypes.byref(need)) == ARG and f(ctypes.byref(_heads()), None) == ARG
    assert tpc.lib().tp_head_norm_rotate_forward(None, A, 64, A, 32, B, 64, C, 32, None) == ARG


# ---- routing and products ----------------------------------------------------------------
def test_route():
    f, b = tpc.lib().tp_route_forward, tpc.lib().tp_route_backward
    fwd = lambda dt=F32, n=4, e=8, k=2, o=0, l=A, s=8, w=B, i=C: f(dt, n, e, k, o, l, s, w, i, None)
    bwd = lambda dt=F32, n=4, e=8, k=2, o=1, l=A, s=8, w=B, i=C, g=D, out=D: b(dt, n, e, k, o, l, s, w, i, g, out, None)
    for call in (fwd, bwd):
        assert call(dt=3) == ARG and call(n=-1) == ARG and call(k=0) == ARG and call(k=9) == ARG and call(o=2) == ARG
        assert call(e=0) == UNSUP and call(e=1025, s=2000) == UNSUP and call(e=64, k=17, s=64) == UNSUP
        assert call(s=7) == ARG and call(n=0, l=None, w=None, i=None) == 0
        for name in ("l", "w", "i"):
            assert call(**{name: None}) == ARG and call(**{name: ODD}) == ARG, name
    assert bwd(g=None) == ARG and bwd(out=None) == ARG and bwd(o=0, l=None, s=0, out=None) == ARG
    assert fwd(n=1 << 40, s=8) == OVER


def test_group_rows():
    f = tpc.lib().tp_group_rows
    call = lambda i=A, n=10000, e=8, p=B, r=C, ws=D, nws=1 << 30: f(i, n, e, p, r, ws, nws, None)
    assert call(n=-1) == ARG and call(e=0) == UNSUP and call(e=1025) == UNSUP and call(n=1 << 31) == OVER
    assert call(ws=None) == WS and call(nws=8) == WS
    for name in ("i", "p", "r"):
        assert call(**{name: None}) == ARG and call(**{name: ODD}) == ARG, name
    need = ctypes.c_size_t()
    assert tpc.lib().tp_group_workspace(10000, 8, None) == ARG
    assert tpc.lib().tp_group_workspace(100, 8, ctypes.byref(need)) == 0 and need.value == 0


def _grouped(**kw):
    v = dict(dtype=F32, n_groups=3, n_in=16, n_out=8, n_slots=4096, fan=1, x_rows=0, y_rows=0, ptr=A.value, rows=A.value, w=A.value)
    v.update(kw)
    return blocks._Grouped(*v.values())


def _lin(x=A, xs=16, bias=None, act=0, y=B, ys=8, pre=None, **kw):
    return tpc.lib().tp_grouped_linear_forward(ctypes.byref(_grouped(**kw)), x, xs, bias, act, y, ys, pre, None)


def _back(gz=A, gs=8, x=A, xs=16, pre=None, ps=0, gx=B, gxs=16, gw=C, gb=D, ws=D, nws=1 << 40, **kw):
    return tpc.lib().tp_grouped_linear_backward(ctypes.byref(_grouped(**kw)), gz, gs, x, xs, pre, ps, gx, gxs, gw, gb, ws, nws, None)


BAD_GROUPED = [dict(dtype=2), dict(n_slots=-1), dict(n_in=0), dict(n_out=0), dict(fan=0), dict(fan=3), dict(x_rows=2), dict(y_rows=-1),
               dict(ptr=None), dict(rows=None), dict(w=None), dict(ptr=0x10001), dict(rows=0x10002), dict(w=0x10001)]


@pytest.mark.parametrize("bad", BAD_GROUPED, ids=str)
def test_grouped_descriptions(bad):
    assert _lin(**bad) == ARG and _back(**bad) == ARG


def test_grouped():
    assert _lin(n_groups=0) == UNSUP and _lin(n_groups=1025) == UNSUP and _lin(n_in=1 << 21, xs=1 << 21) == UNSUP
    assert _lin(n_slots=1 << 31) == OVER
    assert _lin(xs=15) == ARG and _lin(ys=7) == ARG and "stride" in err()
    for name in ("x", "y"):
        assert _lin(**{name: None}) == ARG and _lin(**{name: ODD}) == ARG, name
    assert _lin(bias=ODD) == ARG and _lin(act=2) == ARG and _lin(pre=C) == ARG and "activation" in err()
    assert _lin(act=1, pre=ODD) == ARG
    assert _lin(n_slots=0, x=None, y=None, ptr=None, rows=None, w=None) == 0
    for name in ("gz", "x"):
        assert _back(**{name: None}) == ARG and _back(**{name: ODD}) == ARG, name
    for name in ("gx", "gw", "gb", "pre"):
        assert _back(**{name: ODD, "ps": 16}) == ARG, name
    assert _back(gs=7) == ARG and _back(xs=15) == ARG and _back(gxs=15) == ARG and _back(pre=A, ps=15) == ARG
    assert _back(gw=None) == ARG and "grad_bias" in err()
    assert _back(gx=None, gw=None, gb=None) == 0
    assert _back(fan=2, pre=A, ps=16) == ARG and "one slot" in err()
    assert _back(fan=2, gxs=24) == ARG and "contiguous" in err()
    assert _back(nws=16, n_slots=1 << 20) == WS and _back(ws=None, n_slots=1 << 20) == WS and _back(fan=2, ws=None) == WS
    assert _back(ws=ctypes.c_void_p(0x10008)) == ARG
    f, need = tpc.lib().tp_grouped_linear_workspace, ctypes.c_size_t()
    assert f(None, 1, 1, ctypes.byref(need)) == ARG and f(ctypes.byref(_grouped()), 1, 1, None) == ARG
    assert f(ctypes.byref(_grouped(fan=2)), 1, 0, ctypes.byref(need)) == 0 and need.value == 4096 * 16 * 4


def test_combine():
    f, b = tpc.lib().tp_combine_forward, tpc.lib().tp_combine_backward
    fwd = lambda dt=F32, n=4, k=2, c=8, y=A, w=B, out=C: f(dt, n, k, c, y, w, out, None)
    bwd = lambda dt=F32, n=4, k=2, c=8, go=A, y=A, w=B, gy=C, gw=D: b(dt, n, k, c, go, y, w, gy, gw, None)
    for call in (fwd, bwd):
        assert call(dt=2) == ARG and call(n=-1) == ARG and call(k=0) == ARG and call(c=0) == ARG and call(n=1 << 61) == OVER
        assert call(y=None) == ARG and call(y=ODD) == ARG and call(w=ODD) == ARG and call(n=0, y=None) == 0
    assert fwd(out=None) == ARG and bwd(w=None) == ARG and bwd(gy=None) == ARG and bwd(gw=None) == ARG and bwd(go=None) == ARG


# ---- AdamW ----------------------------------------------------------------------------------
def _adamw(n=2, sizes=(300, 5), grads=(0x10000, 0x20000), norm=None, ws=D, nws=1 << 30, **kw):
    s = (ctypes.c_int64 * n)(*sizes)
    v = dict(bits=32, grad_dtype=F32, n_tensors=n, sizes=ctypes.addressof(s), table=A.value, m=A.value, v=B.value, m_unit=None,
             v_unit=None, beta1=0.9, beta2=0.999, eps=1e-8, lr=1e-3, max_norm=0.0, lr_at=None, seed=0, scalars=A.value)
    v.update(kw)
    g = None if grads is None else (ctypes.c_void_p * n)(*grads)
    return tpc.lib().tp_adamw_step(ctypes.byref(blocks._AdamW(*v.values())), g, norm, ws, nws, None)


BAD_ADAMW = [dict(grad_dtype=2), dict(n_tensors=-1), dict(sizes=None), dict(sizes=(300, -5)), dict(beta1=1.0), dict(beta1=-0.1),
             dict(beta2=NAN), dict(beta2=1.0), dict(eps=-1.0), dict(eps=INF), dict(eps=NAN), dict(lr=NAN), dict(lr=INF), dict(max_norm=-1.0),
             dict(max_norm=NAN), dict(scalars=None), dict(table=None), dict(m=None), dict(v=None), dict(grads=None), dict(bits=8),
             dict(grads=(0x10000, None)), dict(grads=(0x10002, 0x20000)), dict(table=0x10008), dict(m=0x10004), dict(v=0x10001),
             dict(scalars=0x10004), dict(ws=ctypes.c_void_p(0x10004)), dict(norm=A), dict(norm=ODD, max_norm=1.0), dict(lr_at=0x10001)]


@pytest.mark.parametrize("bad", BAD_ADAMW, ids=str)
def test_adamw_step(bad):
    if bad.get("sizes", 1) is None:
        v = blocks._AdamW(32, F32, 2, None, A.value, A.value, B.value, None, None, 0.9, 0.999, 1e-8, 1e-3, 0.0, None, 0, A.value)
        assert tpc.lib().tp_adamw_step(ctypes.byref(v), (ctypes.c_void_p * 2)(1, 2), None, D, 1, None) == ARG
    else:
        assert _adamw(**bad) == ARG


def test_adamw():
    L = tpc.lib()
    assert _adamw(bits=16) == UNSUP and _adamw(max_norm=1.0, nws=0) == WS and _adamw(max_norm=1.0, ws=None) == WS
    assert _adamw(sizes=(1 << 39, 1)) == OVER and L.tp_adamw_step(None, None, None, None, 0, None) == ARG
    t, v, w = ctypes.c_size_t(), ctypes.c_int64(), ctypes.c_size_t()
    sizes = (ctypes.c_int64 * 3)(1, 256, 257)
    assert L.tp_adamw_sizes(3, sizes, ctypes.byref(t), ctypes.byref(v), ctypes.byref(w)) == 0 and v.value == 256 + 256 + 512
    assert L.tp_adamw_sizes(3, sizes, None, ctypes.byref(v), ctypes.byref(w)) == ARG
    assert L.tp_adamw_sizes(-1, sizes, ctypes.byref(t), ctypes.byref(v), ctypes.byref(w)) == ARG
    assert L.tp_adamw_sizes(3, None, ctypes.byref(t), ctypes.byref(v), ctypes.byref(w)) == ARG
    host = ctypes.create_string_buffer(t.value)
    p = lambda *a: (ctypes.c_void_p * 3)(*a)
    good = p(A.value, B.value, C.value)
    assert L.tp_adamw_table(3, sizes, good, None, None, host) == 0
    assert L.tp_adamw_table(3, sizes, None, None, None, host) == ARG and L.tp_adamw_table(3, sizes, good, None, None, None) == ARG
    assert L.tp_adamw_table(3, sizes, p(A.value, None, C.value), None, None, host) == ARG
    assert L.tp_adamw_table(3, sizes, p(0x10002, B.value, C.value), None, None, host) == ARG
    assert L.tp_adamw_table(3, sizes, good, p(0x10001, None, None), None, host) == ARG
    assert L.tp_adamw_table(3, sizes, good, None, (ctypes.c_float * 3)(0, NAN, 0), host) == ARG
    f = L.tp_adamw_values
    assert f(0, -256, A, B, C, None) == ARG and f(0, 100, A, B, C, None) == ARG and f(0, 0, None, None, None, None) == 0
    assert f(0, 256, None, B, C, None) == ARG and f(0, 256, A, ODD, C, None) == ARG and f(0, 256, ctypes.c_void_p(0x10004), B, C, None) == ARG


# ---- the binding ------------------------------------------------------------------------------
torch = pytest.importorskip("torch")


@pytest.fixture
def nowhere(monkeypatch):
    calls = []
    monkeypatch.setattr(blocks, "_code", lambda t, name: ({torch.float32: 0, torch.bfloat16: 1}[t.dtype], 0))
    monkeypatch.setattr(blocks, "_rows", lambda t, name, dtype, shape, dev: (0x10000, 8))
    monkeypatch.setattr(blocks, "_need", lambda t, name, dtype, shape, dev: 0x10000)
    monkeypatch.setattr(blocks, "_call", lambda *a: calls.append(a))
    return calls


def meta(*shape, dtype=torch.float32):
    return torch.empty(*shape, dtype=dtype, device="meta")


def test_sizes_beyond_32_bits(nowhere):
    big = 1 << 32
    x = meta(1, big + 8, 8)
    for q, k, match in ((x, meta(1, 1, 8), "heads"), (meta(1, 1, 8), x, "key_heads"), (meta(1, 1, big + 8), meta(1, 1, big + 8), "head_dim")):
        with pytest.raises(ValueError, match=match):
            blocks.head_norm_rotate_forward(q, k)
    q = meta(4, 1, 8)
    with pytest.raises(ValueError, match="axes"):
        blocks.head_norm_rotate_forward(q, q, pos=meta(4, big + 3), freq=meta(4, big + 3, dtype=torch.float64))
    with pytest.raises(ValueError, match="groups"):
        blocks.route_forward(meta(1, big + 4), 2)
    with pytest.raises(ValueError, match="k"):
        blocks.route_forward(meta(1, 4), big + 2)
    g = blocks.Groups(meta(4, dtype=torch.int32), meta(8, dtype=torch.int32), 1)
    for shape, match in (((big + 3, 1, 1), "groups"), ((3, big + 1, 1), "n_in"), ((3, 1, big + 1), "n_out")):
        with pytest.raises(ValueError, match=match):
            blocks.grouped_linear_forward(meta(8, 8), meta(*shape), g)
    with pytest.raises(ValueError, match="columns"):
        blocks.combine_forward(meta(1, big + 1), meta(1, 1))
    assert not nowhere


def test_wrong_arguments(nowhere):
    q = meta(4, 2, 8)
    for kw in (dict(gamma_q=q), dict(pos=q), dict(pos=meta(4), freq=meta(4, 1)), dict(pos=meta(4, 1, dtype=torch.int64), freq=meta(4, 1))):
        with pytest.raises((ValueError, TypeError)):
            blocks.head_norm_rotate_forward(q, q, **kw)
    with pytest.raises(ValueError):
        blocks.head_norm_rotate_backward(q, q, q, q, want_pos=True)
    g = blocks.Groups(meta(4, dtype=torch.int32), meta(8, dtype=torch.int32), 1)
    w = meta(3, 8, 4)
    for kw in (dict(x_rows="rows"), dict(y_rows=1), dict(act="relu"), dict(want_pre=True)):
        with pytest.raises(ValueError):
            blocks.grouped_linear_forward(meta(8, 8), w, g, **kw)
    with pytest.raises(ValueError):
        blocks.grouped_linear_backward(meta(8, 4), meta(8, 8), w, g, want_w=False, want_bias=True)
    with pytest.raises(ValueError):
        blocks.grouped_linear_forward(meta(8, 8), w, g._replace(fan=3))
    for p, kw in (([], {}), ([meta(3)], dict(bits=16)), ([meta(3)], dict(seed=-1)), ([meta(3)], dict(weight_decay=[0, 1])),
                  ([meta(3)], dict(copies=[None, None]))):
        with pytest.raises(ValueError):
            blocks.AdamW(p, **kw)
    assert not nowhere


def test_tensors_on_the_host_are_refused():
    t = torch.zeros(4, 2, 8)
    with pytest.raises(ValueError, match="GPU"):
        tpc.head_norm_rotate_forward(t, t)
    with pytest.raises(ValueError, match="GPU"):
        tpc.group_rows(torch.zeros(4, dtype=torch.int32), 2)
    with pytest.raises(ValueError, match="GPU"):
        tpc.AdamW([torch.zeros(4)])


def test_rotary_frequencies():
    f = tpc.rotary_frequencies(8)
    assert f.dtype == torch.float64 and torch.allclose(f[:, 0], 1e4 ** (-torch.arange(8).double() / 8))
    assert torch.equal(tpc.rotary_frequencies(8, stretch=4.0), f / 4)
    part = tpc.rotary_frequencies(8, stretch=4.0, trained=1000.0, few=1.0, many=32.0)
    turns = f * 1000 / 6.283185307179586
    assert torch.equal(part[turns > 32], f[turns > 32]) and torch.allclose(part[turns < 1], f[turns < 1] / 4)
    mid = (turns >= 1) & (turns <= 32)
    assert ((part <= f) & (part >= f / 4 * (1 - 1e-12)))[mid].all()
    three = tpc.rotary_frequencies(7, axes=3)
    assert three.shape == (7, 3) and ((three != 0).sum(1) == 1).all() and three[1, 1] == 1 and three[3, 0] == 1e4 ** (-1 / 3)
    for kw in (dict(n_pairs=-1), dict(n_pairs=4, axes=0), dict(n_pairs=4, stretch=0.0), dict(n_pairs=4, trained=0.0),
               dict(n_pairs=4, trained=9.0, few=3.0, many=2.0)):
        with pytest.raises(ValueError):
            tpc.rotary_frequencies(**kw)
