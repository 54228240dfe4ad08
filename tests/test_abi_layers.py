"""Refusals of the attention, layer norm and dropout entry points: every case is
caught on the host before a HIP call, so these run without a GPU."""
import ctypes

import pytest

import tensor_product_convolution_amd as tpc
from tensor_product_convolution_amd import layers

import os

pytestmark = pytest.mark.skipif(not os.path.exists(tpc.LIB_PATH),
                                reason="libtpconv.so not built (run __graft_entry__.build())")

A, B, C, D, ODD = (ctypes.c_void_p(x) for x in (0x10000, 0x20000, 0x30000, 0x40000, 0x10001))
F32, BF16 = 0, 1
ARG, UNSUP, OVER, WS = -1, -3, -4, -5


def err():
    return tpc.lib().tp_conv_last_error().decode()


def test_dropout_refusals():
    f = tpc.lib().tp_dropout_apply
    d = layers._Dropout(0.1, 1, 2)
    r = ctypes.byref(d)
    assert f(7, 8, A, None, r, B, None) == ARG and "element type" in err()
    assert f(F32, -1, A, None, r, B, None) == ARG
    assert f(F32, 8, A, None, None, B, None) == ARG
    assert f(F32, 8, None, None, r, B, None) == ARG
    assert f(F32, 8, A, None, r, None, None) == ARG
    assert f(F32, 8, ODD, None, r, B, None) == ARG and "misaligned" in err()
    assert f(F32, 1 << 41, A, None, r, B, None) == OVER
    for p in (-0.1, 1.0, 1.5, float("nan")):
        bad = layers._Dropout(p, 1, 2)
        assert f(F32, 8, A, None, ctypes.byref(bad), B, None) == ARG and "probability" in err()
        assert f(F32, 0, None, None, ctypes.byref(bad), None, None) == ARG
    assert f(F32, 0, None, None, r, None, None) == 0          # nothing to do
    with pytest.raises(ValueError):
        tpc.Dropout(0.1, -1).cstruct()
    with pytest.raises(ValueError):
        tpc.Dropout(0.1, 0, 1 << 64).cstruct()


def _fwd(dtype=F32, rows=4, cols=8, x=A, xs=8, res=None, drop=None, gamma=B, beta=B, eps=1e-5, y=C, ys=8, h=None,
         mean=D, rstd=D):
    return tpc.lib().tp_layer_norm_forward(dtype, rows, cols, x, xs, res, drop, gamma, beta, eps, y, ys, h, mean, rstd,
                                           None)


def test_norm_forward_refusals():
    r = ctypes.byref(layers._Dropout(0.1, 1, 2))
    assert _fwd(dtype=3) == ARG
    assert _fwd(rows=-1) == ARG
    assert _fwd(cols=0, xs=0, ys=0) == UNSUP
    assert _fwd(cols=8193, xs=9000, ys=9000) == UNSUP
    assert _fwd(xs=7) == ARG and "stride" in err()
    assert _fwd(ys=7) == ARG
    for e in (-1e-5, float("nan"), float("inf")):
        assert _fwd(eps=e) == ARG and "eps" in err()
    for name in ("x", "gamma", "beta", "y", "mean", "rstd"):
        assert _fwd(**{name: None}) == ARG, name
        assert _fwd(**{name: ODD}) == ARG, name
    assert _fwd(res=A) == ARG                                  # a residual needs h
    assert _fwd(h=A) == ARG and _fwd(drop=r) == ARG            # and the others need a residual
    assert _fwd(res=A, h=B, drop=ctypes.byref(layers._Dropout(1.0, 1, 2))) == ARG
    assert _fwd(rows=0, x=None, gamma=None, beta=None, y=None, mean=None, rstd=None) == 0


def _bwd(dtype=F32, rows=4000, cols=8, gy=A, gs=8, h=A, hs=8, gamma=B, mean=D, rstd=D, res=None, drop=None, gh=C,
         gx=None, gg=B, gb=B, ws=D, nws=1 << 30):
    return tpc.lib().tp_layer_norm_backward(dtype, rows, cols, gy, gs, h, hs, gamma, mean, rstd, res, drop, gh, gx, gg,
                                            gb, ws, nws, None)


def test_norm_backward_refusals():
    need = ctypes.c_size_t()
    assert tpc.lib().tp_layer_norm_workspace(F32, 4000, 8, ctypes.byref(need)) == 0 and need.value > 0
    assert tpc.lib().tp_layer_norm_workspace(F32, 4000, 8, None) == ARG
    assert tpc.lib().tp_layer_norm_workspace(9, 4000, 8, ctypes.byref(need)) == ARG
    assert tpc.lib().tp_layer_norm_workspace(F32, -1, 8, ctypes.byref(need)) == ARG
    assert _bwd(nws=16) == WS and _bwd(ws=None) == WS
    assert _bwd(gs=7) == ARG and _bwd(hs=7) == ARG
    for name in ("gy", "h", "gamma", "mean", "rstd", "gh"):
        assert _bwd(**{name: None}) == ARG, name
    for name in ("gy", "h", "gamma", "mean", "rstd", "gh", "gg", "res", "ws"):
        assert _bwd(**{name: ODD}) == ARG, name
    assert _bwd(gg=None) == ARG and _bwd(gb=None) == ARG       # both or none
    assert _bwd(gx=A) == ARG and "drop" in err()
    assert _bwd(dtype=2) == ARG and _bwd(cols=0) == UNSUP and _bwd(rows=-4) == ARG


def _desc(**kw):
    v = dict(dtype=BF16, n_nodes=64, n_segments=2, n_heads=4, n_kv_heads=2, head_dim=16, seg_ptr=A.value, key_mask=None,
             pos=A.value, bias=A.value, n_buckets=32, steps=4, r_min=0.5, scale=0.25)
    v.update(kw)
    return layers._Attn(*v.values())


def _attn(q=A, qs=64, k=A, ks=32, v=A, vs=32, out=B, os=64, lse=C, **kw):
    return tpc.lib().tp_attn_forward(ctypes.byref(_desc(**kw)), q, qs, k, ks, v, vs, out, os, lse, None)


BAD = [dict(dtype=5), dict(n_nodes=-1), dict(n_segments=-1), dict(n_segments=0), dict(n_heads=0), dict(n_kv_heads=0),
       dict(n_heads=5), dict(scale=float("nan")), dict(scale=float("inf")), dict(steps=3), dict(steps=0), dict(r_min=0.0),
       dict(r_min=float("nan")), dict(r_min=1e30), dict(n_buckets=-1), dict(seg_ptr=None), dict(pos=None),
       dict(bias=None), dict(seg_ptr=0x10001)]


@pytest.mark.parametrize("bad", BAD, ids=str)
def test_attention_description_refusals(bad):
    assert _attn(**bad) == ARG


def test_attention_refusals():
    for d in (0, 4, 12, 136):
        assert _attn(head_dim=d, qs=4096, ks=4096, vs=4096, os=4096) == UNSUP, d
    assert _attn(n_buckets=65) == UNSUP
    assert _attn(n_heads=2048, n_kv_heads=2048, qs=1 << 20, ks=1 << 20, vs=1 << 20, os=1 << 20) == UNSUP
    assert _attn(n_nodes=2 ** 31 - 1, n_segments=2 ** 31 - 1) == OVER
    for name in ("q", "k", "v", "out"):
        assert _attn(**{name: None}) == ARG, name
        assert _attn(**{name: ctypes.c_void_p(0x10008)}) == ARG and "16-byte" in err(), name
    for name in ("qs", "ks", "vs", "os"):
        assert _attn(**{name: 24}) == ARG and "stride" in err(), name
        assert _attn(**{name: 68}) == ARG and "16-byte" in err(), name
    assert tpc.lib().tp_attn_forward(None, A, 64, A, 32, A, 32, B, 64, C, None) == ARG
    assert _attn(n_nodes=0, q=None, k=None, v=None, out=None, lse=None, seg_ptr=None, pos=None, bias=None) == 0


def _attn_bwd(q=A, k=A, v=A, out=A, go=A, gq=B, gk=B, gv=B, lse=C, gb=D, ws=D, nws=1 << 30, s=64, t=32, **kw):
    return tpc.lib().tp_attn_backward(ctypes.byref(_desc(**kw)), q, s, k, t, v, t, out, s, lse, go, s, gq, s, gk, t, gv, t,
                                      gb, ws, nws, None)


@pytest.mark.parametrize("bad", BAD, ids=str)
def test_attention_backward_description_refusals(bad):
    assert _attn_bwd(**bad) == ARG


def test_attention_backward_refusals():
    need = ctypes.c_size_t()
    f = tpc.lib().tp_attn_backward_workspace
    assert f(ctypes.byref(_desc()), ctypes.byref(need)) == 0 and need.value >= 4 * 64 * 4
    assert f(ctypes.byref(_desc()), None) == ARG and f(None, ctypes.byref(need)) == ARG
    assert f(ctypes.byref(_desc(head_dim=9)), ctypes.byref(need)) == UNSUP
    assert _attn_bwd(nws=16) == WS and _attn_bwd(ws=None) == WS
    for name in ("q", "k", "v", "out", "go", "gq", "gk", "gv", "lse"):
        assert _attn_bwd(**{name: None}) == ARG, name
    assert _attn_bwd(n_buckets=0, pos=None, bias=None) == ARG and "grad_bias" in err()
    assert _attn_bwd(gq=ctypes.c_void_p(0x10008)) == ARG
    assert _attn_bwd(ws=ctypes.c_void_p(0x10008)) == ARG
