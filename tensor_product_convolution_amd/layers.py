"""Layers around the convolution: attention between the atoms of each structure
with a learned bias by interatomic distance, layer norm and dropout.

Argument marshalling only, like the rest of the binding: conventions, formulas
and errors are those of ``include/tpconv.h``.  Tensors are float32 or bfloat16;
strided rows are taken as they are where the C entry point takes a stride.
"""
import ctypes
from typing import NamedTuple

from . import _check, _need, _ptr, _stream, _torch, lib

TP_F32, TP_BF16 = 0, 1


class _Dropout(ctypes.Structure):
    _fields_ = [("p", ctypes.c_double), ("seed", ctypes.c_uint64), ("offset", ctypes.c_uint64)]


class _Attn(ctypes.Structure):
    _fields_ = [("dtype", ctypes.c_int32), ("n_nodes", ctypes.c_int32), ("n_segments", ctypes.c_int32),
                ("n_heads", ctypes.c_int32), ("n_kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("seg_ptr", ctypes.c_void_p), ("key_mask", ctypes.c_void_p), ("pos", ctypes.c_void_p),
                ("bias", ctypes.c_void_p), ("n_buckets", ctypes.c_int32), ("steps", ctypes.c_int32),
                ("r_min", ctypes.c_float), ("scale", ctypes.c_float)]


class Dropout(NamedTuple):
    """Probability, seed and offset of a dropout: the same triple draws the same mask."""
    p: float
    seed: int
    offset: int = 0

    def cstruct(self):
        if not 0 <= self.seed < 1 << 64 or not 0 <= self.offset < 1 << 64:
            raise ValueError("seed and offset must be unsigned 64-bit integers")
        return _Dropout(self.p, self.seed, self.offset)


def _code(t, name):
    torch = _torch()
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch tensor")
    if t.device.type != "cuda":
        raise ValueError(f"{name} must live on the GPU")
    if t.dtype is torch.float32:
        return TP_F32
    if t.dtype is torch.bfloat16:
        return TP_BF16
    raise TypeError(f"{name} must be float32 or bfloat16, got {t.dtype}")


def _same(t, name, like):
    if t.device != like.device:
        raise ValueError(f"{name} is on {t.device}, expected {like.device}")
    return t


def _rows(t, name, like, shape):
    """A tensor of rows (dense but for the row stride) of the type and device of ``like``."""
    if not isinstance(t, type(like)) and not isinstance(t, _torch().Tensor):
        raise TypeError(f"{name} must be a torch tensor")
    if t.dtype is not like.dtype:
        raise TypeError(f"{name} must be {like.dtype}, got {t.dtype}")
    if tuple(t.shape) != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {shape}")
    _same(t, name, like)
    want = 1
    for s, n in zip(t.stride()[:0:-1], shape[:0:-1]):
        if n != 1 and s != want:
            raise ValueError(f"{name}: rows must be contiguous")
        want *= n
    if shape[0] <= 1:
        return want                     # the stride of a single row says nothing
    return t.stride(0)


# ---- dropout -------------------------------------------------------------------
def _dropout(x, drop, residual, out):
    torch = _torch()
    dt = _code(x, "x")
    _need(x, "x", x.dtype)
    if residual is not None:
        _same(_need(residual, "residual", x.dtype, x.shape), "residual", x)
    if out is None:
        out = torch.empty_like(x)
    _same(_need(out, "out", x.dtype, x.shape), "out", x)
    _check(lib().tp_dropout_apply(dt, x.numel(), _ptr(x), _ptr(residual), ctypes.byref(drop.cstruct()), _ptr(out),
                                  _stream(x.device)))
    return out


def dropout_forward(x, drop, residual=None, out=None):
    """dropout(x) (+ residual); ``drop`` is a Dropout.  No mask is stored."""
    return _dropout(x, drop, residual, out)


def dropout_backward(grad_out, drop, out=None):
    """Gradient with respect to x of dropout_forward with the same ``drop``."""
    return _dropout(grad_out, drop, None, out)


# ---- layer norm ------------------------------------------------------------------
def _norm_forward(x, residual, gamma, beta, drop, eps):
    torch = _torch()
    dt = _code(x, "x")
    if x.dim() != 2:
        raise ValueError("x must be [rows, columns]")
    n, c = x.shape
    xs = _rows(x, "x", x, (n, c))
    _same(_need(gamma, "gamma", torch.float32, (c,)), "gamma", x)
    _same(_need(beta, "beta", torch.float32, (c,)), "beta", x)
    y = torch.empty((n, c), dtype=x.dtype, device=x.device)
    stats = torch.empty((2, n), dtype=torch.float32, device=x.device)
    mean, rstd = stats[0], stats[1]
    h = None
    if residual is not None:
        _same(_need(residual, "residual", x.dtype, (n, c)), "residual", x)
        h = torch.empty_like(y)
    _check(lib().tp_layer_norm_forward(dt, n, c, _ptr(x), xs, _ptr(residual),
                                       None if drop is None else ctypes.byref(drop.cstruct()), _ptr(gamma), _ptr(beta),
                                       eps, _ptr(y), c, _ptr(h), _ptr(mean), _ptr(rstd), _stream(x.device)))
    return y, mean, rstd, h


def layer_norm_forward(x, gamma, beta, eps=1e-5):
    """(y, mean, rstd) of the norm of the rows of x [rows, columns]; x may be a
    column range of wider rows (the scalar block of node rows)."""
    return _norm_forward(x, None, gamma, beta, None, eps)[:3]


def layer_norm_residual_forward(x, residual, gamma, beta, drop=None, eps=1e-5):
    """(y, mean, rstd, h) with h = dropout(x) + residual, normalised, in one pass."""
    if residual is None:
        raise ValueError("residual is missing")
    return _norm_forward(x, residual, gamma, beta, drop, eps)


def _norm_backward(grad_y, h, gamma, mean, rstd, grad_res, drop, want_x, want_weights):
    torch = _torch()
    dt = _code(h, "h")
    if h.dim() != 2:
        raise ValueError("h must be [rows, columns]")
    n, c = h.shape
    hs = _rows(h, "h", h, (n, c))
    gs = _rows(grad_y, "grad_y", h, (n, c))
    _same(_need(gamma, "gamma", torch.float32, (c,)), "gamma", h)
    _same(_need(mean, "mean", torch.float32, (n,)), "mean", h)
    _same(_need(rstd, "rstd", torch.float32, (n,)), "rstd", h)
    if grad_res is not None:
        _same(_need(grad_res, "grad_h", h.dtype, (n, c)), "grad_h", h)
    gh = torch.empty((n, c), dtype=h.dtype, device=h.device)
    gx = torch.empty_like(gh) if want_x else None
    gg = gb = ws = None
    nbytes = 0
    if want_weights:
        need = ctypes.c_size_t()
        _check(lib().tp_layer_norm_workspace(dt, n, c, ctypes.byref(need)))
        nbytes = need.value
        gg = torch.empty(c, dtype=torch.float32, device=h.device)
        gb = torch.empty(c, dtype=torch.float32, device=h.device)
        if nbytes:
            ws = torch.empty(nbytes, dtype=torch.uint8, device=h.device)
    _check(lib().tp_layer_norm_backward(dt, n, c, _ptr(grad_y), gs, _ptr(h), hs, _ptr(gamma), _ptr(mean), _ptr(rstd),
                                        _ptr(grad_res), None if drop is None else ctypes.byref(drop.cstruct()),
                                        _ptr(gh), _ptr(gx), _ptr(gg), _ptr(gb), _ptr(ws), nbytes, _stream(h.device)))
    return gh, gx, gg, gb


def layer_norm_backward(grad_y, x, gamma, mean, rstd, want_weights=True):
    """(grad_x, grad_gamma, grad_beta) of layer_norm_forward; the latter two are
    None without ``want_weights``."""
    gx, _, gg, gb = _norm_backward(grad_y, x, gamma, mean, rstd, None, None, False, want_weights)
    return gx, gg, gb


def layer_norm_residual_backward(grad_y, h, gamma, mean, rstd, drop=None, grad_h=None, want_weights=True):
    """(grad_x, grad_residual, grad_gamma, grad_beta) of layer_norm_residual_forward;
    ``grad_h``: the gradient that reaches h past the norm.  Without a dropout grad_x is
    grad_residual itself."""
    gr, gx, gg, gb = _norm_backward(grad_y, h, gamma, mean, rstd, grad_h, drop, drop is not None, want_weights)
    return (gr if gx is None else gx), gr, gg, gb


# ---- attention -------------------------------------------------------------------
def _describe(q, k, v, seg_ptr, pos, bias, r_min, steps, key_mask, scale):
    """(tp_attn, strides of q, k, v) after the checks that need the tensors."""
    torch = _torch()
    dt = _code(q, "q")
    if q.dim() != 3 or not isinstance(k, torch.Tensor) or k.dim() != 3:
        raise ValueError("q must be [nodes, heads, head_dim], k and v [nodes, key heads, head_dim]")
    n, hq, d = q.shape
    hk = k.shape[1]
    qs = _rows(q, "q", q, (n, hq, d))
    ks = _rows(k, "k", q, (n, hk, d))
    vs = _rows(v, "v", q, (n, hk, d))
    _same(_need(seg_ptr, "seg_ptr", torch.int32), "seg_ptr", q)
    if seg_ptr.dim() != 1 or seg_ptr.shape[0] < 1:
        raise ValueError("seg_ptr must hold the number of structures + 1 offsets")
    nb = 0
    if (pos is None) != (bias is None):
        raise ValueError("pos and bias go together")
    if bias is not None:
        _same(_need(pos, "pos", torch.float32, (n, 3)), "pos", q)
        if not isinstance(bias, torch.Tensor) or bias.dim() != 2 or bias.shape[1] < 1:
            raise ValueError("bias must be [heads, buckets]")
        nb = bias.shape[1]
        _same(_need(bias, "bias", q.dtype, (hq, nb)), "bias", q)
    if key_mask is not None:
        if isinstance(key_mask, torch.Tensor) and key_mask.dtype is torch.bool:
            key_mask = key_mask.view(torch.uint8)
        _same(_need(key_mask, "key_mask", torch.uint8, (n,)), "key_mask", q)
    if scale is None:
        scale = d ** -0.5 if d else 1.0
    p = lambda t: None if t is None else t.data_ptr()
    a = _Attn(dt, n, seg_ptr.shape[0] - 1, hq, hk, d, p(seg_ptr), p(key_mask), p(pos), p(bias), nb, steps, r_min, scale)
    return a, qs, ks, vs


def attn_forward(q, k, v, seg_ptr, pos=None, bias=None, r_min=0.5, steps=4, key_mask=None, scale=None, out=None):
    """(out [nodes, heads, head_dim], lse [heads, nodes]) of attention within each
    structure of a packed batch.

    q [nodes, heads, head_dim], k, v [nodes, key heads, head_dim] (views of one
    projected row are fine); seg_ptr int32 [structures + 1] node offsets; pos [nodes, 3]
    and bias [heads, buckets]: learned bias by distance bucket; key_mask [nodes]
    (uint8 or bool, 0 = masked); scale defaults to head_dim ** -0.5."""
    torch = _torch()
    a, qs, ks, vs = _describe(q, k, v, seg_ptr, pos, bias, r_min, steps, key_mask, scale)
    n, hq, d = q.shape
    if out is None:
        out = torch.empty((n, hq, d), dtype=q.dtype, device=q.device)
    os = _rows(out, "out", q, (n, hq, d))
    lse = torch.empty((hq, n), dtype=torch.float32, device=q.device)
    _check(lib().tp_attn_forward(ctypes.byref(a), _ptr(q), qs, _ptr(k), ks, _ptr(v), vs, _ptr(out), os, _ptr(lse),
                                 _stream(q.device)))
    return out, lse


def attn_backward(q, k, v, seg_ptr, out, lse, grad_out, pos=None, bias=None, r_min=0.5, steps=4, key_mask=None,
                  scale=None, outs=None, want_bias=True):
    """(grad_q, grad_k, grad_v, grad_bias) of attn_forward; grad_bias is None without a
    bias or with ``want_bias`` false.  ``outs``: (grad_q, grad_k, grad_v) to fill, e.g. the
    views of one projected row's gradient."""
    torch = _torch()
    a, qs, ks, vs = _describe(q, k, v, seg_ptr, pos, bias, r_min, steps, key_mask, scale)
    n, hq, d = q.shape
    hk = k.shape[1]
    os = _rows(out, "out", q, (n, hq, d))
    gs = _rows(grad_out, "grad_out", q, (n, hq, d))
    _same(_need(lse, "lse", torch.float32, (hq, n)), "lse", q)
    if outs is None:
        outs = tuple(torch.empty((n, h, d), dtype=q.dtype, device=q.device) for h in (hq, hk, hk))
    gq, gk, gv = outs
    gqs = _rows(gq, "grad_q", q, (n, hq, d))
    gks = _rows(gk, "grad_k", q, (n, hk, d))
    gvs = _rows(gv, "grad_v", q, (n, hk, d))
    gb = torch.empty_like(bias) if bias is not None and want_bias else None
    need = ctypes.c_size_t()
    _check(lib().tp_attn_backward_workspace(ctypes.byref(a), ctypes.byref(need)))
    ws = torch.empty(need.value, dtype=torch.uint8, device=q.device) if need.value else None
    _check(lib().tp_attn_backward(ctypes.byref(a), _ptr(q), qs, _ptr(k), ks, _ptr(v), vs, _ptr(out), os, _ptr(lse),
                                  _ptr(grad_out), gs, _ptr(gq), gqs, _ptr(gk), gks, _ptr(gv), gvs, _ptr(gb), _ptr(ws),
                                  need.value, _stream(q.device)))
    return gq, gk, gv, gb
