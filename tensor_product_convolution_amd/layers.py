"""Layers around the convolution: attention between the atoms of each structure
with a learned bias by interatomic distance, layer norm and dropout.

Argument marshalling only, like the rest of the binding: conventions, formulas
and errors are those of ``include/tpconv.h``.  Tensors are float32 or bfloat16;
strided rows are taken as they are where the C entry point takes a stride.
"""
import ctypes
from typing import NamedTuple

import torch

from . import TPError, lib

TP_F32, TP_BF16 = 0, 1
_CODES = {torch.float32: TP_F32, torch.bfloat16: TP_BF16}
_raw_stream = torch._C._cuda_getCurrentRawStream


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


# The smallest calls are bound by the host, so the checks take one pass over the
# attributes and pointers go to ctypes as plain integers.
def _code(t, name):
    """Element type code and device number of an operand."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch tensor")
    code = _CODES.get(t.dtype)
    if code is None:
        raise TypeError(f"{name} must be float32 or bfloat16, got {t.dtype}")
    dev = t.get_device()
    if dev < 0:
        raise ValueError(f"{name} must live on the GPU")
    return code, dev


def _refuse(t, name, dtype, shape, dev):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch tensor")
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.get_device() != dev:
        raise ValueError(f"{name} is on {t.device}, expected cuda:{dev}")
    raise ValueError(f"{name} must be contiguous")


def _need(t, name, dtype, shape, dev):
    """The address of a contiguous tensor of this type, shape and device."""
    if (isinstance(t, torch.Tensor) and t.dtype is dtype and t.is_contiguous() and t.shape == shape
            and t.get_device() == dev):
        return t.data_ptr()
    _refuse(t, name, dtype, shape, dev)


def _rows(t, name, dtype, shape, dev):
    """(address, row stride) of a tensor whose rows are dense, whatever their stride."""
    if not (isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape and t.get_device() == dev):
        _refuse(t, name, dtype, shape, dev)
    strides = t.stride()
    want = 1
    for i in range(len(shape) - 1, 0, -1):
        if strides[i] != want and shape[i] != 1:
            raise ValueError(f"{name}: rows must be contiguous")
        want *= shape[i]
    # the stride of a single row says nothing
    return t.data_ptr(), strides[0] if shape[0] > 1 else want


_INT32_MAX = 2 ** 31 - 1


# ctypes cuts an integer to the lower bits of a narrower argument without a word
def _too_large(**sizes):
    name, n = max(sizes.items(), key=lambda kv: kv[1])
    raise ValueError(f"{name}: {n} is more than 32 bits hold")


def _call(dev, f, *args):
    """The C entry point on the current stream of device ``dev``."""
    if torch._C._cuda_getDevice() == dev:
        status = f(*args, _raw_stream(dev))
    else:
        with torch.cuda.device(dev):
            status = f(*args, _raw_stream(dev))
    if status:
        raise TPError(status, lib().tp_conv_last_error().decode())


def _check(status):
    if status:
        raise TPError(status, lib().tp_conv_last_error().decode())


# ---- dropout -------------------------------------------------------------------
def _dropout(x, drop, residual, out):
    code, dev = _code(x, "x")
    dtype, shape = x.dtype, x.shape
    px = _need(x, "x", dtype, shape, dev)
    pr = None if residual is None else _need(residual, "residual", dtype, shape, dev)
    if out is None:
        out = torch.empty_like(x)
    po = _need(out, "out", dtype, shape, dev)
    _call(dev, lib().tp_dropout_apply, code, x.numel(), px, pr, ctypes.byref(drop.cstruct()), po)
    return out


def dropout_forward(x, drop, residual=None, out=None):
    """dropout(x) (+ residual); ``drop`` is a Dropout.  No mask is stored."""
    return _dropout(x, drop, residual, out)


def dropout_backward(grad_out, drop, out=None):
    """Gradient with respect to x of dropout_forward with the same ``drop``."""
    return _dropout(grad_out, drop, None, out)


# ---- layer norm ------------------------------------------------------------------
def _norm_forward(x, residual, gamma, beta, drop, eps):
    code, dev = _code(x, "x")
    if x.dim() != 2:
        raise ValueError("x must be [rows, columns]")
    dtype, shape = x.dtype, x.shape
    n, c = shape
    if c > _INT32_MAX:
        _too_large(columns=c)
    px, xs = _rows(x, "x", dtype, shape, dev)
    pg = _need(gamma, "gamma", torch.float32, (c,), dev)
    pb = _need(beta, "beta", torch.float32, (c,), dev)
    y = x.new_empty(shape)
    mean, rstd = x.new_empty((2, n), dtype=torch.float32).unbind(0)
    h = pr = ph = None
    if residual is not None:
        pr = _need(residual, "residual", dtype, shape, dev)
        h = torch.empty_like(y)
        ph = h.data_ptr()
    _call(dev, lib().tp_layer_norm_forward, code, n, c, px, xs, pr, None if drop is None else ctypes.byref(drop.cstruct()),
          pg, pb, eps, y.data_ptr(), c, ph, mean.data_ptr(), rstd.data_ptr())
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
    code, dev = _code(h, "h")
    if h.dim() != 2:
        raise ValueError("h must be [rows, columns]")
    dtype, shape = h.dtype, h.shape
    n, c = shape
    if c > _INT32_MAX:
        _too_large(columns=c)
    ph, hs = _rows(h, "h", dtype, shape, dev)
    py, ys = _rows(grad_y, "grad_y", dtype, shape, dev)
    pg = _need(gamma, "gamma", torch.float32, (c,), dev)
    pm = _need(mean, "mean", torch.float32, (n,), dev)
    ps = _need(rstd, "rstd", torch.float32, (n,), dev)
    pr = None if grad_res is None else _need(grad_res, "grad_h", dtype, shape, dev)
    gh = h.new_empty(shape)
    gx = torch.empty_like(gh) if want_x else None
    gg = gb = ws = pgg = pgb = pws = None
    nbytes = 0
    if want_weights:
        need = ctypes.c_size_t()
        _check(lib().tp_layer_norm_workspace(code, n, c, ctypes.byref(need)))
        nbytes = need.value
        gg, gb = h.new_empty((2, c), dtype=torch.float32).unbind(0)
        pgg, pgb = gg.data_ptr(), gb.data_ptr()
        if nbytes:
            ws = h.new_empty(nbytes, dtype=torch.uint8)
            pws = ws.data_ptr()
    _call(dev, lib().tp_layer_norm_backward, code, n, c, py, ys, ph, hs, pg, pm, ps, pr,
          None if drop is None else ctypes.byref(drop.cstruct()), gh.data_ptr(), None if gx is None else gx.data_ptr(),
          pgg, pgb, pws, nbytes)
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
    """(tp_attn, device, addresses and strides of q, k, v) after the checks that need the tensors."""
    code, dev = _code(q, "q")
    if q.dim() != 3 or not isinstance(k, torch.Tensor) or k.dim() != 3:
        raise ValueError("q must be [nodes, heads, head_dim], k and v [nodes, key heads, head_dim]")
    dtype = q.dtype
    n, hq, d = q.shape
    hk = k.shape[1]
    rows = (*_rows(q, "q", dtype, (n, hq, d), dev), *_rows(k, "k", dtype, (n, hk, d), dev),
            *_rows(v, "v", dtype, (n, hk, d), dev))
    if not isinstance(seg_ptr, torch.Tensor) or seg_ptr.dim() != 1 or seg_ptr.shape[0] < 1:
        raise ValueError("seg_ptr must hold the number of structures + 1 offsets")
    m = seg_ptr.shape[0]
    pseg = _need(seg_ptr, "seg_ptr", torch.int32, (m,), dev)
    nb = 0
    pp = pb = pk = None
    if (pos is None) != (bias is None):
        raise ValueError("pos and bias go together")
    if bias is not None:
        pp = _need(pos, "pos", torch.float32, (n, 3), dev)
        if not isinstance(bias, torch.Tensor) or bias.dim() != 2 or bias.shape[1] < 1:
            raise ValueError("bias must be [heads, buckets]")
        nb = bias.shape[1]
        pb = _need(bias, "bias", dtype, (hq, nb), dev)
    if key_mask is not None:
        if isinstance(key_mask, torch.Tensor) and key_mask.dtype is torch.bool:
            key_mask = key_mask.view(torch.uint8)
        pk = _need(key_mask, "key_mask", torch.uint8, (n,), dev)
    if scale is None:
        scale = d ** -0.5 if d else 1.0
    if max(n, m - 1, hq, hk, d, nb, abs(steps)) > _INT32_MAX:
        _too_large(nodes=n, structures=m - 1, heads=hq, key_heads=hk, head_dim=d, buckets=nb, steps=abs(steps))
    return _Attn(code, n, m - 1, hq, hk, d, pseg, pk, pp, pb, nb, steps, r_min, scale), dev, rows


def attn_forward(q, k, v, seg_ptr, pos=None, bias=None, r_min=0.5, steps=4, key_mask=None, scale=None, out=None):
    """(out [nodes, heads, head_dim], lse [heads, nodes]) of attention within each
    structure of a packed batch.

    q [nodes, heads, head_dim], k, v [nodes, key heads, head_dim] (views of one
    projected row are fine); seg_ptr int32 [structures + 1] node offsets; pos [nodes, 3]
    and bias [heads, buckets]: learned bias by distance bucket; key_mask [nodes]
    (uint8 or bool, 0 = masked); scale defaults to head_dim ** -0.5."""
    a, dev, rows = _describe(q, k, v, seg_ptr, pos, bias, r_min, steps, key_mask, scale)
    shape = q.shape
    if out is None:
        out = q.new_empty(shape)
    lse = q.new_empty((shape[1], shape[0]), dtype=torch.float32)
    _call(dev, lib().tp_attn_forward, ctypes.byref(a), *rows, *_rows(out, "out", q.dtype, shape, dev), lse.data_ptr())
    return out, lse


def attn_backward(q, k, v, seg_ptr, out, lse, grad_out, pos=None, bias=None, r_min=0.5, steps=4, key_mask=None,
                  scale=None, outs=None, want_bias=True):
    """(grad_q, grad_k, grad_v, grad_bias) of attn_forward; grad_bias is None without a
    bias or with ``want_bias`` false.  ``outs``: (grad_q, grad_k, grad_v) to fill, e.g. the
    views of one projected row's gradient."""
    a, dev, rows = _describe(q, k, v, seg_ptr, pos, bias, r_min, steps, key_mask, scale)
    dtype = q.dtype
    n, hq, d = q.shape
    hk = k.shape[1]
    if outs is None:
        outs = [q.new_empty((n, h, d)) for h in (hq, hk, hk)]
    gq, gk, gv = outs
    gb = torch.empty_like(bias) if bias is not None and want_bias else None
    need = ctypes.c_size_t()
    _check(lib().tp_attn_backward_workspace(ctypes.byref(a), ctypes.byref(need)))
    ws = q.new_empty(need.value, dtype=torch.uint8) if need.value else None
    _call(dev, lib().tp_attn_backward, ctypes.byref(a), *rows, *_rows(out, "out", dtype, (n, hq, d), dev),
          _need(lse, "lse", torch.float32, (hq, n), dev), *_rows(grad_out, "grad_out", dtype, (n, hq, d), dev),
          *_rows(gq, "grad_q", dtype, (n, hq, d), dev), *_rows(gk, "grad_k", dtype, (n, hk, d), dev),
          *_rows(gv, "grad_v", dtype, (n, hk, d), dev), None if gb is None else gb.data_ptr(),
          None if ws is None else ws.data_ptr(), need.value)
    return gq, gk, gv, gb
