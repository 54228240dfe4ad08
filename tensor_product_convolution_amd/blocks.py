"""Around the attention block: the norm and position rotation of queries and keys, routing
and products grouped by chemical element or expert, and the AdamW step.

Argument marshalling only, like the rest of the binding: conventions, formulas
and errors are those of ``include/tpconv.h``.  Tensors are float32 or bfloat16;
strided rows are taken as they are where the C entry point takes a stride.
"""
import array
import ctypes
import math
from typing import NamedTuple

import torch

from . import lib
from .layers import _INT32_MAX, _call, _check, _code, _need, _rows, _too_large

_TENSORS = {torch.Tensor, torch.nn.Parameter}
_dtype_of, _shape_of = torch.Tensor.dtype.__get__, torch.Tensor.shape.__get__
_is_contiguous, _device_of, _address_of = torch.Tensor.is_contiguous, torch.Tensor.get_device, torch.Tensor.data_ptr
_ROWS = {"source": 0, "grouped": 1}
_ACTS = {None: 0, "silu": 1}
_POS = {torch.float32: 0, torch.int32: 1}


class _Heads(ctypes.Structure):
    _fields_ = [("dtype", ctypes.c_int32), ("n_heads", ctypes.c_int32), ("n_kv_heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("n_rows", ctypes.c_int64), ("gamma_q", ctypes.c_void_p),
                ("gamma_k", ctypes.c_void_p), ("eps", ctypes.c_float), ("pos_type", ctypes.c_int32),
                ("axes", ctypes.c_int32), ("pos", ctypes.c_void_p), ("freq", ctypes.c_void_p),
                ("n_pairs", ctypes.c_int32), ("interleaved", ctypes.c_int32)]


class _Grouped(ctypes.Structure):
    _fields_ = [("dtype", ctypes.c_int32), ("n_groups", ctypes.c_int32), ("n_in", ctypes.c_int32),
                ("n_out", ctypes.c_int32), ("n_slots", ctypes.c_int64), ("fan", ctypes.c_int32),
                ("x_rows", ctypes.c_int32), ("y_rows", ctypes.c_int32), ("ptr", ctypes.c_void_p),
                ("rows", ctypes.c_void_p), ("w", ctypes.c_void_p)]


class _AdamW(ctypes.Structure):
    _fields_ = [("bits", ctypes.c_int32), ("grad_dtype", ctypes.c_int32), ("n_tensors", ctypes.c_int32),
                ("sizes", ctypes.c_void_p), ("table", ctypes.c_void_p), ("m", ctypes.c_void_p), ("v", ctypes.c_void_p),
                ("m_unit", ctypes.c_void_p), ("v_unit", ctypes.c_void_p), ("beta1", ctypes.c_double),
                ("beta2", ctypes.c_double), ("eps", ctypes.c_double), ("lr", ctypes.c_double),
                ("max_norm", ctypes.c_double), ("lr_at", ctypes.c_void_p), ("seed", ctypes.c_uint64),
                ("scalars", ctypes.c_void_p)]


def _workspace(t, nbytes):
    return t.new_empty(nbytes, dtype=torch.uint8) if nbytes else None


def _at(t):
    return None if t is None else t.data_ptr()


# ---- norm and rotation of queries and keys ---------------------------------------------
def rotary_frequencies(n_pairs, axes=1, base=1e4, stretch=1.0, trained=None, few=1.0, many=32.0, device=None):
    """Frequencies [n_pairs, axes] (float64) that fall geometrically from 1 to 1 / base, for
    head_norm_rotate_forward: pair i turns with axis i % axes.

    stretch: the length to serve over the length trained for; all frequencies are divided by it.
    With ``trained`` (that length) only the slow ones are, by parts (Peng, Quesnelle, Fan and Shippole, 2023): a pair that makes more than ``many``
    turns over it keeps its frequency, one with fewer than ``few`` is divided by ``stretch``, those
    between go over linearly in the number of turns."""
    if n_pairs < 0 or axes < 1 or not stretch > 0 or not base > 0:
        raise ValueError("n_pairs must not be negative; axes, base and stretch must be positive")
    each = (n_pairs + axes - 1) // axes
    i = torch.arange(n_pairs, dtype=torch.float64)
    f = base ** (-(i // axes) / max(1, each))
    slow = torch.ones_like(f)
    if trained is not None:
        if not trained > 0 or not 0 <= few < many:
            raise ValueError("trained must be positive, 0 <= few < many")
        slow = 1.0 - ((f * trained / (2 * math.pi) - few) / (many - few)).clamp(0.0, 1.0)
    f = f * ((1.0 - slow) + slow / stretch)
    out = torch.zeros(n_pairs, axes, dtype=torch.float64)
    if n_pairs:
        out[i.long(), i.long() % axes] = f
    return out.to(device) if device is not None else out


def _heads(q, k, gamma_q, gamma_k, pos, freq, interleaved, eps):
    """(tp_heads, device, addresses and strides of q and k)"""
    code, dev = _code(q, "q")
    if q.dim() != 3 or not isinstance(k, torch.Tensor) or k.dim() != 3:
        raise ValueError("q must be [rows, heads, head_dim], k [rows, key heads, head_dim]")
    n, hq, d = q.shape
    hk = k.shape[1]
    if max(hq, hk, d) > _INT32_MAX:
        _too_large(heads=hq, key_heads=hk, head_dim=d)
    rows = (*_rows(q, "q", q.dtype, (n, hq, d), dev), *_rows(k, "k", q.dtype, (n, hk, d), dev))
    if (gamma_q is None) != (gamma_k is None):
        raise ValueError("gamma_q and gamma_k go together")
    if (pos is None) != (freq is None):
        raise ValueError("pos and freq go together")
    gq = gk = pp = pf = None
    if gamma_q is not None:
        gq = _need(gamma_q, "gamma_q", torch.float32, (d,), dev)
        gk = _need(gamma_k, "gamma_k", torch.float32, (d,), dev)
    kind = axes = pairs = 0
    if pos is not None:
        if not isinstance(pos, torch.Tensor) or pos.dtype not in _POS or pos.dim() != 2:
            raise TypeError("pos must be float32 or int32 [rows, axes]")
        if not isinstance(freq, torch.Tensor) or freq.dim() != 2:
            raise ValueError("freq must be [pairs, axes]")
        kind, axes, pairs = _POS[pos.dtype], pos.shape[1], freq.shape[0]
        if max(axes, pairs) > _INT32_MAX:
            _too_large(axes=axes, pairs=pairs)
        pp = _need(pos, "pos", pos.dtype, (n, axes), dev)
        pf = _need(freq, "freq", torch.float64, (pairs, axes), dev)
    return _Heads(code, hq, hk, d, n, gq, gk, eps, kind, axes, pp, pf, pairs, int(bool(interleaved))), dev, rows


def head_norm_rotate_forward(q, k, gamma_q=None, gamma_k=None, pos=None, freq=None, interleaved=False, eps=1e-6, outs=None):
    """(q, k) with each head normed (gamma_q, gamma_k float32 [head_dim]; None: not) and its first
    2 pairs values turned by pos @ freq.T (pos [rows, axes] float32 or int32, freq [pairs, axes]
    float64; None: not).

    q [rows, heads, head_dim], k [rows, key heads, head_dim] may be views of one projected row;
    ``outs``: (q, k) to fill, also q and k themselves."""
    h, dev, rows = _heads(q, k, gamma_q, gamma_k, pos, freq, interleaved, eps)
    qo, ko = (q.new_empty(q.shape), q.new_empty(k.shape)) if outs is None else outs
    _call(dev, lib().tp_head_norm_rotate_forward, ctypes.byref(h), *rows, *_rows(qo, "q_out", q.dtype, q.shape, dev),
          *_rows(ko, "k_out", q.dtype, k.shape, dev))
    return qo, ko


def head_norm_rotate_backward(grad_qo, grad_ko, q, k, gamma_q=None, gamma_k=None, pos=None, freq=None, interleaved=False,
                              eps=1e-6, want_pos=False, want_weights=True, outs=None):
    """(grad_q, grad_k, grad_gamma_q, grad_gamma_k, grad_pos) of head_norm_rotate_forward, None for
    what is not there or not wanted.  ``outs``: (grad_q, grad_k) to fill."""
    h, dev, rows = _heads(q, k, gamma_q, gamma_k, pos, freq, interleaved, eps)
    gq, gk = (q.new_empty(q.shape), q.new_empty(k.shape)) if outs is None else outs
    gamma = gamma_q is not None and want_weights
    ggq = ggk = gpos = ws = None
    nbytes = 0
    if gamma:
        need = ctypes.c_size_t()
        _check(lib().tp_head_norm_rotate_workspace(ctypes.byref(h), ctypes.byref(need)))
        nbytes = need.value
        ws = _workspace(q, nbytes)
        ggq, ggk = q.new_empty((2, q.shape[2]), dtype=torch.float32).unbind(0)
    if want_pos:
        if pos is None:
            raise ValueError("want_pos without pos")
        gpos = torch.empty_like(pos, dtype=torch.float32)
    dt = q.dtype
    _call(dev, lib().tp_head_norm_rotate_backward, ctypes.byref(h), *_rows(grad_qo, "grad_qo", dt, q.shape, dev),
          *_rows(grad_ko, "grad_ko", dt, k.shape, dev), *rows, *_rows(gq, "grad_q", dt, q.shape, dev),
          *_rows(gk, "grad_k", dt, k.shape, dev), _at(ggq), _at(ggk), _at(gpos), _at(ws), nbytes)
    return gq, gk, ggq, ggk, gpos


# ---- routing and products by group -------------------------------------------------------
class Groups(NamedTuple):
    """Slots in group order, from group_rows: ``rows`` int32 [slots], ``ptr`` int32 [groups + 1],
    ``fan`` slots for each source row."""
    ptr: torch.Tensor
    rows: torch.Tensor
    fan: int


def route_forward(logits, k, over_all=False):
    """(weight float32, index int32), [rows, k], of the k largest logits of each row of
    logits [rows, groups]: softmax over the chosen, or with ``over_all`` over all groups."""
    code, dev = _code(logits, "logits")
    if logits.dim() != 2:
        raise ValueError("logits must be [rows, groups]")
    n, e = logits.shape
    if max(e, k) > _INT32_MAX:
        _too_large(groups=e, k=k)
    pl, stride = _rows(logits, "logits", logits.dtype, (n, e), dev)
    weight = logits.new_empty((n, max(k, 0)), dtype=torch.float32)
    index = logits.new_empty((n, max(k, 0)), dtype=torch.int32)
    _call(dev, lib().tp_route_forward, code, n, e, k, int(bool(over_all)), pl, stride, weight.data_ptr(), index.data_ptr())
    return weight, index


def route_backward(grad_weight, logits, weight, index, over_all=False):
    """Gradient with respect to the logits of route_forward."""
    code, dev = _code(logits, "logits")
    if logits.dim() != 2 or not isinstance(weight, torch.Tensor) or weight.dim() != 2:
        raise ValueError("logits must be [rows, groups], weight [rows, k]")
    n, e = logits.shape
    k = weight.shape[1]
    if max(e, k) > _INT32_MAX:
        _too_large(groups=e, k=k)
    pl, stride = _rows(logits, "logits", logits.dtype, (n, e), dev)
    out = logits.new_empty((n, e))
    _call(dev, lib().tp_route_backward, code, n, e, k, int(bool(over_all)), pl, stride,
          _need(weight, "weight", torch.float32, (n, k), dev), _need(index, "index", torch.int32, (n, k), dev),
          _need(grad_weight, "grad_weight", torch.float32, (n, k), dev), out.data_ptr())
    return out


def group_rows(index, n_groups):
    """Groups of the slots ``index`` (int32, [rows] or [rows, k]): chemical elements of atoms, or
    route_forward's choices.  An index that is no group leaves its slot out."""
    if not isinstance(index, torch.Tensor):
        raise TypeError("index must be a torch tensor")
    if index.dim() not in (1, 2) or (index.dim() == 2 and index.shape[1] < 1):
        raise ValueError("index must be [rows] or [rows, k]")
    dev = index.get_device()
    if dev < 0:
        raise ValueError("index must live on the GPU")
    n, fan = index.numel(), 1 if index.dim() == 1 else index.shape[1]
    pi = _need(index, "index", torch.int32, index.shape, dev)
    if n_groups > _INT32_MAX:
        _too_large(groups=n_groups)
    need = ctypes.c_size_t()
    _check(lib().tp_group_workspace(n, n_groups, ctypes.byref(need)))
    ptr, rows, ws = index.new_empty(n_groups + 1), index.new_empty(n), _workspace(index, need.value)
    _call(dev, lib().tp_group_rows, pi, n, n_groups, ptr.data_ptr(), rows.data_ptr(), _at(ws), need.value)
    return Groups(ptr, rows, fan)


def _grouped(w, groups, x_rows, y_rows):
    """(tp_grouped, device, rows of x, rows of y)"""
    code, dev = _code(w, "w")
    if w.dim() != 3:
        raise ValueError("w must be [groups, in, out]")
    e, i, o = w.shape
    if max(e, i, o) > _INT32_MAX:
        _too_large(groups=e, n_in=i, n_out=o)
    pw = _need(w, "w", w.dtype, w.shape, dev)
    for name, r in (("x_rows", x_rows), ("y_rows", y_rows)):
        if r not in _ROWS:
            raise ValueError(f"{name} must be 'source' or 'grouped'")
    n, fan = groups.rows.shape[0], groups.fan
    if fan < 1 or n % fan:
        raise ValueError("groups: slots must be a multiple of fan")
    g = _Grouped(code, e, i, o, n, fan, _ROWS[x_rows], _ROWS[y_rows], _need(groups.ptr, "groups.ptr", torch.int32, (e + 1,), dev),
                 _need(groups.rows, "groups.rows", torch.int32, (n,), dev), pw)
    return g, dev, n // fan if x_rows == "source" else n, n


def grouped_linear_forward(x, w, groups, bias=None, act=None, x_rows="source", y_rows="source", want_pre=False):
    """act(x w[group] + bias[group]) for each slot of ``groups``, [slots, out]; with ``want_pre`` also
    what the activation was taken of, for the backward.

    w [groups, in, out], bias [groups, out]; act None or "silu".  x_rows "source": x [rows, in],
    each row read by its slots; "grouped": one row for each slot, in group order.  y_rows
    "source": rows of the result by slot, "grouped": in group order.  Slots that belong to no group
    get zeros."""
    g, dev, nx, n = _grouped(w, groups, x_rows, y_rows)
    if act not in _ACTS:
        raise ValueError("act must be None or 'silu'")
    if want_pre and act is None:
        raise ValueError("want_pre goes with an activation")
    px, xs = _rows(x, "x", w.dtype, (nx, g.n_in), dev)
    pb = None if bias is None else _need(bias, "bias", w.dtype, (g.n_groups, g.n_out), dev)
    y = w.new_empty((n, g.n_out))
    pre = torch.empty_like(y) if want_pre else None
    _call(dev, lib().tp_grouped_linear_forward, ctypes.byref(g), px, xs, pb, _ACTS[act], y.data_ptr(), g.n_out, _at(pre))
    return (y, pre) if want_pre else y


def grouped_linear_backward(grad_z, x, w, groups, x_rows="source", y_rows="source", pre=None, want_x=True, want_w=True,
                            want_bias=False):
    """(grad_x, grad_w, grad_bias) from ``grad_z``, the gradient of x w + bias (rows as y_rows says);
    None for what is not wanted.  ``pre``: where x = silu(pre), grad_x is the gradient of pre."""
    g, dev, nx, n = _grouped(w, groups, x_rows, y_rows)
    dt = w.dtype
    pg, gs = _rows(grad_z, "grad_z", dt, (n, g.n_out), dev)
    px, xs = _rows(x, "x", dt, (nx, g.n_in), dev)
    pp, ps = (None, 0) if pre is None else _rows(pre, "pre", dt, (nx, g.n_in), dev)
    if want_bias and not want_w:
        raise ValueError("want_bias goes with want_w")
    gx = w.new_empty((nx, g.n_in)) if want_x else None
    gw = torch.empty_like(w) if want_w else None
    gb = w.new_empty((g.n_groups, g.n_out)) if want_bias else None
    need = ctypes.c_size_t()
    _check(lib().tp_grouped_linear_workspace(ctypes.byref(g), int(want_x), int(want_w), ctypes.byref(need)))
    ws = _workspace(w, need.value)
    _call(dev, lib().tp_grouped_linear_backward, ctypes.byref(g), pg, gs, px, xs, pp, ps, _at(gx), g.n_in, _at(gw), _at(gb),
          _at(ws), need.value)
    return gx, gw, gb


def _choices(y, weight):
    code, dev = _code(y, "y")
    if y.dim() != 2 or not isinstance(weight, torch.Tensor) or weight.dim() != 2:
        raise ValueError("y must be [rows * k, columns], weight [rows, k]")
    n, k = weight.shape
    c = y.shape[1]
    if max(k, c) > _INT32_MAX:
        _too_large(k=k, columns=c)
    return code, dev, n, k, c, _need(y, "y", y.dtype, (n * k, c), dev), _need(weight, "weight", torch.float32, (n, k), dev)


def combine_forward(y, weight):
    """Sum over a row's choices: out[n] = sum_j weight[n, j] y[n k + j]."""
    code, dev, n, k, c, py, pw = _choices(y, weight)
    out = y.new_empty((n, c))
    _call(dev, lib().tp_combine_forward, code, n, k, c, py, pw, out.data_ptr())
    return out


def combine_backward(grad_out, y, weight):
    """(grad_y, grad_weight) of combine_forward."""
    code, dev, n, k, c, py, pw = _choices(y, weight)
    gy, gw = torch.empty_like(y), torch.empty_like(weight)
    _call(dev, lib().tp_combine_backward, code, n, k, c, _need(grad_out, "grad_out", y.dtype, (n, c), dev), py, pw,
          gy.data_ptr(), gw.data_ptr())
    return gy, gw


# ---- the AdamW step ------------------------------------------------------------------------
class AdamW:
    """AdamW over ``params`` (contiguous float32 tensors on one GPU, updated in place), all in a few
    launches a step.

    weight_decay: one number, or one for each tensor.  max_norm: the gradients are scaled down to this
    2-norm over all of them (None: not; float("inf"): the norm is only returned), and a step whose
    norm is not finite changes nothing.  bits: 32, or 8 for states of one byte a value (rounded at
    random, from ``seed`` and the step's number; without max_norm a gradient that is not finite leaves zeros there).  copies: bfloat16 tensors (or None) that get the new
    parameters too.  lr: a number, or a float32 tensor of one value on the GPU, read by every step: the
    way to change it under a captured graph.

    The states of tensor i lie from ``offsets[i]`` on in ``exp_avg`` and ``exp_avg_sq`` (with bits 8 codes,
    whose units of 256 values each are ``exp_avg_unit`` and ``exp_avg_sq_unit``).  One optimiser serves
    one stream at a time.  Parameters and copies stay where they are: copy new values into them; a step after
    their ``.data`` was set to another tensor is refused."""

    def __init__(self, params, lr=1e-3, betas=(0.9, 0.999), eps=1e-8, weight_decay=0.01, max_norm=None, bits=32, copies=None,
                 seed=0):
        params = list(params)
        if not params:
            raise ValueError("no parameters")
        if bits not in (8, 32):
            raise ValueError("bits must be 8 or 32")
        if not 0 <= seed < 1 << 64:
            raise ValueError("seed must be an unsigned 64-bit integer")
        _, self._dev = _code(params[0], "params[0]")
        n = self._n = len(params)
        where = [_need(p, f"params[{i}]", torch.float32, p.shape, self._dev) for i, p in enumerate(params)]
        copies = [None] * n if copies is None else list(copies)
        decay = [float(weight_decay)] * n if isinstance(weight_decay, (int, float)) else [float(d) for d in weight_decay]
        if len(copies) != n or len(decay) != n:
            raise ValueError("copies and weight_decay need one entry for each parameter")
        low = [None if c is None else _need(c, f"copies[{i}]", torch.bfloat16, params[i].shape, self._dev)
               for i, c in enumerate(copies)]
        end = 0                            # a value in two tensors would be updated twice, by whichever comes last
        for first, last in sorted((t.data_ptr(), t.data_ptr() + t.nbytes) for t in (*params, *copies) if t is not None and t.numel()):
            if first < end:
                raise ValueError("a parameter or copy is there twice, or two overlap")
            end = last
        # the table holds addresses: of memory that stays the optimiser's even where a tensor is given other
        self._written = [t for t in (*params, *copies) if t is not None]
        self._places, self._held = list(map(_address_of, self._written)), [t.detach() for t in self._written]
        self.params, self.copies, self.bits, self.betas, self.eps, self.max_norm = params, copies, bits, betas, eps, max_norm
        self.lr, self.seed = lr, seed
        self.numels = [p.numel() for p in params]
        self._shapes = [p.shape for p in params]
        self._sizes = (ctypes.c_int64 * n)(*self.numels)
        self.offsets, at = [], 0
        for k in self.numels:
            self.offsets.append(at)
            at += (k + 255) // 256 * 256
        table, values, ws = ctypes.c_size_t(), ctypes.c_int64(), ctypes.c_size_t()
        _check(lib().tp_adamw_sizes(n, self._sizes, ctypes.byref(table), ctypes.byref(values), ctypes.byref(ws)))
        host = torch.empty(max(16, table.value), dtype=torch.uint8)
        pointers = ctypes.c_void_p * n
        _check(lib().tp_adamw_table(n, self._sizes, pointers(*where), pointers(*low), (ctypes.c_float * n)(*decay),
                                    host.data_ptr()))
        new = lambda k, dt: torch.zeros(k, dtype=dt, device=params[0].device)
        self._table = host.to(params[0].device)
        code, total = (torch.float32 if bits == 32 else torch.uint8), values.value
        self.exp_avg, self.exp_avg_sq = new(total, code), new(total, code)
        self.exp_avg_unit = self.exp_avg_sq_unit = None
        if bits == 8:
            self.exp_avg_unit, self.exp_avg_sq_unit = new(total // 256, torch.float32), new(total // 256, torch.float32)
        self._scalars = new(64, torch.uint8)
        self._ws = new(max(16, ws.value), torch.uint8)
        self._ws_bytes = ws.value
        # the arrays that the description points to live as long as it does; the rates are set by each step
        self._desc = _AdamW(bits, 0, n, ctypes.addressof(self._sizes), self._table.data_ptr(), self.exp_avg.data_ptr(),
                            self.exp_avg_sq.data_ptr(), _at(self.exp_avg_unit), _at(self.exp_avg_sq_unit), 0.0, 0.0, 0.0, 0.0, 0.0,
                            None, 0, self._scalars.data_ptr())

    def step(self, grads, lr=None):
        """One step with ``grads``, contiguous tensors of the parameters' shapes, all float32 or all
        bfloat16 (None is refused: a step moves every parameter).  Returns their norm (a float32 tensor of one value), or None without max_norm."""
        if len(grads) != self._n:
            raise ValueError(f"{len(grads)} gradients for {self._n} parameters")
        code, _ = _code(grads[0], "grads[0]")
        dt, dev, n = grads[0].dtype, self._dev, self._n
        # one pass over all tensors for each property: the host's time is most of a small step's
        if not (set(map(type, grads)) <= _TENSORS and list(map(_dtype_of, grads)).count(dt) == n
                and list(map(_shape_of, grads)) == self._shapes and all(map(_is_contiguous, grads))
                and list(map(_device_of, grads)).count(dev) == n):
            for i, (g, shape) in enumerate(zip(grads, self._shapes)):
                _need(g, f"grads[{i}]", dt, shape, dev)
        if list(map(_address_of, self._written)) != self._places:
            raise ValueError("a parameter or copy has moved since the optimiser was made (its .data was set)")
        where = array.array("Q", map(_address_of, grads))
        lr = self.lr if lr is None else lr
        lr_at = None
        if isinstance(lr, torch.Tensor):
            lr_at, lr = _need(lr, "lr", torch.float32, lr.shape if lr.numel() == 1 else (1,), dev), 0.0
        norm = None
        if self.max_norm is not None:
            if not self.max_norm > 0:
                raise ValueError("max_norm must be positive")
            norm = self._table.new_empty((), dtype=torch.float32)
        a = self._desc
        a.grad_dtype, a.lr, a.lr_at, a.max_norm = code, lr, lr_at, 0.0 if norm is None else self.max_norm
        a.beta1, a.beta2 = self.betas
        a.eps, a.seed = self.eps, self.seed
        _call(dev, lib().tp_adamw_step, ctypes.byref(a), where.buffer_info()[0], _at(norm), self._ws.data_ptr(), self._ws_bytes)
        torch.autograd.graph.increment_version(self._written)  # a graph that saved one of them is not right any more
        return norm

    def moments(self):
        """(exp_avg, exp_avg_sq) over all tensors as float32 values: the states themselves with bits 32,
        new tensors with bits 8."""
        if self.bits == 32:
            return self.exp_avg, self.exp_avg_sq
        out = []
        for second, codes, units in ((0, self.exp_avg, self.exp_avg_unit), (1, self.exp_avg_sq, self.exp_avg_sq_unit)):
            v = torch.empty_like(codes, dtype=torch.float32)
            _call(self._dev, lib().tp_adamw_values, second, codes.numel(), codes.data_ptr(), units.data_ptr(), v.data_ptr())
            out.append(v)
        return tuple(out)

    def state(self):
        """What a checkpoint holds: (steps done, exp_avg, exp_avg_sq[, their units]), for load().  Waits
        for the GPU."""
        held = (self.exp_avg, self.exp_avg_sq, self.exp_avg_unit, self.exp_avg_sq_unit)
        return (int(self._scalars[:8].view(torch.int64)), *[t.clone() for t in held if t is not None])

    def load(self, step, *held):
        """Takes up the states of state()."""
        mine = [t for t in (self.exp_avg, self.exp_avg_sq, self.exp_avg_unit, self.exp_avg_sq_unit) if t is not None]
        if len(held) != len(mine):
            raise ValueError(f"{len(mine)} state tensors, got {len(held)}")
        if step < 0:
            raise ValueError("step must not be negative")
        for t, h in zip(mine, held):
            if h.dtype != t.dtype or h.shape != t.shape:
                raise ValueError(f"a state is {h.dtype} {tuple(h.shape)}, expected {t.dtype} {tuple(t.shape)}")
            t.copy_(h)
        self._scalars[:8].view(torch.int64).fill_(step)
