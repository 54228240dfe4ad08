"""Float64 reference of what stands around the attention block: norm and rotation of queries
and keys, routing and products by group, the AdamW step.

Written from the definitions; the formulas are in ``include/tpconv.h``.  Everything is
float64 except what the definitions round: the unit of 8-bit states.
"""
import numpy as np

from .layers import philox_words


def _f(t):
    return np.asarray(t, dtype=np.float64)


# ---- norm and rotation of queries and keys ---------------------------------------------
def pair_places(n_pairs, interleaved):
    i = np.arange(n_pairs)
    return (2 * i, 2 * i + 1) if interleaved else (i, i + n_pairs)


def _angles(pos, freq):
    return (_f(pos)[:, None, :] * _f(freq)[None]).sum(-1)[:, None, :]      # [rows, 1, pairs]


def head_forward(x, gamma, pos, freq, interleaved, eps):
    """One side: x [rows, heads, dim], gamma and pos may be None."""
    x = _f(x)
    y = x.copy()
    if gamma is not None:
        y = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * _f(gamma)
    if pos is not None:
        t = _angles(pos, freq)
        a, b = pair_places(len(freq), interleaved)
        ya, yb = y[..., a], y[..., b]
        y[..., a], y[..., b] = ya * np.cos(t) - yb * np.sin(t), ya * np.sin(t) + yb * np.cos(t)
    return y


def head_backward(g, x, gamma, pos, freq, interleaved, eps):
    """(grad_x, grad_gamma, grad_pos) of one side."""
    g, x = _f(g), _f(x)
    h, gpos, gg = g.copy(), None, None
    r = np.ones(x.shape[:2] + (1,)) if gamma is None else 1 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    z = x * r
    y = z if gamma is None else z * _f(gamma)
    if pos is not None:
        t = _angles(pos, freq)
        a, b = pair_places(len(freq), interleaved)
        h[..., a], h[..., b] = g[..., a] * np.cos(t) + g[..., b] * np.sin(t), g[..., b] * np.cos(t) - g[..., a] * np.sin(t)
        gpos = (h[..., b] * y[..., a] - h[..., a] * y[..., b]).sum(1) @ _f(freq)
    if gamma is not None:
        gg = (h * z).sum((0, 1))
        s = h * _f(gamma)
        h = r * (s - z * (s * z).mean(-1, keepdims=True))
    return h, gg, gpos


# ---- routing -------------------------------------------------------------------------------
def route(logits, k, over_all=False):
    """(weight, index)"""
    l = _f(logits)
    n, e = l.shape
    weight, index = np.zeros((n, k)), np.full((n, k), -1)
    for r in range(n):
        live = [i for i in range(e) if l[r, i] > -np.inf]                  # neither -inf nor NaN
        best = sorted(live, key=lambda i: (-l[r, i], i))[:k]
        if not best:
            continue
        p = np.exp(l[r] - l[r, best[0]])
        weight[r, :len(best)] = p[best] / p[live if over_all else best].sum()
        index[r, :len(best)] = best
    return weight, index


def route_backward(grad_weight, logits, weight, index, over_all=False):
    l, w, g = _f(logits), _f(weight), _f(grad_weight)
    out = np.zeros(l.shape)
    for r in range(l.shape[0]):
        at = index[r] >= 0
        if not at.any():
            continue
        chosen, wr, gr = index[r][at], w[r][at], g[r][at]
        out[r, chosen] = wr * gr
        if over_all:
            live = l[r] > -np.inf
            p = np.where(live, np.exp(np.where(live, l[r], 0) - l[r][live].max()), 0)
            out[r] -= p / p.sum() * (wr * gr).sum()
        else:
            out[r, chosen] -= wr * (wr * gr).sum()
    return out


def group_rows(index, n_groups):
    """(ptr, rows)"""
    i = np.asarray(index).reshape(-1)
    g = np.where((i >= 0) & (i < n_groups), i, n_groups)
    return np.searchsorted(np.sort(g), np.arange(n_groups + 1)), np.argsort(g, kind="stable")


# ---- products by group ----------------------------------------------------------------------
def silu(z):
    with np.errstate(over="ignore"):
        return z / (1 + np.exp(-z))


def silu_slope(z):
    with np.errstate(over="ignore"):
        s = 1 / (1 + np.exp(-z))
    return s * (1 + z * (1 - s))


def _rows(ptr, rows, fan, order):
    """Row of each slot of the grouped order, and of what it is read or written to."""
    return np.arange(len(rows)) if order == "grouped" else rows // fan


def grouped_forward(x, w, ptr, rows, fan, bias, x_rows, y_rows):
    """z, rows as y_rows says; zeros for slots without a group."""
    x, w = _f(x), _f(w)
    z = np.zeros((len(rows), w.shape[2]))
    at, to = _rows(ptr, rows, fan, x_rows), _rows(ptr, rows, 1, y_rows)
    for e in range(w.shape[0]):
        s = slice(ptr[e], ptr[e + 1])
        z[to[s]] = x[at[s]] @ w[e] + (0 if bias is None else _f(bias)[e])
    return z


def grouped_backward(gz, x, w, ptr, rows, fan, x_rows, y_rows, pre=None):
    """(grad_x, grad_w, grad_bias)"""
    gz, x, w = _f(gz), _f(x), _f(w)
    gx, gw, gb = np.zeros(x.shape), np.zeros(w.shape), np.zeros((w.shape[0], w.shape[2]))
    at, to = _rows(ptr, rows, fan, x_rows), _rows(ptr, rows, 1, y_rows)
    for e in range(w.shape[0]):
        s = slice(ptr[e], ptr[e + 1])
        np.add.at(gx, at[s], gz[to[s]] @ w[e].T)
        gw[e] = x[at[s]].T @ gz[to[s]]
        gb[e] = gz[to[s]].sum(0)
    return (gx if pre is None else gx * silu_slope(_f(pre))), gw, gb


# ---- the AdamW step --------------------------------------------------------------------------
BLOCK = 256


def code_values(second):
    """Values of the codes of an 8-bit state over its unit, lowest first."""
    octaves = 31 if second else 15
    c = np.arange(8 * octaves + 8)
    return np.where(c < 8, c * 2.0 ** (-2 - octaves), 2.0 ** (c // 8 - octaves) * (1 + c % 8 / 8))


def decode(codes, units, second):
    c, v = np.asarray(codes).astype(int), code_values(second)
    x = v[c] if second else np.where(c >= 128, -1.0, 1.0) * v[c & 127]
    return x * np.repeat(_f(units), BLOCK)


def encode(x, second, u):
    """(codes, units) of values x; u [0, 1) of each."""
    x = _f(x)
    units = np.minimum(np.abs(x).reshape(-1, BLOCK).max(1) / 1.875, 2.0 ** 127).astype(np.float32)
    wide = np.repeat(_f(units), BLOCK)
    a = np.divide(np.abs(x), wide, out=np.zeros_like(x), where=wide > 0)
    v = code_values(second)
    low = np.minimum(np.searchsorted(v, a, side="right") - 1, len(v) - 2)
    code = np.minimum(low + ((a - v[low]) / (v[low + 1] - v[low]) + u >= 1), len(v) - 1)
    if second:
        code = np.where(a > 0, np.maximum(code, 1), code)
    else:
        code = code + np.where((x < 0) & (code > 0), 128, 0)
    return code.astype(np.uint8), units


def adamw(p, g, m, v, t, lr, beta1, beta2, eps, decay, factor=1.0):
    """(p, m, v) after step t (1 for the first) on arrays of one layout."""
    g = _f(g) * factor
    m, v = beta1 * _f(m) + (1 - beta1) * g, beta2 * _f(v) + (1 - beta2) * g * g
    with np.errstate(divide="ignore", invalid="ignore"):
        step = (m / (1 - beta1 ** t)) / (np.sqrt(v / (1 - beta2 ** t)) + eps)
    return _f(p) * (1 - lr * _f(decay)) - lr * step, m, v


def rounding(n, seed, t):
    """u of the first and of the second moments, n values each."""
    w = np.array(philox_words(n, seed, t), dtype=np.int64)
    return (w & 0xFFFF) / 65536.0, (w >> 16) / 65536.0
