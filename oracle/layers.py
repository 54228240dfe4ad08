"""Float64 reference of the layers around the convolution: attention within each
structure with a bias by distance bucket, layer norm and dropout.

Written from the definitions; the formulas are in ``include/tpconv.h``.  Everything
is float64 except what the definitions place in float32: the squared distance that
selects a bucket and the dropout factor.
"""
import numpy as np

LOWEST = -1e30          # scores at or below count as masked


def buckets(pos, r_min, steps, n_buckets):
    """[n, n] bucket of every pair of rows of pos (float32 [n, 3]); a distance that is not a
    number has no bits to go by and counts as bucket 0."""
    p = np.asarray(pos, dtype=np.float32)
    shift = 23 - int(np.log2(steps))
    with np.errstate(invalid="ignore", over="ignore"):
        d = p[:, None, :] - p[None, :, :]
        sq = d * d                                          # float32, rounded each
        d2 = (sq[..., 0] + sq[..., 1]) + sq[..., 2]
    r = np.float32(r_min)
    base = int((r * r).view(np.int32)) >> shift
    return np.where(np.isnan(d2), 0, np.clip((d2.view(np.int32).astype(np.int64) >> shift) - base, 0, n_buckets - 1))


def _probs(q, k, b, live, scale):
    """(probabilities, lse) of one head of one structure; rows without a key are zero."""
    s = scale * (q @ k.T) + b
    s = np.where(live[None, :] & ~(s <= LOWEST), s, -np.inf)
    m = s.max(axis=1, initial=-np.inf)
    some = m > -np.inf
    e = np.exp(s - np.where(some, m, 0.0)[:, None])
    l = e.sum(axis=1)
    with np.errstate(divide="ignore"):
        lse = np.where(some, np.where(some, m, 0.0) + np.log(l), -np.inf)
    return e / np.where(some, l, 1.0)[:, None], lse


def _each(q, k, v, seg_ptr, pos, bias, r_min, steps, key_mask, scale):
    f = lambda t: np.asarray(t, dtype=np.float64)
    q, k, v = f(q), f(k), f(v)
    hq, rep = q.shape[1], q.shape[1] // k.shape[1]
    scale = q.shape[2] ** -0.5 if scale is None else scale
    for b in range(len(seg_ptr) - 1):
        sl = slice(int(seg_ptr[b]), int(seg_ptr[b + 1]))
        n = sl.stop - sl.start
        if n == 0:
            continue
        live = np.ones(n, bool) if key_mask is None else np.asarray(key_mask[sl]) != 0
        bk = None if bias is None else buckets(pos[sl], r_min, steps, bias.shape[1])
        for h in range(hq):
            g = h // rep
            # a masked key's rows are never multiplied
            kk = np.where(live[:, None], k[sl, g], 0.0)
            vv = np.where(live[:, None], v[sl, g], 0.0)
            bb = 0.0 if bias is None else f(bias)[h][bk]
            p, lse = _probs(q[sl, h], kk, bb, live, scale)
            yield sl, h, g, bk, live, q[sl, h], kk, vv, p, lse, scale


def attn_forward(q, k, v, seg_ptr, pos=None, bias=None, r_min=0.5, steps=4, key_mask=None, scale=None):
    """(out, lse) as tp_attn_forward."""
    out = np.zeros(q.shape)
    lse = np.zeros((q.shape[1], q.shape[0]))
    for sl, h, g, bk, live, qq, kk, vv, p, t, sc in _each(q, k, v, seg_ptr, pos, bias, r_min, steps, key_mask, scale):
        out[sl, h] = p @ vv
        lse[h, sl] = t
    return out, lse


def attn_backward(q, k, v, seg_ptr, grad_out, pos=None, bias=None, r_min=0.5, steps=4, key_mask=None, scale=None):
    """(grad_q, grad_k, grad_v, grad_bias) as tp_attn_backward."""
    gq, gk, gv = np.zeros(q.shape), np.zeros(k.shape), np.zeros(v.shape)
    gb = None if bias is None else np.zeros(bias.shape)
    go = np.asarray(grad_out, dtype=np.float64)
    for sl, h, g, bk, live, qq, kk, vv, p, t, sc in _each(q, k, v, seg_ptr, pos, bias, r_min, steps, key_mask, scale):
        d = go[sl, h]
        dp = d @ vv.T
        ds = p * (dp - (p * dp).sum(axis=1, keepdims=True))
        gq[sl, h] = sc * (ds @ kk)
        gk[sl, g] += np.where(live[:, None], sc * (ds.T @ qq), 0.0)
        gv[sl, g] += np.where(live[:, None], p.T @ d, 0.0)
        if gb is not None:
            np.add.at(gb[h], bk, ds)
    return gq, gk, gv, gb


def layer_norm_forward(h, gamma, beta, eps):
    """(y, mean, rstd)"""
    h = np.asarray(h, dtype=np.float64)
    mean = h.mean(axis=1)
    rstd = 1.0 / np.sqrt(((h - mean[:, None]) ** 2).mean(axis=1) + eps)
    return (h - mean[:, None]) * rstd[:, None] * np.asarray(gamma, dtype=np.float64) + np.asarray(beta, dtype=np.float64), mean, rstd


def layer_norm_backward(grad_y, h, gamma, eps):
    """(grad_h, grad_gamma, grad_beta)"""
    gy = np.asarray(grad_y, dtype=np.float64)
    _, mean, rstd = layer_norm_forward(h, gamma, gamma, eps)
    z = (np.asarray(h, dtype=np.float64) - mean[:, None]) * rstd[:, None]
    t = gy * np.asarray(gamma, dtype=np.float64)
    gh = rstd[:, None] * (t - t.mean(axis=1, keepdims=True) - z * (t * z).mean(axis=1, keepdims=True))
    return gh, (gy * z).sum(axis=0), gy.sum(axis=0)


def philox_block(blk, seed, offset):
    """The four 32-bit words of Philox 4x32-10 (Salmon et al., SC 2011) with the key
    `seed` and the counter (blk, offset), as Python integers."""
    c = [blk & 0xFFFFFFFF, blk >> 32, offset & 0xFFFFFFFF, offset >> 32]
    k = [seed & 0xFFFFFFFF, seed >> 32]
    for _ in range(10):
        a, b = 0xD2511F53 * c[0], 0xCD9E8D57 * c[2]
        c = [(b >> 32) ^ c[1] ^ k[0], b & 0xFFFFFFFF, (a >> 32) ^ c[3] ^ k[1], a & 0xFFFFFFFF]
        k = [(k[0] + 0x9E3779B9) & 0xFFFFFFFF, (k[1] + 0xBB67AE85) & 0xFFFFFFFF]
    return c


def philox_words(n, seed, offset):
    """Word e is word e % 4 of block e // 4, for e < n."""
    return [w for blk in range((n + 3) // 4) for w in philox_block(blk, seed, offset)][:n]


def dropout_factor(shape, p, seed, offset):
    """1 / (1 - p) (rounded to float32) where an element is kept, else 0."""
    n = int(np.prod(shape))
    w = np.array(philox_words(n, seed, offset), dtype=np.uint64).reshape(shape)
    return np.where(w >= int(p * 2.0 ** 32), np.float64(np.float32(1.0 / (1.0 - p))), 0.0)
