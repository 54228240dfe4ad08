"""What is measured of the operators around the convolution: attention over the
atoms of each structure with a distance-bucket bias, layer norm and dropout.

Each case runs one operator as a training or evaluation program calls it.  With
``own`` false the operators are computed in their plain form (elementary torch
operations in 32 bits, rounded once at the end); with ``own`` true by the
library's kernels.  ``exact`` gives the same values from the definitions in 64
bits.  Sizes follow the repository's workloads: 32, 1,536, 4,096, 32,768 and
100,000 atoms, 8 to 128 channels per degree, node rows of 288 to 1,152 values.
"""
import math
import random

import numpy as np
import torch

own = False

DT = {"f32": torch.float32, "bf16": torch.bfloat16}
PAIRS = 16384 * 16384 * 8          # pairs times heads of the largest listed case
EPS = 1e-5


# ---- the cases ---------------------------------------------------------------
def _attn(name, dtype, step, sizes, lo, hi, count, hq, hkv, d, buckets=32, masked=0.0):
    return dict(name=name, op="attn", dtype=dtype, step=step, sizes=sizes, lo=lo, hi=hi, count=count,
                hq=hq, hkv=hkv, d=d, buckets=buckets, masked=masked)


def _norm(name, dtype, step, rows, cols, stride, fused, p):
    return dict(name=name, op="norm", dtype=dtype, step=step, rows=rows, cols=cols, stride=stride,
                fused=fused, p=p)


def _drop(name, dtype, step, rows, cols, p):
    return dict(name=name, op="dropout", dtype=dtype, step=step, rows=rows, cols=cols, p=p)


def listed():
    return [
        # one small structure in an MD loop: the call's latency
        _attn("attn_32atoms_f32_fwd", "f32", False, 1, 32, 32, 1, 4, 4, 16),
        # the 1,536-atom structure, a training step in either type
        _attn("attn_1536_bf16_step", "bf16", True, 1, 1536, 1536, 1, 8, 8, 32),
        _attn("attn_1536_f32_step", "f32", True, 1, 1536, 1536, 1, 8, 8, 16),
        # a training batch of small molecules of uneven size, shared key heads,
        # some atoms masked (ghosts)
        _attn("attn_molecules_bf16_step", "bf16", True, 7, 5, 120, 512, 8, 2, 32, 64, 0.05),
        # an odd structure with an odd head width, evaluated
        _attn("attn_1001_f32_fwd", "f32", False, 1, 1001, 1001, 1, 5, 5, 40, 20, 0.1),
        # 4,096 atoms, one shared key head, 32-bit training step
        _attn("attn_4096_f32_step", "f32", True, 1, 4096, 4096, 1, 4, 1, 64, 64),
        # the largest: one 16,384-atom structure, evaluated
        _attn("attn_16384_bf16_fwd", "bf16", False, 1, 16384, 16384, 1, 8, 8, 64, 64),
        # the norm of the scalar block (128 of 1,152 values) of 100,000 node rows
        _norm("norm_scalars_f32_step", "f32", True, 100000, 128, 1152, False, 0.0),
        # latency of a small norm
        _norm("norm_32x64_f32_fwd", "f32", False, 32, 64, 64, False, 0.0),
        # residual, dropout and norm together over whole rows of 1,024 values
        _norm("norm_fused_bf16_step", "bf16", True, 32768, 1024, 1024, True, 0.1),
        # dropout onto the residual: rows of the 1,536-atom workload, and the
        # 100,000-atom rows with the gradient
        _drop("dropout_1536_f32_fwd", "f32", False, 1536, 288, 0.1),
        _drop("dropout_100000_bf16_step", "bf16", True, 100000, 1152, 0.1),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    dtype, step = rng.choice(["f32", "bf16"]), rng.random() < 0.6
    op = rng.choice(["attn", "attn", "norm", "dropout"])
    if op == "attn":
        hkv = rng.choice([1, 2, 4, 5, 8])
        hq = min(16, hkv * rng.choice([1, 1, 2, 4])) // hkv * hkv
        d = rng.choice([8, 16, 24, 32, 40, 64, 96, 128])
        # a softmax over one key has no gradient: training draws start at 16 atoms
        least = 16 if step else 1
        hi = _log(rng, 2 * least, 8192)
        lo = max(least, int(hi * rng.uniform(0.1, 1.0)))
        # training steps do about 3.5 times the work of an evaluation, wide heads
        # more than narrow ones
        cost = (3.5 if step else 1.0) * max(1.0, d / 64) * (4 if dtype == "f32" else 1)
        room = max(1, min(1024, int(PAIRS / cost / (hi * hi * hq))))
        while hi * hi * hq * cost > PAIRS:
            hi, lo = max(2 * least, hi // 2), max(least, lo // 2)
        count = _log(rng, 1, room)
        c = _attn("", dtype, step, rng.randrange(1 << 20), lo, hi, count, hq, hkv, d,
                  rng.choice([8, 20, 32, 64]), rng.choice([0.0, 0.05, 0.5]))
    elif op == "norm":
        cols = _log(rng, 8, 4096)
        rows = _log(rng, 1, max(1, min(100000, 60000000 // cols)))
        fused = rng.random() < 0.5
        # strided rows where the elements stay within a fixed amount of memory
        stride = cols if rng.random() < 0.5 or rows * cols > 10000000 else cols + rng.randrange(0, 4 * cols)
        c = _norm("", dtype, step, rows, cols, stride, fused, rng.choice([0.05, 0.1, 0.5]) if fused else 0.0)
    else:
        cols = _log(rng, 8, 4096)
        rows = _log(rng, 1, max(1, min(100000, 115000000 // cols)))
        c = _drop("", dtype, step, rows, cols, rng.choice([0.0, 0.05, 0.1, 0.5]))
    del c["name"]
    return c


def _lengths(case):
    """Atoms of each structure: fixed by the case."""
    r = random.Random(case["sizes"])
    return [r.randint(case["lo"], case["hi"]) for _ in range(case["count"])]


# ---- what a program has in hand before the call --------------------------------
def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    dt = DT[case["dtype"]]

    def normal(*shape, dtype=dt):
        return torch.randn(*shape, device="cuda", generator=g).to(dtype)

    if case["op"] == "attn":
        n = _lengths(case)
        N, hq, hkv, d = sum(n), case["hq"], case["hkv"], case["d"]
        # queries, keys and values are views of one projected row per atom
        qkv = normal(N, (hq + 2 * hkv) * d)
        q = qkv[:, :hq * d].view(N, hq, d)
        k = qkv[:, hq * d:(hq + hkv) * d].view(N, hkv, d)
        v = qkv[:, (hq + hkv) * d:].view(N, hkv, d)
        seg = torch.tensor(np.concatenate([[0], np.cumsum(n)]), dtype=torch.int32, device="cuda")
        # atoms at a number density of 0.05 per cubic Angstrom
        box = (max(n) / 0.05) ** (1.0 / 3.0)
        pos = torch.rand(N, 3, device="cuda", generator=g) * box
        s = dict(case=case, q=q, k=k, v=v, seg=seg, longest=max(n), pos=pos, r_min=0.5, steps=4,
                 bias=0.5 * torch.randn(hq, case["buckets"], device="cuda", generator=g), mask=None)
        s["bias"] = s["bias"].to(dt)
        if case["masked"]:
            s["mask"] = (torch.rand(N, device="cuda", generator=g) >= case["masked"]).to(torch.uint8)
        if case["step"]:
            s["grad"] = normal(N, hq, d)
        return s
    rows, cols = case["rows"], case["cols"]
    s = dict(case=case, p=case["p"], seed=int(seed) * 2654435761 % (1 << 62), offset=int(seed) % 1000)
    if case["op"] == "dropout":
        s.update(x=normal(rows, cols), residual=normal(rows, cols))
        if case["step"]:
            s["grad"] = normal(rows, cols)
        return s
    # feature rows with a mean and a size of their own
    x = torch.randn(rows, case["stride"], device="cuda", generator=g)
    x = x.mul_(torch.rand(rows, 1, device="cuda", generator=g) + 0.5).add_(
        torch.randn(rows, 1, device="cuda", generator=g)).to(dt)
    s.update(x=x[:, :cols], gamma=1 + 0.1 * normal(cols, dtype=torch.float32),
             beta=0.1 * normal(cols, dtype=torch.float32), residual=None)
    if case["fused"]:
        s["residual"] = normal(rows, cols)
    if case["step"]:
        s["grad"] = normal(rows, cols)
        # the gradient that reaches the residual past the norm
        s["grad_h"] = normal(rows, cols) if case["fused"] else None
    return s


# ---- the plain forms -----------------------------------------------------------
def _mulhilo(a, b):
    """High and low 32 bits of the product of a constant and 32-bit words held in int64."""
    p = a * b                                   # wraps modulo 2^64
    return (p >> 32) & 0xFFFFFFFF, p & 0xFFFFFFFF


def _round(c, k):
    h0, l0 = _mulhilo(0xD2511F53, c[0])
    h1, l1 = _mulhilo(0xCD9E8D57, c[2])
    return (h1 ^ c[1] ^ k[0], l1, h0 ^ c[3] ^ k[1], l0), ((k[0] + 0x9E3779B9) & 0xFFFFFFFF,
                                                          (k[1] + 0xBB67AE85) & 0xFFFFFFFF)


def _factor(shape, p, seed, offset, device):
    """1 / (1 - p) where an element is kept, 0 where it is dropped."""
    n = shape[0] * shape[1]
    b = torch.arange((n + 3) // 4, device=device)
    c = (b & 0xFFFFFFFF, b >> 32, torch.full_like(b, offset & 0xFFFFFFFF), torch.full_like(b, offset >> 32))
    k = (seed & 0xFFFFFFFF, seed >> 32)
    c, k = _round(*_round(*_round(*_round(*_round(c, k)))))
    c, k = _round(*_round(*_round(*_round(*_round(c, k)))))
    w = torch.stack(c, 1).reshape(-1)[:n].reshape(shape)
    return (w >= int(p * 4294967296.0)).float() * float(np.float32(1.0 / (1.0 - p)))


def _plain_dropout(s):
    f = _factor(s["x"].shape, s["p"], s["seed"], s["offset"], s["x"].device)
    out = [(s["x"].float() * f + s["residual"].float()).to(s["x"].dtype)]
    if "grad" in s:
        out.append((s["grad"].float() * f).to(s["x"].dtype))
    return out


def _plain_norm(s):
    x, dt = s["x"].float(), s["x"].dtype
    f = None
    if s["residual"] is not None:
        f = _factor(x.shape, s["p"], s["seed"], s["offset"], x.device)
        h = (x * f + s["residual"].float()).to(dt)      # the new residual stream, an output of its own
        x = h.float()
    mean = x.mean(1)
    c = x - mean[:, None]
    rstd = 1.0 / torch.sqrt((c * c).mean(1) + EPS)
    xhat = c * rstd[:, None]
    out = [(xhat * s["gamma"] + s["beta"]).to(dt), mean, rstd]
    if f is not None:
        out.append(h)
    if "grad" in s:
        gy = s["grad"].float()
        t = gy * s["gamma"]
        gh = rstd[:, None] * (t - t.mean(1, keepdim=True) - xhat * (t * xhat).mean(1, keepdim=True))
        if f is not None:
            gh = gh + s["grad_h"].float()
            out.append((gh * f).to(dt))
        out += [gh.to(dt), (gy * xhat).sum(0), gy.sum(0)]
    return out


def _plain_attn(s):
    case, dt = s["case"], s["q"].dtype
    seg, L, hq, hkv = s["seg"].long(), s["longest"], case["hq"], case["hkv"]
    ar = torch.arange(L, device="cuda")
    real = ar < (seg[1:] - seg[:-1])[:, None]                         # [B, L]
    at = (seg[:-1, None] + ar).clamp(max=s["q"].shape[0] - 1)
    back = real.reshape(-1).nonzero()[:, 0]

    def rows(t):                                                      # [B, H, L, D] in 32 bits
        return t.float()[at].transpose(1, 2)

    def packed(t):                                                    # back to [N, H, D]
        return t.transpose(1, 2).reshape(-1, t.shape[1], t.shape[3])[back].to(dt)

    q, k, v = rows(s["q"]), rows(s["k"]), rows(s["v"])
    rep = hq // hkv
    kq, vq = k.repeat_interleave(rep, 1), v.repeat_interleave(rep, 1)
    p = s["pos"][at]
    d = p[:, :, None, :] - p[:, None, :, :]
    d2 = d[..., 0] * d[..., 0] + d[..., 1] * d[..., 1] + d[..., 2] * d[..., 2]
    shift = 23 - int(math.log2(s["steps"]))
    base = int(np.float32(s["r_min"] * s["r_min"]).view(np.int32)) >> shift
    bucket = ((d2.view(torch.int32) >> shift) - base).clamp(0, case["buckets"] - 1).long()
    del d, d2
    keys = real if s["mask"] is None else real & (s["mask"].bool()[at])
    scale = 1.0 / math.sqrt(case["d"])
    S = torch.matmul(q, kq.transpose(2, 3)) * scale + s["bias"].float()[:, bucket].transpose(0, 1)
    S = S.masked_fill(~keys[:, None, None, :], -math.inf)
    m = S.amax(3, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    P = torch.exp(S - m)
    del S
    l = P.sum(3, keepdim=True)
    P = P / torch.where(l == 0, torch.ones_like(l), l)
    lse = (m + torch.log(l))[..., 0].transpose(1, 2).reshape(-1, hq)[back].t().contiguous()
    out = [packed(torch.matmul(P, vq)), lse]
    if "grad" in s:
        g = rows(s["grad"]) * real[:, None, :, None]
        dv = torch.matmul(P.transpose(2, 3), g)
        dP = torch.matmul(g, vq.transpose(2, 3))
        dS = P * (dP - (P * dP).sum(3, keepdim=True))
        del P, dP
        dq = torch.matmul(dS, kq) * scale
        dk = torch.matmul(dS.transpose(2, 3), q) * scale
        B = q.shape[0]
        db = torch.zeros(B, hq, L, case["buckets"], device="cuda")
        db.scatter_add_(3, bucket[:, None].expand(B, hq, L, L), dS)
        D = case["d"]
        out += [packed(dq), packed(dk.reshape(B, hkv, rep, L, D).sum(2)),
                packed(dv.reshape(B, hkv, rep, L, D).sum(2)), db.sum((0, 2)).to(dt)]
    return out


# ---- one pass ------------------------------------------------------------------
def run(s):
    op = s["case"]["op"]
    if not own:
        return {"attn": _plain_attn, "norm": _plain_norm, "dropout": _plain_dropout}[op](s)
    import tensor_product_convolution_amd as tpc
    if op == "attn":
        kw = dict(pos=s["pos"], bias=s["bias"], r_min=s["r_min"], steps=s["steps"], key_mask=s["mask"])
        out, lse = tpc.attn_forward(s["q"], s["k"], s["v"], s["seg"], **kw)
        if "grad" not in s:
            return [out, lse]
        return [out, lse, *tpc.attn_backward(s["q"], s["k"], s["v"], s["seg"], out, lse, s["grad"], **kw)]
    drop = tpc.Dropout(s["p"], s["seed"], s["offset"])
    if op == "dropout":
        out = [tpc.dropout_forward(s["x"], drop, residual=s["residual"])]
        if "grad" in s:
            out.append(tpc.dropout_backward(s["grad"], drop))
        return out
    if s["residual"] is None:
        y, mean, rstd = tpc.layer_norm_forward(s["x"], s["gamma"], s["beta"], eps=EPS)
        if "grad" not in s:
            return [y, mean, rstd]
        return [y, mean, rstd, *tpc.layer_norm_backward(s["grad"], s["x"], s["gamma"], mean, rstd)]
    y, mean, rstd, h = tpc.layer_norm_residual_forward(s["x"], s["residual"], s["gamma"], s["beta"], drop, eps=EPS)
    if "grad" not in s:
        return [y, mean, rstd, h]
    return [y, mean, rstd, h, *tpc.layer_norm_residual_backward(s["grad"], h, s["gamma"], mean, rstd, drop,
                                                                grad_h=s["grad_h"])]


# ---- the work that the definitions ask for ---------------------------------------
def work(case):
    size = 4 if case["dtype"] == "f32" else 2
    if case["op"] == "attn":
        n = _lengths(case)
        N, pairs, hq, hkv, d = sum(n), sum(v * v for v in n), case["hq"], case["hkv"], case["d"]
        rows = N * d * size
        nbytes = rows * (2 * hq + 2 * hkv) + 4 * N * hq + 12 * N + 4 * len(n)
        flops = 4.0 * d * hq * pairs
        if case["step"]:                         # reads the gradient, writes three
            nbytes += rows * (2 * hq + 2 * hkv)
            flops += 10.0 * d * hq * pairs
        return {"bytes": nbytes, "flops": flops}
    e = case["rows"] * case["cols"]
    if case["op"] == "dropout":
        return {"bytes": e * size * (5 if case["step"] else 3), "flops": 2.0 * e * (1 + case["step"])}
    streams = (4 if case["fused"] else 2) + ((4 if case["fused"] else 2) if case["step"] else 0)
    return {"bytes": e * size * streams + 8 * case["rows"] + 8 * case["cols"], "flops": e * (8.0 + 14.0 * case["step"])}


# ---- the definitions in 64 bits ----------------------------------------------------
def _exact_keep(n, p, seed, offset):
    """The kept elements, by the generator's definition in unsigned words."""
    m32 = np.uint64(0xFFFFFFFF)
    blk = np.arange(-(-n // 4), dtype=np.uint64)
    c = [blk & m32, blk >> np.uint64(32), np.full_like(blk, offset & 0xFFFFFFFF), np.full_like(blk, offset >> 32)]
    k0, k1 = seed & 0xFFFFFFFF, seed >> 32
    for _ in range(10):
        a, b = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        c = [(b >> np.uint64(32)) ^ c[1] ^ np.uint64(k0), b & m32, (a >> np.uint64(32)) ^ c[3] ^ np.uint64(k1), a & m32]
        k0, k1 = (k0 + 0x9E3779B9) % 2 ** 32, (k1 + 0xBB67AE85) % 2 ** 32
    w = np.empty((blk.size, 4), dtype=np.uint64)
    for i in range(4):
        w[:, i] = c[i]
    return torch.from_numpy(w.reshape(-1)[:n] >= np.uint64(math.floor(p * 2.0 ** 32))).cuda()


def exact(case, seed):
    s = prepare(case, seed)
    f64 = torch.float64
    if case["op"] == "attn":
        return _exact_attn(case, s)
    rows, cols = case["rows"], case["cols"]
    x = s["x"].to(f64)
    if case["op"] == "dropout":
        keep = _exact_keep(rows * cols, s["p"], s["seed"], s["offset"]).view(rows, cols) / (1.0 - s["p"])
        res = [x * keep + s["residual"]]
        return res + [s["grad"].to(f64) * keep] if case["step"] else res
    res, keep = [], None
    if case["fused"]:
        keep = _exact_keep(rows * cols, s["p"], s["seed"], s["offset"]).view(rows, cols) / (1.0 - s["p"])
        h = x * keep + s["residual"]
        x = h.to(s["x"].dtype).to(f64)           # the norm is that of the stored row
        res = [h]
    var, mean = torch.var_mean(x, dim=1, correction=0)
    rstd = (var + EPS).rsqrt()
    z = (x - mean.unsqueeze(1)) * rstd.unsqueeze(1)
    res = [z * s["gamma"].to(f64) + s["beta"].to(f64), mean, rstd] + res
    if case["step"]:
        gy = s["grad"].to(f64)
        gz = gy * s["gamma"].to(f64)
        proj = (gz.sum(1, keepdim=True) + z * (gz * z).sum(1, keepdim=True)) / cols
        gx = (gz - proj) * rstd.unsqueeze(1)
        if case["fused"]:
            gx = gx + s["grad_h"].to(f64)
            res.append(gx * keep)
        res += [gx, (gy * z).sum(0), gy.sum(0)]
    return res


def _exact_attn(case, s):
    f64, step = torch.float64, case["step"]
    n, hq, hkv, D, nb = _lengths(case), case["hq"], case["hkv"], case["d"], case["buckets"]
    if len(n) * hq > 10000:
        return None
    N, scale = sum(n), case["d"] ** -0.5
    shift = {1: 23, 2: 22, 4: 21, 8: 20}[s["steps"]]
    first = int(np.array([s["r_min"] ** 2], dtype=np.float32).view(np.int32)[0]) >> shift
    z = lambda *a: torch.zeros(*a, dtype=f64, device="cuda")
    out, lse = z(N, hq, D), z(hq, N)
    dq, dk, dv, db = z(N, hq, D), z(N, hkv, D), z(N, hkv, D), z(hq, nb)
    lo = 0
    for m in n:
        sl = slice(lo, lo + m)
        lo += m
        x, y, w = s["pos"][sl].unbind(1)         # the bucket is defined on float32 distances
        ex, ey, ez = (t[:, None] - t[None] for t in (x, y, w))
        code = ((ex * ex + ey * ey) + ez * ez).view(torch.int32)
        b = torch.clamp((code >> shift) - first, min=0, max=nb - 1)
        live = torch.ones(m, dtype=torch.bool, device="cuda") if s["mask"] is None else s["mask"][sl] != 0
        for h in range(hq):
            c = h // (hq // hkv)
            Q, K, V = s["q"][sl, h].to(f64), s["k"][sl, c].to(f64)[live], s["v"][sl, c].to(f64)[live]
            if K.shape[0] == 0:
                lse[h, sl] = -math.inf
                continue
            bl = b[:, live].long()
            S = Q @ K.T * scale + s["bias"][h].to(f64)[bl]
            t = torch.logsumexp(S, 1)
            P = torch.exp(S - t[:, None])
            del S
            lse[h, sl], O = t, P @ V
            out[sl, h] = O
            if step:
                G = s["grad"][sl, h].to(f64)
                dS = P * (G @ V.T - (G * O).sum(1, keepdim=True))
                dq[sl, h] = dS @ K * scale
                dk[sl, c] += z(m, D).index_copy_(0, live.nonzero()[:, 0], dS.T @ Q * scale)
                dv[sl, c] += z(m, D).index_copy_(0, live.nonzero()[:, 0], P.T @ G)
                db[h] += torch.bincount(bl.reshape(-1), weights=dS.reshape(-1), minlength=nb)
    return [out, lse, dq, dk, dv, db] if step else [out, lse]
