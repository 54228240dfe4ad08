"""What is measured of the operators before, behind and around the attention block:
the norm and position rotation of queries and keys, products grouped by chemical
element or by expert with the router in front, and the AdamW step that trains them.

Each case runs one operator, or the run of them that a program makes, as a training or
evaluation program does.  With ``own`` false the operators are computed in their plain
form (elementary torch operations in 32 bits, each operator's outputs rounded once);
with ``own`` true by the library's kernels.  ``exact`` gives the same values from the
definitions in 64 bits.  Sizes follow the repository's workloads: 32, 1,536, 4,096,
32,768 and 100,000 atoms, 8 to 128 channels per degree, node rows of up to 1,152 values.
"""
import math

import numpy as np
import torch

own = False

DT = {"f32": torch.float32, "bf16": torch.bfloat16}
EPS = 1e-6
HEAD_VALUES = 100000 * 20 * 64 * 5         # values that the largest listed case of its kind moves
SPECIES_FLOPS = 100000 * 128 * 128 * 6     # products of the largest listed case of its kind, times the type's cost
EXPERT_FLOPS = 65536 * 1024 * 4096 * 2
EXPERT_WEIGHTS = 64 * 1024 * 4096
ADAM_VALUES = 64000000
BLOCK = 256                                # state values that share a scale; tensors start at multiples of it
BETA1, BETA2, ADAM_EPS = 0.9, 0.999, 1e-8


# ---- the cases ---------------------------------------------------------------
def _heads(name, dtype, step, rows, hq, hk, d, rot, axes, reach, interleaved, norm):
    return dict(name=name, op="heads", dtype=dtype, step=step, rows=rows, hq=hq, hk=hk, d=d, rot=rot, axes=axes,
                reach=reach, interleaved=interleaved, norm=norm)


def _species(name, dtype, step, rows, cin, cout, kinds, tilt):
    return dict(name=name, op="species", dtype=dtype, step=step, rows=rows, cin=cin, cout=cout, kinds=kinds, tilt=tilt)


def _experts(name, dtype, step, rows, width, hidden, experts, k, tilt):
    return dict(name=name, op="experts", dtype=dtype, step=step, rows=rows, width=width, hidden=hidden, experts=experts,
                k=k, tilt=tilt)


def _adamw(name, bits, grads, count, total, clip, low):
    return dict(name=name, op="adamw", bits=bits, grads=grads, count=count, total=total, clip=clip, low=low)


def listed():
    return [
        # one small structure in an MD loop: the call's latency
        _heads("heads_32_f32_fwd", "f32", False, 32, 4, 4, 16, 16, 3, 9.0, False, True),
        # the 1,536-atom structure, a training step with the gradient of the positions
        _heads("heads_1536_bf16_step", "bf16", True, 1536, 8, 8, 32, 32, 3, 32.0, False, True),
        # the largest: 100,000 atoms, shared key heads, adjacent pairs
        _heads("heads_100000_bf16_step", "bf16", True, 100000, 16, 4, 64, 48, 3, 126.0, True, True),
        # rotation alone of part of odd heads, by far integer positions along a chain
        _heads("heads_far_f32_fwd", "f32", False, 8191, 5, 5, 40, 24, 1, 2.0e8, False, False),
        # a linear layer with weights by chemical element: a training step of the 1,536-atom structure
        _species("species_1536_f32_step", "f32", True, 1536, 128, 128, 4, 1.0),
        # the same over 100,000 atoms of an inorganic mix, most elements rare
        _species("species_100000_f32_step", "f32", True, 100000, 128, 128, 89, 2.0),
        # odd widths, one evaluation
        _species("species_1001_bf16_fwd", "bf16", False, 1001, 136, 75, 7, 1.0),
        # experts for a molecule of 16 atoms in an MD loop: the weights' bytes
        _experts("experts_16_bf16_fwd", "bf16", False, 16, 1024, 4096, 32, 2, 0.5),
        # a training step of the 4,096-atom structure
        _experts("experts_4096_bf16_step", "bf16", True, 4096, 512, 2048, 8, 2, 0.5),
        # the largest: 32,768 atoms, 64 experts, evaluated
        _experts("experts_32768_bf16_fwd", "bf16", False, 32768, 1024, 4096, 64, 2, 0.5),
        # the optimiser of a small potential: 40 tensors, the call's latency
        _adamw("adamw_40_tensors_f32", 32, "f32", 40, 300000, 1.0, False),
        # of a large one, 8-bit states, bfloat16 gradients and working copies
        _adamw("adamw_64m_8bit", 8, "bf16", 300, 64000000, 1.0, True),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    dtype, step = rng.choice(["f32", "bf16"]), rng.random() < 0.6
    op = rng.choice(["heads", "species", "experts", "experts", "adamw"])
    if op == "heads":
        hk = rng.choice([1, 2, 4, 5, 8])
        hq = min(16, hk * rng.choice([1, 1, 2, 4])) // hk * hk
        d = rng.choice([8, 16, 24, 32, 40, 64, 96, 128])
        rot = 2 * rng.randint(1, d // 2) if rng.random() < 0.4 else d
        room = HEAD_VALUES // ((hq + hk) * d * (5 if step else 2) * (2 if dtype == "f32" else 1))
        axes = rng.choice([1, 3, 3])
        c = _heads("", dtype, step, _log(rng, 1, max(1, min(100000, room))), hq, hk, d, rot, axes,
                   2.0 ** rng.uniform(3, 28) if axes == 1 else rng.uniform(5, 200), rng.random() < 0.5, rng.random() < 0.8)
    elif op == "species":
        cin, cout, kinds = _log(rng, 8, 512), _log(rng, 8, 512), rng.randint(1, 118)
        room = SPECIES_FLOPS // (cin * cout * (6 if step else 2))
        c = _species("", dtype, step, _log(rng, 1, max(1, min(100000, room))), cin, cout, kinds, rng.choice([0.0, 1.0, 2.0]))
    elif op == "experts":
        width, hidden, experts = _log(rng, 32, 1024), _log(rng, 32, 4096), _log(rng, 2, 128)
        while experts * width * hidden * (2 if dtype == "f32" else 1) * (3 if step else 1) > EXPERT_WEIGHTS:
            experts, hidden = max(2, experts * 2 // 3), max(32, hidden * 2 // 3)
        k = min(experts, rng.choice([1, 2, 2, 4, 8]))
        room = EXPERT_FLOPS // (2 * width * hidden * k * (3 if step else 1) * (4 if dtype == "f32" else 1))
        tilt = rng.choice([0.0, 0.5, 2.0])
        if tilt > 1.0:                     # one expert may get every row, and the plain form pads all to it
            room = min(room, 1500000000 // (experts * max(width, hidden)))
        c = _experts("", dtype, step, _log(rng, 1, max(1, min(32768, room))), width, hidden, experts, k, tilt)
    else:
        bits, count = rng.choice([8, 32]), _log(rng, 1, 400)
        c = _adamw("", bits, dtype, count, _log(rng, max(1000, 4 * count), ADAM_VALUES // (4 if bits == 32 else 1)),
                   rng.choice([0.0, 1.0]), rng.random() < 0.5)
    del c["name"]
    return c


def _sizes(case):
    """Elements of each tensor: a few large matrices, many small vectors; fixed by the case."""
    r = np.random.RandomState(case["count"])
    share = r.pareto(0.8, case["count"]) + 0.01
    return np.maximum(1, share / share.sum() * case["total"]).astype(np.int64).tolist()


# ---- what a program has in hand before the call --------------------------------
def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))

    def normal(*shape, dtype=torch.float32, size=1.0):
        return (torch.randn(*shape, device="cuda", generator=g) * size).to(dtype)

    def uniform(*shape):
        return torch.rand(*shape, device="cuda", generator=g)

    s = dict(case=case)
    if case["op"] == "adamw":
        return _prepare_adamw(s, seed, normal, uniform)
    dt, rows = DT[case["dtype"]], case["rows"]
    if case["op"] == "heads":
        hq, hk, d, axes, pairs = case["hq"], case["hk"], case["d"], case["axes"], case["rot"] // 2
        # queries and keys are views of one projected row per atom, with the values behind them
        row = normal(rows, (hq + 2 * hk) * d, dtype=dt)
        s.update(q=row[:, :hq * d].view(rows, hq, d), k=row[:, hq * d:(hq + hk) * d].view(rows, hk, d))
        if axes == 1:                      # places along a chain, frequencies that fall geometrically
            s["pos"] = (uniform(rows, 1).double() * case["reach"]).to(torch.int32)
            s["freq"] = (1e4 ** (-torch.arange(pairs, device="cuda", dtype=torch.float64) / pairs)).view(pairs, 1)
        else:                              # atoms in a box, wave vectors up to 3 per Angstrom
            s["pos"] = uniform(rows, axes) * case["reach"]
            s["freq"] = normal(pairs, axes).double()
        s["gq"] = s["gk"] = None
        if case["norm"]:
            s.update(gq=1 + normal(d, size=0.1), gk=1 + normal(d, size=0.1))
        if case["step"]:
            s.update(grad_q=normal(rows, hq, d, dtype=dt), grad_k=normal(rows, hk, d, dtype=dt))
    elif case["op"] == "species":
        cin, cout, kinds = case["cin"], case["cout"], case["kinds"]
        share = torch.arange(1, kinds + 1, device="cuda").double() ** -case["tilt"]
        edge = (share.cumsum(0) / share.sum()).float()
        s["kind"] = torch.searchsorted(edge, uniform(rows)).clamp(max=kinds - 1).to(torch.int32)
        s.update(x=normal(rows, cin, dtype=dt), w=normal(kinds, cin, cout, dtype=dt, size=cin ** -0.5),
                 b=normal(kinds, cout, dtype=dt, size=0.1))
        if case["step"]:
            s["grad"] = normal(rows, cout, dtype=dt)
    else:
        width, hidden, n = case["width"], case["hidden"], case["experts"]
        s.update(x=normal(rows, width, dtype=dt), logits=(normal(rows, n) + case["tilt"] * normal(n)).to(dt),
                 w1=normal(n, width, hidden, dtype=dt, size=width ** -0.5), b1=normal(n, hidden, dtype=dt, size=0.1),
                 w2=normal(n, hidden, width, dtype=dt, size=hidden ** -0.5))
        if case["step"]:
            s["grad"] = normal(rows, width, dtype=dt)
    return s


def _prepare_adamw(s, seed, normal, uniform):
    """Parameters in the middle of a training run, as views of one arena in which each
    tensor starts at a multiple of BLOCK; the states lie in arenas of the same layout."""
    case = s["case"]
    n = _sizes(case)
    start = np.concatenate([[0], np.cumsum([-(-v // BLOCK) * BLOCK for v in n])]).tolist()
    total = start[-1]
    sizes = torch.tensor(n, device="cuda")
    first = torch.tensor(start, device="cuda")
    owner = torch.repeat_interleave(torch.arange(len(n), device="cuda"), first[1:] - first[:-1], output_size=total)
    live = torch.arange(total, device="cuda") - first[owner] < sizes[owner]
    scale = torch.exp(normal(len(n)))[owner]                  # gradients of a size of their own in each tensor
    decay = [0.0 if i % 3 else 0.01 for i in range(len(n))]   # weights decay, biases and norms do not
    s.update(p=normal(total, size=0.1) * live, decay=torch.tensor(decay, device="cuda")[owner],
             t=100, lr=1e-3, seed=int(seed) * 2654435761 % (1 << 62))
    s["g"] = (normal(total, size=1e-3) * scale * live).to(DT[case["grads"]])
    m, v = normal(total, size=3e-4) * scale * live, (1e-6 * scale * scale * live) * (0.2 + uniform(total))
    if case["bits"] == 8:                                     # codes and scales as a step left them
        for name, value, top in (("m", m, 127), ("v", v, 255)):
            b = value.view(-1, BLOCK).double()
            unit = (b.abs().amax(1) / 1.875).float()
            code = _encode(b / torch.where(unit == 0, torch.ones_like(unit), unit).double()[:, None], top, 0.5)
            s.update({name: code.view(-1), name + "_unit": unit})
    else:
        s.update(m=m, v=v)
    del m, v, scale, owner
    s["low"] = s["p"].to(torch.bfloat16) if case["low"] else None
    views = lambda a: None if a is None else [a[i:i + k] for i, k in zip(start, n)]
    s["grads"] = views(s["g"])
    if own:
        import tensor_product_convolution_amd as tpc
        s["opt"] = tpc.AdamW(views(s["p"]), lr=s["lr"], betas=(BETA1, BETA2), eps=ADAM_EPS, weight_decay=decay,
                             max_norm=case["clip"] or None, bits=case["bits"], copies=views(s["low"]), seed=s["seed"])
        s["opt"].load(s["t"], *[s[k] for k in ("m", "v", "m_unit", "v_unit") if k in s])
    return s


# ---- the plain forms -----------------------------------------------------------
def _rotation(s):
    """cos and sin of every row and pair; far positions lose their angle in 32 bits."""
    angle = s["pos"].double() @ s["freq"].t()
    return torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]


def _split(x, case):
    """First and second values of the pairs."""
    p = case["rot"] // 2
    return (x[..., 0:2 * p:2], x[..., 1:2 * p:2]) if case["interleaved"] else (x[..., :p], x[..., p:2 * p])


def _join(a, b, x, case):
    r = torch.stack([a, b], -1).flatten(-2) if case["interleaved"] else torch.cat([a, b], -1)
    return torch.cat([r, x[..., case["rot"]:]], -1)


def _plain_heads(s):
    case, dt = s["case"], s["q"].dtype
    cos, sin = _rotation(s)
    out, grads, weights, turn = [], [], [], 0.0
    for name in ("q", "k"):
        x, w = s[name].float(), s["g" + name]
        r = torch.ones_like(x[..., :1]) if w is None else 1.0 / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS)
        z = x * r
        y = z if w is None else z * w
        a, b = _split(y, case)
        out.append(_join(a * cos - b * sin, a * sin + b * cos, y, case).to(dt))
        if not case["step"]:
            continue
        g = s["grad_" + name].float()
        ga, gb = _split(g, case)
        ha, hb = ga * cos + gb * sin, gb * cos - ga * sin
        turn = turn + (hb * a - ha * b).sum(1)
        g = _join(ha, hb, g, case)
        if w is not None:
            weights.append((g * z).sum((0, 1)))
            t = g * w
            g = r * (t - z * (t * z).mean(-1, keepdim=True))
        grads.append(g.to(dt))
    if case["step"] and case["axes"] > 1:
        weights.append((turn.double() @ s["freq"]).float())
    return out + grads + weights


def _plain_groups(index, n):
    """Rows in groups, padded to the longest: (slots [n, longest], which are real)."""
    flat = index.reshape(-1).long()
    order = torch.sort(flat, stable=True)[1]
    count = torch.bincount(flat, minlength=n)
    at = torch.arange(int(count.max()), device="cuda")
    real = at < count[:, None]
    return order[(count.cumsum(0) - count)[:, None].add(at).clamp(max=flat.numel() - 1)], real


def _spread(values, slots, real, rows):
    """Padded rows back to the place of their slots."""
    out = torch.zeros(rows, values.shape[2], device="cuda")
    out[slots[real]] = values[real]
    return out


def _plain_species(s):
    dt, rows = s["x"].dtype, s["case"]["rows"]
    slots, real = _plain_groups(s["kind"], s["case"]["kinds"])
    x = s["x"].float()[slots]
    w = s["w"].float()
    out = [_spread(torch.matmul(x, w) + s["b"].float()[:, None], slots, real, rows).to(dt)]
    if "grad" in s:
        g = s["grad"].float()[slots] * real[..., None]
        out += [_spread(torch.matmul(g, w.transpose(1, 2).contiguous()), slots, real, rows).to(dt),
                torch.matmul(x.transpose(1, 2).contiguous(), g).to(dt), g.sum(1).to(dt)]
    return out


def _plain_experts(s):
    case, dt = s["case"], s["x"].dtype
    rows, k, n = case["rows"], case["k"], case["experts"]
    logits = s["logits"].float()
    index = torch.sort(logits, dim=1, descending=True, stable=True)[1][:, :k]
    top = logits.gather(1, index)
    e = torch.exp(top - top.amax(1, keepdim=True))
    weight = e / e.sum(1, keepdim=True)
    slots, real = _plain_groups(index, n)
    x, w1, w2 = s["x"].float()[slots // k], s["w1"].float(), s["w2"].float()
    z = (torch.matmul(x, w1) + s["b1"].float()[:, None]).to(dt).float()   # stored: the backward reads it
    sig = 1.0 / (1.0 + torch.exp(-z))
    h = (z * sig).to(dt).float()
    y = _spread(torch.matmul(h, w2), slots, real, rows * k).to(dt).float().view(rows, k, -1)
    out = [weight, index.to(torch.int32), (weight[..., None] * y).sum(1).to(dt)]
    if "grad" in s:
        go = s["grad"].float()
        gweight = (go[:, None] * y).sum(2)
        gy = (weight[..., None] * go[:, None]).to(dt).float().view(rows * k, -1)[slots] * real[..., None]
        del y
        gw2 = torch.matmul(h.transpose(1, 2).contiguous(), gy)
        gz = (torch.matmul(gy, w2.transpose(1, 2).contiguous()) * (sig * (1.0 + z * (1.0 - sig)))).to(dt).float()
        del sig, z, h
        gx = _spread(torch.matmul(gz, w1.transpose(1, 2).contiguous()), slots, real, rows * k).view(rows, k, -1).sum(1)
        gw1 = torch.matmul(x.transpose(1, 2).contiguous(), gz)
        # differences first: where one weight is nearly 1, gweight less its mean cancels
        gl = weight * ((gweight[:, :, None] - gweight[:, None, :]) * weight[:, None, :]).sum(2)
        out += [gx.to(dt), gw1.to(dt), gz.sum(1).to(dt), gw2.to(dt), torch.zeros_like(logits).scatter_(1, index, gl).to(dt)]
    return out


def _mulhilo(a, b):
    """High and low 32 bits of the product of a constant and 32-bit words held in int64."""
    p = a * b                                   # wraps modulo 2^64
    return (p >> 32) & 0xFFFFFFFF, p & 0xFFFFFFFF


def _round(c, k):
    h0, l0 = _mulhilo(0xD2511F53, c[0])
    h1, l1 = _mulhilo(0xCD9E8D57, c[2])
    return (h1 ^ c[1] ^ k[0], l1, h0 ^ c[3] ^ k[1], l0), ((k[0] + 0x9E3779B9) & 0xFFFFFFFF,
                                                          (k[1] + 0xBB67AE85) & 0xFFFFFFFF)


def _words(n, seed, offset):
    """Word e % 4 of the generator's block e // 4, for e < n (a multiple of 4)."""
    b = torch.arange(n // 4, device="cuda")
    c = (b & 0xFFFFFFFF, b >> 32, torch.full_like(b, offset & 0xFFFFFFFF), torch.full_like(b, offset >> 32))
    k = (seed & 0xFFFFFFFF, seed >> 32)
    c, k = _round(*_round(*_round(*_round(*_round(c, k)))))
    c, k = _round(*_round(*_round(*_round(*_round(c, k)))))
    return torch.stack(c, 1).reshape(-1)


# An 8-bit state holds unit times a small float: three bits of significand, eight codes an
# octave, the lowest octave linear down to zero, the highest code 1.875.  127 codes and a
# sign for the first moment, 255 for the second.
def _encode(a, top, u):
    """Code of a (float64): the place of |a| among the codes plus u in [0, 1), rounded down."""
    size = a.abs()
    low = 2.0 ** (1 - (top >> 3))                             # least value of full precision
    place = (size.view(torch.int64) - int(np.float64(low).view(np.int64))).double() * 2.0 ** -49 + 8.0
    place = torch.where(size < low, size * (8.0 / low), place)
    code = (place + u).floor().clamp(max=top).long()
    if top == 255:                                            # a second moment that is not zero stays so
        code = torch.where(size > 0, code.clamp(min=1), code)
    return (code + torch.where((a < 0) & (code > 0), 128, 0)).to(torch.uint8)


def _decode(code, unit, top):
    """Values of codes, float64."""
    c = code.long() if top == 255 else code.long() & 127
    low = 2.0 ** (1 - (top >> 3))
    v = torch.where(c < 8, c.double() * (low / 8.0), torch.exp2(((c >> 3) - (top >> 3)).double()) * (1.0 + (c & 7).double() / 8.0))
    if top == 127:
        v = torch.where(code >= 128, -v, v)
    return (v.view(-1, BLOCK) * unit.double()[:, None]).view(-1)


def _plain_adamw(s):
    case = s["case"]
    small = case["bits"] == 8
    s["t"] += 1
    t = s["t"]
    g, out = s["g"].float(), []
    if case["clip"]:
        norm = torch.sqrt((s["g"].double() ** 2).sum())
        out.append(norm.float())
        factor = torch.clamp(case["clip"] / norm, max=1.0)    # 0 / 0 does not arise: gradients are drawn
    else:
        factor = torch.ones((), dtype=torch.float64, device="cuda")
    # an 8-bit state's rounding asks which side of a border a value lies on: in 64 bits
    g = g.double() * factor if small else g * factor.float()
    m = _decode(s["m"], s["m_unit"], 127) if small else s["m"]
    v = _decode(s["v"], s["v_unit"], 255) if small else s["v"]
    m = BETA1 * m + (1.0 - BETA1) * g
    v = BETA2 * v + (1.0 - BETA2) * (g * g)
    del g
    step = (m / (1.0 - BETA1 ** t)) / (torch.sqrt(v / (1.0 - BETA2 ** t)) + ADAM_EPS)
    p = s["p"].mul_(1.0 - s["lr"] * s["decay"]).sub_((s["lr"] * step).float())
    del step
    if not small:
        s["m"], s["v"] = m, v
    else:
        w = _words(m.numel(), s["seed"], t)
        for name, x, top, u in (("m", m, 127, w & 0xFFFF), ("v", v, 255, w >> 16)):
            x = x.view(-1, BLOCK)
            unit = (x.abs().amax(1) / 1.875).float()
            a = x / torch.where(unit == 0, torch.ones_like(unit), unit).double()[:, None]
            code = _encode(a, top, u.view(-1, BLOCK).double() / 65536.0).view(-1)
            s[name], s[name + "_unit"] = code, unit
            out.append(_decode(code, unit, top).float())
    out += [p] if small else [p, m, v]
    if s["low"] is not None:
        out.append(s["low"].copy_(p))
    return out


# ---- one pass ------------------------------------------------------------------
def run(s):
    case = s["case"]
    op = case["op"]
    if not own:
        return {"heads": _plain_heads, "species": _plain_species, "experts": _plain_experts, "adamw": _plain_adamw}[op](s)
    import tensor_product_convolution_amd as tpc
    if op == "heads":
        kw = dict(gamma_q=s["gq"], gamma_k=s["gk"], pos=s["pos"], freq=s["freq"], interleaved=case["interleaved"], eps=EPS)
        out = list(tpc.head_norm_rotate_forward(s["q"], s["k"], **kw))
        if case["step"]:
            back = tpc.head_norm_rotate_backward(s["grad_q"], s["grad_k"], s["q"], s["k"], want_pos=case["axes"] > 1, **kw)
            out += [t for t in back if t is not None]
        return out
    if op == "species":
        groups = tpc.group_rows(s["kind"], case["kinds"])
        out = [tpc.grouped_linear_forward(s["x"], s["w"], groups, bias=s["b"])]
        if case["step"]:
            out += tpc.grouped_linear_backward(s["grad"], s["x"], s["w"], groups, want_bias=True)
        return out
    if op == "experts":
        weight, index = tpc.route_forward(s["logits"], case["k"])
        groups = tpc.group_rows(index, case["experts"])
        h = tpc.grouped_linear_forward(s["x"], s["w1"], groups, bias=s["b1"], act="silu", y_rows="grouped", want_pre=case["step"])
        h, z = h if case["step"] else (h, None)
        y = tpc.grouped_linear_forward(h, s["w2"], groups, x_rows="grouped")
        out = [weight, index, tpc.combine_forward(y, weight)]
        if case["step"]:
            gy, gweight = tpc.combine_backward(s["grad"], y, weight)
            gz, gw2, _ = tpc.grouped_linear_backward(gy, h, s["w2"], groups, x_rows="grouped", pre=z)
            gx, gw1, gb1 = tpc.grouped_linear_backward(gz, s["x"], s["w1"], groups, y_rows="grouped", want_bias=True)
            out += [gx, gw1, gb1, gw2, tpc.route_backward(gweight, s["logits"], weight, index)]
        return out
    opt = s["opt"]
    norm = opt.step(s["grads"])
    m, v = opt.moments()                                      # 8-bit states as the values they stand for
    out = [] if norm is None else [norm]
    out += [m, v, s["p"]] if case["bits"] == 8 else [s["p"], m, v]
    return out if s["low"] is None else out + [s["low"]]


# ---- the work that the definitions ask for ---------------------------------------
def _used(groups, slots):
    """Groups that `slots` even draws reach, on average."""
    return groups * (1.0 - (1.0 - 1.0 / groups) ** slots)


def work(case):
    if case["op"] == "adamw":
        n = float(sum(_sizes(case)))
        state = 2.0 + 2 * 4.0 / BLOCK if case["bits"] == 8 else 8.0
        nbytes = n * (8 + 2 * state + (4 if case["grads"] == "f32" else 2) + (2 if case["low"] else 0))
        return {"bytes": nbytes, "flops": n * (16.0 + (2 if case["clip"] else 0))}
    size, rows, step = 4 if case["dtype"] == "f32" else 2, case["rows"], case["step"]
    if case["op"] == "heads":
        e = rows * (case["hq"] + case["hk"]) * case["d"]
        nbytes = e * size * (5 if step else 2) + 4 * rows * case["axes"] * (2 if step and case["axes"] > 1 else 1)
        return {"bytes": nbytes, "flops": e * (8.0 + 22.0 * step)}
    if case["op"] == "species":
        cin, cout, kinds = case["cin"], case["cout"], _used(case["kinds"], rows)
        nbytes = size * (rows * (cin + cout) * (2 if step else 1) + kinds * (cin + 1) * cout) + 4 * rows
        if step:
            nbytes += size * case["kinds"] * (cin + 1) * cout
        return {"bytes": nbytes, "flops": 2.0 * rows * cin * cout * (3 if step else 1)}
    width, hidden, n, slots = case["width"], case["hidden"], case["experts"], rows * case["k"]
    weights = 2.0 * width * hidden + hidden
    nbytes = size * (_used(n, slots) * weights + rows * (width * 2 + n)) + 8 * slots
    if step:
        nbytes += size * (n * weights + rows * (width * 2 + n))
    return {"bytes": nbytes, "flops": 4.0 * slots * width * hidden * (3 if step else 1)}


# ---- the definitions in 64 bits ----------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    return {"heads": _exact_heads, "species": _exact_species, "experts": _exact_experts, "adamw": _exact_adamw}[case["op"]](case, s)


def _exact_heads(case, s):
    f64, step, d, pairs = torch.float64, case["step"], case["d"], case["rot"] // 2
    phase = sum(s["pos"][:, a, None].to(f64) * s["freq"][None, :, a] for a in range(case["axes"]))
    turn = torch.polar(torch.ones_like(phase), phase).unsqueeze(1)                     # [rows, 1, pairs]
    i = torch.arange(pairs, device="cuda")
    at = torch.stack([2 * i, 2 * i + 1] if case["interleaved"] else [i, i + pairs])    # where a pair's values lie
    pick = lambda x: torch.complex(x[..., at[0]].contiguous(), x[..., at[1]].contiguous())

    def put(x, c):
        x = x.clone()
        x[..., at[0]], x[..., at[1]] = c.real, c.imag
        return x

    res, grads, gammas, torque = [], [], [], torch.zeros(case["rows"], pairs, dtype=f64, device="cuda")
    for x, gamma, up in ((s["q"], s["gq"], s.get("grad_q")), (s["k"], s["gk"], s.get("grad_k"))):
        x = x.to(f64)
        if gamma is None:
            unit = y = x
        else:
            length = (x.square().sum(-1, keepdim=True) / d + EPS).sqrt()
            unit = x / length
            y = unit * gamma.to(f64)
        o = pick(y) * turn
        res.append(put(y, o))
        if not step:
            continue
        up = up.to(f64)
        # the angle's gradient: the upstream gradient's part across the rotated pair
        torque += (pick(up) * o.conj()).imag.sum(1)
        gy = put(up, pick(up) * turn.conj())
        if gamma is None:
            grads.append(gy)
            continue
        gammas.append((gy * unit).flatten(0, 1).sum(0))
        gu = gy * gamma.to(f64)
        grads.append((gu - unit * ((gu * unit).sum(-1, keepdim=True) / d)) / length)
    res += grads + gammas
    if step and case["axes"] > 1:
        res.append(torch.stack([(torque * s["freq"][:, a]).sum(1) for a in range(case["axes"])], 1))
    return res


def _exact_species(case, s):
    f64, step = torch.float64, case["step"]
    y = torch.zeros(case["rows"], case["cout"], dtype=f64, device="cuda")
    gx = torch.zeros(case["rows"], case["cin"], dtype=f64, device="cuda")
    gw, gb = torch.zeros(s["w"].shape, dtype=f64, device="cuda"), torch.zeros(s["b"].shape, dtype=f64, device="cuda")
    for e in range(case["kinds"]):
        rows = (s["kind"] == e).nonzero()[:, 0]
        if rows.numel() == 0:
            continue
        x, w = s["x"][rows].to(f64), s["w"][e].to(f64)
        y[rows] = torch.addmm(s["b"][e].to(f64), x, w)
        if step:
            g = s["grad"][rows].to(f64)
            gx[rows], gw[e], gb[e] = g.mm(w.T), x.T.mm(g), g.sum(0)
    return [y, gx, gw, gb] if step else [y]


def _exact_experts(case, s):
    f64, step, rows, k, n = torch.float64, case["step"], case["rows"], case["k"], case["experts"]
    left, index, score = s["logits"].to(f64).clone(), [], []
    for _ in range(k):                                        # the highest left, the lowest index among equals
        best = left.amax(1, keepdim=True)
        at = torch.where(left == best, torch.arange(n, device="cuda"), n).amin(1, keepdim=True)
        index.append(at)
        score.append(best)
        left.scatter_(1, at, -math.inf)
    index = torch.cat(index, 1)
    weight = torch.softmax(torch.cat(score, 1), 1)
    z64 = lambda *shape: torch.zeros(*shape, dtype=f64, device="cuda")
    out, gx, gweight = z64(rows, case["width"]), z64(rows, case["width"]), z64(rows, k)
    gw1, gb1, gw2 = (z64(s[t].shape if step else 1) for t in ("w1", "b1", "w2"))
    for e in range(n):
        row, which = (index == e).nonzero(as_tuple=True)
        if row.numel() == 0:
            continue
        x, a, c, p = s["x"][row].to(f64), s["w1"][e].to(f64), s["w2"][e].to(f64), weight[row, which].unsqueeze(1)
        z = torch.addmm(s["b1"][e].to(f64), x, a)
        h = z * torch.sigmoid(z)
        y = h.mm(c)
        out.index_add_(0, row, p * y)
        if step:
            go = s["grad"][row].to(f64)
            gweight[row, which] = (go * y).sum(1)
            gy = p * go
            gw2[e] = h.T.mm(gy)
            sg = torch.sigmoid(z)
            gz = gy.mm(c.T) * (sg + h * (1 - sg))
            gw1[e], gb1[e] = x.T.mm(gz), gz.sum(0)
            gx.index_add_(0, row, gz.mm(a.T))
    res = [weight, index.to(torch.int32), out]
    if step:
        mean = (weight * gweight).sum(1, keepdim=True)
        res += [gx, gw1, gb1, gw2, z64(rows, n).scatter_(1, index, weight * (gweight - mean))]
    return res


def _exact_words(n, seed, offset):
    """The generator's words by its definition in unsigned arithmetic, on the host."""
    m32 = np.uint64(0xFFFFFFFF)
    blk = np.arange(n // 4, dtype=np.uint64)
    c = [blk & m32, blk >> np.uint64(32), np.full_like(blk, offset & 0xFFFFFFFF), np.full_like(blk, offset >> 32)]
    k0, k1 = seed & 0xFFFFFFFF, seed >> 32
    for _ in range(10):
        a, b = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        c = [(b >> np.uint64(32)) ^ c[1] ^ np.uint64(k0), b & m32, (a >> np.uint64(32)) ^ c[3] ^ np.uint64(k1), a & m32]
        k0, k1 = (k0 + 0x9E3779B9) % 2 ** 32, (k1 + 0xBB67AE85) % 2 ** 32
    w = np.empty((blk.size, 4), dtype=np.int64)
    for i in range(4):
        w[:, i] = c[i]
    return torch.from_numpy(w.reshape(-1)).cuda()


def _code_values(octaves):
    """The values of the codes, lowest first: a linear octave from 0, then eight steps each."""
    low = 2.0 ** (1 - octaves)
    v = [low * i / 8 for i in range(8)] + [low * 2.0 ** o * (1 + i / 8) for o in range(octaves) for i in range(8)]
    return torch.tensor(v, dtype=torch.float64, device="cuda")


def _exact_adamw(case, s):
    f64 = torch.float64
    g, t, res = s["g"].to(f64), s["t"] + 1, []
    if case["clip"]:
        norm = torch.linalg.vector_norm(g)
        res.append(norm)
        g = g * min(1.0, case["clip"] / float(norm))
    small = case["bits"] == 8
    if small:
        tables = _code_values(15), _code_values(31)
        held = []
        for name, table in zip("mv", tables):
            code = s[name].long()
            value = table[code & (table.numel() - 1)] * (1 - 2 * (code >= table.numel()).to(f64))
            held.append(value * s[name + "_unit"].to(f64).repeat_interleave(BLOCK))
    else:
        held = [s["m"].to(f64), s["v"].to(f64)]
    m, v = torch.lerp(g, held[0], BETA1), torch.lerp(g * g, held[1], BETA2)
    p = s["p"].to(f64) * (1 - s["lr"] * s["decay"].to(f64))
    p = p - s["lr"] * (m / (1 - BETA1 ** t)) / ((v / (1 - BETA2 ** t)).sqrt() + ADAM_EPS)
    if small:
        w = _exact_words(m.numel(), s["seed"], t)
        for value, table, u in ((m, tables[0], w % 65536), (v, tables[1], w // 65536)):
            unit = (value.view(-1, BLOCK).abs().max(1).values / 1.875).float().to(f64).repeat_interleave(BLOCK)
            a = torch.where(unit > 0, value.abs() / unit, torch.zeros_like(value))
            below = (torch.bucketize(a, table, right=True) - 1).clamp(max=table.numel() - 2)
            part = (a - table[below]) / (table[below + 1] - table[below])    # of the way to the next code
            code = (below + (part + u.to(f64) / 65536.0 >= 1.0)).clamp(max=table.numel() - 1)
            if table.numel() == 256:
                code = torch.where(a > 0, code.clamp(min=1), code)
            res.append(torch.sign(value) * table[code] * unit)
        res.append(p)
    else:
        res += [p, m, v]
    return res + [p] if s["low"] is not None else res
