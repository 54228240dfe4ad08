"""A training step of a potential's layer with global attention between atoms.

The convolution mixes neighbours; the attention block behind it mixes all atoms of
a structure, through the scalar (0e) channels of the node rows:

    f = convolution(x, Y, w)                    node rows, 0e block first
    y = layer_norm(f[:, :U])                    strided: the 0e block as it lies
    a = attention(y Wq, y Wk, y Wv; bias by distance bucket)
    h, z = dropout(a Wo) + f[:, :U], layer_norm(h)
    energy of a structure per atom = mean over its atoms of z . readout

trained on random targets with plain gradient descent; the gradient reaches every
weight of the block and, through the convolution's backward, x and w.  Run on a GPU:

    python examples/atom_attention.py [steps]
"""
import os
import sys

import numpy as np
import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import tensor_product_convolution_amd as tpc  # noqa: E402

IRREPS, LMAX = "32x0e+32x1o+32x2e", 2
HEADS, KEY_HEADS, DIM, BUCKETS = 4, 2, 16, 32


class Layer:
    """Weights of the attention block and its hand-written forward and backward."""

    def __init__(self, channels, p_drop, gen):
        u, d = channels, DIM
        rand = lambda *s: torch.randn(*s, device="cuda", generator=gen)
        self.w = dict(gamma1=torch.ones(u, device="cuda"), beta1=torch.zeros(u, device="cuda"),
                      qkv=rand(u, (HEADS + 2 * KEY_HEADS) * d) / u ** 0.5, bias=0.1 * rand(HEADS, BUCKETS),
                      out=rand(HEADS * d, u) / (HEADS * d) ** 0.5, gamma2=torch.ones(u, device="cuda"),
                      beta2=torch.zeros(u, device="cuda"), readout=rand(u) / u ** 0.5)
        self.p_drop = p_drop

    def _split(self, row):
        n = row.shape[0]
        return [t.view(n, -1, DIM) for t in row.split([HEADS * DIM, KEY_HEADS * DIM, KEY_HEADS * DIM], dim=1)]

    def forward(self, f, seg, pos, step):
        """(z, what the backward needs) for the scalar block f of the node rows."""
        w = self.w
        y, mean1, rstd1 = tpc.layer_norm_forward(f, w["gamma1"], w["beta1"])
        qkv = y @ w["qkv"]
        q, k, v = self._split(qkv)
        o, lse = tpc.attn_forward(q, k, v, seg, pos=pos, bias=w["bias"])
        drop = tpc.Dropout(self.p_drop, seed=17, offset=step)
        z, mean2, rstd2, h = tpc.layer_norm_residual_forward(o.view(len(f), -1) @ w["out"], f.contiguous(), w["gamma2"],
                                                             w["beta2"], drop)
        return z, (f, y, mean1, rstd1, q, k, v, o, lse, drop, h, mean2, rstd2, seg, pos)

    def backward(self, grad_z, saved):
        """(gradient of f, gradients of the weights but the readout)"""
        f, y, mean1, rstd1, q, k, v, o, lse, drop, h, mean2, rstd2, seg, pos = saved
        w, g, n = self.w, {}, len(f)
        grad_a, grad_f, g["gamma2"], g["beta2"] = tpc.layer_norm_residual_backward(grad_z, h, w["gamma2"], mean2, rstd2, drop)
        g["out"] = o.view(n, -1).t() @ grad_a
        grad_qkv = torch.empty(n, w["qkv"].shape[1], device="cuda")
        *_, g["bias"] = tpc.attn_backward(q, k, v, seg, o, lse, (grad_a @ w["out"].t()).view(n, HEADS, DIM), pos=pos,
                                          bias=w["bias"], outs=self._split(grad_qkv))
        g["qkv"] = y.t() @ grad_qkv
        grad_1, g["gamma1"], g["beta1"] = tpc.layer_norm_backward(grad_qkv @ w["qkv"].t(), f, w["gamma1"], mean1, rstd1)
        return grad_f + grad_1, g


def batch(sizes, neighbours, seed):
    """Random structures: positions at 0.05 atoms per cubic Angstrom, each atom's nearest
    neighbours as edges, and one target energy per atom for each structure."""
    r = np.random.default_rng(seed)
    pos, src, dst, at = [], [], [], 0
    for n in sizes:
        p = r.uniform(0, (n / 0.05) ** (1 / 3), size=(n, 3))
        near = np.argsort(((p[:, None] - p[None]) ** 2).sum(-1), axis=1)[:, 1:neighbours + 1]
        src.append(near.reshape(-1) + at)
        dst.append(np.repeat(np.arange(n), near.shape[1]) + at)
        pos.append(p)
        at += n
    cuda = lambda a, t: torch.tensor(np.concatenate(a) if isinstance(a, list) else a, dtype=t, device="cuda")
    seg = np.concatenate([[0], np.cumsum(sizes)])
    return (cuda(pos, torch.float32), cuda(src, torch.int32), cuda(dst, torch.int32), cuda(seg, torch.int32),
            cuda(r.normal(size=len(sizes)), torch.float32))


def train(steps=20, sizes=(40, 1, 97, 64), p_drop=0.1, rate=0.02, seed=0, report=print):
    """Losses of `steps` steps."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    pos, src, dst, seg, target = batch(sizes, 12, seed)
    n, struct = pos.shape[0], torch.repeat_interleave(torch.arange(len(sizes), device="cuda"), torch.tensor(sizes, device="cuda"))
    plan = tpc.Plan(IRREPS, LMAX, LMAX)
    graph = tpc.graph_launch_order(tpc.graph_build(src, dst, n))
    r = tpc.gather_rows(pos[src.long()] - pos[dst.long()], graph.perm)
    Y = tpc.sph_harm(LMAX, r)
    x = torch.randn(n, plan.xdim, device="cuda", generator=gen)
    w = torch.randn(graph.n_edges, plan.n_paths, plan.mul, device="cuda", generator=gen) / (12 * plan.n_paths) ** 0.5
    layer = Layer(plan.mul, p_drop, gen)
    share = 1 / torch.tensor(sizes, dtype=torch.float32, device="cuda")[struct]
    losses = []
    for step in range(steps):
        rows = tpc.forward(plan, graph, x, Y, w)
        z, saved = layer.forward(rows[:, :plan.mul], seg, pos, step)
        energy = torch.zeros(len(sizes), device="cuda").index_add_(0, struct, share * (z @ layer.w["readout"]))
        error = energy - target
        losses.append(float((error * error).mean()))
        report(f"step {step}: loss {losses[-1]:.5f}")
        grad_atom = share * (2 / len(sizes) * error)[struct]
        grad_scalars, grads = layer.backward(grad_atom[:, None] * layer.w["readout"], saved)
        grads["readout"] = grad_atom @ z
        grad_rows = torch.zeros_like(rows)
        grad_rows[:, :plan.mul] = grad_scalars
        _, _, grad_w = tpc.backward(plan, graph, x, Y, w, grad_rows, want=("w",))
        for name, g in grads.items():
            layer.w[name] -= rate * g
        w -= rate * grad_w
    return losses


if __name__ == "__main__":
    if not torch.cuda.is_available():
        raise SystemExit("needs a GPU")
    train(int(sys.argv[1]) if len(sys.argv) > 1 else 20)
