"""Attention at the ends of what its entry points accept: bucket ranges that pass the
largest float, huge scores, where masked scores begin, infinite operands,
positions that are no numbers.

Tolerances are those derived in test_gpu_attn.py, whose cases these are.
"""
import numpy as np
import pytest

from oracle import layers as ol

from .test_gpu_attn import Case, U, W, tpc  # noqa: F401  (tpc is the module's fixture)

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("r_min,steps,nb", [(1e10, 1, 64), (6.1e9, 1, 64), (1e15, 1, 64), (1e15, 1, 3), (5e14, 2, 64),
                                            (1e15, 4, 64), (1e15, 8, 20)])
def test_bucket_ranges_that_pass_the_largest_float(tpc, dtype, r_min, steps, nb):
    """Distances below the range, inside it and so large that their squares are infinite."""
    print(f"attn bucket range {dtype} {r_min} {steps} {nb}", flush=True)
    c = Case(dtype, [75, 40], 2, 2, 16, nb=nb, steps=steps, r_min=r_min, masked=0.1)
    r = np.random.default_rng(5)
    far = 10.0 ** r.uniform(0, 20, size=(115, 1)) * r.normal(size=(115, 3))
    c.kw["pos"] = torch.tensor(far.astype(np.float32), device="cuda")
    c.check(tpc)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("size", [-5e29, -1e12, -1e9, 1e9, 1e12])
@pytest.mark.parametrize("n", [70, 300])
def test_huge_scores_of_one_size(tpc, dtype, size, n):
    """Every score is one huge bias: out is the mean of v."""
    c = Case(dtype, [n], 2, 2, 16, nb=4, packed=False)
    c.kw["bias"][:] = size
    c.q[:] = 0
    out, lse = tpc.attn_forward(c.q, c.k, c.v, c.segt, **c.kw)
    v, bias = c.v.double(), float(c.kw["bias"][0, 0])
    # n equal probabilities: sums of n terms in float32, one division, the type's rounding
    tol = ((n + 4) * U + (W if dtype == "bf16" else 2 * U)) * v.abs().mean(0)
    assert ((out.double() - v.mean(0)).abs() <= tol).all()
    assert ((lse.double() - bias - np.log(n)).abs() <= 8 * U * abs(bias)).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_huge_scores_of_some_rows_and_tiles(tpc, dtype):
    """Biases of very different sizes in one row: the largest bucket of a row takes it all, wherever
    its tile comes, and rows beside it are not disturbed."""
    c = Case(dtype, [300], 2, 2, 16, nb=4, steps=1, packed=False)
    c.q[:] = 0
    c.kw["bias"][:] = torch.tensor([-1e12, -1e9, 3.0, -np.inf], device="cuda").to(c.kw["bias"].dtype)
    # buckets: r_min = 0.5, one step an octave of d2: 0 below 0.71, 1 to 1, 2 to 1.41, 3 beyond
    pos = torch.zeros(300, 3, device="cuda")
    pos[:, 0] = 10 * (torch.arange(300, device="cuda") % 60)                  # rows p, p + 60 .. share a place
    pos[60:120, 1], pos[180:240, 1] = 0.8, 1.2                                # 1, 2 from the first
    c.kw["pos"] = pos
    out, lse = tpc.attn_forward(c.q, c.k, c.v, c.segt, **c.kw)
    h, kw, _ = c.host()
    ref, rlse = ol.attn_forward(**h, **kw)
    size = np.abs(h["v"]).max()
    tol = 16 * U * size + (W if dtype == "bf16" else 0) * np.abs(ref)
    assert (np.abs(out.double().cpu().numpy() - ref) <= tol).all()
    assert (np.abs(lse.double().cpu().numpy() - rlse) <= 8 * U * np.abs(rlse)).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("low", [-1e9, -3e9, -7e11, -5e29])
@pytest.mark.parametrize("n", [40, 300])
def test_rows_of_huge_negative_scores_leave_finite_gradients(tpc, dtype, low, n):
    """A masked atom far from all others, where a finite large negative bias masks far pairs:
    its row holds such scores only.  It has no upstream gradient, so nothing but its own out
    and lse may differ from a bias of -inf, bit for bit."""
    c = Case(dtype, [n, 33], 4, 2, 32, nb=16, steps=1, box=3.0)
    c.kw["pos"][7] += 1e4
    c.kw["key_mask"] = torch.ones(n + 33, dtype=torch.uint8, device="cuda")
    c.kw["key_mask"][7] = 0
    c.go[7] = 0
    c.kw["bias"][:, 15] = -np.inf
    c.run(tpc)
    want = [c.out.clone(), c.lse.clone(), *(g.clone() for g in c.grads)]
    assert torch.all(c.lse[:, 7] == -np.inf)
    c.kw["bias"][:, 15] = low
    c.run(tpc)
    got = [c.out, c.lse, *c.grads]
    assert torch.isfinite(c.out).all() and torch.isfinite(c.lse).all()
    want[0][7], want[1][:, 7] = c.out[7], c.lse[:, 7]
    for name, g, w in zip(("out", "lse", "grad_q", "grad_k", "grad_v", "grad_bias"), got, want):
        assert torch.equal(g, w), name


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("size", [-5e29, -1e12, -1e9, 1e9, 1e12])
def test_probabilities_of_huge_scores_stay_below_one(tpc, dtype, size):
    """Every score is one huge bias: 32 bits cannot hold the backward's probabilities there, but
    they stay between 0 and 1."""
    n, d = 70, 16
    c = Case(dtype, [n], 2, 2, d, nb=4, packed=False)
    c.kw["bias"][:] = size
    c.q[:] = 0
    c.run(tpc)
    v, go = c.v.double(), c.go.double()
    over = 1 + 2 ** -7
    assert (c.grads[2].double().abs() <= over * go.abs().sum(0)).all()
    # |ds| <= |dp| + |delta| for p <= 1
    ds = (go.abs()[:, None] * (v.abs()[None] + v.abs().mean(0))).sum(-1)
    assert (c.grads[0].double().abs() <= over * d ** -0.5 * torch.einsum("ijh,jhd->ihd", ds, c.k.double().abs())).all()
    assert not c.grads[1].any() and torch.isfinite(c.grads[3]).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_where_masked_scores_begin(tpc, dtype):
    """Scores at or below -1e30 count as masked, those above do not."""
    c = Case(dtype, [50], 2, 2, 16, nb=4, packed=False)
    for size in (-1.01e30, -1e30):
        c.kw["bias"][:] = size
        c.run(tpc)
        assert not c.out.any() and torch.all(c.lse == -np.inf) and not any(g.any() for g in c.grads)
    c.kw["bias"][:] = -9.9e29
    c.run(tpc)
    mean = c.v.double().mean(0)
    tol = (54 * U + (W if dtype == "bf16" else 2 * U)) * c.v.double().abs().mean(0)
    assert ((c.out.double() - mean).abs() <= tol).all() and torch.isfinite(c.lse).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("n", [1, 40, 300])
@pytest.mark.parametrize("bad", [np.inf, -np.inf])
def test_infinite_values_reach_out_as_infinities(tpc, dtype, n, bad):
    """One infinite element of v: the outputs that it enters are infinite, all else, grad_v with
    it, is bit for bit as before."""
    c = Case(dtype, [n, 20], 2, 2, 40, nb=8, packed=False).run(tpc)
    want, lse, gv = c.out.clone(), c.lse.clone(), c.grads[2].clone()
    c.v[n // 2, 1, 11] = bad
    c.run(tpc)
    want[:n, 1, 11] = bad
    assert torch.equal(c.out, want) and torch.equal(c.lse, lse) and torch.equal(c.grads[2], gv)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("n", [40, 300])
def test_infinite_keys_that_give_scores_of_minus_infinity(tpc, dtype, n):
    """Such a key has no weight in any row: out and lse are those of a masked key.  An infinite
    query on the other side of the sign leaves its own row empty."""
    c = Case(dtype, [n, 20], 2, 2, 24, nb=8, packed=False)
    c.q[:, :, 3] = c.q[:, :, 3].abs() + 0.25
    c.kw["key_mask"] = torch.ones(n + 20, dtype=torch.uint8, device="cuda")
    c.kw["key_mask"][n // 2] = 0
    c.run(tpc)
    want = [c.out.clone(), c.lse.clone()]
    c.kw["key_mask"][n // 2] = 1
    c.k[n // 2, :, 3] = -np.inf
    got = tpc.attn_forward(c.q, c.k, c.v, c.segt, **c.kw)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    c.k[:, :, 3] = c.k[:, :, 3].abs() + 0.25
    c.k[n // 2, :, 3] = 1
    c.q[5, :, 3] = -np.inf
    out, lse = tpc.attn_forward(c.q, c.k, c.v, c.segt, **c.kw)
    assert not out[5].any() and torch.all(lse[:, 5] == -np.inf)
    keep = torch.arange(n + 20, device="cuda") != 5
    assert torch.isfinite(out[keep]).all() and torch.isfinite(lse[:, keep]).all()


def test_largest_floats(tpc):
    """Values beyond the largest bfloat16, which rounding to bfloat16 would make infinite, are
    exact: a single key's value comes back bit for bit."""
    c = Case("f32", [1] * 40, 2, 2, 16, packed=False)
    c.q[:] = 0
    c.v[:, 0, :] = torch.finfo(torch.float32).max
    c.v[:, 1, :8] = -3.3961e38
    c.v[:, 1, 8:] = 3.39e38
    c.run(tpc)
    assert torch.equal(c.out, c.v)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_positions_that_are_not_numbers_count_as_the_first_bucket(tpc, dtype):
    """NaN positions, and infinite ones on both sides of a pair."""
    c = Case(dtype, [45, 70], 2, 2, 16, nb=8, box=4.0)
    c.kw["pos"][4] = np.nan
    c.kw["pos"][50, 1] = -np.nan
    c.kw["pos"][60], c.kw["pos"][61] = np.inf, np.inf
    c.check(tpc)
