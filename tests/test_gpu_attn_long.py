"""Attention over structures of more than 1,024 atoms, and the workgroup shapes that serve
them, against the float64 reference: all rows of the first and the last key head.

Workgroup shapes are chosen by the number of 32-row tiles times heads and by the mean
length.  CASES reach, forward and query side: two tiles by four (two for wide heads) parts of the
keys, eight tiles, four tiles (query side of heads of 128), each with one and two heads a wave, the
latter with shared and with separate key heads; key side: two tiles by four and by two
parts of the queries, four tiles by two.  BATCHES: four (two) tiles, two heads with key
heads of their own.

Tolerances are those derived in test_gpu_attn.py.  They hold what float32 products leave out
(three cut pieces, six partial products: below 2^-21, 8 units, of each): a score's 2 D + 8 units
cover it beside the D of the sum, an output's n + 2 D + 32 beside the n.
"""
import pytest

from .test_gpu_attn import Case, tpc  # noqa: F401  (tpc is the module's fixture)

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def check(tpc, c):
    c.run(tpc)
    hk = c.k.shape[1]
    rep = c.q.shape[1] // hk
    g = [0, hk - 1] if hk > 1 else [0]
    h = [i * rep + r for i in g for r in range(rep)]
    s = object.__new__(Case)
    s.lens, s.dtype, s.d, s.seg, s.kw = c.lens, c.dtype, c.d, c.seg, {**c.kw, "bias": c.kw["bias"][h]}
    s.q, s.k, s.v, s.go, s.out, s.lse = c.q[:, h], c.k[:, g], c.v[:, g], c.go[:, h], c.out[:, h], c.lse[h]
    s.grads = (c.grads[0][:, h], c.grads[1][:, g], c.grads[2][:, g], c.grads[3][h])
    s.run = lambda _: s
    s.check(tpc)


# (query heads, key heads, width, buckets)
ONE = [(8, 8, 16, 32), (8, 2, 32, 32), (8, 8, 40, 20), (8, 8, 64, 64), (8, 8, 96, 8), (8, 8, 128, 20), (64, 64, 16, 32),
       (64, 32, 16, 32)]
TWO = [(64, 64, 16, 32), (64, 32, 16, 32), (64, 64, 32, 20), (64, 64, 64, 16), (16, 16, 16, 32), (128, 64, 8, 32),
       (128, 128, 16, 8), (64, 32, 64, 32), (36, 36, 64, 32), (36, 36, 128, 32), (16, 16, 128, 8)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("heads", ONE, ids=str)
def test_one_long_structure(tpc, dtype, heads):
    hq, hk, d, nb = heads
    print(f"attn long {dtype} {heads}", flush=True)
    check(tpc, Case(dtype, [1100], hq, hk, d, nb=nb, seed=3))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("heads", TWO, ids=str)
def test_two_long_structures(tpc, dtype, heads):
    """Masked atoms, whole tiles of them among these."""
    hq, hk, d, nb = heads
    print(f"attn two long {dtype} {heads}", flush=True)
    c = Case(dtype, [1100, 1057], hq, hk, d, nb=nb, masked=0.05, seed=4)
    c.kw["key_mask"][:70] = 0
    c.kw["key_mask"][400:530] = 0
    check(tpc, c)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("heads", [(16, 16, 16, 32), (16, 16, 32, 16)], ids=str)
def test_batches_of_short_structures(tpc, dtype, heads):
    hq, hk, d, nb = heads
    print(f"attn batch {dtype} {heads}", flush=True)
    check(tpc, Case(dtype, [90] * 60 + [1, 0, 200], hq, hk, d, nb=nb, masked=0.05, seed=5))
