"""The float64 reference of the operators around the attention block against differences of
itself, closed forms and its own inverses.  No GPU."""
import numpy as np
import pytest

from oracle import blocks as ob


def slope(f, x, d, h=1e-6):
    return (f(x + h * d) - f(x - h * d)) / (2 * h)


@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("pairs,axes", [(0, 1), (2, 1), (3, 3)])
def test_heads_by_differences(norm, interleaved, pairs, axes):
    r = np.random.default_rng(pairs * 4 + norm)
    x, g = r.normal(size=(4, 3, 7)), r.normal(size=(4, 3, 7))
    gamma = r.normal(size=7) if norm else None
    pos, freq = (r.normal(size=(4, axes)), r.normal(size=(pairs, axes))) if pairs else (None, None)
    f = lambda x, gamma=gamma, pos=pos: (ob.head_forward(x, gamma, pos, freq, interleaved, 1e-3) * g).sum()
    gx, gg, gpos = ob.head_backward(g, x, gamma, pos, freq, interleaved, 1e-3)
    d = r.normal(size=x.shape)
    assert abs(slope(f, x, d) - (gx * d).sum()) < 1e-7
    if norm:
        d = r.normal(size=7)
        assert abs(slope(lambda q: f(x, gamma=q), gamma, d) - (gg * d).sum()) < 1e-7
    if pairs:
        d = r.normal(size=pos.shape)
        assert abs(slope(lambda q: f(x, pos=q), pos, d) - (gpos * d).sum()) < 1e-7


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotated_products_depend_on_differences_alone(interleaved):
    r = np.random.default_rng(1)
    q, k = r.normal(size=(2, 5, 1, 8))
    pos, freq = r.normal(size=(5, 3)), r.normal(size=(4, 3))
    rot = lambda x, p: ob.head_forward(x, None, p, freq, interleaved, 0.0)[:, 0]
    a = rot(q, pos) @ rot(k, pos).T
    assert np.allclose(a, rot(q, pos + [3.0, -1.0, 7.0]) @ rot(k, pos + [3.0, -1.0, 7.0]).T, atol=1e-12)
    assert np.allclose(np.linalg.norm(rot(q, pos), axis=1), np.linalg.norm(q[:, 0], axis=1))


@pytest.mark.parametrize("over_all", [False, True])
def test_route(over_all):
    r = np.random.default_rng(2)
    l = np.round(r.normal(size=(40, 6)), 1)                    # ties
    l[3] = -np.inf
    l[4, 1:] = -np.inf
    l[5, 2] = np.nan
    w, i = ob.route(l, 3, over_all)
    assert (i[3] == -1).all() and (w[3] == 0).all() and list(i[4]) == [0, -1, -1]
    assert not over_all or abs(w[4, 0] - 1) < 1e-15
    for row in range(40):
        for a, b in zip(i[row], i[row][1:]):
            assert b < 0 or l[row, a] > l[row, b] or (l[row, a] == l[row, b] and a < b)
    if not over_all:
        assert np.allclose(w.sum(1), (i[:, 0] >= 0).astype(float))
    l = r.normal(size=(8, 6))
    g = r.normal(size=(8, 3))
    w, i = ob.route(l, 3, over_all)
    d = r.normal(size=l.shape)
    want = slope(lambda x: (ob.route(x, 3, over_all)[0] * g).sum(), l, d)
    assert abs((ob.route_backward(g, l, w, i, over_all) * d).sum() - want) < 1e-7


@pytest.mark.parametrize("x_rows,y_rows,fan", [("source", "source", 1), ("source", "grouped", 2), ("grouped", "source", 2),
                                               ("grouped", "grouped", 1)])
def test_grouped_by_differences(x_rows, y_rows, fan):
    r = np.random.default_rng(fan)
    index = r.integers(-1, 4, size=12)
    ptr, rows = ob.group_rows(index, 4)
    assert ptr[0] == 0 and sorted(rows) == list(range(12))
    for e in range(4):
        assert list(rows[ptr[e]:ptr[e + 1]]) == [s for s in range(12) if index[s] == e]
    x, w, b = r.normal(size=(12 // fan if x_rows == "source" else 12, 3)), r.normal(size=(4, 3, 2)), r.normal(size=(4, 2))
    g = r.normal(size=(12, 2))
    f = lambda x, w=w, b=b: (ob.grouped_forward(x, w, ptr, rows, fan, b, x_rows, y_rows) * g).sum()
    gx, gw, gb = ob.grouped_backward(g, x, w, ptr, rows, fan, x_rows, y_rows)
    for t, grad, call in ((x, gx, f), (w, gw, lambda t: f(x, w=t)), (b, gb, lambda t: f(x, b=t))):
        d = r.normal(size=t.shape)
        assert abs(slope(call, t, d) - (grad * d).sum()) < 1e-7
    z = r.normal(size=50)
    assert np.abs(ob.silu_slope(z) - slope(ob.silu, z, np.ones(50))).max() < 1e-8


def test_codes():
    for second, top in ((False, 128), (True, 256)):
        v = ob.code_values(second)
        assert len(v) == top and v[0] == 0 and v[-1] == 1.875 and (np.diff(v) > 0).all()
        # codes are exact at u = 0 and stay where they are whatever u is
        codes = np.r_[np.arange(top), np.zeros(256 - top % 256 if top % 256 else 0, int)][:256].astype(np.uint8)
        codes[0] = top - 1
        if not second:
            codes[10:100] |= 128
        x = ob.decode(codes, [2.0], second)
        for u in (0.0, 0.9999):
            c, unit = ob.encode(x, second, u)
            assert unit[0] == 2.0 and np.array_equal(c, codes)
    # the mean of the roundings is the value
    x = np.full(256 * 400, 0.3)
    x[::256] = 1.0
    u = np.random.default_rng(0).random(x.size)
    c, unit = ob.encode(x, True, u)
    y = ob.decode(c, unit, True)
    # 102,000 draws between two codes an eighth of an octave apart: 5 standard errors
    assert abs(np.delete(y, np.s_[::256]).mean() - 0.3) < 5 * 0.5 * 0.3 / 8 / 102000 ** 0.5
