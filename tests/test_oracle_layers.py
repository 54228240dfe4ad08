"""The float64 reference of attention, layer norm and dropout against things other
than itself: central differences, torch's float64 softmax and norm on the CPU,
plain loops, the generator's published test vectors and limits."""
import numpy as np
import pytest
import torch

from oracle import layers as ol


def _case(seed, lens, hq, hk, d, nb=0, masked=0.0):
    r = np.random.default_rng(seed)
    n = sum(lens)
    seg = np.concatenate([[0], np.cumsum(lens)])
    c = dict(q=r.normal(size=(n, hq, d)), k=r.normal(size=(n, hk, d)), v=r.normal(size=(n, hk, d)), seg_ptr=seg)
    kw = {}
    if nb:
        kw.update(pos=r.uniform(0, 4, size=(n, 3)).astype(np.float32), bias=r.normal(size=(hq, nb)), r_min=0.5, steps=4)
    if masked:
        kw["key_mask"] = (r.uniform(size=n) >= masked).astype(np.uint8)
    return c, kw, r.normal(size=(n, hq, d))


def test_attention_matches_torch_softmax():
    c, kw, _ = _case(0, [5, 1, 0, 9], 4, 2, 8, nb=20, masked=0.3)
    out, lse = ol.attn_forward(**c, **kw)
    t = lambda a: torch.tensor(np.asarray(a), dtype=torch.float64)
    for b in range(len(c["seg_ptr"]) - 1):
        sl = slice(c["seg_ptr"][b], c["seg_ptr"][b + 1])
        live = torch.tensor(kw["key_mask"][sl] != 0)
        bk = ol.buckets(kw["pos"][sl], 0.5, 4, 20)
        for h in range(4):
            s = t(c["q"][sl, h]) @ t(c["k"][sl, h // 2]).T / 8 ** 0.5 + t(kw["bias"][h][bk])
            s = s.masked_fill(~live, -np.inf)
            if live.any():
                assert np.allclose(out[sl, h], (torch.softmax(s, 1) @ t(c["v"][sl, h // 2])).numpy(), atol=1e-13)
                assert np.allclose(lse[h, sl], torch.logsumexp(s, 1).numpy(), atol=1e-13)
            else:
                assert not out[sl, h].any() and np.all(lse[h, sl] == -np.inf)


@pytest.mark.parametrize("which", ["q", "k", "v", "bias"])
def test_attention_gradients_by_differences(which):
    c, kw, go = _case(1, [4, 6], 4, 2, 8, nb=8, masked=0.2)
    g = dict(zip(("q", "k", "v", "bias"), ol.attn_backward(**c, **kw, grad_out=go)))[which]
    loss = lambda: float((ol.attn_forward(**c, **kw)[0] * go).sum())
    a = c.get(which, kw.get(which))
    for i in np.random.default_rng(2).choice(a.size, size=min(25, a.size), replace=False):
        keep, h = a.flat[i], 1e-5
        a.flat[i] = keep + h
        up = loss()
        a.flat[i] = keep - h
        down = loss()
        a.flat[i] = keep
        # second-order error h^2 f''' / 6 plus rounding 1e-16 |loss| / h
        assert abs((up - down) / (2 * h) - g.flat[i]) < 1e-7


def test_buckets_against_a_plain_loop():
    pos = np.random.default_rng(3).uniform(0, 9, size=(40, 3)).astype(np.float32)
    for steps in (1, 2, 4, 8):
        b = ol.buckets(pos, 0.5, steps, 32)
        for i in range(40):
            for j in range(40):
                d2 = float(((pos[i].astype(np.float64) - pos[j]) ** 2).sum())
                # octave and linear step of d2, counted from those of r_min^2 = 0.25
                want = 0
                if d2 >= 0.25:
                    e = int(np.floor(np.log2(d2)))
                    want = (e + 2) * steps + int((d2 / 2.0 ** e - 1) * steps)
                near = abs(d2 * steps / 2.0 ** np.floor(np.log2(max(d2, 1e-9))) % 1)
                if min(near, 1 - near) > 1e-4:          # away from a step's edge
                    assert b[i, j] == min(want, 31), (d2, steps)


def test_low_scores_count_as_masked():
    c, kw, go = _case(4, [6], 2, 2, 8, nb=4)
    kw["bias"][:, 3] = -np.inf
    a = ol.attn_forward(**c, **kw)
    kw["bias"][:, 3] = -3e38
    b = ol.attn_forward(**c, **kw)
    assert np.array_equal(a[0], b[0]) and np.array_equal(a[1], b[1])
    kw["bias"][:] = -3e38
    out, lse = ol.attn_forward(**c, **kw)
    assert not out.any() and np.all(lse == -np.inf)
    assert not any(g.any() for g in ol.attn_backward(**c, **kw, grad_out=go))


def test_norm_matches_torch_and_differences():
    r = np.random.default_rng(5)
    h, gamma, beta, gy = r.normal(size=(7, 13)) + 2, r.normal(size=13), r.normal(size=13), r.normal(size=(7, 13))
    y, mean, rstd = ol.layer_norm_forward(h, gamma, beta, 1e-5)
    t = [torch.tensor(a, requires_grad=True) for a in (h, gamma, beta)]
    ref = torch.nn.functional.layer_norm(t[0], (13,), t[1], t[2], 1e-5)
    assert np.allclose(y, ref.detach().numpy(), atol=1e-13)
    ref.backward(torch.tensor(gy))
    for got, x in zip(ol.layer_norm_backward(gy, h, gamma, 1e-5), t):
        assert np.allclose(got, x.grad.numpy(), atol=1e-12)
    assert np.allclose(mean, h.mean(1)) and np.allclose(rstd, 1 / np.sqrt(h.var(1) + 1e-5))


def test_generator_published_vectors():
    """The known-answer vectors published with the generator (10 rounds)."""
    m = 2 ** 64 - 1
    assert ol.philox_block(0, 0, 0) == [0x6627e8d5, 0xe169c58d, 0xbc57ac4c, 0x9b00dbd8]
    assert ol.philox_block(m, m, m) == [0x408f276d, 0x41c83b0e, 0xa20bc7c6, 0x6d5451fd]
    assert ol.philox_block(0x85a308d3243f6a88, 0x299f31d0a4093822, 0x0370734413198a2e) == [
        0xd16cfe09, 0x94fdcceb, 0x5001e420, 0x24126ea1]


def test_dropout_rate():
    n, p = 20000, 0.3
    f = ol.dropout_factor((n,), p, 12345, 7)
    # binomial: 5 standard deviations
    assert abs((f == 0).mean() - p) < 5 * np.sqrt(p * (1 - p) / n)
    assert np.all(ol.dropout_factor((50,), 0.0, 1, 2) == 1.0)
