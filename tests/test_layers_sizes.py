"""Sizes beyond the 32 bits of the C entry points are refused by the binding, not cut to
their lower bits.  Without a GPU: the checks of a tensor's place are stubbed, the
tensors have no storage."""
import pytest

torch = pytest.importorskip("torch")

from tensor_product_convolution_amd import layers  # noqa: E402


@pytest.fixture
def nowhere(monkeypatch):
    calls = []
    monkeypatch.setattr(layers, "_code", lambda t, name: (layers._CODES[t.dtype], 0))
    monkeypatch.setattr(layers, "_rows", lambda t, name, dtype, shape, dev: (0x10000, 8))
    monkeypatch.setattr(layers, "_need", lambda t, name, dtype, shape, dev: 0x10000)
    monkeypatch.setattr(layers, "_call", lambda *a: calls.append(a))
    return calls


def meta(*shape, dtype=torch.float32):
    return torch.empty(*shape, dtype=dtype, device="meta")


def test_attention(nowhere):
    seg = meta(2, dtype=torch.int32)
    for n in (1 << 31, (1 << 32) + 5):
        q = meta(n, 1, 8, dtype=torch.bfloat16)
        with pytest.raises(ValueError, match="nodes"):
            layers._describe(q, q, q, seg, None, None, 0.5, 4, None, None)
    q = meta(40, 1, 8)
    with pytest.raises(ValueError, match="structures"):
        layers._describe(q, q, q, meta((1 << 32) + 2, dtype=torch.int32), None, None, 0.5, 4, None, None)
    with pytest.raises(ValueError, match="buckets"):
        layers._describe(q, q, q, seg, meta(40, 3), meta(1, (1 << 32) + 8), 0.5, 4, None, None)
    with pytest.raises(ValueError, match="heads"):
        big = meta(1, (1 << 32) + 1, 8)
        layers._describe(big, big, big, seg, None, None, 0.5, 4, None, None)
    with pytest.raises(ValueError, match="head_dim"):
        big = meta(1, 1, (1 << 32) + 8)
        layers._describe(big, big, big, seg, None, None, 0.5, 4, None, None)
    for steps in ((1 << 32) + 4, 4 - (1 << 32)):
        with pytest.raises(ValueError, match="steps"):
            layers._describe(q, q, q, seg, meta(40, 3), meta(1, 8), 0.5, steps, None, None)
    a, _, _ = layers._describe(q, q, q, seg, None, None, 0.5, 4, None, None)
    assert (a.n_nodes, a.n_segments, a.n_heads, a.n_kv_heads, a.head_dim) == (40, 1, 1, 1, 8)


def test_layer_norm(nowhere):
    x, g = meta(1, (1 << 32) + 8), meta((1 << 32) + 8)
    with pytest.raises(ValueError, match="columns"):
        layers.layer_norm_forward(x, g, g)
    with pytest.raises(ValueError, match="columns"):
        layers.layer_norm_backward(x, x, g, g, g)
    assert not nowhere
