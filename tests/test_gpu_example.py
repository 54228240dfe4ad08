"""The example that trains a convolution with the attention block behind it: its
gradient against differences of its own loss, and a falling loss."""
import importlib.util
import os

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def example():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "atom_attention.py")
    spec = importlib.util.spec_from_file_location("atom_attention", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_loss_falls(example):
    losses = example.train(steps=30, report=lambda s: None)
    assert all(l == l for l in losses)
    # noisy by the dropout: the last third against the first step
    assert sum(losses[-10:]) / 10 < 0.5 * losses[0], losses


def test_gradients_by_differences(example):
    """Directional differences of sum(z * c) in every weight and in f.  Step 2^-8: the
    truncation and the rounding of the loss stay below 2e-2 of the sum of absolute terms."""
    gen = torch.Generator(device="cuda").manual_seed(3)
    sizes = (20, 1, 33)
    pos, _, _, seg, _ = example.batch(sizes, 4, 3)
    n = sum(sizes)
    layer = example.Layer(32, 0.2, gen)
    rows = torch.randn(n, 96, device="cuda", generator=gen)
    f = rows[:, :32]
    c = torch.randn(n, 32, device="cuda", generator=gen)
    loss = lambda: float((layer.forward(f, seg, pos, 5)[0].double() * c.double()).sum())
    z, saved = layer.forward(f, seg, pos, 5)
    grad_f, grads = layer.backward(c, saved)
    for name, g in [("f", grad_f), *grads.items()]:
        t = f if name == "f" else layer.w[name]
        keep, d, h = t.clone(), torch.randn(t.shape, device="cuda", generator=gen), 2.0 ** -8
        t.copy_(keep + h * d)
        up = loss()
        t.copy_(keep - h * d)
        down = loss()
        t.copy_(keep)
        want = float((g.double() * d.double()).sum())
        assert abs((up - down) / (2 * h) - want) < 2e-2 * float((g * d).abs().double().sum()), name
