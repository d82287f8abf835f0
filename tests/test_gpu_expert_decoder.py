"""The example that runs the token moves together: its gradients against the
same layer in plain torch operations in 64 bits, its losses, and its
token-by-token outputs."""

import importlib.util
import os

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "expert_decoder.py")


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("expert_decoder", PATH)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def _plain(example, layer, x, positions):
    """The layer with plain torch operations in place of the moves."""
    freq, axes, pairs = layer.inv_freq.double(), layer.pair_axes.long(), layer.head_dim // 2
    angle = (positions[axes].t().float() * layer.inv_freq).double()[:, None]
    cos, sin = torch.cos(angle), torch.sin(angle)

    def turn(y):
        a, b = y[..., :pairs], y[..., pairs:]
        return torch.cat([a * cos - b * sin, b * cos + a * sin], -1)

    q, k, v = layer.split(x)
    n = x.shape[0]
    x = x + layer.attend(turn(q), turn(k), v, torch.ones(n, n, dtype=torch.bool, device="cuda").tril())
    weights, ids = torch.softmax(x @ layer.router, dim=1).topk(layer.choices, dim=1)
    out = torch.zeros_like(x)
    for e in range(layer.experts):
        w = (weights * (ids == e)).sum(1, keepdim=True)
        out = out + w * (torch.relu(x @ layer.up[e]) @ layer.down[e])
    return x + out


def test_gradients_of_the_layer(example):
    torch.manual_seed(3)
    layer = example.Layer()
    exact = example.Layer(dtype=torch.float64)
    exact.load_state_dict({n: p.double() if p.is_floating_point() and n != "inv_freq" else p for n, p in layer.state_dict().items()})
    x = torch.randn(60, 256, device="cuda")
    positions = example.image_positions(60)
    target = torch.randn(60, 256, device="cuda")
    (layer(x, positions) - target).square().mean().backward()
    (_plain(example, exact, x.double(), positions) - target.double()).square().mean().backward()
    for (name, p), q in zip(layer.named_parameters(), exact.parameters()):
        off = float((p.grad.double() - q.grad).norm() / q.grad.norm())
        # sums of up to some thousand products in 32 bits, a few of them one
        # after another: unit roundoff 6e-8 times a few hundred
        assert off < 2e-5, (name, off)


def test_training_and_generation(example):
    torch.manual_seed(0)
    layer = example.Layer()
    losses = example.train(layer, steps=5)
    assert losses[-1] < losses[0]
    off, size = example.generate(layer)
    assert off < 1e-4 * size
