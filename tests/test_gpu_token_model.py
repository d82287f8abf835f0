"""The example's decoder, which runs the library's calls together: embedding,
rotary, experts and their balance loss trained, and a cache in 8 bits appended
to and read back token by token."""

import importlib.util
import os

import pytest

import bmmc_index_transforms_gb300 as bm

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "expert_decoder.py")


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("expert_decoder", PATH)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def _plain_loss(decoder, ids, positions, weight):
    """The decoder's loss with plain torch operations in place of the calls."""
    axes, pairs = decoder.pair_axes.long(), decoder.head_dim // 2
    angle = (positions[axes].t().float() * decoder.inv_freq.float()).double()[:, None]
    cos, sin = torch.cos(angle), torch.sin(angle)

    def turn(y):
        a, b = y[..., :pairs], y[..., pairs:]
        return torch.cat([a * cos - b * sin, b * cos + a * sin], -1)

    x = decoder.table[ids[:-1]] * decoder.table.shape[1] ** 0.5
    q, k, v = decoder.split(x)
    n, E = x.shape[0], decoder.experts
    x = x + decoder.attend(turn(q), turn(k), v, torch.ones(n, n, dtype=torch.bool, device="cuda").tril())
    p = torch.softmax(x @ decoder.router, dim=1)
    weights, chosen = p.topk(decoder.choices, dim=1)
    share = torch.bincount(chosen.flatten(), minlength=E).double() / chosen.numel()
    out = torch.zeros_like(x)
    for e in range(E):
        w = (weights * (chosen == e)).sum(1, keepdim=True)
        out = out + w * (torch.relu(x @ decoder.up[e]) @ decoder.down[e])
    y = (x + out) @ decoder.table.t()
    return torch.nn.functional.cross_entropy(y, ids[1:]) + weight * E * (share * p.mean(0)).sum()


def test_gradients_of_the_decoder(example):
    torch.manual_seed(5)
    decoder, exact = example.Decoder(), example.Decoder(dtype=torch.float64)
    exact.load_state_dict({n: p.double() if p.is_floating_point() and n != "inv_freq" else p for n, p in decoder.state_dict().items()})
    ids = torch.randint(0, 300, (81,), device="cuda")
    positions = example.image_positions(80)
    a, b = decoder.loss(ids, positions, 0.5), _plain_loss(exact, ids, positions, 0.5)
    assert abs(float(a.detach()) - float(b.detach())) < 2e-5 * abs(float(b.detach()))
    a.backward()
    b.backward()
    for (name, p), (_, q) in zip(decoder.named_parameters(), exact.named_parameters()):
        off = float((p.grad.double() - q.grad).norm() / q.grad.norm())
        # sums of up to some thousand products in 32 bits, a few of them one
        # after another: unit roundoff 6e-8 times a few hundred
        assert off < 2e-5, (name, off)


def test_training_runs(example):
    torch.manual_seed(0)
    losses = example.train_decoder(example.Decoder(), steps=3)
    assert len(losses) == 3 and all(torch.tensor(losses).isfinite())


@pytest.mark.parametrize("dtype", [torch.float8_e4m3fn, torch.int8])
def test_token_by_token_over_a_cache_of_8_bits(example, dtype):
    """What a step reads back is each head within half a step of the type: the
    heads come from products in 32 bits (256 terms, 2**-24 of their sum of
    magnitudes each), and keys are turned (8 * 2**-24 of a pair)."""
    torch.manual_seed(2)
    layer = example.Layer()
    B, n = 3, 40
    x = torch.randn(B, n, 256, device="cuda")
    positions = example.image_positions(n)
    cache = example.Cache(layer, B, n, dtype=dtype)
    for t in range(n):
        y = example.step(layer, cache, x[:, t].contiguous(), positions[:, t:t + 1].expand(3, B).contiguous())
        assert torch.isfinite(y).all()
    keys, values, lengths = cache.read()
    assert lengths == [n] * B
    flat = x.reshape(B * n, 256).double()
    heads = (flat @ layer.qkv.double()).view(B * n, -1, layer.head_dim)
    size = (flat.abs() @ layer.qkv.double().abs()).view(B * n, -1, layer.head_dim)
    _, k, v = heads.split([layer.q_heads, layer.kv_heads, layer.kv_heads], dim=1)
    _, k_size, v_size = size.split([layer.q_heads, layer.kv_heads, layer.kv_heads], dim=1)
    angle = (positions[layer.pair_axes.long()].t().float() * layer.inv_freq).double().repeat(B, 1)[:, None]
    P = layer.head_dim // 2
    a, b = k[..., :P], k[..., P:]
    k = torch.cat([a * torch.cos(angle) - b * torch.sin(angle), b * torch.cos(angle) + a * torch.sin(angle)], -1)
    pair = k_size[..., :P] + k_size[..., P:]
    k_size = torch.cat([pair, pair], -1)
    for got, want, s in ((keys, k, k_size), (values, v, v_size)):
        off = (256 + 8) * 2.0 ** -24 * s
        scale = (want.abs().amax(-1, keepdim=True) + off.amax(-1, keepdim=True)) / (448 if dtype == torch.float8_e4m3fn else 127)
        half = scale / 2 if dtype == torch.int8 else torch.maximum(2.0 ** -4 * (want.abs() + off), 2.0 ** -10 * scale)
        # read back in 32 bits: one more rounding, and 2 * 2**-24 of the value in its quotient
        limit = half * (1 + 2.0 ** -20) + off + 4 * 2.0 ** -24 * (want.abs() + off)
        assert bool(((got.double() - want).abs() <= limit).all())


def test_a_step_captured_in_a_graph(example):
    """Lookup, append and read in one graph, replayed with other tokens."""
    torch.manual_seed(4)
    decoder = example.Decoder()
    B = 4
    cache = example.Cache(decoder, B, 32, dtype=torch.float8_e4m3fn)
    ids = torch.randint(0, 300, (B,), device="cuda")
    rows = 4 * 32

    def run():
        x = decoder.embed(ids)
        q, k, v = decoder.split(x)
        q = bm.paged_append(k, v, cache.k, cache.v, cache.table, cache.lengths, q=q, inv_freq=decoder.inv_freq, **cache.scales)
        cache.lengths += 1
        cache.starts[1:] = torch.cumsum(cache.lengths, 0)
        return (q, *bm.paged_read(cache.k, cache.v, cache.table, cache.starts, rows, dtype=torch.float32, **cache.scales))

    texts = torch.randint(0, 300, (6, B), device="cuda")
    with torch.no_grad():
        want = []
        for text in texts:
            ids.copy_(text)
            want.append([x.clone() for x in run()])
        cache.lengths.zero_()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = run()
        cache.lengths.zero_()
        for text, w in zip(texts, want):
            ids.copy_(text)
            graph.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(x, y) for x, y in zip(got, w))
