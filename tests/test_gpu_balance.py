"""expert_balance and its gradient on the GPU against the definition in 64
bits.

To first order a share of a softmax of E logits over a range r is off by at
most S = (2 * (r + 2) + E + 4) * 2**-24 of itself: the differences from the
largest logit are rounded (r * 2**-24 of the exponential, above and below the
line), an exponential is off by 2 ulp, the sum's E - 1 additions and the
quotient by one rounding each.  All shares are positive, so a sum over n
tokens, with the roundings of its additions, is off by S + n * 2**-24 of
itself.
"""

import pytest

import bmmc_index_transforms_gb300 as bm

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16
U32 = 2.0 ** -24
ROUND = {F32: 2.0 ** -24, F16: 2.0 ** -11, BF16: 2.0 ** -8}
TINY = {F32: 2.0 ** -149, F16: 2.0 ** -24, BF16: 2.0 ** -133}


def _gen(seed):
    g = torch.Generator("cuda")
    g.manual_seed(seed)
    return g


def _definition(logits, ids):
    """(loss, counts, gradient of the loss, bound of the loss, bound of the gradient) in 64 bits."""
    T, E = logits.shape
    x = logits.double()
    routed = (ids >= 0) & (ids < E)
    there = routed.any(1)
    c = torch.bincount(ids[routed].long(), minlength=E)
    n, C = int(there.sum()), max(1, int(c.sum()))
    top = x.amax(1, keepdim=True)
    e = torch.exp(x - torch.where(top.isinf(), 0, top))
    total = e.sum(1, keepdim=True)
    p = torch.where(total > 0, e / total, 0) * there[:, None]
    p = torch.where(there[:, None], p, 0)
    f = c.double() / C
    loss = E * (f * p.sum(0)).sum() / max(1, n)
    dot = (p * f).sum(1, keepdim=True)
    grad = E / max(1, n) * p * (f - dot)
    low = torch.where(x.isinf() | ~there[:, None], float("inf"), x).amin(1, keepdim=True)
    reach = torch.where(there[:, None] & ~low.isinf() & ~top.isinf(), top - low, 0)
    S = (2 * (reach + 2) + E + 4) * U32
    counts = torch.cat([c, c.new_tensor([n])]).int()
    # the products of shares with f and their sum over E: each of dot's terms off by S and E + 2 roundings
    bound = E / max(1, n) * p * ((f + dot) * (S + 8 * U32) + dot * (S + (E + 2) * U32))
    return loss, counts, grad, loss * (float(S.max() if T else 0) + (T + E + 8) * U32), bound


def _check(logits, ids, scale=1.0):
    loss, counts, grad, loss_bound, grad_bound = _definition(logits, ids)
    got, got_counts = bm.expert_balance(logits, ids)
    assert got.dtype == F32 and got.shape == () and got_counts.dtype == torch.int32
    assert torch.equal(got_counts, counts)
    off = abs(float(got) - float(loss))
    assert off <= loss_bound, (off, float(loss_bound))
    by = torch.tensor(scale, device="cuda")
    out = bm.expert_balance_backward(by, logits, ids, got_counts)
    assert out.dtype == logits.dtype and out.shape == logits.shape and torch.isfinite(out).all()
    t = logits.dtype
    limit = abs(scale) * grad_bound * (1 + 1e-3) + (ROUND[t] + 4 * U32) * (abs(scale) * grad.abs()) + TINY[t]
    miss = (out.double() - scale * grad).abs() - limit * (1 + 1e-3)
    assert bool((miss <= 0).all()), float(miss.max())
    again, _ = bm.expert_balance(logits, ids)
    assert torch.equal(again, got) and torch.equal(bm.expert_balance_backward(by, logits, ids, got_counts), out)
    return got, got_counts, out


def _case(g, T, K, E, dtype, empty=0.1, pad=0, ids=torch.int64, shift=0):
    x = 2 * torch.randn(T * (E + pad) + shift, generator=g, device="cuda")
    logits = x.to(dtype)[shift:].view(T, E + pad)[:, :E]
    chosen = torch.rand(T, E, generator=g, device="cuda").topk(K, dim=1)[1]
    chosen.masked_fill_(torch.rand(T, K, generator=g, device="cuda") < empty / 2, -1)
    chosen[torch.rand(T, generator=g, device="cuda") < empty / 2] = E
    return logits, chosen.to(ids)


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("T,K,E,pad,shift", [
    (1, 1, 1, 0, 0), (1, 1, 2, 0, 0), (5, 2, 3, 0, 0), (7, 2, 8, 0, 0), (509, 2, 8, 0, 0), (33, 3, 7, 1, 1), (64, 4, 16, 0, 0),
    (1000, 1, 31, 0, 0), (300, 8, 32, 8, 0), (1021, 4, 61, 0, 0), (2000, 6, 64, 0, 0), (100, 2, 65, 0, 1), (3001, 8, 128, 0, 0),
    (777, 5, 160, 0, 0), (40, 8, 256, 4, 0), (9001, 8, 256, 0, 0), (200, 8, 257, 0, 0), (500, 8, 384, 0, 0), (611, 7, 512, 0, 0), (50, 3, 511, 1, 0),
    (90, 64, 600, 0, 0), (130, 8, 1000, 0, 0), (70, 8, 1024, 8, 0), (30, 2, 1025, 0, 0), (77, 4, 2048, 0, 0), (20, 8, 4095, 0, 0), (65, 8, 4096, 0, 0),
    (20011, 2, 12, 0, 0), (70001, 1, 4, 0, 0),
])
def test_loss_counts_and_gradient(T, K, E, pad, shift, dtype):
    g = _gen(T + E)
    logits, ids = _case(g, T, K, E, dtype, pad=pad, shift=shift)
    _check(logits, ids, 256.0 if dtype == F16 else 0.01)
    _check(logits, ids.int(), -3.0)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_a_balanced_router_has_the_loss_one(dtype):
    """Equal logits and choices dealt out in turn."""
    ids = torch.arange(640, device="cuda").view(320, 2) % 16
    loss, counts, _ = _check(torch.zeros(320, 16, device="cuda", dtype=dtype), ids)
    assert float(loss) == 1.0 and counts.tolist() == [40] * 16 + [320]


def test_nothing_routed():
    logits = torch.full((30, 8), float("nan"), device="cuda")
    ids = torch.full((30, 2), -1, device="cuda")
    loss, counts = bm.expert_balance(logits, ids)
    assert float(loss) == 0.0 and not counts.any()
    assert not bm.expert_balance_backward(torch.ones((), device="cuda"), logits, ids, counts).any()
    loss, counts = bm.expert_balance(logits[:0], ids[:0])
    assert float(loss) == 0.0 and not counts.any()
    assert bm.expert_balance_backward(torch.ones((), device="cuda"), logits[:0], ids[:0], counts).shape == (0, 8)


@pytest.mark.parametrize("E", [8, 61, 256, 700, 1500])
@pytest.mark.parametrize("dtype", [F32, F16, BF16])
def test_masked_experts_and_rows_of_padding(E, dtype):
    """Experts switched off by -inf, rows that are all switched off, the
    type's lowest value, and rows of padding that hold anything."""
    g = _gen(E)
    logits, ids = _case(g, 97, 2, E, dtype, empty=0.0)
    logits = logits.clone()
    logits[:, ::3] = float("-inf")
    logits[5] = float("-inf")
    logits[6] = torch.finfo(dtype).min
    logits[7, 1:] = torch.finfo(dtype).min
    ids[11:14] = -1
    logits[11], logits[12], logits[13] = float("nan"), float("inf"), float("-inf")
    seen = logits.clone()
    seen[11:14] = 0
    loss, counts, _ = _check(seen, ids)
    got, got_counts = bm.expert_balance(logits, ids)
    by = torch.ones((), device="cuda")
    assert torch.equal(got, loss) and torch.equal(got_counts, counts)
    grad = bm.expert_balance_backward(by, logits, ids, counts)
    assert torch.equal(grad, bm.expert_balance_backward(by, seen, ids, counts))
    assert not grad[5].any() and not grad[11:14].any()


@pytest.mark.parametrize("E", [8, 200, 1500])
@pytest.mark.parametrize("value", ["nan", "inf"])
def test_a_bad_logit_shows(E, value):
    g = _gen(E)
    logits, ids = _case(g, 40, 2, E, F32, empty=0.0)
    logits = logits.clone()
    logits[3, E // 2] = float(value)
    loss, counts = bm.expert_balance(logits, ids)
    assert bool(loss.isnan())
    grad = bm.expert_balance_backward(torch.ones((), device="cuda"), logits, ids, counts)
    assert bool(grad[3].isnan().any()) and torch.isfinite(grad[:3]).all() and torch.isfinite(grad[4:]).all()


def test_gradient_by_differences():
    """Central differences of the definition in 64 bits, whose third
    derivative (below 10 here) leaves h**2 * 10 / 6, and whose rounding
    1e-16 / h."""
    g = _gen(1)
    logits, ids = _case(g, 6, 2, 5, F32, empty=0.2)
    _, counts = bm.expert_balance(logits, ids)
    grad = bm.expert_balance_backward(torch.ones((), device="cuda"), logits, ids, counts).double()
    h, x = 1e-4, logits.double()
    bound = _definition(x, ids)[4] + ROUND[F32] * grad.abs() + 4 * U32 * grad.abs()
    for t in range(6):
        for e in range(5):
            up, down = x.clone(), x.clone()
            up[t, e] += h
            down[t, e] -= h
            slope = float(_definition(up, ids)[0] - _definition(down, ids)[0]) / (2 * h)
            assert abs(slope - float(grad[t, e])) <= float(bound[t, e]) + h * h * 10 / 6 + 1e-15 / h


def test_rows_that_share_memory_and_rows_apart():
    g = _gen(2)
    row, ids = torch.randn(1, 24, generator=g, device="cuda"), torch.randint(0, 24, (300, 2), generator=g, device="cuda")
    loss, counts, grad = _check(row.expand(300, 24), ids)
    wide = torch.full((300, 40), 7.0, device="cuda")
    out = bm.expert_balance_backward(torch.ones((), device="cuda"), row.expand(300, 24), ids, counts, out=wide[:, 8:32])
    assert out.data_ptr() == wide[:, 8:].data_ptr() and torch.equal(wide[:, 8:32], grad)
    assert bool((wide[:, :8] == 7).all()) and bool((wide[:, 32:] == 7).all())


def test_a_large_batch():
    g = _gen(9)
    logits, ids = _case(g, 300007, 8, 64, BF16, empty=0.02, ids=torch.int32)
    _check(logits, ids, 0.01)


def test_captured_and_replayed_on_two_streams():
    g = _gen(4)
    cases = [_case(g, 4001, 4, 60, F32) for _ in range(2)]
    by = torch.full((), 0.5, device="cuda")

    def both(c, **kw):
        loss, counts = bm.expert_balance(*c, **kw)
        return loss, counts, bm.expert_balance_backward(by, *c, counts, **kw)

    want = [[x.clone() for x in both(c)] for c in cases]
    held = [x.clone() for x in cases[0]]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = both(held)
    for c, w in zip(cases, want):
        for a, b in zip(held, c):
            a.copy_(b)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, w))
    streams, outs = [torch.cuda.Stream() for _ in range(2)], []
    for _ in range(20):
        outs += [both(c, stream=st) for c, st in zip(cases, streams)]
    torch.cuda.synchronize()
    for i, o in enumerate(outs):
        assert all(torch.equal(a, b) for a, b in zip(o, want[i % 2]))
