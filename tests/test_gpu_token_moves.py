"""The token moves (expert_sort, expert_dispatch, expert_combine and its
gradient, rotary, paged_append) on the GPU against their definitions in 64
bits.

Maps and pure moves are compared exactly.  Computed values have a bound from
the definition: products and sums in 32 bits (unit roundoff 2**-24 for each
operation, in any order), the 2 ulp of CUDA's sinf and cosf, and one rounding
to the result's type.
"""

import numpy as np
import pytest

import bmmc_index_transforms_gb300 as bm

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16
U32 = 2.0 ** -24
ROUND = {F32: 2.0 ** -24, F16: 2.0 ** -11, BF16: 2.0 ** -8}   # relative, to nearest
TINY = {F32: 2.0 ** -149, F16: 2.0 ** -24, BF16: 2.0 ** -133}  # absolute, where results are subnormal


def _gen(seed):
    g = torch.Generator("cuda")
    g.manual_seed(seed)
    return g


def _randn(g, *shape, dtype=F32):
    return torch.randn(*shape, generator=g, device="cuda").to(dtype)


def _within(got, want, bound, dtype):
    """|got - want| <= bound + one rounding to dtype, everywhere."""
    got = got.double()
    limit = bound + ROUND[dtype] * (want.abs() + bound) + TINY[dtype]
    off = (got - want).abs()
    assert torch.isfinite(got).all()
    assert bool((off <= limit).all()), f"off by up to {float((off - limit).max())} more than the bound"


# ---- sort --------------------------------------------------------------------

def _sorted_by_definition(ids, experts):
    flat = ids.reshape(-1).astype(object) if ids.dtype == object else ids.reshape(-1)
    key = np.where((flat >= 0) & (flat < experts), flat, experts)
    order = np.argsort(key, kind="stable")
    slot = np.empty(flat.size, dtype=np.int64)
    slot[order] = np.arange(flat.size)
    slot = np.where(key < experts, slot, ~slot)
    source = np.where(key[order] < experts, order, ~order)
    offsets = np.array([np.count_nonzero(key < e) for e in range(experts + 1)])
    return slot.reshape(ids.shape), source, offsets


def _check_sort(ids, experts):
    slot, source, offsets = bm.expert_sort(ids, experts)
    want = _sorted_by_definition(ids.cpu().numpy(), experts)
    for got, w, name in zip((slot, source, offsets), want, ("slot", "source", "offsets")):
        assert got.dtype == torch.int32
        assert np.array_equal(got.cpu().numpy(), w), name


@pytest.mark.parametrize("dtype", [torch.int32, torch.int64])
@pytest.mark.parametrize("tokens,choices,experts", [
    (0, 2, 3), (1, 1, 1), (1, 8, 8), (31, 1, 5), (33, 3, 7), (48, 8, 128), (1024, 8, 1), (1024, 8, 256), (1025, 8, 256),
    (777, 5, 4096), (9001, 6, 300), (4096, 2, 2048), (70001, 8, 257), (262147, 4, 3), (600, 64, 511),
])
def test_sort(tokens, choices, experts, dtype):
    g = _gen(tokens + choices)
    ids = torch.randint(-1, experts + 1, (tokens, choices), generator=g, device="cuda", dtype=dtype)
    _check_sort(ids, experts)


@pytest.mark.parametrize("tokens", [1024, 1025, 4096, 4097, 8191, 20000, 32768, 32769, 40961])
@pytest.mark.parametrize("experts", [3, 200, 1024, 4096])
def test_sort_around_the_sizes_of_tiles(tokens, experts):
    g = _gen(tokens + experts)
    ids = torch.randint(0, experts, (tokens, 1), generator=g, device="cuda")
    ids[torch.rand(tokens, 1, generator=g, device="cuda") < 0.1] = -1
    _check_sort(ids, experts)


@pytest.mark.parametrize("tokens", [5, 2000, 40000])
def test_sort_one_sided(tokens):
    """Every choice the same expert, none routed, and an expert without any."""
    for value in (0, 6, 7, -1, 99):
        _check_sort(torch.full((tokens, 3), value, dtype=torch.int32, device="cuda"), 7)
    ids = torch.arange(tokens * 3, device="cuda").view(tokens, 3) % 7
    _check_sort(torch.where(ids == 3, 4, ids), 7)


def test_sort_wide_ids():
    """64-bit ids whose low 32 bits name an expert are not routed."""
    ids = torch.tensor([[2**32 + 1, 1], [-(2**32) + 2, 2], [2**63 - 1, -(2**63)], [0, 3]], device="cuda")
    _check_sort(ids, 4)


# ---- dispatch, combine and their gradients ------------------------------------

def _routing(g, tokens, choices, experts, out=0.2):
    """slot of random choices, some of them and one token's whole row not routed."""
    ids = torch.randint(0, experts, (tokens, choices), generator=g, device="cuda")
    ids[torch.rand(tokens, choices, generator=g, device="cuda") < out] = -1
    if tokens > 2:
        ids[tokens // 2] = -1
    return bm.expert_sort(ids, experts)[0]


def _picked(slot, num_rows):
    """(routed and kept, row) of every choice."""
    row = torch.where(slot >= 0, slot, ~slot).long()
    return (slot >= 0) & (row < num_rows), row


SHAPES = [(1, 1, 1), (1, 8, 4096), (3, 2, 7), (17, 4, 64), (64, 8, 1030), (33, 6, 2048), (130, 1, 5120), (9, 64, 136),
          (5, 3, 16400), (300, 2, 33), (513, 5, 72)]


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("tokens,choices,hidden", SHAPES)
def test_dispatch(tokens, choices, hidden, dtype):
    g = _gen(hidden)
    slot = _routing(g, tokens, choices, 5)
    x = _randn(g, tokens, hidden, dtype=dtype)
    for num_rows in {tokens * choices, tokens * choices // 2, 0}:
        got = bm.expert_dispatch(x, slot, num_rows)
        keep, row = _picked(slot, num_rows)
        want = torch.zeros(num_rows, hidden, dtype=dtype, device="cuda")
        want[row[keep]] = x[:, None].expand(-1, choices, -1)[keep]
        assert torch.equal(got, want)


def _combine64(rows, slot, weights, num_rows):
    """(result, sum of the terms' magnitudes)"""
    keep, row = _picked(slot, num_rows)
    w = torch.ones_like(slot, dtype=torch.float64) if weights is None else weights.double()
    terms = torch.zeros(*slot.shape, rows.shape[1], dtype=torch.float64, device="cuda")
    terms[keep] = w[keep][:, None] * rows[row[keep]].double()
    return terms.sum(1), terms.abs().sum(1)


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("weight", ["none", "f32", "rows"])
@pytest.mark.parametrize("tokens,choices,hidden", SHAPES)
def test_combine(tokens, choices, hidden, weight, dtype):
    g = _gen(hidden + 1)
    slot = _routing(g, tokens, choices, 5)
    n = tokens * choices
    rows = _randn(g, n, hidden, dtype=dtype)
    w = None if weight == "none" else torch.rand(tokens, choices, generator=g, device="cuda").to(
        F32 if weight == "f32" else dtype)
    for num_rows in {n, (n + 1) // 2}:
        got = bm.expert_combine(rows[:num_rows], slot, w)
        want, size = _combine64(rows, slot, w, num_rows)
        _within(got, want, (choices + 1) * U32 * size, dtype)
        empty = ~_picked(slot, num_rows)[0].any(1)
        assert not got[empty].any()


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("weight", ["f32", "rows"])
@pytest.mark.parametrize("tokens,choices,hidden", SHAPES)
def test_combine_backward(tokens, choices, hidden, weight, dtype):
    g = _gen(hidden + 2)
    slot = _routing(g, tokens, choices, 5)
    n = tokens * choices
    rows, grad = _randn(g, n, hidden, dtype=dtype), _randn(g, tokens, hidden, dtype=dtype)
    w = torch.rand(tokens, choices, generator=g, device="cuda").to(F32 if weight == "f32" else dtype)
    for num_rows in {n, (n + 1) // 2}:
        grad_rows, grad_w = bm.expert_combine_backward(grad, rows[:num_rows], slot, w)
        keep, row = _picked(slot, num_rows)
        want = torch.zeros(num_rows, hidden, dtype=torch.float64, device="cuda")
        want[row[keep]] = (w.double()[..., None] * grad.double()[:, None])[keep]
        _within(grad_rows, want, U32 * want.abs(), dtype)
        products = torch.zeros(tokens, choices, hidden, dtype=torch.float64, device="cuda")
        products[keep] = rows[row[keep]].double() * grad.double()[:, None].expand(-1, choices, -1)[keep]
        _within(grad_w, products.sum(2), (hidden + 1) * U32 * products.abs().sum(2), w.dtype)
        assert not grad_w[~keep].any()


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("tokens,choices,hidden,pad,shift", [
    (700, 2, 4095, 0, 0), (700, 2, 4096, 0, 0), (700, 1, 4092, 8, 0), (1300, 3, 2050, 1, 1), (300, 8, 4093, 0, 3), (5000, 2, 1031, 2, 0),
    (5000, 4, 516, 0, 0), (200, 2, 12345, 0, 1), (6000, 9, 515, 0, 0), (2500, 7, 1025, 3, 2),
])
def test_large_calls_of_rows_that_lie_anyhow(tokens, choices, hidden, pad, shift, dtype):
    """Rows of any width, alignment and gap in calls that fill the machine,
    some choices not routed or dropped: dispatch, combine and its gradient."""
    g = _gen(hidden + pad)
    slot = _routing(g, tokens, choices, 11)
    n = tokens * choices

    def spread(k, values=None):
        base = torch.full((k * (hidden + pad) + shift + 8,), 5.0, dtype=dtype, device="cuda")
        view = base[shift:shift + k * (hidden + pad)].view(k, hidden + pad)[:, :hidden]
        if values is not None:
            view.copy_(values)
        return base, view

    x, rows = _randn(g, tokens, hidden, dtype=dtype), _randn(g, n, hidden, dtype=dtype)
    w = torch.rand(tokens, choices, generator=g, device="cuda")
    xs, rs = spread(tokens, x)[1], spread(n, rows)[1]
    for num_rows in (n, n - n // 3):
        keep, row = _picked(slot, num_rows)
        base, out = spread(num_rows)
        bm.expert_dispatch(xs, slot, num_rows, out=out)
        want = torch.zeros(num_rows, hidden, dtype=dtype, device="cuda")
        want[row[keep]] = x[:, None].expand(-1, choices, -1)[keep]
        assert torch.equal(out, want)
        out.fill_(5.0)
        assert bool((base == 5.0).all())
        base, out = spread(tokens)
        bm.expert_combine(rs[:num_rows], slot, w, out=out)
        want, size = _combine64(rows, slot, w, num_rows)
        _within(out, want, (choices + 1) * U32 * size, dtype)
        out.fill_(5.0)
        assert bool((base == 5.0).all())
        grad_rows, grad_w = bm.expert_combine_backward(xs, rs[:num_rows], slot, w)
        want = torch.zeros(num_rows, hidden, dtype=torch.float64, device="cuda")
        want[row[keep]] = (w.double()[..., None] * x.double()[:, None])[keep]
        _within(grad_rows, want, U32 * want.abs(), dtype)
        products = torch.zeros(tokens, choices, hidden, dtype=torch.float64, device="cuda")
        products[keep] = rows[row[keep]].double() * x.double()[:, None].expand(-1, choices, -1)[keep]
        _within(grad_w, products.sum(2), (hidden + 1) * U32 * products.abs().sum(2), F32)
        assert not grad_w[~keep].any()


def test_gradients_against_differences():
    """combine is linear in the rows and in the weights, so a difference of
    two results over a step is the gradient up to rounding."""
    g = _gen(5)
    T, K, H = 11, 3, 24
    slot = _routing(g, T, K, 4)
    rows, grad = _randn(g, T * K, H), _randn(g, T, H)
    w = torch.rand(T, K, generator=g, device="cuda")
    grad_rows, grad_w = bm.expert_combine_backward(grad, rows, slot, w)
    loss = lambda r, u: float((bm.expert_combine(r, slot, u).double() * grad.double()).sum())  # noqa: E731
    size = float((_combine64(rows, slot, w, T * K)[1] * grad.double().abs()).sum())
    # two losses, each off by (K + 2) roundings of its terms, over a step of 1
    bound = 2 * (K + 2) * U32 * (size + 8 * H)
    at = loss(rows, w)
    for i in range(0, T * K, 4):
        t, k = divmod(i, K)
        u = w.clone()
        u[t, k] += 1.0
        assert abs(loss(rows, u) - at - float(grad_w[t, k])) <= bound
        r = rows.clone()
        r[i, i % H] += 1.0
        assert abs(loss(r, w) - at - float(grad_rows[i, i % H])) <= bound
    # dispatch: x -> rows; its gradient by x is the plain sum
    x, gr = _randn(g, T, H), _randn(g, T * K, H)
    gx = bm.expert_combine(gr, slot)
    loss = lambda v: float((bm.expert_dispatch(v, slot).double() * gr.double()).sum())  # noqa: E731
    at, bound = loss(x), 4 * U32 * float((x.abs().sum() + 8 * H) * 8)
    for t in range(T):
        y = x.clone()
        y[t, t % H] += 1.0
        assert abs(loss(y) - at - float(gx[t, t % H])) <= bound


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("hidden,pad,shift", [(64, 8, 0), (64, 3, 0), (63, 1, 1), (40, 0, 1), (2050, 6, 2)])
def test_strided_rows(hidden, pad, shift, dtype):
    """Rows with gaps and any alignment: the same values as dense ones, the
    gaps kept."""
    g = _gen(9)
    T, K = 21, 3
    slot = _routing(g, T, K, 4)
    w = torch.rand(T, K, generator=g, device="cuda")

    def spread(n, fill):
        base = torch.full((n * (hidden + pad) + shift + 8,), fill, dtype=dtype, device="cuda")
        return base, base[shift:shift + n * (hidden + pad)].view(n, hidden + pad)[:, :hidden]

    x, rows = _randn(g, T, hidden, dtype=dtype), _randn(g, T * K, hidden, dtype=dtype)
    xs, rs = spread(T, 9.0)[1], spread(T * K, 9.0)[1]
    xs.copy_(x)
    rs.copy_(rows)
    for inp, n, call in ((xs, T * K, lambda out: bm.expert_dispatch(xs, slot, out=out)),
                         (rs, T, lambda out: bm.expert_combine(rs, slot, w, out=out))):
        base, out = spread(n, 7.0)
        call(out)
        dense = bm.expert_dispatch(x, slot) if inp is xs else bm.expert_combine(rows, slot, w)
        assert torch.equal(out, dense)
        out.fill_(7.0)
        assert bool((base == 7.0).all())
    a, b = bm.expert_combine_backward(xs, rs, slot, w), bm.expert_combine_backward(x, rows, slot, w)
    assert torch.equal(a[0], b[0])
    # the sums run over other words: the bound of two sums in 32 bits
    size = (rows.abs().double().sum(1).max() * x.abs().double().max())
    assert float((a[1] - b[1]).abs().max()) <= 2 * (hidden + 1) * U32 * float(size)


def test_broadcast_rows():
    g = _gen(10)
    slot = _routing(g, 40, 4, 4)
    x = _randn(g, 1, 72, dtype=BF16)
    assert torch.equal(bm.expert_dispatch(x.expand(40, 72), slot), bm.expert_dispatch(x.repeat(40, 1), slot))
    w = torch.rand(40, 4, generator=g, device="cuda")
    rows = _randn(g, 160, 72, dtype=BF16)
    a, b = (bm.expert_combine_backward(v, rows, slot, w) for v in (x.expand(40, 72), x.repeat(40, 1)))
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    assert torch.equal(bm.expert_combine(x.expand(160, 72), slot, w), bm.expert_combine(x.repeat(160, 1), slot, w))


def test_rows_that_are_not_routed_are_not_read():
    """NaN and infinities in rows of choices that are not routed, and in
    weights there, reach no result."""
    g = _gen(11)
    T, K, H = 30, 4, 200
    slot = _routing(g, T, K, 3, out=0.5)
    keep, row = _picked(slot, T * K)
    rows, grad, w = _randn(g, T * K, H), _randn(g, T, H), torch.rand(T, K, generator=g, device="cuda")
    clean = (bm.expert_combine(rows, slot, w), *bm.expert_combine_backward(grad, rows, slot, w))
    rows[row[~keep]] = float("nan")
    w[~keep] = float("inf")
    grad[T // 2] = float("nan")  # a token without any routed choice
    dirty = (bm.expert_combine(rows, slot, w), *bm.expert_combine_backward(grad, rows, slot, w))
    for a, b in zip(clean, dirty):
        assert torch.equal(a, b)


def test_infinities_and_nan_pass_through_where_they_are_routed():
    slot = torch.tensor([[0, 1], [2, 3]], dtype=torch.int32, device="cuda")
    rows = torch.tensor([[float("inf")], [1.0], [float("nan")], [2.0]], device="cuda")
    out = bm.expert_combine(rows, slot, torch.ones(2, 2, device="cuda"))
    assert float(out[0]) == float("inf") and torch.isnan(out[1]).all()
    big = torch.full((2, 8), 60000.0, dtype=F16, device="cuda")  # a sum above the type's range
    assert torch.isinf(bm.expert_combine(big, torch.tensor([[0, 1]], dtype=torch.int32, device="cuda"))).all()


def test_maps_that_name_no_row():
    """Entries beyond the rows move nothing and read nothing."""
    T, K, H = 4, 2, 40
    top = 2**31 - 1
    slot = torch.tensor([[0, top], [~top, 1], [8, -(2**31)], [~8, 7]], dtype=torch.int32, device="cuda")
    x = torch.ones(T, H, device="cuda")
    out = torch.full((T * K, H), 5.0, device="cuda")
    bm.expert_dispatch(x, slot, out=out)
    assert out[:, 0].tolist() == [1, 1, 5, 5, 5, 5, 5, 1]
    assert bm.expert_combine(out, slot)[:, 0].tolist() == [1, 1, 0, 1]
    grad_rows, grad_w = bm.expert_combine_backward(x, out, slot, torch.ones(T, K, device="cuda"))
    assert grad_w.tolist() == [[H, 0], [0, H], [0, 0], [0, H]]


def test_offsets_beyond_32_bits():
    T, K, H = 150000, 4, 4096  # 2.46e9 elements, 4.9 GB
    slot = torch.arange(T * K, dtype=torch.int32, device="cuda").flip(0).view(T, K)
    x = (torch.arange(T, device="cuda") % 251).to(BF16)[:, None].expand(T, H).contiguous()
    rows = bm.expert_dispatch(x, slot)
    want = (torch.arange(T * K, device="cuda").flip(0) // K % 251).to(BF16)
    for column in (0, 1, H - 1):
        assert torch.equal(rows[:, column], want)
    out = bm.expert_combine(rows, slot)
    want = 4 * (torch.arange(T, device="cuda") % 251).double()
    _within(out[:, H - 1], want, 0.0, BF16)
    del out
    grad_rows, grad_w = bm.expert_combine_backward(x, rows, slot, torch.ones(T, K, device="cuda"))
    assert torch.equal(grad_rows[::997], rows[::997]) and torch.equal(grad_rows[-9:], rows[-9:])
    # whole numbers below 2**24 * 16 in sums of 4096 equal terms
    d = (torch.arange(T, device="cuda") % 251).double()
    _within(grad_w[:, 3], d * d * H, (H + 1) * U32 * d * d * H, F32)


# ---- rotary ------------------------------------------------------------------

def _turn64(x, positions, freq, pair_axes, interleaved, inverse=False):
    """(result, |a| + |b| of each element's pair): the angle is the product in
    32 bits, the rest in 64."""
    P = freq.numel()
    axis = torch.zeros(P, dtype=torch.long, device="cuda") if pair_axes is None else pair_axes.long()
    there = (axis >= 0) & (axis < positions.shape[0])
    at = torch.where(there[:, None], positions[axis.clamp(0, positions.shape[0] - 1)], 0).t()
    angle = (at.float() * freq).double()[:, None] * (-1 if inverse else 1)
    c, s, y, size = torch.cos(angle), torch.sin(angle), x.double().clone(), torch.zeros_like(x, dtype=torch.float64)
    i, j = (slice(0, 2 * P, 2), slice(1, 2 * P, 2)) if interleaved else (slice(0, P), slice(P, 2 * P))
    a, b = y[..., i].clone(), y[..., j].clone()
    y[..., i], y[..., j] = a * c - b * s, b * c + a * s
    size[..., i] = size[..., j] = a.abs() + b.abs()
    return y, size


TURN = 8 * U32  # 2 ulp of sine and cosine, the products' and the sum's roundings


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("tokens,heads,dim,pairs,axes", [
    (1, 1, 2, 1, 1), (1, 32, 128, 64, 1), (7, 3, 10, 3, 1), (65, 16, 64, 32, 1), (130, 2, 80, 40, 3), (33, 5, 96, 32, 3),
    (9, 4, 66, 33, 2), (1000, 8, 128, 64, 3), (3, 1, 8192, 4096, 2), (700, 2, 256, 20, 1), (40000, 1, 32, 16, 2),
    (5, 70, 12, 2, 2), (2000, 24, 72, 36, 3),
])
def test_rotary(tokens, heads, dim, pairs, axes, interleaved, dtype):
    g = _gen(dim + pairs)
    x = _randn(g, tokens, heads, dim, dtype=dtype)
    freq = 10000.0 ** (-torch.arange(pairs, device="cuda") / pairs)
    positions = torch.randint(0, 131072, (axes, tokens), generator=g, device="cuda")
    positions[:, 0] = 0
    pair_axes = None if axes == 1 else torch.randint(-1, axes + 1, (pairs,), generator=g, device="cuda", dtype=torch.int32)
    for inverse in (False, True):
        want, size = _turn64(x, positions, freq, pair_axes, interleaved, inverse)
        for p in (positions, positions.int()):
            got = bm.rotary(x, p if axes > 1 else p[0], freq, pair_axes, interleaved=interleaved, inverse=inverse)
            _within(got, want, TURN * size, dtype)
            assert torch.equal(got[..., 2 * pairs:], x[..., 2 * pairs:])
            assert torch.equal(got[0], x[0])  # position 0


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("tokens,heads,dim,pairs", [
    (1, 1, 16, 1), (3, 5, 128, 37), (6000, 3, 128, 37), (5000, 1, 24, 11), (70, 40, 64, 3), (33, 2, 512, 255), (9, 3, 520, 131),
    (4, 2, 1024, 509), (5, 2, 1032, 3), (777, 9, 96, 25), (20000, 2, 8, 3),
])
def test_rotary_pairs_across_words(tokens, heads, dim, pairs, interleaved, dtype):
    """Rows that allow wide words and pairs that do not lie in them; dense and
    as slices, out of place, head-major and in place."""
    g = _gen(dim + pairs)
    fused = _randn(g, tokens, heads + 1, dim, dtype=dtype)
    x = fused[:, 1:]
    freq = 1000.0 ** (-torch.arange(pairs, device="cuda") / pairs)
    at = torch.randint(-9, 4096, (2, tokens), generator=g, device="cuda")
    axes = (torch.arange(pairs, device="cuda") % 3).int()  # one axis that is not there
    want, size = _turn64(x, at, freq, axes, interleaved)
    got = bm.rotary(x, at, freq, axes, interleaved=interleaved)
    _within(got, want, TURN * size, dtype)
    assert torch.equal(got[..., 2 * pairs:], x[..., 2 * pairs:])
    out = torch.empty(heads, tokens, dim, dtype=dtype, device="cuda").transpose(0, 1)
    assert torch.equal(bm.rotary(x.contiguous(), at, freq, axes, interleaved=interleaved, out=out), got)
    keep = fused[:, 0].clone()
    bm.rotary(x, at, freq, axes, interleaved=interleaved, out=x)
    assert torch.equal(x, got) and torch.equal(fused[:, 0], keep)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("dim,offset", [(64, 0), (64, 1), (36, 0), (35, 3)])
def test_rotary_views(dim, offset, dtype, interleaved):
    """Slices of a fused projection, head-major outputs, in place: the values
    of the dense call."""
    g = _gen(dim)
    T, H, pairs = 50, 6, 16
    fused = _randn(g, T, (H + 4) * dim + 5, dtype=dtype)
    x = fused[:, offset:offset + H * dim].view(T, H, dim)
    freq = 1.0 / (1 + torch.arange(pairs, device="cuda").float())
    at = torch.randint(-5, 3000, (T,), generator=g, device="cuda")
    want = bm.rotary(x.contiguous(), at, freq, interleaved=interleaved)
    assert torch.equal(bm.rotary(x, at, freq, interleaved=interleaved), want)
    out = torch.empty(H, T, dim, dtype=dtype, device="cuda").transpose(0, 1)
    assert torch.equal(bm.rotary(x, at, freq, interleaved=interleaved, out=out), want)
    assert torch.equal(bm.rotary(out, at, freq, interleaved=interleaved), bm.rotary(want, at, freq, interleaved=interleaved))
    keep = fused.clone()
    bm.rotary(x, at, freq, interleaved=interleaved, out=x)
    assert torch.equal(x, want)
    fused[:, offset:offset + H * dim] = keep[:, offset:offset + H * dim]
    assert torch.equal(fused, keep)


def test_rotary_gradient_against_differences():
    g = _gen(3)
    T, H, D, pairs = 6, 2, 10, 4
    x, grad = _randn(g, T, H, D), _randn(g, T, H, D)
    freq = torch.rand(pairs, generator=g, device="cuda")
    at = torch.randint(0, 500, (2, T), generator=g, device="cuda")
    axes = torch.tensor([0, 1, 1, 0], dtype=torch.int32, device="cuda")
    for interleaved in (False, True):
        call = lambda v, **kw: bm.rotary(v, at, freq, axes, interleaved=interleaved, **kw)  # noqa: E731
        back = call(grad, inverse=True)
        loss = lambda v: float((call(v).double() * grad.double()).sum())  # noqa: E731
        bound = 2 * TURN * 2 * float((x.abs().sum() + 1) * grad.abs().max())
        base = loss(x)
        for i in range(0, T * H * D, 7):
            y = x.clone()
            y.view(-1)[i] += 1.0
            assert abs(loss(y) - base - float(back.reshape(-1)[i])) <= bound


# ---- append to a paged cache ---------------------------------------------------

def _append_case(g, B, counts, page, Hq, Hk, Dk, Dv, dtype, head_major, cached, spare=3):
    """Inputs of an append whose sequences have counts[b] new tokens."""
    counts = torch.tensor(counts, device="cuda")
    T = int(counts.sum())
    starts = torch.cat([counts.new_zeros(1), counts.cumsum(0)]).int()
    lengths = torch.randint(0, cached + 1, (B,), generator=g, device="cuda").int()
    need = (lengths + counts + page - 1) // page
    columns = int(need.max()) + 1
    pages = int(need.sum()) + spare
    table = torch.full((B, columns), -1, dtype=torch.int32, device="cuda")
    order = torch.randperm(pages, generator=g, device="cuda").int()
    used = 0
    for b in range(B):
        n = int(need[b])
        table[b, :n] = order[used:used + n]
        used += n
    shape = lambda D: (pages, Hk, page, D) if head_major else (pages, page, Hk, D)  # noqa: E731
    caches = [torch.full(shape(D), 3.0, dtype=dtype, device="cuda") for D in (Dk, Dv)]
    k, v = _randn(g, T, Hk, Dk, dtype=dtype), _randn(g, T, Hk, Dv, dtype=dtype)
    q = _randn(g, T, Hq, Dk, dtype=dtype) if Hq else None
    return dict(k=k, v=v, q=q, starts=starts, lengths=lengths, table=table, caches=caches, page=page, head_major=head_major)


def _append64(c, positions, freq, pair_axes, interleaved):
    """Entries written: (page, slot, token) in order, and the turned keys and
    queries with their bounds' sizes; plain loops over the tokens."""
    starts, lengths, table = c["starts"].tolist(), c["lengths"].tolist(), c["table"].tolist()
    T, pages, page = c["k"].shape[0], c["caches"][0].shape[0], c["page"]
    where, place = [], [0] * T
    for b in range(len(lengths)):
        for t in range(max(0, starts[b]), min(T, starts[b + 1])):
            e = lengths[b] + t - starts[b]
            place[t] = e
            if e // page < len(table[b]) and 0 <= table[b][e // page] < pages:
                where.append((table[b][e // page], e % page, t))
    if positions is None:
        positions = torch.tensor([place], device="cuda")
    if freq is None:
        freq = torch.zeros(1, device="cuda")
    turned = [None if x is None else _turn64(x, positions, freq, pair_axes, interleaved) for x in (c["k"], c["q"])]
    return where, turned


def _check_append(c, freq=None, positions=None, pair_axes=None, interleaved=False, starts=True, **kw):
    before = [m.clone() for m in c["caches"]]
    where, (k64, q64) = _append64(c, positions, freq, pair_axes, interleaved)
    out = bm.paged_append(c["k"], c["v"], *c["caches"], c["table"], c["lengths"], starts=c["starts"] if starts else None,
                          q=c["q"], positions=positions, inv_freq=freq, pair_axes=pair_axes, interleaved=interleaved,
                          head_major=c["head_major"], **kw)
    dtype = c["k"].dtype
    p, s, t = (torch.tensor(v, dtype=torch.long, device="cuda") for v in zip(*where)) if where else \
        (torch.empty(0, dtype=torch.long, device="cuda"),) * 3
    for m, old, want, size in ((c["caches"][0], before[0], *k64), (c["caches"][1], before[1], c["v"].double(), None)):
        seen = m.transpose(1, 2) if c["head_major"] else m
        old = (old.transpose(1, 2) if c["head_major"] else old).clone()
        if size is None:
            assert torch.equal(seen[p, s].double(), want[t])
        else:
            _within(seen[p, s], want[t], TURN * size[t], dtype)
        old[p, s] = seen[p, s]
        assert torch.equal(seen, old), "an entry that no token has was written"
    if c["q"] is None:
        assert out is None
    else:
        _within(out, q64[0], TURN * q64[1], dtype)
    return out


FREQ = {n: 100.0 ** (-np.arange(n, dtype=np.float32) / n) for n in (4, 8, 16, 32, 64)}


def _freq(n):
    return torch.from_numpy(FREQ[n]).cuda()


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("head_major", [False, True])
@pytest.mark.parametrize("B,page,Hq,Hk,Dk,Dv,pairs,cached", [
    (1, 1, 0, 1, 8, 8, 4, 0), (1, 16, 8, 1, 128, 128, 64, 100), (70, 16, 32, 8, 128, 128, 64, 50), (300, 64, 4, 4, 64, 64, 32, 200),
    (5, 3, 6, 3, 20, 12, 8, 9), (17, 100, 2, 2, 36, 34, 16, 150),
])
def test_append_one_token_each(B, page, Hq, Hk, Dk, Dv, pairs, cached, head_major, dtype):
    c = _append_case(_gen(B), B, [1] * B, page, Hq, Hk, Dk, Dv, dtype, head_major, cached)
    _check_append(c, _freq(pairs), starts=False)
    _check_append(c, _freq(pairs), interleaved=True)
    _check_append(c)  # no rotation


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("counts,page,cached", [
    ([5], 16, 0), ([0, 3, 0, 0, 40, 1], 16, 20), ([16, 16, 16], 16, 0), ([33, 0, 129, 7], 1, 5), ([1] * 100 + [0] * 60 + [3] * 100, 7, 30),
    ([2000, 1, 3001], 64, 1000), ([0, 0, 0, 9], 100, 250),
])
def test_append_ragged(counts, page, cached, interleaved, dtype):
    g = _gen(len(counts))
    c = _append_case(g, len(counts), counts, page, 4, 2, 64, 64, dtype, False, cached)
    _check_append(c, _freq(32), interleaved=interleaved)
    T = c["k"].shape[0]
    positions = torch.randint(0, 4096, (3, T), generator=g, device="cuda")
    axes = (torch.arange(16, device="cuda") % 3).int()
    _check_append(c, _freq(16), positions, axes, interleaved)
    _check_append(c, _freq(16), positions.int(), axes, interleaved)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("head_major", [False, True])
@pytest.mark.parametrize("counts,Dk,Dv,pairs", [
    ([1], 64, 64, 5), ([1] * 130, 128, 128, 37), ([30, 0, 7], 96, 32, 25), ([4000, 0, 2100], 64, 72, 31), ([2, 1], 512, 1024, 13),
])
def test_append_pairs_across_words(counts, Dk, Dv, pairs, head_major, interleaved, dtype):
    g = _gen(Dk + pairs)
    c = _append_case(g, len(counts), counts, 16, 6, 2, Dk, Dv, dtype, head_major, 40)
    freq = 100.0 ** (-torch.arange(pairs, device="cuda") / pairs)
    _check_append(c, freq, interleaved=interleaved, starts=max(counts) > 1)
    c["table"][0, 0] = -1
    T = c["k"].shape[0]
    positions = torch.randint(0, 4096, (2, T), generator=g, device="cuda")
    _check_append(c, freq, positions, (torch.arange(pairs, device="cuda") % 2).int(), interleaved)


def test_append_skips_tokens_without_a_page():
    """Pages that are not there, entries beyond the table, tokens outside
    every sequence: nothing is written for them; the queries are turned."""
    g = _gen(1)
    c = _append_case(g, 4, [6, 9, 0, 8], 4, 3, 2, 16, 16, F32, False, 6)
    c["table"][0, 1] = -1
    c["table"][1] = c["caches"][0].shape[0]  # one past the pool
    c["table"][3, 0] = -(2**31)
    c["table"] = c["table"][:, :3]  # rows that are not dense, and fewer entries than sequence 3 needs
    c["lengths"][3] = 6
    _check_append(c, _freq(8))
    c["starts"] += 2  # two tokens before the first sequence, the last ones cut off
    _check_append(c, _freq(8))
    c["starts"] -= 4  # starts before the first token; tokens behind the last sequence
    _check_append(c, _freq(8))
    empty = dict(c, table=c["table"][:, :0])
    _check_append(empty, _freq(8))


def test_append_lengths_that_run_over():
    """Entry numbers near 2**31 need 64 bits and have no page here."""
    c = _append_case(_gen(2), 2, [3, 3], 4, 1, 1, 8, 8, F32, False, 0)
    c["lengths"][:] = torch.tensor([2**31 - 2, -2], dtype=torch.int32)
    before = [m.clone() for m in c["caches"]]
    c["table"][:] = 0
    bm.paged_append(c["k"], c["v"], *c["caches"], c["table"], c["lengths"], starts=c["starts"], inv_freq=_freq(4))
    first = c["caches"][1][0, 0]  # entry 0 of sequence 1 is its third token
    assert torch.equal(first, c["v"][5])
    for m, old in zip(c["caches"], before):
        assert torch.equal(m[0, 1:], old[0, 1:]) and torch.equal(m[1:], old[1:])


def test_append_fused_views():
    """q, k and v as slices of one projection, keys and values in one cache
    allocation, queries in place."""
    g = _gen(4)
    c = _append_case(g, 3, [10, 0, 30], 16, 8, 2, 64, 64, BF16, False, 40)
    T = c["k"].shape[0]
    qkv = _randn(g, T, 12 * 64, dtype=BF16)
    heads = qkv.view(T, 12, 64)
    both = torch.full((c["caches"][0].shape[0], 2, 16, 2, 64), 3.0, dtype=BF16, device="cuda")
    c.update(q=heads[:, :8], k=heads[:, 8:10], v=heads[:, 10:], caches=[both[:, 0], both[:, 1]])
    want = _check_append(c, _freq(32)).clone()
    rest = qkv[:, 8 * 64:].clone()
    got = bm.paged_append(c["k"], c["v"], *c["caches"], c["table"], c["lengths"], starts=c["starts"], q=c["q"], q_out=c["q"],
                          inv_freq=_freq(32))
    assert got.data_ptr() == qkv.data_ptr() and torch.equal(got, want) and torch.equal(qkv[:, 8 * 64:], rest)


def test_append_offsets_beyond_32_bits():
    page, H, D = 16, 8, 256
    pages = 2**32 // (page * H * D) + 10  # over 2**32 elements
    k_cache = torch.zeros(pages, page, H, D, dtype=BF16, device="cuda")
    v_cache = torch.zeros_like(k_cache)
    k, v = torch.ones(2, H, D, dtype=BF16, device="cuda"), torch.full((2, H, D), 2.0, dtype=BF16, device="cuda")
    table = torch.tensor([[pages - 1], [0]], dtype=torch.int32, device="cuda")
    lengths = torch.tensor([15, 3], dtype=torch.int32, device="cuda")
    bm.paged_append(k, v, k_cache, v_cache, table, lengths)
    for m, value in ((k_cache, 1.0), (v_cache, 2.0)):
        assert bool((m[pages - 1, 15] == value).all()) and bool((m[0, 3] == value).all())
        for part in m.split(pages // 16 + 1):
            part = part.clone()
            if part.shape[0] and part[0, 3, 0, 0] != 0:
                part[0, 3] = 0
            if part[-1, 15, 0, 0] != 0:
                part[-1, 15] = 0
            assert not part.any()


def test_append_nothing():
    c = _append_case(_gen(6), 2, [0, 0], 4, 2, 1, 8, 8, F32, False, 3)
    out = _check_append(c, _freq(4))
    assert out.shape == (0, 2, 8)


# ---- streams, graphs, the same bits ----------------------------------------------

def _everything(s):
    slot, source, offsets = bm.expert_sort(s["ids"], 16)
    rows = bm.expert_dispatch(s["x"], slot)
    out = bm.expert_combine(rows, slot, s["w"])
    grads = bm.expert_combine_backward(s["x"], rows, slot, s["w"])
    heads = out.view(-1, 4, 64)
    turned = bm.rotary(heads, s["at"], s["freq"])
    bm.paged_append(turned, heads, *s["caches"], s["table"], s["lengths"], starts=s["starts"], inv_freq=s["freq"])
    return [slot, source, offsets, rows, out, *grads, turned, *s["caches"]]


def _state(T=3000):
    g = _gen(8)
    caches = [torch.zeros(T // 16 + 4, 16, 4, 64, dtype=BF16, device="cuda") for _ in range(2)]
    return dict(ids=torch.randint(-1, 16, (T, 4), generator=g, device="cuda"), x=_randn(g, T, 256, dtype=BF16),
                w=torch.rand(T, 4, generator=g, device="cuda"), at=torch.arange(T, device="cuda"), freq=_freq(32),
                caches=caches, table=torch.arange(T // 16 + 4, device="cuda").int().view(1, -1),
                lengths=torch.tensor([5], device="cuda").int(), starts=torch.tensor([0, T], device="cuda").int())


def test_same_bits_on_other_streams_and_in_graphs():
    s = _state()
    want = [x.clone() for x in _everything(s)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for m in s["caches"]:
        m.zero_()
    with torch.cuda.stream(side):
        side.wait_stream(torch.cuda.default_stream())
        got = _everything(s)
    side.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = _everything(s)
    for x in got:
        x.zero_()
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def test_stream_argument():
    """A call given a stream waits for that stream's work, not the current one's."""
    s = _state(500)
    slot = bm.expert_sort(s["ids"], 16)[0]
    want = bm.expert_dispatch(s["x"], slot)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    x = torch.zeros_like(s["x"])
    out = torch.empty_like(want)
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)
        x.copy_(s["x"])
    bm.expert_dispatch(x, slot, out=out, stream=side)
    side.synchronize()
    assert torch.equal(out, want)


def test_sort_on_a_given_stream_keeps_its_workspace():
    """The workspace of a sort on another stream is not handed out again
    before that stream is done with it."""
    g = _gen(21)
    ids = torch.randint(0, 300, (30000, 4), generator=g, device="cuda")
    want = [x.clone() for x in bm.expert_sort(ids, 300)]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for stream in (side, side.cuda_stream):
        with torch.cuda.stream(side):
            torch.cuda._sleep(20_000_000)
        got = bm.expert_sort(ids, 300, stream=stream)
        for _ in range(50):  # whatever is free on the current stream is written over meanwhile
            torch.full((40 * 304,), -7, dtype=torch.int32, device="cuda")
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)


def test_no_tokens():
    """Calls without any token write nothing and give empty results."""
    slot = torch.empty(0, 4, dtype=torch.int32, device="cuda")
    x = torch.empty(0, 8, device="cuda")
    assert bm.expert_dispatch(x, slot).shape == (0, 8)
    assert bm.expert_combine(x, slot).shape == (0, 8)
    grad_rows, grad_w = bm.expert_combine_backward(x, x, slot, torch.empty(0, 4, device="cuda"))
    assert grad_rows.shape == (0, 8) and grad_w.shape == (0, 4)
    out = bm.rotary(torch.empty(0, 2, 8, device="cuda"), torch.empty(0, dtype=torch.int64, device="cuda"), _freq(4))
    assert out.shape == (0, 2, 8)
    # tokens, but no row that is kept
    slot = bm.expert_sort(torch.zeros(5, 2, dtype=torch.int32, device="cuda"), 3)[0]
    assert not bm.expert_combine(torch.empty(0, 8, device="cuda"), slot).any()
    assert not bm.expert_combine_backward(torch.ones(5, 8, device="cuda"), torch.empty(0, 8, device="cuda"), slot,
                                          torch.ones(5, 2, device="cuda"))[1].any()


def test_pinned_host_memory():
    """The C entry points take pinned host memory, as those of the permutes do."""
    from bmmc_index_transforms_gb300 import _capi

    L = _capi.lib()
    g = _gen(12)
    T, K, H = 37, 3, 136
    ids = torch.randint(-1, 5, (T, K), generator=g, device="cuda", dtype=torch.int32)
    x, w = _randn(g, T, H, dtype=BF16), torch.rand(T, K, generator=g, device="cuda")
    slot = bm.expert_sort(ids, 5)[0]
    rows = bm.expert_dispatch(x, slot)
    host = lambda v: v.cpu().pin_memory()  # noqa: E731
    h_ids, h_x, h_w = host(ids), host(x), host(w)
    new = lambda *s, dtype: torch.zeros(*s, dtype=dtype).pin_memory()  # noqa: E731
    h_slot, h_source, h_offsets = new(T, K, dtype=torch.int32), new(T * K, dtype=torch.int32), new(6, dtype=torch.int32)
    h_rows, h_out = new(T * K, H, dtype=BF16), new(T, H, dtype=BF16)
    st = torch.cuda.current_stream().cuda_stream
    assert L.expert_sort(h_ids.data_ptr(), 4, T, K, 5, h_slot.data_ptr(), h_source.data_ptr(), h_offsets.data_ptr(), None, 0,
                         st) == _capi.OK
    assert L.expert_dispatch(h_x.data_ptr(), H, h_slot.data_ptr(), T, K, H, _capi.BF16, h_rows.data_ptr(), H, T * K,
                             st) == _capi.OK
    assert L.expert_combine(h_rows.data_ptr(), H, T * K, h_slot.data_ptr(), h_w.data_ptr(), _capi.F32, T, K, H, _capi.BF16,
                            h_out.data_ptr(), H, st) == _capi.OK
    at, f = torch.arange(T, device="cuda"), _freq(4)
    h_at, h_f, h_turned = host(at), host(f), new(T, 17, 8, dtype=BF16)
    args = _capi.ROTARY_ARGS.pack(T, _capi.BF16, h_x.data_ptr(), 17, 8, H, 8, h_turned.data_ptr(), 17, 8, H, 8, h_f.data_ptr(),
                                  0, h_at.data_ptr(), 8, 1, 0, 4, 0)
    assert L.rotary(args, st) == _capi.OK
    torch.cuda.synchronize()
    assert torch.equal(h_slot, slot.cpu()) and torch.equal(h_rows, rows.cpu())
    assert torch.equal(h_out, bm.expert_combine(rows, slot, w).cpu())
    assert torch.equal(h_turned, bm.rotary(x.view(T, 17, 8), at, f).cpu())


def test_tensors_elsewhere_are_refused():
    x = torch.zeros(4, 8)
    slot = torch.zeros(4, 2, dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError, match="current device"):
        bm.expert_dispatch(x, slot)
    with pytest.raises(bm.BmmcError, match="overlap"):
        y = torch.zeros(20, 8, device="cuda")
        bm.expert_combine(y[:8], slot, out=y[6:10])
    x = x.cuda()
    with pytest.raises(ValueError, match="shape"):
        bm.expert_dispatch(x, slot, out=x.half())
    h, at, f = torch.zeros(3, 2, 8, device="cuda"), torch.zeros(3, dtype=torch.int32, device="cuda"), torch.zeros(4, device="cuda")
    with pytest.raises(ValueError, match="type"):
        bm.rotary(h, at, f, out=h.half())
    cache, table = torch.zeros(5, 4, 2, 8, device="cuda"), torch.zeros(3, 2, dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError, match="without q"):
        bm.paged_append(h, h, cache, cache.clone(), table, at, q_out=h.clone())


@pytest.mark.parametrize("choices", [2, 5, 8, 9])
@pytest.mark.parametrize("shift", [0, 1, 2])
def test_widest_rows(shift, choices):
    """The largest hidden of 32 bits, in words of 16 and 8 bytes and across
    words: every form's grid holds it."""
    g = _gen(shift)
    T, H = 2, 1 << 24
    n = T * choices
    slot = torch.randperm(n, generator=g, device="cuda").int().view(T, choices)
    base = torch.randint(-8, 9, (n * H + 4,), generator=g, device="cuda", dtype=torch.int8).float()
    rows = base[shift:shift + n * H].view(n, H)
    w = torch.randint(1, 4, (T, choices), generator=g, device="cuda").float()
    want = torch.zeros(T, H, device="cuda")  # whole numbers: exact in 32 bits in any order
    for k in range(choices):
        want += w[:, k, None] * rows[slot[:, k].long()]
    assert torch.equal(bm.expert_combine(rows, slot, w), want)
    got = bm.expert_dispatch(rows[:T], slot)
    for k in range(choices):
        assert torch.equal(got[slot[:, k].long()], rows[:T])
    del got
    grad = base[shift:shift + T * H].view(T, H).sign()
    grad_rows, grad_w = bm.expert_combine_backward(grad, rows, slot, w)
    for k in range(choices):
        row = slot[:, k].long()
        assert torch.equal(grad_rows[row], w[:, k, None] * grad)
        # sums of whole numbers below 2**24 * 8, some of them rounded on the way
        exact = (rows[row].double() * grad.double()).sum(1)
        size = (rows[row].double() * grad.double()).abs().sum(1)
        # a thread adds its 2**24 / 128 products, 32 lanes and 4 warps follow
        _within(grad_w[:, k], exact, (2 ** 17 + 40) * U32 * size, F32)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("counts", [[1] * 70, [0, 130, 7, 40]])
@pytest.mark.parametrize("between", ["pages", "entries", "heads", "elements"])
@pytest.mark.parametrize("head_major", [False, True])
def test_append_to_caches_that_lie_between_each_other(head_major, between, counts, dtype):
    """Keys and values in one allocation, page by page, entry by entry, head
    by head or side by side in a head's row."""
    g = _gen(len(counts))
    for Dk, Dv in ((64, 64), (64, 40), (66, 33)):
        if Dk != Dv and between != "elements":
            continue
        c = _append_case(g, len(counts), counts, 16, 4, 2, Dk, Dv, dtype, head_major, 50)
        pages, a, b, _ = c["caches"][0].shape  # a, b: entries and heads, or heads and entries
        if between == "elements":
            one = torch.full((pages, a, b, Dk + Dv), 3.0, dtype=dtype, device="cuda")
            c["caches"] = [one[..., :Dk], one[..., Dk:]]
        else:
            axis = {"pages": 1, "entries": 3 if head_major else 2, "heads": 2 if head_major else 3}[between]
            shape = [pages, a, b, Dk]
            shape.insert(axis, 2)
            one = torch.full(shape, 3.0, dtype=dtype, device="cuda")
            c["caches"] = [one.select(axis, 0), one.select(axis, 1)]
        _check_append(c, _freq(16), starts=max(counts) > 1)
        _check_append(c, _freq(32), interleaved=True)


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("tokens,choices,hidden,pads,shift", [
    (700, 2, 4095, (0, 0), 0), (700, 1, 4093, (3, 8), 1), (1300, 3, 2050, (1, 0), 1), (300, 8, 4092, (0, 4), 3),
    (300, 8, 4093, (2, 5), 2), (5000, 2, 1031, (2, 2), 0), (200, 2, 12345, (0, 7), 1), (40, 4, 16400, (1, 0), 1),
    (2500, 7, 1025, (3, 0), 2), (6000, 9, 515, (0, 0), 0), (20000, 8, 513, (0, 1), 0), (40000, 2, 260, (0, 0), 0), (700, 2, 4096, (0, 0), 0),
    (400, 8, 4096, (8, 0), 0), (3, 5, 16400, (0, 1), 1), (1, 1, 1, (0, 0), 0), (33, 6, 2047, (0, 0), 3), (9, 64, 131, (1, 0), 0),
])
def test_sums_of_whole_numbers_are_exact(tokens, choices, hidden, pads, shift, dtype):
    """No element of a row is left out or taken twice at a row's ends, where
    the parts of a row or the words of a pack meet: all products are small
    whole numbers other than zero, so that sums in 32 bits are exact in any
    order (below 2**24) and every element counts."""
    g = _gen(hidden + choices)
    slot = _routing(g, tokens, choices, 11)
    n = tokens * choices

    def whole(k, pad):
        v = torch.randint(1, 4, (k * (hidden + pad) + shift,), generator=g, device="cuda")
        v = v * (2 * torch.randint(0, 2, v.shape, generator=g, device="cuda") - 1)
        return v.to(dtype)[shift:].view(k, hidden + pad)[:, :hidden]

    grad, rows = whole(tokens, pads[0]), whole(n, pads[1])
    w = torch.randint(1, 5, (tokens, choices), generator=g, device="cuda").float()
    keep, row = _picked(slot, n)
    want_w, want_rows = torch.zeros_like(w), torch.zeros(n, hidden, device="cuda")
    want = torch.zeros(tokens, hidden, device="cuda")
    for k in range(choices):
        t = keep[:, k].nonzero().flatten()
        picked = rows[row[t, k]].float()
        want_w[t, k] = (picked.double() * grad[t].double()).sum(1).float()
        want_rows[row[t, k]] = w[t, k, None] * grad[t].float()
        want[t] += w[t, k, None] * picked
    assert float(want_w.abs().max()) < 2 ** 24
    for weights in (w, w.to(dtype)):
        grad_rows, grad_w = bm.expert_combine_backward(grad, rows, slot, weights)
        assert torch.equal(grad_w, want_w.to(weights.dtype))
        assert torch.equal(grad_rows, want_rows.to(dtype))
        assert torch.equal(bm.expert_combine(rows, slot, weights), want.to(dtype))
