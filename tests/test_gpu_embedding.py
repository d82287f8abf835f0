"""embedding_lookup and embedding_backward on the GPU against their
definitions in 64 bits.

A lookup is one product in 32 bits and one rounding.  A sum of m rows in 32
bits, in any order, is off by at most (m - 1) * 2**-24 of the sum of the
magnitudes, to first order; the product with the scale adds one rounding, and
so does the sum with what accumulate finds.  Sums of small whole numbers are
exact.
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


def _within(got, want, bound, dtype):
    limit = bound + ROUND[dtype] * (want.abs() + bound) + TINY[dtype]
    off = (got.double() - want).abs()
    assert torch.isfinite(got).all()
    assert bool((off <= limit).all()), f"off by up to {float((off - limit).max())} more than the bound"


def _ids(g, tokens, vocab, kind, dtype=torch.int64):
    """Tokens, some of which name no row."""
    if kind == "one":  # all the same
        ids = torch.full((tokens,), vocab // 2, device="cuda")
    elif kind == "none":
        ids = torch.full((tokens,), -1, device="cuda")
    elif kind == "few":  # runs of every length, long ones among them
        few = torch.randint(0, vocab, (5,), generator=g, device="cuda")
        ids = few[torch.randint(0, 5, (tokens,), generator=g, device="cuda")]
    elif kind == "rare":  # as frequent as words are
        u = torch.rand(tokens, generator=g, device="cuda", dtype=torch.float64)
        ids = (torch.exp(u * float(torch.log(torch.tensor(vocab + 1.0)))) - 1).long().clamp(max=vocab - 1)
    else:
        ids = torch.randint(0, vocab, (tokens,), generator=g, device="cuda")
    if tokens > 3 and kind != "one":
        ids[1], ids[tokens // 2], ids[-1] = -1, vocab, 2**31 - 1
        if dtype == torch.int64:
            ids[2] = 2**32  # whose low half names row 0
    return ids.to(dtype)


def _rows(g, n, hidden, dtype, pad=0, shift=0, whole=False):
    """Rows `pad` elements apart, the first one `shift` elements from an aligned address."""
    x = torch.randn(n * (hidden + pad) + shift, generator=g, device="cuda")
    if whole:
        x = (x * 3).round().clamp(-4, 4)
    return x.to(dtype)[shift:].view(n, hidden + pad)[:, :hidden]


def _named(ids, vocab):
    at = ((ids >= 0) & (ids < vocab)).nonzero().flatten()
    return at, ids[at].long()


SHAPES = [
    # tokens, vocab, hidden, pad, shift
    (1, 1, 1, 0, 0), (1, 3, 8, 0, 0), (2, 5, 4096, 0, 0), (31, 7, 64, 8, 0), (33, 1000, 1031, 0, 0), (500, 300, 1028, 4, 0),
    (257, 50021, 96, 0, 3), (64, 32768, 4096, 0, 0), (777, 100, 12, 0, 1), (100, 9, 4097, 2, 1), (3000, 70000, 20, 0, 0),
]


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("tokens,vocab,hidden,pad,shift", SHAPES)
def test_lookup(tokens, vocab, hidden, pad, shift, dtype):
    g = _gen(hidden)
    table = _rows(g, vocab, hidden, dtype, pad, shift)
    for id_type in (torch.int32, torch.int64):
        ids = _ids(g, tokens, vocab, "any", id_type)
        at, row = _named(ids, vocab)
        for scale in (1.0, 0.125, 45.25):
            want = torch.zeros(tokens, hidden, dtype=torch.float64, device="cuda")
            want[at] = table[row].double() * scale
            got = bm.embedding_lookup(table, ids, scale=scale)
            assert got.dtype == dtype and got.shape == (tokens, hidden)
            _within(got, want, U32 * want.abs(), dtype)
            if scale == 1.0:
                assert torch.equal(got.double(), want)
    # into rows of an array with a stride of its own, whose other elements stay
    wide = torch.full((tokens, hidden + 5), 7.0, dtype=dtype, device="cuda")
    assert bm.embedding_lookup(table, ids, out=wide[:, 2:2 + hidden]).data_ptr() == wide[:, 2:].data_ptr()
    assert torch.equal(wide[:, 2:2 + hidden].double(), torch.zeros(tokens, hidden, device="cuda").double().index_copy(0, at, table[row].double()))
    assert bool((wide[:, :2] == 7).all()) and bool((wide[:, 2 + hidden:] == 7).all())


def test_lookup_of_nothing_and_in_an_empty_table():
    table = torch.randn(4, 8, device="cuda")
    assert bm.embedding_lookup(table, torch.zeros(0, dtype=torch.int64, device="cuda")).shape == (0, 8)
    out = bm.embedding_lookup(table[:0], torch.zeros(3, dtype=torch.int64, device="cuda"))
    assert out.shape == (3, 8) and not out.any()


def test_lookup_rows_that_share_memory():
    row = torch.randn(1, 72, device="cuda")
    got = bm.embedding_lookup(row.expand(5, 72), torch.tensor([4, 0, 5, 2], device="cuda"))
    assert torch.equal(got, torch.where(torch.tensor([1, 1, 0, 1], device="cuda")[:, None] > 0, row, 0))


def test_lookup_keeps_infinities_and_nan_where_they_are():
    table = torch.tensor([[1.0, float("inf")], [float("nan"), 2.0], [3.0, 4.0]], device="cuda")
    got = bm.embedding_lookup(table, torch.tensor([2, -1, 0, 1], device="cuda"), scale=2.0)
    assert got[0].tolist() == [6.0, 8.0] and got[1].tolist() == [0.0, 0.0] and got[2].tolist() == [2.0, float("inf")]
    assert bool(got[3, 0].isnan()) and float(got[3, 1]) == 4.0


def test_offsets_beyond_32_bits():
    vocab, hidden = 140001, 32768  # over 2**32 elements
    table = torch.zeros(vocab, hidden, dtype=BF16, device="cuda")
    table[vocab - 1], table[131072] = 2, 3
    ids = torch.tensor([vocab - 1, 0, 131072, vocab - 1], device="cuda")
    got = bm.embedding_lookup(table, ids)
    for t, value in enumerate((2, 0, 3, 2)):
        assert bool((got[t] == value).all())
    del table
    grad = bm.embedding_backward(got, ids, vocab)
    assert bool((grad[vocab - 1] == 4).all()) and bool((grad[131072] == 3).all())
    grad[vocab - 1] = 0
    grad[131072] = 0
    for part in grad.split(10000):
        assert not part.any()


def _want_backward(grad, ids, vocab, scale):
    at, row = _named(ids, vocab)
    want = torch.zeros(vocab, grad.shape[1], dtype=torch.float64, device="cuda")
    size, m = torch.zeros_like(want), torch.zeros(vocab, 1, dtype=torch.float64, device="cuda")
    want.index_add_(0, row, grad[at].double())
    size.index_add_(0, row, grad[at].double().abs())
    m.index_add_(0, row, torch.ones(at.numel(), 1, dtype=torch.float64, device="cuda"))
    return want * scale, (m + 1) * U32 * size * abs(scale), m[:, 0] > 0


def _check_backward(grad, ids, vocab, scale=1.0):
    want, bound, there = _want_backward(grad, ids, vocab, scale)
    for dtype in {grad.dtype, F32}:
        got = bm.embedding_backward(grad, ids, vocab, scale=scale, dtype=dtype)
        assert got.dtype == dtype and got.shape == want.shape
        _within(got, want, bound, dtype)
        assert not got[~there].any()
        assert torch.equal(got, bm.embedding_backward(grad, ids, vocab, scale=scale, dtype=dtype))  # the same bits
        held = torch.randn(got.shape, device="cuda").to(dtype)
        more = held.clone()
        assert bm.embedding_backward(grad, ids, scale=scale, out=more, accumulate=True) is more
        total = held.double() + want
        _within(more, torch.where(there[:, None], total, held.double()), bound + U32 * (total.abs() + bound), dtype)
        assert torch.equal(more[~there], held[~there])


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("kind", ["any", "rare", "few"])
@pytest.mark.parametrize("tokens,vocab,hidden,pad,shift", SHAPES)
def test_backward(tokens, vocab, hidden, pad, shift, kind, dtype):
    g = _gen(tokens + hidden)
    grad = _rows(g, tokens, hidden, dtype, pad, shift)
    _check_backward(grad, _ids(g, tokens, vocab, kind, torch.int32), vocab)
    _check_backward(grad, _ids(g, tokens, vocab, kind), vocab, 0.75)


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("kind", ["any", "rare", "few", "one", "none"])
@pytest.mark.parametrize("tokens,vocab,hidden", [
    (31, 4, 8), (32, 4, 8), (33, 4, 8), (63, 2, 17), (64, 2, 17), (65, 2, 17), (96, 1, 130), (97, 3, 33), (128, 3, 129),
    (1000, 10, 40), (1024, 2000, 256), (4095, 100, 24), (4096, 100, 24), (4097, 100, 24), (8193, 1500, 16),
    (20000, 131072, 8), (65536, 1023, 8), (65537, 1024, 4), (70001, 1 << 20, 3), (700003, 300, 2),
])
def test_backward_of_whole_numbers_is_exact(tokens, vocab, hidden, kind, dtype):
    """Around the sizes of chunks, tiles and digits: no row is left out or
    taken twice.  16-bit results are held to the rounding of the exact sum."""
    g = _gen(tokens)
    grad = _rows(g, tokens, hidden, dtype, whole=True)
    ids = _ids(g, tokens, vocab, kind)
    at, row = _named(ids, vocab)
    want = torch.zeros(vocab, hidden, dtype=torch.float64, device="cuda").index_add_(0, row, grad[at].double())
    assert torch.equal(bm.embedding_backward(grad, ids, vocab, dtype=F32), want.float())
    got = bm.embedding_backward(grad, ids, vocab, scale=0.5)
    assert torch.equal(got, (want * 0.5).float().to(dtype))
    out = torch.ones(vocab, hidden, device="cuda")
    bm.embedding_backward(grad, ids, out=out, accumulate=True)
    assert torch.equal(out, (want + 1).float())


def test_backward_is_the_transpose_by_differences():
    """<lookup(table + h d) - lookup(table - h d), grad> / 2h = <d, backward(grad)>, on whole numbers."""
    g = _gen(3)
    table, d, grad = (_rows(g, n, 40, F32, whole=True) for n in (50, 50, 300))
    ids = _ids(g, 300, 50, "any")
    h, scale = 2.0, 4.0
    up, down = (bm.embedding_lookup(table + s * h * d, ids, scale=scale) for s in (1, -1))
    left = float(((up - down).double() * grad.double()).sum()) / (2 * h)
    assert left == float((d.double() * bm.embedding_backward(grad, ids, 50, scale=scale).double()).sum())


def test_backward_into_rows_apart():
    g = _gen(4)
    grad, ids = _rows(g, 200, 50, F32, whole=True), _ids(g, 200, 30, "any")
    wide = torch.full((30, 61), 7.0, device="cuda")
    bm.embedding_backward(grad, ids, out=wide[:, 3:53])
    assert torch.equal(wide[:, 3:53], bm.embedding_backward(grad, ids, 30))
    assert bool((wide[:, :3] == 7).all()) and bool((wide[:, 53:] == 7).all())


def test_backward_of_broadcast_rows():
    g = _gen(5)
    ids = _ids(g, 500, 20, "few")
    row = _rows(g, 1, 64, F32, whole=True)
    assert torch.equal(bm.embedding_backward(row.expand(500, 64), ids, 20),
                       bm.embedding_backward(row.expand(500, 64).contiguous(), ids, 20))


def test_backward_of_nothing():
    none = torch.zeros(0, dtype=torch.int64, device="cuda")
    out = torch.ones(5, 8, device="cuda")
    bm.embedding_backward(torch.zeros(0, 8, device="cuda"), none, out=out, accumulate=True)
    assert bool((out == 1).all())
    assert not bm.embedding_backward(torch.zeros(0, 8, device="cuda"), none, out=out).any()
    assert bm.embedding_backward(torch.ones(3, 8, device="cuda"), torch.zeros(3, dtype=torch.int32, device="cuda"), 0).shape == (0, 8)


def test_backward_leaves_out_nan_of_padding():
    grad = torch.tensor([[1.0, 2.0], [float("nan"), float("inf")], [3.0, 4.0], [float("inf"), 1.0]], device="cuda")
    got = bm.embedding_backward(grad, torch.tensor([1, -1, 1, 0], device="cuda"), 3)
    assert got.tolist() == [[float("inf"), 1.0], [4.0, 6.0], [0.0, 0.0]]


@pytest.mark.parametrize("shift", [0, 1])
def test_widest_rows(shift):
    g = _gen(shift)
    hidden, ids = 1 << 24, torch.tensor([1, 1, 0], device="cuda")
    base = torch.randint(-8, 9, (3 * hidden + 4,), generator=g, device="cuda", dtype=torch.int8).float()
    grad = base[shift:shift + 3 * hidden].view(3, hidden)
    got = bm.embedding_backward(grad, ids, 2)
    assert torch.equal(got[1], grad[0] + grad[1]) and torch.equal(got[0], grad[2])
    assert torch.equal(bm.embedding_lookup(got, ids), got[ids])
    many = torch.zeros(100, dtype=torch.int64, device="cuda")  # a run over several chunks
    assert torch.equal(bm.embedding_backward(grad[:1].expand(100, hidden), many, 1)[0], 100 * grad[0])


def test_captured_replayed_and_on_two_streams():
    g = _gen(6)
    T, V, H = 5000, 700, 136
    table, ids = _rows(g, V, H, F32, whole=True), _ids(g, T, V, "rare")
    grad = _rows(g, T, H, F32, whole=True)

    def both():
        x = bm.embedding_lookup(table, ids, scale=2.0)
        return x, bm.embedding_backward(grad, ids, V)

    want = [x.clone() for x in both()]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = both()
    for k in (1, -1):
        table *= k
        grad *= k
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b * k)
    streams = [torch.cuda.Stream() for _ in range(2)]
    table *= -1
    grad *= -1
    torch.cuda.synchronize()
    outs = []
    for _ in range(20):
        for st in streams:
            outs.append((bm.embedding_lookup(table, ids, scale=2.0, stream=st), bm.embedding_backward(grad, ids, V, stream=st)))
    torch.cuda.synchronize()
    for pair in outs:
        for a, b in zip(pair, want):
            assert torch.equal(a, b)


def test_ids_that_change_under_a_captured_call():
    """The number of rows of a call is fixed, what they are is not."""
    g = _gen(7)
    T, V, H = 3000, 50, 24
    grad, ids = _rows(g, T, H, F32, whole=True), _ids(g, T, V, "any")
    bm.embedding_backward(grad, ids, V)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = bm.embedding_backward(grad, ids, V)
    for kind in ("one", "none", "few", "rare"):
        ids.copy_(_ids(g, T, V, kind))
        graph.replay()
        at, row = _named(ids, V)
        want = torch.zeros(V, H, dtype=torch.float64, device="cuda").index_add_(0, row, grad[at].double())
        assert torch.equal(got, want.float())


@pytest.mark.parametrize("T", [700, 40000])
@pytest.mark.parametrize("accumulate", [False, True])
def test_backward_captured_and_behind_other_work(T, accumulate):
    """The sort as one block and as several launches, captured and replayed
    behind a kernel that writes the gradient, and before one that reads the result."""
    g = _gen(T)
    V, H = 300, 72
    grad, ids = _rows(g, T, H, BF16, whole=True), _ids(g, T, V, "rare")
    at, row = _named(ids, V)
    want = torch.zeros(V, H, dtype=torch.float64, device="cuda").index_add_(0, row, grad[at].double()).float()
    held, out = torch.empty_like(grad), torch.zeros(V, H, device="cuda")
    total = torch.zeros(V, H, device="cuda")

    def run():
        held.copy_(grad)
        bm.embedding_backward(held, ids, out=out, accumulate=accumulate)
        total.add_(out)
        held.zero_()

    run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for _ in range(3):
            run()
    out.zero_()
    total.zero_()
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, 6 * want if accumulate else want)
    assert torch.equal(total, 21 * want if accumulate else 6 * want)
