"""Calls on a stream that is not the current one, whose outputs and workspaces
they make themselves: nothing of theirs shares memory with work that is still
queued on the current stream, before the call or after it."""

import pytest

import bmmc_index_transforms_gb300 as bm

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

DELAY = 20_000_000  # clocks, some 10 ms: far longer than the host takes for what follows


def _state():
    g = torch.Generator("cuda").manual_seed(1)
    T, K, H = 20000, 4, 136  # the sort needs a workspace
    randn = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    ids = torch.randint(-1, 300, (T, K), generator=g, device="cuda")
    s = dict(ids=ids, slot=bm.expert_sort(ids, 300)[0], x=randn(T, H), rows=randn(T * K, H),
             w=torch.rand(T, K, generator=g, device="cuda"), heads=randn(T, 2, 68), at=torch.arange(T, device="cuda").int(),
             zero=torch.zeros(T, dtype=torch.int32, device="cuda"), freq=torch.rand(32, generator=g, device="cuda"), table=torch.arange(T, device="cuda").int().view(T, 1),
             caches=[torch.zeros(T, 1, 2, 68, device="cuda") for _ in range(2)])
    torch.cuda.synchronize()
    return s


CALLS = {
    "sort": lambda s, st: bm.expert_sort(s["ids"], 300, stream=st),
    "dispatch": lambda s, st: [bm.expert_dispatch(s["x"], s["slot"], stream=st)],
    "combine": lambda s, st: [bm.expert_combine(s["rows"], s["slot"], s["w"], stream=st)],
    "combine_backward": lambda s, st: bm.expert_combine_backward(s["x"], s["rows"], s["slot"], s["w"], stream=st),
    "rotary": lambda s, st: [bm.rotary(s["heads"], s["at"], s["freq"], stream=st)],
    "append": lambda s, st: [bm.paged_append(s["heads"], s["heads"], *s["caches"], s["table"], s["zero"], q=s["heads"],
                                             inv_freq=s["freq"], stream=st)],
    "contiguous": lambda s, st: [bm.contiguous(s["x"].t(), st)],
}


def _like(outputs, value):
    """Tensors of the sizes of the outputs, and of what a sort works in, twice each."""
    sizes = [x.numel() * x.element_size() // 4 for x in outputs] * 2 + [n * 304 for n in range(20, 160, 4)]
    return [torch.full((n,), value, dtype=torch.int32, device="cuda") for n in sizes]


@pytest.fixture(params=sorted(CALLS))
def case(request):
    s, call = _state(), CALLS[request.param]
    want = [x.clone() for x in call(s, None)]
    torch.cuda.synchronize()
    return s, call, want


@pytest.fixture(params=["stream", "handle"])
def side(request):
    st = torch.cuda.Stream()
    return st, st if request.param == "stream" else st.cuda_stream


def test_memory_that_the_current_stream_still_reads(case, side):
    s, call, want = case
    call(s, side[1])  # nothing is set up for the first time below
    freed = _like(want, 3)
    kept = _like(want, 0)
    torch.cuda.synchronize()
    torch.cuda._sleep(DELAY)
    for y, x in zip(kept, freed):
        y.copy_(x)
    del x, freed  # free for new tensors of the current stream, which reads them first
    got = call(s, side[1])
    torch.cuda.synchronize()
    for y in kept:
        assert bool((y == 3).all())
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def test_outputs_that_are_dropped(case, side):
    s, call, want = case
    call(s, side[1])
    torch.cuda.synchronize()
    with torch.cuda.stream(side[0]):
        torch.cuda._sleep(DELAY)
    call(s, side[1])  # dropped before it has begun
    later = _like(want, 7)
    torch.cuda.synchronize()
    for y in later:
        assert bool((y == 7).all())


def test_sorts_on_two_streams_at_once(side):
    """Each has a workspace of its own, also right behind a call on the other."""
    s = _state()
    want = [x.clone() for x in bm.expert_sort(s["ids"], 300)]
    other = torch.randint(0, 300, s["ids"].shape, device="cuda")
    want_other = [x.clone() for x in bm.expert_sort(other, 300)]
    torch.cuda.synchronize()
    for _ in range(30):
        a = bm.expert_sort(s["ids"], 300)
        b = bm.expert_sort(other, 300, stream=side[1])
        torch.cuda.synchronize()
        for got, w in zip((*a, *b), (*want, *want_other)):
            assert torch.equal(got, w)


def test_the_default_stream_by_its_handle():
    """Handle 0 is the default stream's, also where another one is current."""
    s = _state()
    want = bm.expert_dispatch(s["x"], s["slot"])
    torch.cuda.synchronize()
    with torch.cuda.stream(torch.cuda.Stream()):
        got = bm.expert_dispatch(s["x"], s["slot"], stream=0)
    torch.cuda.synchronize()
    assert torch.equal(got, want)
