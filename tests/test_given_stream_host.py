"""A call that is given a stream makes its outputs and workspaces as that
stream's memory: shown without a GPU, with the library, the allocations and
torch's streams replaced by ones that keep a record."""

import contextlib

import pytest

import bmmc_index_transforms_gb300 as bm
from bmmc_index_transforms_gb300 import _build, token_moves as tm

torch = pytest.importorskip("torch")

CURRENT, GIVEN = 0x100, 0x200


class OnDevice:
    """A host tensor that says it is on cuda:0."""

    def __init__(self, x):
        self.x = x

    def __getattr__(self, name):
        return getattr(self.x, name)

    def get_device(self):
        return 0


class Handle:
    cuda_stream = GIVEN


@pytest.fixture
def made(monkeypatch):
    """The streams on which the calls of this test make tensors."""
    _build.build()
    tm._setup()
    now, log = [CURRENT], []

    @contextlib.contextmanager
    def stream(s):
        now.append(s)
        yield
        now.pop()

    def empty(*size, **kw):
        log.append(now[-1])
        kw["device"] = "cpu"
        return OnDevice(torch.zeros(*size, **kw))

    class Library:
        def __getattr__(self, name):
            def call(*a):
                if name == "expert_sort_workspace":
                    a[-1].value = 64
                return 0
            return call

    monkeypatch.setattr(tm, "_empty", empty)
    monkeypatch.setattr(tm, "_library", Library())
    monkeypatch.setattr(tm, "_raw_stream", lambda device: CURRENT)
    monkeypatch.setattr(tm, "_current_device", lambda: 0)
    monkeypatch.setattr(tm, "_workspaces", {})
    monkeypatch.setattr(torch, "empty", empty)
    monkeypatch.setattr(torch.cuda, "stream", stream)
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle: handle)
    monkeypatch.setattr(torch.cuda, "default_stream", lambda: 0)
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda *a: None)
    return log


def _calls(stream):
    new = lambda *s, dtype=torch.float32: OnDevice(torch.zeros(*s, dtype=dtype))  # noqa: E731
    slot, x, rows, w = new(4, 2, dtype=torch.int32), new(4, 8), new(8, 8), new(4, 2)
    heads, at, freq = new(4, 2, 8), new(4, dtype=torch.int32), new(4)
    cache, table = new(5, 4, 2, 8), new(4, 2, dtype=torch.int32)
    bm.expert_sort(new(4, 2, dtype=torch.int64), 4, stream=stream)
    bm.expert_dispatch(x, slot, stream=stream)
    bm.expert_combine(rows, slot, w, stream=stream)
    bm.expert_combine_backward(x, rows, slot, w, stream=stream)
    bm.rotary(heads, at, freq, stream=stream)
    bm.paged_append(heads, heads, cache, cache, table, at, q=heads, inv_freq=freq, stream=stream)


MADE = 4 + 1 + 1 + 2 + 1 + 1


@pytest.mark.parametrize("stream,owner", [(None, CURRENT), (CURRENT, CURRENT), (GIVEN, GIVEN), (Handle(), GIVEN), (0, 0)])
def test_new_tensors_are_the_given_streams(made, stream, owner):
    _calls(stream)
    assert made == [owner] * MADE


@pytest.mark.parametrize("stream,owner", [(None, CURRENT), (GIVEN, GIVEN), (Handle(), GIVEN), (0, 0)])
def test_the_copy_of_a_view_is_the_given_streams(made, monkeypatch, stream, owner):
    given = []
    monkeypatch.setattr(bm, "lmad_copy_tensor", lambda src, dst, st: given.append(st))
    x = OnDevice(torch.zeros(4, 6).t())
    x.is_cuda = True
    assert bm.contiguous(x, stream).shape == (6, 4)
    assert made == [owner] and given == [stream]
