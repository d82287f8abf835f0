"""Embeddings, the balance loss and 8-bit caches reach their shared arrays
through the views that the bounds-checked build tests, and make what they
return on the stream they are given."""

import pytest
from test_given_stream_host import CURRENT, GIVEN, Handle, OnDevice, made  # noqa: F401
from test_shared_views import test_shared_arrays_are_reached_through_views as reached_through_views

import bmmc_index_transforms_gb300 as bm
from bmmc_index_transforms_gb300 import token_moves as tm

torch = pytest.importorskip("torch")


@pytest.mark.parametrize("name,arrays", [("embedding.cu", 6), ("balance.cu", 8), ("paged_cache8.cu", 12)])
def test_shared_arrays(name, arrays):
    reached_through_views(name, arrays)


class Library:
    """Every workspace is of 64 bytes."""

    def __getattr__(self, name):
        def call(*a):
            if name.endswith("_workspace"):
                a[-1].value = 64
            return 0
        return call


@pytest.mark.parametrize("stream,owner", [(None, CURRENT), (CURRENT, CURRENT), (GIVEN, GIVEN), (Handle(), GIVEN), (0, 0)])
def test_new_tensors_are_the_given_streams(made, monkeypatch, stream, owner):  # noqa: F811
    monkeypatch.setattr(tm, "_library", Library())
    new = lambda *s, dtype=torch.float32: OnDevice(torch.zeros(*s, dtype=dtype))  # noqa: E731
    x, ids, choices = new(4, 8), new(4, dtype=torch.int64), new(4, 2, dtype=torch.int32)
    bm.embedding_lookup(x, ids, stream=stream)
    bm.embedding_backward(x, ids, 9, stream=stream)
    bm.expert_balance(x, choices, stream=stream)
    bm.expert_balance_backward(new(1), x, choices, new(9, dtype=torch.int32), stream=stream)
    cache, scales, table = new(5, 4, 2, 8, dtype=torch.int8), new(5, 4, 2), new(4, 2, dtype=torch.int32)
    heads, lengths = new(4, 2, 8), new(4, dtype=torch.int32)
    bm.paged_append(heads, heads, cache, cache, table, lengths, q=heads, k_scales=scales, v_scales=scales, stream=stream)
    bm.paged_read(cache, cache, table, new(5, dtype=torch.int32), 6, k_scales=scales, v_scales=scales, dtype=torch.float16,
                  stream=stream)
    assert made == [owner] * (1 + 2 + 3 + 1 + 1 + 2)
