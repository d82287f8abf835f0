"""Embeddings, the balance loss and 8-bit caches at the ends of the ranges that
their calls allow, on the GPU against the definitions."""

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from test_gpu_paged_cache8 import BF16, E4M3, F16, F32, I8, _case, _check_append, _check_read, _gen  # noqa: E402


@pytest.mark.parametrize("head_major", [False, True])
@pytest.mark.parametrize("cache,dtype", [(E4M3, BF16), (I8, F32), (None, F16)])
@pytest.mark.parametrize("heads,dim", [(65, 8191), (274, 4095), (274, 8190), (2052, 2047), (4121, 1023), (16400, 1023), (2048, 8192)])
def test_entries_of_many_wide_heads(heads, dim, cache, dtype, head_major):
    """More than 2**16 words an entry, up to 2**24 elements: every word is its
    own head's, with its own head's scale."""
    c = _case(_gen(heads), [2, 1], 2, 0, heads, dim, dim, dtype, cache or E4M3, head_major, 2, spare=1)
    if cache is None:
        c["caches"] = [torch.randn(m.shape, device="cuda").to(dtype) for m in c["caches"]]
    else:
        _check_append(c)
    _check_read(c, dtype, c["lengths"])
