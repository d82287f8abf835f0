"""Embeddings, the balance loss and 8-bit caches at the ends of the ranges that
their calls allow, on the GPU against the definitions."""

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from test_gpu_paged_cache8 import BF16, E4M3, F16, F32, I8, _case, _check_append, _check_read, _freq, _gen  # noqa: E402


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


def _pool(c, layout, D):
    """The case's caches and scales as views of one pool of bytes: pages of
    entries (or, head_major, of heads), each head's values and scale in the
    `layout`'s order; what it gives between them belongs to nobody."""
    cache, head_major = c["caches"][0].dtype, c["head_major"]
    pages, a, b = c["caches"][0].shape[:3]  # page and heads, in their order
    page, heads = (b, a) if head_major else (a, b)
    if layout in ("behind each head", "behind each head, in words"):
        gap = 16 if layout.endswith("words") else 4
        pool = torch.full((pages, 2, a, b, D + gap), 0x5a, dtype=torch.uint8, device="cuda")
        values = [pool[:, i, ..., :D] for i in range(2)]
        scales = [pool.view(F32)[:, i, ..., D // 4] for i in range(2)]
    elif layout == "keys, values and both scales together":
        pool = torch.full((pages, a, b, 2 * D + 8), 0x5a, dtype=torch.uint8, device="cuda")
        values = [pool[..., :D], pool[..., D:2 * D]]
        scales = [pool.view(F32)[..., D // 2 + i] for i in range(2)]
    elif layout == "behind each entry":
        pool = torch.full((pages, 2, page, heads * (D + 4)), 0x5a, dtype=torch.uint8, device="cuda")
        values = [pool[:, i, :, :heads * D].unflatten(2, (heads, D)) for i in range(2)]
        scales = [pool.view(F32)[:, i, :, heads * D // 4:] for i in range(2)]
        if head_major:
            values, scales = [x.transpose(1, 2) for x in values], [x.transpose(1, 2) for x in scales]
    elif layout == "scales in turn by head":
        both = torch.full((pages, a, b, 2), 7.0, device="cuda")
        pool, values, scales = both, c["caches"], [both[..., i] for i in range(2)]
    else:
        assert layout == "scales in turn by entry"
        both = torch.full((pages, a, 2, b), 7.0, device="cuda")
        pool, values, scales = both, c["caches"], [both[:, :, i] for i in range(2)]
    if values is not c["caches"]:
        values = [x.view(cache) for x in values]
    return pool, dict(c, caches=values, scales=scales)


@pytest.mark.parametrize("head_major", [False, True])
@pytest.mark.parametrize("cache,dtype", [(E4M3, BF16), (I8, F32)])
@pytest.mark.parametrize("counts,page,Hk,D", [([1] * 9, 16, 8, 128), ([40, 0, 3], 8, 2, 64), ([7, 5], 4, 3, 36), ([2], 1, 1, 256)])
@pytest.mark.parametrize("layout", ["behind each head", "behind each head, in words", "keys, values and both scales together",
                                    "behind each entry", "scales in turn by head", "scales in turn by entry"])
def test_scales_between_the_values(layout, counts, page, Hk, D, cache, dtype, head_major):
    """A pool of pages that holds values and scales: an append writes these and
    nothing else of it, and a read finds them."""
    apart = _case(_gen(D + Hk), counts, page, 4, Hk, D, D, dtype, cache, head_major, 20)
    pool, c = _pool(apart, layout, D)
    for old, new in zip(apart["caches"] + apart["scales"], c["caches"] + c["scales"]):
        if old is not new:
            (new.view(torch.uint8) if new.element_size() == 1 else new).copy_(old.view(torch.uint8) if old.element_size() == 1 else old)
    mine = torch.zeros(pool.numel() * pool.element_size(), dtype=torch.bool, device="cuda")
    for x in (c["caches"] if layout.startswith(("behind", "keys")) else []) + c["scales"]:
        at = torch.arange(x.element_size(), device="cuda") + (x.data_ptr() - pool.data_ptr())
        for n, s in zip(x.shape, x.stride()):
            at = (at[:, None] + torch.arange(n, device="cuda") * s * x.element_size()).flatten()
        assert not mine[at].any()
        mine[at] = True
    before = pool.view(torch.uint8).flatten().clone()
    _check_append(c, _freq(D // 2))
    _check_append(c)
    assert torch.equal(pool.view(torch.uint8).flatten()[~mine], before[~mine])
    _check_read(c, dtype, c["lengths"])
