"""paged_read's number of rows and given results, as far as the binding looks
at them."""

import pytest

import bmmc_index_transforms_gb300 as bm

torch = pytest.importorskip("torch")


def _read(*a, **kw):
    """The refusal of a call on host tensors; one that is fine is refused for these alone."""
    cache, scales = torch.zeros(5, 4, 2, 8, dtype=torch.int8), torch.zeros(5, 4, 2)
    table, starts = torch.zeros(3, 2, dtype=torch.int32), torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError) as e:
        bm.paged_read(cache, cache, table, starts, *a, k_scales=scales, v_scales=scales, **kw)
    return str(e.value)


def test_a_negative_number_of_rows_is_refused():
    assert "num_rows -1 is negative" in _read(-1, dtype=torch.float16)
    assert "current device" in _read(0, dtype=torch.float16)


def test_one_result_may_be_given():
    """The other one is new, of its rows and type."""
    out = torch.zeros(6, 2, 8, dtype=torch.float16)
    assert "current device" in _read(k_out=out)
    assert "current device" in _read(v_out=out)
    assert "num_rows" in _read(dtype=torch.float16)


@pytest.mark.gpu
@pytest.mark.parametrize("given", ["k_out", "v_out"])
def test_one_given_result_on_the_gpu(given):
    cache = torch.randint(-127, 128, (5, 4, 2, 8), dtype=torch.int8, device="cuda")
    scales = torch.rand(5, 4, 2, device="cuda")
    table = torch.arange(4, dtype=torch.int32, device="cuda").view(2, 2)
    starts = torch.tensor([0, 5, 8], dtype=torch.int32, device="cuda")
    kw = dict(k_scales=scales, v_scales=scales)
    want = bm.paged_read(cache, cache, table, starts, 9, dtype=torch.float16, **kw)
    out = torch.full((9, 2, 8), 7.0, dtype=torch.float16, device="cuda")
    got = bm.paged_read(cache, cache, table, starts, **{given: out}, **kw)
    assert got[given == "v_out"] is out
    assert all(g.dtype == torch.float16 and torch.equal(g, w) for g, w in zip(got, want))
