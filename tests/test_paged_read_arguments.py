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
