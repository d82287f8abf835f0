"""Outputs of rotary and paged_append that may share bytes with the maps that
the call reads (positions, frequencies, axes, starts, lengths, table) are
refused, as those that may share bytes with the heads are.  On the host:
addresses are only looked at."""

import pytest

from bmmc_index_transforms_gb300 import _build, _capi

pytestmark = pytest.mark.no_gpu  # calls that are accepted would be launched

S, Q, C = 1 << 32, 1 << 34, 1 << 36
ALIAS = _capi.ERR_ALIAS


@pytest.fixture(scope="module", autouse=True)
def lib():
    _build.build()
    return _capi.lib()


# tokens type, x and out: data heads dim token head, turns: freq axes positions bytes axes axis_stride pairs flags
ROTARY = [10, 2, 1 << 20, 4, 64, 256, 64, Q, 4, 64, 256, 64, S, S + 1024, S + 4096, 4, 3, 16, 32, 0]
FREQ, AXES, POSITIONS, AXIS_STRIDE = 12, 13, 14, 17
OUT = Q, Q + 10 * 256 * 2  # [lo, hi) of its bytes


def _rotary(lib, change):
    a = list(ROTARY)
    for i, v in change.items():
        a[i] = v
    return lib.rotary(_capi.ROTARY_ARGS.pack(*a), None)


@pytest.mark.parametrize("which,size", [(FREQ, 32 * 4), (AXES, 32 * 4), (POSITIONS, (2 * 16 + 10) * 4)])
def test_rotary(lib, which, size):
    accepted = _rotary(lib, {})  # as far as the check of the pointers, or the launch, which need a device
    assert accepted not in (ALIAS, _capi.ERR_INVALID_ARG, _capi.ERR_MISALIGNED)
    lo, hi = OUT
    for at in (lo, lo + 256, hi - 4, lo - size + 4):
        assert _rotary(lib, {which: at}) == ALIAS
    for at in (hi, lo - size):
        assert _rotary(lib, {which: at}) == accepted


def test_positions_of_the_last_axis(lib):
    """The ranges reach from the first axis to the last."""
    assert _rotary(lib, {POSITIONS: OUT[0] - 4096, AXIS_STRIDE: 512 - 4}) == ALIAS


# tokens type | k, v, q, q_out | turns | starts lengths sequences | table stride columns pages page_size | caches
APPEND = ([8, 2, 1 << 20, 2, 64, 128, 64, 1 << 21, 2, 64, 128, 64, 1 << 22, 4, 64, 256, 64, Q, 4, 64, 256, 64]
          + [S, S + 512, S + 1024, 8, 2, 8, 32, 0] + [S + 2048, S + 4096, 8] + [S + 8192, 6, 4, 32, 16]
          + [C, 2048, 128, 64, C + (1 << 24), 2048, 128, 64])
MAPS = {"freq": (22, 128), "axes": (23, 128), "positions": (24, 128), "starts": (30, 36), "lengths": (31, 32),
        "table": (33, (7 * 6 + 4) * 4)}
OUTPUTS = {"q_out": (Q, Q + 8 * 256 * 2), "k_cache": (C, C + 32 * 2048 * 2),
           "v_cache": (C + (1 << 24), C + (1 << 24) + 32 * 2048 * 2)}


def _append(lib, change):
    a = list(APPEND)
    for i, v in change.items():
        a[i] = v
    return lib.paged_append(_capi.PAGED_APPEND_ARGS.pack(*a), None)


@pytest.mark.parametrize("name", MAPS)
@pytest.mark.parametrize("output", OUTPUTS)
def test_append(lib, name, output):
    accepted = _append(lib, {})
    assert accepted not in (ALIAS, _capi.ERR_INVALID_ARG, _capi.ERR_MISALIGNED)
    (which, size), (lo, hi) = MAPS[name], OUTPUTS[output]
    align = 8 if name == "positions" else 4
    for at in (lo, lo + 512, hi - align, lo - size + align):
        assert _append(lib, {which: at}) == ALIAS
    for at in (hi, lo - size):
        assert _append(lib, {which: at}) == accepted


def test_append_without_maps(lib):
    """Maps that are not there meet nothing."""
    accepted = _append(lib, {})
    assert _append(lib, {23: 0}) == accepted
    assert _append(lib, {24: 0, 25: 0}) == accepted
    assert _append(lib, {30: 0}) == accepted
    assert _append(lib, {22: 0, 23: 0, 24: 0, 28: 0}) == accepted
