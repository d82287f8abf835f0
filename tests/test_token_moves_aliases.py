"""Outputs of rotary and paged_append that may share bytes with the maps that
the call reads (positions, frequencies, axes, starts, lengths, table) are
refused, as those that may share bytes with the heads are; key and value
caches that lie between each other are told apart.  On the host: addresses
are only looked at."""

import random

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


def _bytes(at, pages, page, heads, dim, strides):
    """Every byte of a cache of 16-bit elements."""
    return {at + 2 * (p * strides[0] + s * strides[1] + h * strides[2] + d) + b
            for p in range(pages) for s in range(page) for h in range(heads) for d in range(dim) for b in (0, 1)}


@pytest.mark.parametrize("pages,page,heads,dk,dv,strides,distance", [
    (3, 4, 2, 8, 8, (64, 16, 8), 64 * 3),    # one cache behind the other
    (3, 4, 2, 8, 8, (128, 16, 8), 64),       # pages in turn
    (3, 4, 2, 8, 8, (128, 32, 8), 16),       # entries in turn
    (3, 4, 2, 8, 8, (128, 32, 16), 8),       # heads in turn
    (3, 4, 2, 8, 6, (112, 28, 14), 8),       # heads of different widths in turn
    (3, 4, 2, 8, 8, (128, 16, 64), 8),       # (by head first: entries in turn)
    (3, 4, 2, 8, 8, (128, 8, 64), 32),       # (by head first: heads in turn)
    (1, 1, 2, 8, 8, (5, 3, 16), 8),          # strides of single pages and entries do not count
    (3, 4, 2, 8, 8, (128, 32, 16), -8), (3, 4, 2, 8, 8, (128, 32, 8), -16), (3, 4, 2, 8, 8, (128, 16, 8), -64),
    (3, 4, 2, 8, 8, (128, 32, 16), 7), (3, 4, 2, 8, 8, (128, 32, 16), 9), (3, 4, 2, 8, 8, (128, 32, 8), 15),
    (3, 4, 2, 8, 8, (128, 32, 8), 24), (3, 4, 2, 8, 8, (128, 16, 8), 63), (3, 4, 2, 8, 8, (128, 16, 8), 8), (3, 4, 2, 8, 8, (128, 32, 16), 0),
    (3, 4, 2, 8, 9, (128, 32, 16), 8), (3, 4, 2, 9, 7, (128, 32, 16), 8), (3, 4, 2, 9, 8, (130, 32, 16), 8), (3, 4, 2, 8, 8, (130, 32, 16), 8),
    (3, 4, 2, 8, 8, (128, 32, 16), 8 + 32 * 3), (3, 4, 2, 8, 8, (128, 32, 16), 8 - 128),
])
def test_caches_that_lie_between_each_other(lib, pages, page, heads, dk, dv, strides, distance):
    at = 1 << 36
    shared = _bytes(at, pages, page, heads, dk, strides) & _bytes(at + 2 * distance, pages, page, heads, dv, strides)
    accepted = _append(lib, {})
    change = {3: heads, 4: dk, 8: heads, 9: dv, 14: dk, 19: dk, 28: 3, 36: pages, 37: page, 38: at, 42: at + 2 * distance}
    change.update(dict(zip((39, 40, 41), strides)))
    change.update(dict(zip((43, 44, 45), strides)))
    assert _append(lib, change) == (ALIAS if shared else accepted)


@pytest.mark.parametrize("stride", [39, 40, 41])
def test_caches_of_other_strides_are_not_told_apart(lib, stride):
    """Even where they share nothing, as here by their last page's gap."""
    a = {36: 2, 37: 2, 39: 4096, 40: 512, 41: 64, 42: C + 256, 43: 4096, 44: 512, 45: 64}
    assert _append(lib, a) == _append(lib, {})
    a[stride] += {39: 512, 40: 64, 41: 64}[stride]
    assert _append(lib, a) == ALIAS


def test_any_caches(lib):
    """Caches at any distance, with any gaps: those that share a byte are
    refused; those that share none and lie in each other's gaps are not."""
    rng = random.Random(5)
    accepted = _append(lib, {})
    seen = {True: 0, False: 0}
    for _ in range(4000):
        dk, dv = rng.randint(1, 5), rng.randint(1, 5)
        sizes = [rng.randint(1, 3) for _ in range(3)]
        strides, span = [0, 0, 0], max(dk, dv)
        order = rng.sample(range(3), 3)
        for i in order:
            strides[i] = span + rng.choice([0, 0, 1, span, span + 3])
            span += (sizes[i] - 1) * strides[i]
        distance = rng.choice([rng.randint(-span, span)] + [rng.choice([1, -1]) * max(x // 2, 1) for x in strides])
        at = 1 << 36
        shared = bool(_bytes(at, *sizes, dk, strides) & _bytes(at + 2 * distance, *sizes, dv, strides))
        change = {3: sizes[2], 4: dk, 8: sizes[2], 9: dv, 14: dk, 19: dk, 22: 0, 23: 0, 24: 0, 28: 0, 36: sizes[0],
                  37: sizes[1], 38: at, 42: at + 2 * distance}
        change.update(dict(zip((39, 40, 41), strides)))
        change.update(dict(zip((43, 44, 45), strides)))
        got = _append(lib, change)
        assert got in (accepted, ALIAS)
        if shared:
            assert got == ALIAS, (sizes, strides, dk, dv, distance)
        elif got == ALIAS:
            seen[False] += 1
        else:
            seen[True] += 1
    assert seen[True] > 1000 and seen[False] < seen[True] // 10, seen
