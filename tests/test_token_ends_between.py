"""Scales of 8-bit caches that lie between the caches' values and between each
other: accepted where no byte is shared and the arrays lie in each other's gaps,
refused where one is.  On the host: addresses are only looked at."""

import random

import pytest

from bmmc_index_transforms_gb300 import _build, _capi

pytestmark = pytest.mark.no_gpu  # calls that are accepted would be launched

P, Q, S, C = 1 << 20, 1 << 30, 1 << 32, 1 << 36
ALIAS, INVALID = _capi.ERR_ALIAS, _capi.ERR_INVALID_ARG


@pytest.fixture(scope="module", autouse=True)
def lib():
    _build.build()
    return _capi.lib()


def _append(lib, sizes, dims, caches, scales):
    """caches, scales: (address, strides in bytes) of keys and values each."""
    pages, page, heads = sizes
    a = [8, 2]
    for at, dim in ((P, dims[0]), (P + (1 << 16), dims[1])):
        a += [at, heads, dim, heads * dim, dim]
    a += [0] * 10 + [0] * 8 + [0, S + 4096, 8] + [S + 8192, 4, 4, pages, page]
    for at, strides in caches:
        a += [at, *strides]
    a += [_capi.E4M3]
    for at, strides in scales:
        a += [at, *(s // 4 for s in strides)]
    return lib.paged_append_quantised(_capi.PAGED_APPEND_QUANTISED_ARGS.pack(*a), None)


def _bytes(sizes, run, at, strides):
    return {at + p * strides[0] + s * strides[1] + h * strides[2] + b
            for p in range(sizes[0]) for s in range(sizes[1]) for h in range(sizes[2]) for b in range(run)}


def _shared(sizes, dims, caches, scales):
    sets = [_bytes(sizes, d, *c) for d, c in zip(dims, caches)] + [_bytes(sizes, 4, *s) for s in scales]
    return any(sets[i] & sets[j] for i in range(4) for j in range(i))


def _accepted(lib):
    apart = [(C, (64, 16, 8)), (C + 4096, (64, 16, 8))], [(C + 8192, (32, 8, 4)), (C + 12288, (32, 8, 4))]
    status = _append(lib, (2, 3, 2), (8, 8), *apart)  # as far as the check of the pointers, which needs a device
    assert status not in (_capi.OK, ALIAS, INVALID)
    return status


LAYOUTS = {
    # sizes, dims, strides of k, v, k's scales, v's, and where they start
    "a scale behind each head": ((3, 4, 2), (16, 16), [(160, 40, 20)] * 4, [0, 480, 16, 496]),
    "both heads and both scales together": ((3, 4, 2), (16, 12), [(288, 72, 36)] * 4, [0, 16, 28, 32]),
    "scales ahead of the heads": ((3, 4, 2), (16, 16), [(160, 40, 20)] * 4, [4, 484, 0, 480]),
    "an entry's scales behind its heads": ((3, 4, 2), (16, 16), [(160, 40, 16)] * 2 + [(160, 40, 4)] * 2, [0, 480, 32, 512]),
    "by head, an entry's scale behind it": ((3, 4, 2), (16, 16), [(160, 20, 80)] * 4, [0, 480, 16, 496]),
    "by head, a head's scales behind its entries": ((3, 4, 2), (16, 16), [(160, 16, 80)] * 2 + [(160, 4, 80)] * 2, [0, 480, 64, 544]),
    "key and value scales in turn, by head": ((3, 4, 2), (8, 8), [(64, 16, 8)] * 2 + [(64, 16, 8)] * 2, [0, 4096, 8192, 8196]),
    "key and value scales in turn, by entry": ((3, 4, 2), (8, 8), [(64, 16, 8)] * 2 + [(64, 16, 4)] * 2, [0, 4096, 8192, 8200]),
    "key and value scales in turn, by page": ((3, 4, 2), (8, 8), [(64, 16, 8)] * 2 + [(64, 8, 4)] * 2, [0, 4096, 8192, 8224]),
    "all of a page in one run": ((3, 4, 2), (8, 8), [(192, 16, 8)] * 2 + [(192, 8, 4)] * 2, [0, 64, 128, 160]),
    "a page of one entry": ((4, 1, 2), (16, 16), [(40, 999, 20)] * 2 + [(40, 4, 20)] * 2, [0, 160, 16, 176]),
    "one head": ((3, 4, 1), (16, 16), [(160, 40, 7)] * 2 + [(160, 40, 4)] * 2, [0, 16, 32, 36]),
}


@pytest.mark.parametrize("name", LAYOUTS)
def test_layouts(lib, name):
    sizes, dims, strides, at = LAYOUTS[name]
    place = lambda at: ([(C + at[0], strides[0]), (C + at[1], strides[1])],  # noqa: E731
                        [(C + at[2], strides[2]), (C + at[3], strides[3])])
    assert not _shared(sizes, dims, *place(at))
    assert _append(lib, sizes, dims, *place(at)) == _accepted(lib)
    refused = 0
    for i in range(4):
        for step in (-8, -4, 4, 8):
            moved = list(at)
            moved[i] += step
            if _shared(sizes, dims, *place(moved)):
                assert _append(lib, sizes, dims, *place(moved)) == ALIAS, (i, step)
                refused += 1
    assert refused >= 4


def test_any_scales(lib):
    """Caches and scales with any gaps, at any distances."""
    rng = random.Random(9)
    accepted = _accepted(lib)
    seen = {ALIAS: 0, accepted: 0, "told apart": 0, "not told apart": 0}
    for _ in range(6000):
        sizes = tuple(rng.randint(1, 3) for _ in range(3))
        dims = rng.choice([4, 8, 6, 3]), rng.choice([4, 8, 5])
        order = rng.sample(range(3), 3)

        def nest(run):
            strides, span = [0, 0, 0], run
            for i in order:
                strides[i] = -(-span // 4) * 4 + rng.choice([0, 0, 4, 8, span // 4 * 4 + 8])
                span += (sizes[i] - 1) * strides[i]
            return strides, span

        common, span = nest(max(dims) + rng.choice([0, 4, 8]))
        arrays = []
        for run in (*dims, 4, 4):
            strides = list(common)
            if rng.random() < 0.2:
                strides, _ = nest(run)
            elif rng.random() < 0.3:  # the fastest dimension without gaps
                strides[order[0]] = -(-run // 4) * 4
            arrays.append((C + (0 if not arrays else rng.choice([rng.randint(0, span) // 4 * 4, rng.randint(0, 16) * 4, rng.choice(common)])),
                           tuple(strides)))
        caches, scales = arrays[:2], arrays[2:]
        if rng.random() < 0.5:
            caches[1] = (C + (1 << 20), caches[1][1])
        got = _append(lib, sizes, dims, caches, scales)
        assert got in (accepted, ALIAS), got
        seen[got] += 1
        if _shared(sizes, dims, caches, scales):
            assert got == ALIAS, (sizes, dims, arrays)
        else:
            seen["told apart" if got == accepted else "not told apart"] += 1
    assert seen[accepted] > 300 and seen[ALIAS] > 300, seen
    print(seen)
