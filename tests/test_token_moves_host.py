"""Refusals of the token moves, through the C ABI and the binding: every bad
argument is turned down on the host, before any device work."""

import ctypes

import pytest

import bmmc_index_transforms_gb300 as bm
from bmmc_index_transforms_gb300 import _build, _capi

torch = pytest.importorskip("torch")

P = 1 << 20   # addresses that are only looked at
Q = 1 << 30
S = 1 << 32


@pytest.fixture(scope="module", autouse=True)
def lib():
    _build.build()
    return _capi.lib()


INVALID, UNSUPPORTED, MISALIGNED, ALIAS, NO_SCRATCH = (_capi.ERR_INVALID_ARG, _capi.ERR_UNSUPPORTED_ELEM,
                                                       _capi.ERR_MISALIGNED, _capi.ERR_ALIAS, _capi.ERR_NO_SCRATCH)


def _workspace(lib, *a):
    size = ctypes.c_size_t(7)
    return lib.expert_sort_workspace(*a, size), size.value


def test_sort_workspace(lib):
    assert _workspace(lib, 0, 1, 1) == (_capi.OK, 0)
    assert _workspace(lib, 48, 8, 128) == (_capi.OK, 0)
    status, size = _workspace(lib, 100000, 8, 256)
    assert status == _capi.OK and 0 < size <= 1 << 20
    assert _workspace(lib, 2**31 - 1, 1, 4096)[0] == _capi.OK
    for bad in ((-1, 1, 1), (1, 0, 1), (1, 65, 1), (2**31, 1, 1), (2**30, 2, 1), (2**62, 64, 1), (1, 1, 0), (1, 1, 4097)):
        assert _workspace(lib, *bad) == (INVALID, 0)
    assert lib.expert_sort_workspace(1, 1, 1, None) == INVALID


@pytest.mark.parametrize("change,status", [
    ({0: None}, INVALID), ({1: 2}, UNSUPPORTED), ({2: -1}, INVALID), ({3: 0}, INVALID), ({4: 0}, INVALID), ({5: None}, INVALID),
    ({6: None}, INVALID), ({7: None}, INVALID), ({0: P + 2}, MISALIGNED), ({5: Q + 1}, MISALIGNED), ({6: Q}, ALIAS), ({5: P + 8}, ALIAS),
    ({7: P}, ALIAS), ({2: 100000}, NO_SCRATCH), ({2: 100000, 8: S + 4096, 9: 100}, NO_SCRATCH),
])
def test_sort_refusals(lib, change, status):
    a = [P, 4, 10, 2, 8, Q, Q + (1 << 24), S, None, 0, None]
    for i, v in change.items():
        a[i] = v
    assert lib.expert_sort(*a) == status


#          x  stride slot tokens choices hidden type rows row_stride n_rows stream
DISPATCH = [P, 64, S, 10, 2, 64, 2, Q, 64, 20, None]


@pytest.mark.parametrize("change,status", [
    ({0: None}, INVALID), ({2: None}, INVALID), ({7: None}, INVALID), ({1: -1}, INVALID), ({8: 63}, INVALID), ({3: -1}, INVALID),
    ({4: 0}, INVALID), ({4: 65}, INVALID), ({5: 0}, INVALID), ({5: 1 << 25}, INVALID), ({6: 3}, UNSUPPORTED), ({6: -1}, UNSUPPORTED),
    ({9: 21}, INVALID), ({9: -1}, INVALID), ({3: 2**62}, INVALID), ({1: 2**41}, INVALID), ({8: 2**62}, INVALID),
    ({0: P + 1}, MISALIGNED), ({7: Q + 1}, MISALIGNED), ({2: S + 2}, MISALIGNED), ({7: P + 128}, ALIAS), ({2: Q + 64}, ALIAS),
])
def test_dispatch_refusals(lib, change, status):
    a = list(DISPATCH)
    for i, v in change.items():
        a[i] = v
    assert lib.expert_dispatch(*a) == status


#         rows stride n_rows slot weights wtype tokens choices hidden type out out_stride stream
COMBINE = [P, 64, 20, S, S + 4096, 0, 10, 2, 64, 2, Q, 64, None]


@pytest.mark.parametrize("change,status", [
    ({0: None}, INVALID), ({3: None}, INVALID), ({10: None}, INVALID), ({5: 1}, UNSUPPORTED), ({9: 7}, UNSUPPORTED), ({2: 21}, INVALID),
    ({11: 60}, INVALID), ({1: -64}, INVALID), ({4: S + 4097}, MISALIGNED), ({10: P}, ALIAS), ({4: Q + 4}, ALIAS), ({3: Q}, ALIAS),
])
def test_combine_refusals(lib, change, status):
    a = list(COMBINE)
    for i, v in change.items():
        a[i] = v
    assert lib.expert_combine(*a) == status


#          grad stride rows stride n_rows slot weights wtype tokens choices hidden type grad_rows stride grad_weights stream
BACKWARD = [P, 64, P + (1 << 16), 64, 20, S, S + 4096, 0, 10, 2, 64, 2, Q, 64, S + 8192, None]


@pytest.mark.parametrize("change,status", [
    ({0: None}, INVALID), ({2: None}, INVALID), ({5: None}, INVALID), ({6: None}, INVALID), ({12: None}, INVALID), ({14: None}, INVALID),
    ({7: 1}, UNSUPPORTED), ({13: 63}, INVALID), ({12: P}, ALIAS), ({14: S + 4096}, ALIAS), ({14: Q + 8}, ALIAS), ({14: S + 8193}, MISALIGNED),
])
def test_combine_backward_refusals(lib, change, status):
    a = list(BACKWARD)
    for i, v in change.items():
        a[i] = v
    assert lib.expert_combine_backward(*a) == status


# tokens type, x: data heads dim token head, out: the same, turns: freq axes positions bytes axes stride pairs flags
ROTARY = [10, 2, P, 4, 64, 256, 64, Q, 4, 64, 256, 64, S, 0, S + 4096, 4, 1, 0, 32, 0]


def test_slices_of_one_array_are_told_apart(lib):
    """Overlapping ranges of interleaved slices are no alias (they get as far
    as the pointers' check, which needs a device), slices that meet are."""
    a = list(ROTARY)
    a[5] = a[10] = 1024
    a[7] = P + 512
    assert lib.rotary(_capi.ROTARY_ARGS.pack(*a), None) not in (_capi.OK, ALIAS, INVALID)
    a[7] = P + 510
    assert lib.rotary(_capi.ROTARY_ARGS.pack(*a), None) == ALIAS
    a[7] = P + 2048 - 128
    assert lib.rotary(_capi.ROTARY_ARGS.pack(*a), None) == ALIAS


@pytest.mark.parametrize("change,status", [
    ({0: -1}, INVALID), ({1: 9}, UNSUPPORTED), ({2: 0}, INVALID), ({3: 0}, INVALID), ({4: 0}, INVALID), ({4: 8193}, INVALID),
    ({3: 1 << 20}, INVALID), ({5: -1}, INVALID), ({8: 3}, INVALID), ({9: 32}, INVALID), ({10: 255}, INVALID), ({11: 63}, INVALID),
    ({7: P + 64}, ALIAS), ({7: P, 10: 512}, ALIAS), ({2: P + 1}, MISALIGNED), ({12: 0, 18: 0}, INVALID), ({14: 0}, INVALID),
    ({15: 2}, UNSUPPORTED), ({16: 0}, INVALID), ({16: 33}, INVALID), ({17: -1}, INVALID), ({18: 33}, INVALID), ({18: 0}, INVALID),
    ({19: 4}, INVALID), ({13: S + 2}, MISALIGNED), ({14: S + 2}, MISALIGNED),
])
def test_rotary_refusals(lib, change, status):
    a = list(ROTARY)
    for i, v in change.items():
        a[i] = v
    assert lib.rotary(_capi.ROTARY_ARGS.pack(*a), None) == status
    assert lib.rotary(None, None) == INVALID


C = 1 << 36
# tokens type | k, v, q, q_out | turns | starts lengths sequences | table stride columns pages page_size | caches
APPEND = ([8, 2, P, 2, 64, 128, 64, P + (1 << 16), 2, 64, 128, 64, P + (1 << 18), 4, 64, 256, 64, Q, 4, 64, 256, 64]
          + [S, 0, 0, 0, 0, 0, 32, 0] + [0, S + 4096, 8] + [S + 8192, 4, 4, 32, 16]
          + [C, 2048, 128, 64, C + (1 << 24), 2048, 128, 64])


@pytest.mark.parametrize("change,status", [
    ({0: -1}, INVALID), ({1: 5}, UNSUPPORTED), ({2: 0}, INVALID), ({8: 3}, INVALID), ({14: 32}, INVALID), ({17: 0}, INVALID),
    ({18: 2}, INVALID), ({22: 0}, INVALID), ({28: 33}, INVALID), ({29: 2}, INVALID), ({31: 0}, INVALID), ({32: 7}, INVALID), ({32: -1}, INVALID),
    ({33: 0}, INVALID), ({34: -1}, INVALID), ({37: 0}, INVALID), ({36: -1}, INVALID), ({38: 0}, INVALID), ({39: 2047}, INVALID), ({40: 100}, INVALID),
    ({41: 63}, INVALID), ({42: C}, ALIAS), ({38: P}, ALIAS), ({42: Q}, ALIAS), ({17: P}, ALIAS), ({38: C + 1}, MISALIGNED), ({31: S + 1}, MISALIGNED),
])
def test_append_refusals(lib, change, status):
    a = list(APPEND)
    for i, v in change.items():
        a[i] = v
    assert lib.paged_append(_capi.PAGED_APPEND_ARGS.pack(*a), None) == status
    assert lib.paged_append(None, None) == INVALID


def test_arrays_beyond_any_memory(lib):
    """Strides that are fine by themselves, with so many rows that byte
    offsets would leave 64 bits."""
    n = 2**31 - 1
    assert lib.expert_dispatch(P, 2**40, S, n, 1, 64, 2, Q, 64, n, None) == INVALID
    assert lib.expert_dispatch(P, 64, S, n, 1, 64, 2, Q, 2**40, n, None) == INVALID
    assert lib.expert_combine(P, 2**40, n, S, None, 0, n, 1, 64, 2, Q, 64, None) == INVALID
    assert lib.expert_combine_backward(P, 2**40, P, 64, n, S, S, 0, n, 1, 64, 2, Q, 64, S, None) == INVALID
    a = list(ROTARY)
    a[0], a[5], a[10] = n, 2**40, 2**40
    assert lib.rotary(_capi.ROTARY_ARGS.pack(*a), None) == INVALID
    a = list(APPEND)
    a[36], a[39] = n, 2**40
    assert lib.paged_append(_capi.PAGED_APPEND_ARGS.pack(*a), None) == INVALID


def test_nothing_to_do_is_fine(lib):
    a = list(APPEND)
    a[0] = 0
    assert lib.paged_append(_capi.PAGED_APPEND_ARGS.pack(*a), None) == _capi.OK
    a = list(ROTARY)
    a[0] = 0
    assert lib.rotary(_capi.ROTARY_ARGS.pack(*a), None) == _capi.OK
    assert lib.expert_dispatch(None, 64, None, 0, 2, 64, 2, None, 64, 0, None) == _capi.OK
    assert lib.expert_combine(None, 64, 0, None, None, 0, 0, 2, 64, 2, None, 64, None) == _capi.OK


def test_binding_refusals():
    x, slot = torch.zeros(4, 8), torch.zeros(4, 2, dtype=torch.int32)
    cases = [
        (lambda: bm.expert_sort(slot.float(), 4), "experts must be"), (lambda: bm.expert_sort(slot.t(), 4), "experts must be"),
        (lambda: bm.expert_sort(slot, 4), "current device"), (lambda: bm.expert_dispatch(x, slot.long()), "slot must be"),
        (lambda: bm.expert_dispatch(x[:3], slot), "shape"), (lambda: bm.expert_dispatch(x.t(), slot), "dense rows"),
        (lambda: bm.expert_dispatch(x, slot, 9), "num_rows"),
        (lambda: bm.expert_dispatch(x, slot), "current device"), (lambda: bm.expert_combine(torch.zeros(9, 8), slot), "9 rows"),
        (lambda: bm.expert_combine(torch.zeros(8, 8), slot, torch.zeros(4, 3)), "slot's shape"),
        (lambda: bm.expert_combine(torch.zeros(8, 8), slot, torch.zeros(4, 2).half()), "float32 or of the rows' type"),
        (lambda: bm.expert_combine_backward(x.half(), torch.zeros(8, 8), slot, torch.zeros(4, 2)), "type of rows"),
    ]
    h, f, at = torch.zeros(3, 2, 8), torch.zeros(4), torch.zeros(3, dtype=torch.int32)
    cases += [
        (lambda: bm.rotary(h[0], at, f), "tokens, heads, dim"), (lambda: bm.rotary(h, at[:2], f), "positions must"),
        (lambda: bm.rotary(h, at.float(), f), "positions must"), (lambda: bm.rotary(h, at, f.double()), "inv_freq must"),
        (lambda: bm.rotary(h, at, f, torch.zeros(3, dtype=torch.int32)), "pair_axes must"),
        (lambda: bm.rotary(h, None, f), "needed"), (lambda: bm.rotary(h, at, f), "current device"),
    ]
    cache, table, n = torch.zeros(5, 4, 2, 8), torch.zeros(3, 2, dtype=torch.int32), torch.zeros(3, dtype=torch.int32)
    call = bm.paged_append
    cases += [
        (lambda: call(h, h[:2], cache, cache, table, n), "tokens of the other"), (lambda: call(h, h, cache[0], cache, table, n), "4-D"),
        (lambda: call(h, h, cache, cache[:4], table, n), "does not fit"), (lambda: call(h, h, cache, cache, table, n, head_major=True), "does not fit"),
        (lambda: call(h, h, cache, cache, table.long(), n), "page_table must"), (lambda: call(h, h, cache, cache, table, n[:2]), "lengths must"),
        (lambda: call(h, h, cache, cache, table[:2], n[:2]), "need starts"), (lambda: call(h, h, cache, cache, table, n, starts=n), "starts must"),
        (lambda: call(h, h, cache, cache, table, n, positions=at), "need inv_freq"),
        (lambda: call(h, h, cache, cache, table, n), "current device"),
    ]
    for refused, message in cases:
        with pytest.raises(ValueError, match=message):
            refused()
