"""Refusals of embeddings, the balance loss and 8-bit caches, through the C ABI
and the binding: every bad argument is turned down on the host, before any
device work."""

import ctypes

import pytest

import bmmc_index_transforms_gb300 as bm
from bmmc_index_transforms_gb300 import _build, _capi

torch = pytest.importorskip("torch")

P = 1 << 20   # addresses that are only looked at
Q = 1 << 30
S = 1 << 32
C = 1 << 36


@pytest.fixture(scope="module", autouse=True)
def lib():
    _build.build()
    return _capi.lib()


OK, INVALID, UNSUPPORTED, MISALIGNED, ALIAS, NO_SCRATCH = (
    _capi.OK, _capi.ERR_INVALID_ARG, _capi.ERR_UNSUPPORTED_ELEM, _capi.ERR_MISALIGNED, _capi.ERR_ALIAS, _capi.ERR_NO_SCRATCH)


def _changed(a, change):
    a = list(a)
    for i, v in change.items():
        a[i] = v
    return a


#         table stride vocab ids bytes tokens hidden type scale out stride stream
LOOKUP = [P, 64, 100, S, 8, 10, 64, 2, 1.0, Q, 64, None]


@pytest.mark.parametrize("change,status", [
    ({0: None}, INVALID), ({3: None}, INVALID), ({9: None}, INVALID), ({1: -1}, INVALID), ({10: 63}, INVALID), ({2: -1}, INVALID),
    ({2: 2**31}, INVALID), ({4: 2}, UNSUPPORTED), ({5: -1}, INVALID), ({5: 2**31}, INVALID), ({6: 0}, INVALID), ({6: (1 << 24) + 1}, INVALID),
    ({7: 3}, UNSUPPORTED), ({7: 4}, UNSUPPORTED), ({7: -1}, UNSUPPORTED), ({1: 2**41}, INVALID), ({2: 2**31 - 2, 1: 2**40}, INVALID),
    ({0: P + 1}, MISALIGNED), ({9: Q + 1}, MISALIGNED), ({3: S + 4}, MISALIGNED), ({9: P + 128}, ALIAS), ({3: Q + 64}, ALIAS),
])
def test_lookup_refusals(lib, change, status):
    assert lib.embedding_lookup(*_changed(LOOKUP, change)) == status


#           grad stride ids bytes tokens hidden type scale accumulate out stride vocab out_type workspace bytes stream
BACKWARD = [P, 64, S, 8, 10, 64, 2, 1.0, 0, Q, 64, 100, 0, C, 1 << 20, None]


@pytest.mark.parametrize("change,status", [
    ({0: None}, INVALID), ({2: None}, INVALID), ({9: None}, INVALID), ({1: -1}, INVALID), ({10: 63}, INVALID), ({11: -1}, INVALID),
    ({3: 1}, UNSUPPORTED), ({4: -1}, INVALID), ({5: 0}, INVALID), ({6: 5}, UNSUPPORTED), ({12: 1}, UNSUPPORTED), ({6: 0, 12: 2}, UNSUPPORTED),
    ({12: 3}, UNSUPPORTED), ({13: None}, NO_SCRATCH), ({14: 16}, NO_SCRATCH), ({0: P + 1}, MISALIGNED), ({9: Q + 2}, MISALIGNED),
    ({2: S + 4}, MISALIGNED), ({13: C + 8}, MISALIGNED), ({9: P}, ALIAS), ({2: Q}, ALIAS), ({13: Q}, ALIAS), ({13: P}, ALIAS), ({13: S}, ALIAS),
])
def test_backward_refusals(lib, change, status):
    assert lib.embedding_backward(*_changed(BACKWARD, change)) == status


def test_backward_workspace(lib):
    def ask(*a):
        size = ctypes.c_size_t(7)
        return lib.embedding_backward_workspace(*a, size), size.value

    assert ask(0, 100, 64) == (OK, 0) and ask(10, 0, 64) == (OK, 0)
    status, size = ask(10, 100, 64)
    assert status == OK and 80 <= size <= 1 << 16
    for tokens in (1, 31, 32, 8192, 8193, 32768, 32769, 10**6, 2**31 - 1):
        status, size = ask(tokens, 2**31 - 2, 1 << 24)
        assert status == OK and size >= 8 * tokens
    for bad in ((-1, 1, 1), (2**31, 1, 1), (1, -1, 1), (1, 2**31 - 1, 1), (1, 1, 0), (1, 1, (1 << 24) + 1)):
        assert ask(*bad) == (INVALID, 0)
    assert lib.embedding_backward_workspace(1, 1, 1, None) == INVALID


#          logits stride type ids bytes tokens choices experts loss counts workspace bytes stream
BALANCE = [P, 64, 2, S, 8, 10, 2, 64, Q, Q + 4096, None, 0, None]


@pytest.mark.parametrize("change,status", [
    ({0: None}, INVALID), ({3: None}, INVALID), ({8: None}, INVALID), ({9: None}, INVALID), ({1: -1}, INVALID), ({2: 3}, UNSUPPORTED),
    ({4: 1}, UNSUPPORTED), ({5: -1}, INVALID), ({6: 0}, INVALID), ({6: 65}, INVALID), ({7: 0}, INVALID), ({7: 4097}, INVALID),
    ({5: 2**30, 6: 2}, INVALID), ({5: 10**6}, NO_SCRATCH), ({5: 10**6, 10: C, 11: 100}, NO_SCRATCH), ({5: 10**6, 10: C + 4, 11: 1 << 30}, MISALIGNED),
    ({0: P + 1}, MISALIGNED), ({3: S + 4}, MISALIGNED), ({8: Q + 2}, MISALIGNED), ({9: Q}, ALIAS), ({8: P}, ALIAS), ({9: S}, ALIAS),
])
def test_balance_refusals(lib, change, status):
    assert lib.expert_balance(*_changed(BALANCE, change)) == status


#                   grad logits stride type ids bytes tokens choices experts counts out stride stream
BALANCE_BACKWARD = [C, P, 64, 2, S, 8, 10, 2, 64, C + 4096, Q, 64, None]


@pytest.mark.parametrize("change,status", [
    ({0: None}, INVALID), ({1: None}, INVALID), ({4: None}, INVALID), ({9: None}, INVALID), ({10: None}, INVALID), ({2: -1}, INVALID),
    ({11: 63}, INVALID), ({3: 3}, UNSUPPORTED), ({5: 2}, UNSUPPORTED), ({7: 65}, INVALID), ({8: 4097}, INVALID), ({0: C + 2}, MISALIGNED),
    ({10: Q + 1}, MISALIGNED), ({10: P}, ALIAS), ({10: S}, ALIAS), ({10: C + 4096}, ALIAS), ({10: C}, ALIAS),
])
def test_balance_backward_refusals(lib, change, status):
    assert lib.expert_balance_backward(*_changed(BALANCE_BACKWARD, change)) == status


# tokens type | k, v, q, q_out | turns | starts lengths sequences | table stride columns pages page_size | caches | cache_type, scales
APPEND = ([8, 2, P, 2, 64, 128, 64, P + (1 << 16), 2, 64, 128, 64, P + (1 << 18), 4, 64, 256, 64, Q, 4, 64, 256, 64]
          + [S, 0, 0, 0, 0, 0, 32, 0] + [0, S + 4096, 8] + [S + 8192, 4, 4, 32, 16]
          + [C, 2048, 128, 64, C + (1 << 24), 2048, 128, 64] + [3, C + (1 << 28), 32, 2, 1, C + (1 << 29), 32, 2, 1])


@pytest.mark.parametrize("change,status", [
    ({0: -1}, INVALID), ({1: 5}, UNSUPPORTED), ({1: 3}, UNSUPPORTED), ({2: 0}, INVALID), ({8: 3}, INVALID), ({14: 32}, INVALID), ({29: 2}, INVALID),
    ({31: 0}, INVALID), ({37: 0}, INVALID), ({38: 0}, INVALID), ({39: 2047}, INVALID), ({42: C}, ALIAS), ({38: P}, ALIAS), ({17: P}, ALIAS),
    ({46: 2}, UNSUPPORTED), ({46: 5}, UNSUPPORTED), ({47: 0}, INVALID), ({48: 31}, INVALID), ({49: 1}, INVALID), ({50: 0}, INVALID), ({51: 0}, INVALID),
    ({47: C + (1 << 28) + 2}, MISALIGNED), ({47: C}, ALIAS), ({51: C + (1 << 24)}, ALIAS), ({51: C + (1 << 28)}, ALIAS), ({47: P}, ALIAS), ({47: Q}, ALIAS),
    ({47: S}, ALIAS), ({51: S + 4096}, ALIAS), ({51: S + 8192}, ALIAS), ({47: P + (1 << 18)}, ALIAS), ({48: 2**41}, INVALID),
])
def test_append_refusals(lib, change, status):
    a = _changed(APPEND, change)
    assert lib.paged_append_quantised(_capi.PAGED_APPEND_QUANTISED_ARGS.pack(*a), None) == status
    assert lib.paged_append_quantised(None, None) == INVALID


# tokens type cache_type | k, v | starts firsts sequences | table stride columns pages page_size | k_cache v_cache k_scales v_scales
READ = ([20, 2, 3, P, 2, 64, 128, 64, P + (1 << 16), 2, 64, 128, 64] + [S, S + 1024, 4] + [S + 4096, 4, 4, 32, 16]
        + [C, 2048, 128, 64, C + (1 << 24), 2048, 128, 64, C + (1 << 28), 32, 2, 1, C + (1 << 29), 32, 2, 1])


@pytest.mark.parametrize("change,status", [
    ({0: -1}, INVALID), ({1: 3}, UNSUPPORTED), ({2: 0}, UNSUPPORTED), ({2: 5}, UNSUPPORTED), ({2: 2}, INVALID), ({3: 0}, INVALID), ({9: 3}, INVALID),
    ({6: 64}, INVALID), ({13: 0}, INVALID), ({15: -1}, INVALID), ({16: 0}, INVALID), ({17: -1}, INVALID), ({20: 0}, INVALID), ({19: -1}, INVALID),
    ({21: 0}, INVALID), ({22: -1}, INVALID), ({29: 0}, INVALID), ({33: 0}, INVALID), ({30: -1}, INVALID), ({29: C + (1 << 28) + 1}, MISALIGNED),
    ({3: P + 1}, MISALIGNED), ({13: S + 2}, MISALIGNED), ({14: S + 1026}, MISALIGNED), ({8: P}, ALIAS), ({3: C}, ALIAS), ({8: C + (1 << 28)}, ALIAS),
    ({3: S}, ALIAS), ({3: S + 1024}, ALIAS), ({3: S + 4096}, ALIAS), ({8: C + (1 << 24) + 64}, ALIAS), ({2: 2, 21: C + 1, 29: 0, 33: 0}, MISALIGNED),
])
def test_read_refusals(lib, change, status):
    a = _changed(READ, change)
    assert lib.paged_read(_capi.PAGED_READ_ARGS.pack(*a), None) == status
    assert lib.paged_read(None, None) == INVALID


def test_nothing_to_do_is_fine(lib):
    assert lib.embedding_lookup(*_changed(LOOKUP, {0: None, 3: None, 5: 0, 9: None})) == OK
    assert lib.embedding_backward(*_changed(BACKWARD, {4: 0, 8: 1, 0: None, 2: None})) == OK
    assert lib.embedding_backward(*_changed(BACKWARD, {11: 0, 9: None})) == OK
    assert lib.expert_balance_backward(*_changed(BALANCE_BACKWARD, {6: 0, 1: None})) == OK
    assert lib.paged_append_quantised(_capi.PAGED_APPEND_QUANTISED_ARGS.pack(*_changed(APPEND, {0: 0})), None) == OK
    assert lib.paged_read(_capi.PAGED_READ_ARGS.pack(*_changed(READ, {0: 0})), None) == OK


@pytest.mark.no_gpu
def test_results_and_caches_that_lie_between_each_other(lib):
    """As far as the check of the pointers, which needs a device."""
    refused = (OK, ALIAS, INVALID)
    # results head by head in one array
    a = _changed(READ, {5: 64, 6: 256, 7: 128, 8: P + 128, 10: 64, 11: 256, 12: 128})
    assert lib.paged_read(_capi.PAGED_READ_ARGS.pack(*a), None) not in refused
    assert lib.paged_read(_capi.PAGED_READ_ARGS.pack(*_changed(a, {8: P + 126})), None) == ALIAS
    # caches page by page, whose elements are bytes
    a = _changed(APPEND, {39: 4096, 43: 4096, 42: C + 2048})
    assert lib.paged_append_quantised(_capi.PAGED_APPEND_QUANTISED_ARGS.pack(*a), None) not in refused
    assert lib.paged_append_quantised(_capi.PAGED_APPEND_QUANTISED_ARGS.pack(*_changed(a, {42: C + 2047})), None) == ALIAS


def test_binding_refusals():
    x, ids = torch.zeros(4, 8), torch.zeros(4, dtype=torch.int64)
    look, back = bm.embedding_lookup, bm.embedding_backward
    cases = [
        (lambda: look(x, ids.float()), "ids must be"), (lambda: look(x, ids[None]), "ids must be"), (lambda: look(x.t(), ids), "dense rows"),
        (lambda: look(x.double(), ids), "supported"), (lambda: look(x, ids), "current device"),
        (lambda: back(x, ids[:3], 5), "3 ids"), (lambda: back(x.long(), ids, 5), "supported"), (lambda: back(x, ids, 5), "current device"),
    ]
    choices = torch.zeros(4, 2, dtype=torch.int64)
    counts, one = torch.zeros(9, dtype=torch.int32), torch.zeros(())
    cases += [
        (lambda: bm.expert_balance(x, choices[:3]), "experts must be"), (lambda: bm.expert_balance(x, choices.float()), "experts must be"),
        (lambda: bm.expert_balance(x.long(), choices), "supported"), (lambda: bm.expert_balance(x, choices), "current device"),
        (lambda: bm.expert_balance_backward(one.double(), x, choices, counts), "one element"),
        (lambda: bm.expert_balance_backward(torch.zeros(2), x, choices, counts), "one element"),
        (lambda: bm.expert_balance_backward(one, x, choices, counts[:8]), "counts must"),
        (lambda: bm.expert_balance_backward(one, x, choices, counts), "current device"),
    ]
    h, n, table = torch.zeros(3, 2, 8), torch.zeros(3, dtype=torch.int32), torch.zeros(3, 2, dtype=torch.int32)
    cache, scales = torch.zeros(5, 4, 2, 8, dtype=torch.int8), torch.zeros(5, 4, 2)
    sides = dict(k_scales=scales, v_scales=scales)
    append, read = bm.paged_append, bm.paged_read
    cases += [
        (lambda: append(h, h, cache, cache, table, n), "k_scales"), (lambda: append(h, h, cache, cache, table, n, k_scales=scales), "v_scales"),
        (lambda: append(h, h, cache, cache, table, n, k_scales=scales[:4], v_scales=scales), "k_scales"),
        (lambda: append(h, h, cache, cache, table, n, k_scales=scales.half(), v_scales=scales), "k_scales"),
        (lambda: append(h, h, cache, cache.float(), table, n, **sides), "4-D"), (lambda: append(h, h, cache.float(), cache.float(), table, n, **sides), "8 bits"),
        (lambda: append(h, h, cache, cache, table, n, **sides), "current device"),
    ]
    starts = torch.zeros(4, dtype=torch.int32)
    cases += [
        (lambda: read(cache, cache, table, starts, 5), "read back"), (lambda: read(cache, cache, table, starts, dtype=torch.float16, **sides), "num_rows"),
        (lambda: read(cache.float(), cache.float(), table, starts, 5, dtype=torch.float16), "read back"),
        (lambda: read(cache[0], cache, table, starts, 5), "4-D"), (lambda: read(cache, cache, table.long(), starts, 5, dtype=torch.float16), "page_table must"),
        (lambda: read(cache, cache, table, starts[:3], 5, dtype=torch.float16), "starts must"),
        (lambda: read(cache, cache, table, starts, 5, firsts=starts, dtype=torch.float16), "firsts must"),
        (lambda: read(cache, cache, table, starts, 5, dtype=torch.float16, **sides), "current device"),
    ]
    for refused, message in cases:
        with pytest.raises(ValueError, match=message):
            refused()
