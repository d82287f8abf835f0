"""Caches of 8 bits: paged_append with scales, and paged_read, on the GPU.

What is not turned is compared exactly with the definition's own products and
quotients in 32 bits.  A turned key y is off by at most 8 * 2**-24 * (|a| +
|b|) of its pair (two products, a sum, sine and cosine within 2 ulp); its
value times its scale is then at most half a step of the 8-bit type away: 2**-4
of |y| or, for small ones, 2**-10 scales (e4m3), half a scale (whole numbers),
of what is rounded: y times the scale's reciprocal, each rounded to 32 bits,
which together move y / scale by 2 * 2**-24 of itself (and a little more of
second order), or 2 * 2**-24 * |y| times the scale.
"""

import pytest

import bmmc_index_transforms_gb300 as bm

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16
E4M3, I8 = torch.float8_e4m3fn, torch.int8
U32 = 2.0 ** -24
ROUND = {F32: 2.0 ** -24, F16: 2.0 ** -11, BF16: 2.0 ** -8}
TINY = {F32: 2.0 ** -149, F16: 2.0 ** -24, BF16: 2.0 ** -133}
MOST = {E4M3: 448.0, I8: 127.0}


def _gen(seed):
    g = torch.Generator("cuda")
    g.manual_seed(seed)
    return g


def _bytes(x):
    return x.view(torch.uint8) if x.dtype in MOST else x


def _freq(pairs):
    return 100.0 ** (-torch.arange(pairs, device="cuda") / max(1, pairs))


def _case(g, counts, page, Hq, Hk, Dk, Dv, dtype, cache, head_major, cached, spare=3):
    """New heads for sequences with `counts` new tokens each, pages in any order."""
    B, T = len(counts), sum(counts)
    lengths = torch.randint(0, cached + 1, (B,), generator=g, device="cuda")
    new = torch.tensor(counts, device="cuda")
    need = (lengths + new + page - 1) // page
    total = int(need.sum()) + spare
    columns = max(1, int(need.max()))
    pool = torch.randperm(total, generator=g, device="cuda").int()
    table = torch.full((B, columns), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(need.tolist()):
        table[b, :n] = pool[at:at + n]
        at += n
    c = dict(lengths=lengths.int(), starts=torch.cat([new.new_zeros(1), new.cumsum(0)]).int(), table=table, page=page,
             head_major=head_major, T=T)
    heads = torch.randn(T, Hq + 2 * Hk, max(Dk, Dv), generator=g, device="cuda").to(dtype)
    c["q"] = heads[:, :Hq, :Dk] if Hq else None
    c["k"], c["v"] = heads[:, Hq:Hq + Hk, :Dk], heads[:, Hq + Hk:, :Dv]
    lead = (total, Hk, page) if head_major else (total, page, Hk)
    c["caches"] = [torch.randint(0, 100, (*lead, D), generator=g, device="cuda", dtype=torch.uint8).view(cache) for D in (Dk, Dv)]
    c["scales"] = [torch.rand(lead, generator=g, device="cuda") for _ in range(2)]
    return c


def _entries(x, head_major):
    """[pages * page, heads, ...] of a cache or its scales."""
    x = _bytes(x)
    return (x.transpose(1, 2) if head_major else x).flatten(0, 1)


def _where(c, t_of_seq=None):
    """(token, row of _entries) of the tokens that have a page, and every token's place."""
    T, page, pages = c["T"], c["page"], c["caches"][0].shape[0]
    t = torch.arange(T, device="cuda")
    starts = c["starts"].long()
    seq = torch.searchsorted(starts[:-1].contiguous(), t, right=True) - 1
    ok = (seq >= 0) & (t < starts[(seq + 1).clamp(min=0)])
    place = torch.where(ok, c["lengths"].long()[seq.clamp(min=0)] + t - starts[seq.clamp(min=0)], 0)
    column = place // page
    inside = ok & (column < c["table"].shape[1])
    entry = torch.where(inside, c["table"].long()[seq.clamp(min=0), column.clamp(max=c["table"].shape[1] - 1)], -1)
    ok = inside & (entry >= 0) & (entry < pages)
    return ok.nonzero().flatten(), (entry * page + place % page)[ok], place


def _turned(x, angle, interleaved):
    """(the turned heads in 64 bits, how far they may be off)"""
    x = x.double()
    P = angle.shape[1] if angle is not None else 0
    off = torch.zeros_like(x)
    if not P:
        return x, off
    y = x.clone()
    a, b = (slice(0, 2 * P, 2), slice(1, 2 * P, 2)) if interleaved else (slice(0, P), slice(P, 2 * P))
    cos, sin = torch.cos(angle)[:, None], torch.sin(angle)[:, None]
    y[..., a], y[..., b] = x[..., a] * cos - x[..., b] * sin, x[..., b] * cos + x[..., a] * sin
    size = 8 * U32 * (x[..., a].abs() + x[..., b].abs())
    off[..., a], off[..., b] = size, size
    return y, off


def _quantised(x, cache):
    """(codes, scales) by the definition, in 32 bits."""
    scale = (x.float().abs().amax(-1) * torch.tensor(1.0 / MOST[cache], device="cuda")).clamp(min=2.0 ** -126)
    y = x.float() * (torch.ones_like(scale) / scale)[..., None]
    y = y.clamp(-MOST[cache], MOST[cache])
    return (y.round() if cache == I8 else y).to(cache), scale


def _check_append(c, freq=None, interleaved=False, positions=None, axes=None, starts=True, in_place=False):
    cache = c["caches"][0].dtype
    before = [x.clone() for x in c["caches"] + c["scales"]]
    q = c["q"].clone() if c["q"] is not None else None
    got_q = bm.paged_append(c["k"], c["v"], *c["caches"], c["table"], c["lengths"], starts=c["starts"] if starts else None, q=q,
                            q_out=q if in_place else None, positions=positions, inv_freq=freq, pair_axes=axes,
                            interleaved=interleaved, head_major=c["head_major"], k_scales=c["scales"][0], v_scales=c["scales"][1])
    at, row, place = _where(c)
    angle = None
    if freq is not None:
        if positions is None:
            p = place.float()[:, None] * (torch.ones_like(freq) if axes is None else (axes == 0).float())
        else:
            p = positions[axes.long()].t().float() if axes is not None else positions.view(-1, 1).float()
        angle = (p * freq).double()
    for i, x in enumerate((c["k"], c["v"])):
        turn = angle if i == 0 else None
        old, old_scale = (_entries(before[j], c["head_major"]) for j in (i, 2 + i))
        new, new_scale = (_entries(m, c["head_major"]) for m in (c["caches"][i], c["scales"][i]))
        rest = torch.ones(old.shape[0], dtype=torch.bool, device="cuda")
        rest[row] = False
        assert torch.equal(new[rest], old[rest]) and torch.equal(new_scale[rest], old_scale[rest])
        if turn is None:
            codes, scale = _quantised(x[at], cache)
            assert torch.equal(new_scale[row], scale)
            assert torch.equal(new[row], _bytes(codes))
            continue
        y, off = (m[at] for m in _turned(x, turn, interleaved))
        scale = new_scale[row].double()
        most, slack = y.abs().amax(-1) / MOST[cache], off.amax(-1) / MOST[cache]
        assert bool(((scale - most).abs() <= slack + 4 * U32 * most + 2.0 ** -126).all())
        value = new[row].view(cache).double() * scale[..., None]
        step = scale[..., None] / 2 if cache == I8 else torch.maximum(2.0 ** -4 * (y.abs() + off), 2.0 ** -10 * scale[..., None])
        # |value - y| <= step(y') + |y' - y|, y' = y + off and the two roundings of y' / scale: 2 * U32 * |y'|;
        # the step of y' is within 2**-20 of y's
        assert bool(((value - y).abs() <= (step + off) * (1 + 2.0 ** -20) + 2 * U32 * (y.abs() + off)).all())
    if q is None:
        assert got_q is None
        return
    want, off = _turned(c["q"], angle, interleaved)
    d = c["q"].dtype
    assert got_q.dtype == d and (not in_place or got_q.data_ptr() == q.data_ptr())
    assert bool(((got_q.double() - want).abs() <= off + ROUND[d] * (want.abs() + off) + TINY[d]).all())


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("cache", [E4M3, I8])
@pytest.mark.parametrize("head_major", [False, True])
@pytest.mark.parametrize("B,page,Hq,Hk,Dk,Dv,pairs,cached", [
    (1, 1, 0, 1, 8, 8, 4, 0), (1, 16, 8, 1, 128, 128, 64, 100), (70, 16, 32, 8, 128, 128, 64, 50), (300, 64, 4, 4, 64, 64, 32, 200),
    (5, 3, 6, 3, 20, 12, 8, 9), (17, 100, 2, 2, 36, 34, 16, 150), (3, 16, 2, 2, 10, 7, 5, 20), (9, 8, 4, 1, 256, 256, 100, 30), (2, 4, 2, 1, 1000, 514, 400, 5),
    (4, 16, 2, 16, 1, 1, 0, 9), (33, 16, 8, 8, 80, 96, 40, 60), (6, 16, 1, 1, 66, 33, 33, 40), (40, 16, 4, 2, 192, 128, 32, 40),
])
def test_append_one_token_each(B, page, Hq, Hk, Dk, Dv, pairs, cached, head_major, cache, dtype):
    c = _case(_gen(B), [1] * B, page, Hq, Hk, Dk, Dv, dtype, cache, head_major, cached)
    _check_append(c, starts=False)
    if pairs:
        _check_append(c, _freq(pairs), starts=False, in_place=True)
        _check_append(c, _freq(pairs), interleaved=True)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("cache", [E4M3, I8])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("counts,page,cached,D", [
    ([5], 16, 0, 64), ([0, 3, 0, 0, 40, 1], 16, 20, 64), ([16, 16, 16], 16, 0, 128), ([33, 0, 129, 7], 1, 5, 96),
    ([1] * 100 + [0] * 60 + [3] * 100, 7, 30, 32), ([2000, 1, 3001], 64, 1000, 128), ([0, 0, 0, 9], 100, 250, 80), ([4000, 0, 2100], 16, 40, 66),
])
def test_append_ragged(counts, page, cached, D, interleaved, cache, dtype):
    g = _gen(len(counts))
    c = _case(g, counts, page, 4, 2, D, D, dtype, cache, False, cached)
    _check_append(c, _freq(D // 2), interleaved)
    positions = torch.randint(0, 4096, (3, c["T"]), generator=g, device="cuda")
    axes = (torch.arange(D // 4, device="cuda") % 3).int()
    _check_append(c, _freq(D // 4), interleaved, positions, axes)
    _check_append(c, _freq(D // 2 - 3), interleaved, positions[:1].int())


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("Dk,Dv,pairs", [(512, 256, 256), (520, 264, 256), (1024, 1032, 512), (8192, 8190, 4096), (4097, 8191, 1025)])
def test_append_and_read_of_wide_heads(Dk, Dv, pairs, interleaved):
    c = _case(_gen(Dk), [3, 0, 5], 4, 2, 2, Dk, Dv, BF16, E4M3, False, 6)
    _check_append(c, _freq(pairs), interleaved)
    _check_append(c)
    _check_read(c, F32, c["lengths"])


@pytest.mark.parametrize("cache", [E4M3, I8])
def test_append_skips_tokens_without_a_page(cache):
    c = _case(_gen(1), [6, 9, 0, 8], 4, 3, 2, 16, 16, F32, cache, False, 6)
    c["table"][0, 1] = -1
    c["table"][1] = c["caches"][0].shape[0]  # one past the pool
    c["table"][3, 0] = -(2**31)
    c["table"] = c["table"][:, :3]  # rows that are not dense, and fewer entries than sequence 3 needs
    c["lengths"][3] = 6
    _check_append(c, _freq(8))
    c["starts"] += 2  # two tokens before the first sequence, the last ones cut off
    _check_append(c, _freq(8))
    c["starts"] -= 4  # starts before the first token; tokens behind the last sequence
    _check_append(c, _freq(8))


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("cache", [E4M3, I8])
@pytest.mark.parametrize("D", [64, 66, 33])
def test_heads_of_zeros_tiny_values_infinities_and_nan(D, cache, dtype):
    g = _gen(D)
    c = _case(g, [8], 16, 0, 1, D, D, dtype, cache, False, 0)
    x = torch.randn(8, 1, D, generator=g, device="cuda").to(dtype)
    x[0] = 0
    x[1] = torch.finfo(dtype).smallest_normal * 2.0 ** -3  # subnormal, and for f32 and bf16 below the least scale
    x[2] *= torch.finfo(dtype).max / 8
    x[3, 0, 5], x[4, 0, 6], x[5, 0, 7] = float("inf"), float("-inf"), float("nan")
    x[6] = 0
    x[6, 0, D - 1] = -torch.finfo(dtype).max
    for freq in (None, _freq(D // 2)):
        keys = x if freq is None else torch.randn_like(x)
        bm.paged_append(keys, x, *c["caches"], c["table"], c["lengths"], starts=c["starts"], inv_freq=freq,
                        k_scales=c["scales"][0], v_scales=c["scales"][1])
        at, row, _ = _where(c)
        fine = torch.tensor([0, 1, 2, 6, 7], device="cuda")
        codes, scale = _quantised(x[fine], cache)
        values, scales = _entries(c["caches"][1], False)[row], _entries(c["scales"][1], False)[row]
        assert torch.equal(values[fine], _bytes(codes)) and torch.equal(scales[fine], scale)
        assert bool(scales[3:6].isnan().all())
        if freq is None:
            assert torch.equal(_entries(c["caches"][0], False)[row], values)
        k, v = bm.paged_read(*c["caches"], c["table"], c["starts"], 8, k_scales=c["scales"][0], v_scales=c["scales"][1], dtype=F32)
        assert bool(v[3:6].isnan().all()) and torch.isfinite(v[fine]).all() and not v[0].any()
        assert float(v[6, 0, D - 1]) < 0 and not v[6, 0, :D - 1].any()


def test_append_fused_views_and_scales_beside_each_other():
    """q, k and v as slices of one projection, both caches and both scales in
    one allocation, queries in place."""
    g = _gen(4)
    c = _case(g, [10, 0, 30], 16, 8, 2, 64, 64, BF16, E4M3, False, 40)
    heads = torch.randn(c["T"], 12, 64, generator=g, device="cuda").to(BF16)
    pages = c["caches"][0].shape[0]
    both = torch.zeros(pages, 2, 16, 2, 64, dtype=torch.uint8, device="cuda").view(E4M3)
    scales = torch.zeros(2, pages, 16, 2, device="cuda")
    c.update(q=heads[:, :8], k=heads[:, 8:10], v=heads[:, 10:], caches=[both[:, 0], both[:, 1]], scales=[scales[0], scales[1]])
    _check_append(c, _freq(32))
    rest = heads[:, 8:].clone()
    want = bm.paged_append(c["k"], c["v"], *c["caches"], c["table"], c["lengths"], starts=c["starts"], q=c["q"], inv_freq=_freq(32),
                           k_scales=scales[0], v_scales=scales[1])
    got = bm.paged_append(c["k"], c["v"], *c["caches"], c["table"], c["lengths"], starts=c["starts"], q=c["q"], q_out=c["q"],
                          inv_freq=_freq(32), k_scales=scales[0], v_scales=scales[1])
    assert got.data_ptr() == heads.data_ptr() and torch.equal(got, want) and torch.equal(heads[:, 8:], rest)


# ---- read ------------------------------------------------------------------------

def _check_read(c, dtype, firsts=None, rows=None):
    """Reads the case's sequences back; lengths stand for the first entries."""
    rows = c["T"] if rows is None else rows
    cache = c["caches"][0].dtype
    scales = dict(k_scales=c["scales"][0], v_scales=c["scales"][1]) if cache in MOST else {}
    got = bm.paged_read(*c["caches"], c["table"], c["starts"], rows, firsts=firsts, dtype=dtype, head_major=c["head_major"], **scales)
    at, row, _ = _where(dict(c, T=rows, lengths=torch.zeros_like(c["lengths"]) if firsts is None else firsts))
    for i in range(2):
        x = _entries(c["caches"][i], c["head_major"])[row].view(cache)
        want = torch.zeros(rows, x.shape[1], x.shape[2], dtype=dtype, device="cuda")
        if cache in MOST:
            x = (x.float() * _entries(c["scales"][i], c["head_major"])[row][..., None]).to(dtype)
        want[at] = x
        assert got[i].dtype == dtype and torch.equal(got[i], want)
    return got


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("cache", [E4M3, I8, None])
@pytest.mark.parametrize("head_major", [False, True])
@pytest.mark.parametrize("counts,page,Hk,Dk,Dv,cached", [
    ([1], 16, 1, 8, 8, 0), ([1] * 40, 16, 8, 128, 128, 30), ([5, 0, 60, 17], 16, 4, 96, 96, 0), ([0, 0, 300, 1], 1, 2, 64, 64, 40),
    ([3, 9], 4, 3, 20, 12, 5), ([100, 1], 100, 2, 36, 34, 150), ([7], 16, 2, 10, 7, 20), ([50, 2], 8, 1, 256, 256, 30), ([6], 4, 1, 1000, 514, 5),
    ([9, 3], 16, 16, 1, 1, 9), ([2000, 0, 3001], 64, 8, 128, 128, 100), ([33, 5], 16, 8, 80, 96, 60), ([400], 16, 2, 66, 33, 40),
])
def test_read(counts, page, Hk, Dk, Dv, cached, head_major, cache, dtype):
    c = _case(_gen(len(counts) + Dk), counts, page, 0, Hk, Dk, Dv, dtype, cache or E4M3, head_major, cached)
    if cache is None:  # values of the result's own type are moved as they are
        c["caches"] = [torch.randn(m.shape, device="cuda").to(dtype) for m in c["caches"]]
    _check_read(c, dtype)
    _check_read(c, dtype, c["lengths"], c["T"] + 5)
    c["table"][0, 0] = -1
    c["table"][-1, -1] = c["caches"][0].shape[0]
    _check_read(c, dtype, c["lengths"])


@pytest.mark.parametrize("cache", [E4M3, BF16])
def test_read_rows_of_no_sequence_and_entries_without_a_page(cache):
    c = _case(_gen(2), [6, 9, 0, 8], 4, 0, 2, 16, 16, BF16, E4M3, False, 6)
    if cache == BF16:
        c["caches"] = [torch.randn(m.shape, device="cuda").to(BF16) for m in c["caches"]]
    c["table"] = c["table"][:, :2]
    firsts = torch.tensor([0, 2**31 - 3, -2, -5], dtype=torch.int32, device="cuda")
    _check_read_zeros(c, firsts)
    c["starts"] += 3
    _check_read_zeros(c, firsts)
    c["starts"] -= 5
    _check_read_zeros(c, firsts)
    c["table"] = c["table"][:, :0]
    got = bm.paged_read(*c["caches"], c["table"], c["starts"], 40, dtype=BF16, **_scales(c))
    assert not got[0].any() and not got[1].any()


def _scales(c):
    return dict(k_scales=c["scales"][0], v_scales=c["scales"][1]) if c["caches"][0].dtype in MOST else {}


def _check_read_zeros(c, firsts):
    got = bm.paged_read(*c["caches"], c["table"], c["starts"], 40, firsts=firsts, dtype=BF16, **_scales(c))
    pages, page = c["caches"][0].shape[:2]
    starts, table = c["starts"].tolist(), c["table"].tolist()
    for r in range(40):
        b = max((i for i in range(4) if starts[i] <= r), default=-1)
        e = firsts.tolist()[b] + r - starts[b]
        there = b >= 0 and r < starts[b + 1] and 0 <= e and e // page < len(table[b]) and 0 <= table[b][e // page] < pages
        for i in range(2):
            want = torch.zeros_like(got[i][r])
            if there:
                x = _bytes(c["caches"][i])[table[b][e // page], e % page].view(c["caches"][i].dtype)
                want = x if x.dtype == BF16 else (x.float() * c["scales"][i][table[b][e // page], e % page][:, None]).to(BF16)
            assert torch.equal(got[i][r], want), r


def test_read_pages_that_are_shared_and_given_outputs():
    g = _gen(3)
    c = _case(g, [20, 20, 7], 8, 0, 2, 64, 64, F16, I8, True, 0)
    c["table"][1] = c["table"][0]
    k, v = _check_read(c, F16)
    assert torch.equal(k[:20], k[20:40])
    kv = torch.full((47, 2, 3, 72), 7.0, dtype=F16, device="cuda")
    a, b = bm.paged_read(*c["caches"], c["table"], c["starts"], k_out=kv[:, :, 0, :64], v_out=kv[:, :, 2, 8:], head_major=True, **_scales(c))
    assert a.data_ptr() == kv.data_ptr() and torch.equal(a, k) and torch.equal(b, v)
    assert bool((kv[:, :, 1] == 7).all()) and bool((kv[:, :, 0, 64:] == 7).all()) and bool((kv[:, :, 2, :8] == 7).all())


def test_read_nothing():
    c = _case(_gen(6), [0, 0], 4, 2, 1, 8, 8, F32, E4M3, False, 3)
    k, v = _check_read(c, F32)
    assert k.shape == (0, 1, 8)
    _check_append(c, _freq(4))
    k, v = bm.paged_read(*c["caches"], c["table"][:0], c["starts"][:1], 3, dtype=F32, **_scales(c))
    assert not k.any() and not v.any()


def test_offsets_beyond_32_bits():
    page, H, D = 16, 8, 256
    pages = 2**32 // (page * H * D) + 10  # over 2**32 bytes
    caches = [torch.zeros(pages, page, H, D, dtype=torch.int8, device="cuda") for _ in range(2)]
    scales = [torch.zeros(pages, page, H, device="cuda") for _ in range(2)]
    k, v = torch.ones(2, H, D, dtype=BF16, device="cuda"), torch.full((2, H, D), 2.0, dtype=BF16, device="cuda")
    table = torch.tensor([[pages - 1], [0]], dtype=torch.int32, device="cuda")
    lengths = torch.tensor([15, 3], dtype=torch.int32, device="cuda")
    bm.paged_append(k, v, *caches, table, lengths, k_scales=scales[0], v_scales=scales[1])
    for m, s, value in zip(caches, scales, (1.0, 2.0)):
        for at in ((pages - 1, 15), (0, 3)):
            assert bool((m[at] == 127).all()) and bool((s[at] == torch.tensor(value) * torch.tensor(1 / 127)).all())
            m[at] = 0
        assert not any(bool(part.any()) for part in m.split(10000))
        m[pages - 1, 15] = 127
    starts = torch.tensor([0, 1, 1], dtype=torch.int32, device="cuda")
    got = bm.paged_read(*caches, table, starts, 1, firsts=lengths, k_scales=scales[0], v_scales=scales[1], dtype=BF16)
    assert bool((got[0] == 1).all()) and bool((got[1] == 2).all())


def test_read_back_of_what_was_appended_in_a_graph():
    """A decoding loop: append one token each, read all back; captured once
    and replayed, and the calls on two streams at once."""
    g = _gen(7)
    c = _case(g, [1] * 12, 8, 4, 2, 64, 64, BF16, E4M3, False, 40)
    freq, rows = _freq(32), 12 * 50
    starts = torch.zeros(13, dtype=torch.int32, device="cuda")

    def step(stream=None):
        q = bm.paged_append(c["k"], c["v"], *c["caches"], c["table"], c["lengths"], q=c["q"], inv_freq=freq, stream=stream, **_scales(c))
        starts[1:] = torch.cumsum(c["lengths"] + 1, 0)
        return (q, *bm.paged_read(*c["caches"], c["table"], starts, rows, dtype=BF16, stream=stream, **_scales(c)))

    want = [x.clone() for x in step()]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for x in c["caches"]:
        _bytes(x)[:] = 1
    before = [x.clone() for x in c["caches"]]
    step()
    want = [x.clone() for x in step()]
    for x, old in zip(c["caches"], before):
        _bytes(x).copy_(_bytes(old))
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    outs, streams = [], [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(10):
        for st in streams:
            outs.append(bm.paged_read(*c["caches"], c["table"], starts, rows, dtype=BF16, stream=st, **_scales(c)))
    torch.cuda.synchronize()
    for o in outs:
        assert torch.equal(o[0], want[1]) and torch.equal(o[1], want[2])
