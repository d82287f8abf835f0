"""The operators of a decoder layer that move tokens by maps known only on the device, as cases to measure:

  sort              expert_sort: the choices of a router, sorted by expert
  dispatch          expert_dispatch: each token's row copied to the rows of its choices
  combine           expert_combine: the rows of a token's choices added up with the router's weights
  dispatch_backward expert_combine without weights, which is the gradient of dispatch
  combine_backward  expert_combine_backward: the gradients of combine by the rows and by the weights
  rotary            rotary: positions of one or several axes rotated into queries or keys; inverse for the gradient
  append            paged_append: keys and values written to a paged cache, keys and queries rotated on the way

A case is a dict of plain values; "op" is one of the names above."""
import math

import torch

own = False  # False: the plain form below; True: the calls of bmmc_index_transforms_gb300

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "f16": 2, "bf16": 2}


def listed():
    return [
        # one decoding step of 48 sequences, some slots of the batch empty: the router's choices as topk gives them
        {"name": "sort decode", "op": "sort", "tokens": 48, "choices": 8, "experts": 128, "ids": "i64", "empty": 0.1},
        # a full training or prefill batch
        {"name": "sort batch", "op": "sort", "tokens": 65521, "choices": 8, "experts": 256, "ids": "i32", "empty": 0.02},
        # a decoding step's rows to their experts: latency
        {"name": "dispatch decode", "op": "dispatch", "type": "bf16", "tokens": 32, "choices": 4, "experts": 32, "hidden": 2048, "empty": 0.1},
        # a prefill batch's rows to their experts: bandwidth, eight rows written for one read
        {"name": "dispatch batch", "op": "dispatch", "type": "bf16", "tokens": 16384, "choices": 8, "experts": 128, "hidden": 4096, "empty": 0.02},
        # a decoding step's rows back, weighted
        {"name": "combine decode", "op": "combine", "type": "bf16", "weights": "f32", "tokens": 32, "choices": 8, "experts": 128, "hidden": 4096, "empty": 0.1},
        # the gradient by the tokens in a training step in 32 bits, odd sizes
        {"name": "dispatch backward odd f32", "op": "dispatch_backward", "type": "f32", "tokens": 40961, "choices": 2, "experts": 8, "hidden": 1031, "empty": 0.05},
        # a small training micro-batch in half precision, weights in the rows' type
        {"name": "combine backward small", "op": "combine_backward", "type": "f16", "weights": "rows", "tokens": 509, "choices": 2, "experts": 8, "hidden": 1024, "empty": 0.02},
        # a training batch: the largest of the list
        {"name": "combine backward batch", "op": "combine_backward", "type": "bf16", "weights": "f32", "tokens": 16384, "choices": 8, "experts": 64, "hidden": 4096, "empty": 0.02},
        # queries of one decoding step, one axis: latency
        {"name": "rotary decode", "op": "rotary", "type": "f16", "tokens": 64, "heads": 16, "dim": 64, "rotary_dim": 64, "axes": 1, "interleaved": False, "inverse": False, "fused": True},
        # the gradient of image and video tokens' queries in 32 bits: three axes, adjacent pairs, part of the head rotated
        {"name": "rotary backward 3 axes", "op": "rotary", "type": "f32", "tokens": 10007, "heads": 12, "dim": 96, "rotary_dim": 64, "axes": 3, "interleaved": True, "inverse": True, "fused": False},
        # one token for each of 256 sequences: a decoding step's append, the queries rotated with it
        {"name": "append decode", "op": "append", "type": "bf16", "sequences": 256, "tokens": 256, "q_heads": 32, "kv_heads": 8, "dim": 128, "rotary_dim": 128, "axes": 1, "interleaved": False, "page": 16, "cached": 500, "head_major": False},
        # prompts of uneven lengths appended to what they had, three axes
        {"name": "append prompts", "op": "append", "type": "bf16", "sequences": 13, "tokens": 16001, "q_heads": 32, "kv_heads": 8, "dim": 128, "rotary_dim": 128, "axes": 3, "interleaved": False, "page": 64, "cached": 3000, "head_major": True},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["sort", "dispatch", "combine", "dispatch_backward", "combine_backward", "rotary", "rotary", "append", "append"])
    type_ = rng.choice(["f32", "f16", "bf16", "bf16"])
    if op == "sort":
        experts = _log(rng, 2, 512)
        return {"op": op, "tokens": _log(rng, 1, 65536), "choices": rng.randint(1, min(8, experts)), "experts": experts, "ids": rng.choice(["i32", "i64"]), "empty": rng.choice([0.0, 0.05, 0.5])}
    if op in ("dispatch", "combine", "dispatch_backward", "combine_backward"):
        experts = _log(rng, 2, 256)
        choices = rng.randint(1, min(8, experts))
        # a multiple of 8 mostly, as models have it; else any width
        hidden = _log(rng, 8, 1024) * 8 if rng.random() < 0.75 else _log(rng, 1, 4097)
        hidden += 8 if hidden == 3072 else 0
        most = (16384 * 8 * 4096 * 2) // (choices * hidden * SIZE[type_])
        c = {"op": op, "type": type_, "tokens": _log(rng, 1, max(1, min(65536, most))), "choices": choices, "experts": experts, "hidden": hidden, "empty": rng.choice([0.0, 0.05, 0.3])}
        if op in ("combine", "combine_backward"):
            c["weights"] = rng.choice(["f32", "rows"])
        return c
    dim = rng.choice([32, 64, 80, 96, 128, 192, 256, 66, 10])
    rotary_dim = dim if rng.random() < 0.6 else 2 * rng.randint(1, dim // 2)
    axes = min(rng.choice([1, 1, 2, 3]), rotary_dim // 2)
    c = {"op": op, "type": type_, "dim": dim, "rotary_dim": rotary_dim, "axes": axes, "interleaved": rng.random() < 0.4}
    if op == "rotary":
        heads = _log(rng, 1, 64)
        most = (16384 * 8 * 4096) // (heads * dim * SIZE[type_])
        return {**c, "tokens": _log(rng, 1, min(65536, most)), "heads": heads, "inverse": rng.random() < 0.5, "fused": rng.random() < 0.5}
    kv_heads = _log(rng, 1, 16)
    q_heads = kv_heads * rng.choice([0, 1, 4, 8])
    sequences = _log(rng, 1, 512)
    tokens = sequences if rng.random() < 0.5 else max(sequences, _log(rng, 1, 16384))
    return {**c, "sequences": sequences, "tokens": tokens, "q_heads": q_heads, "kv_heads": kv_heads, "page": rng.choice([1, 16, 64, 100]), "cached": _log(rng, 1, max(1, min(4096, 65536 // sequences))), "head_major": rng.random() < 0.5}


# ---- inputs ------------------------------------------------------------------------------------------------------

def _route(case, g):
    """A router's choices: distinct experts by score, some experts more popular than others, the last tokens of the
    batch empty and a few choices more left out."""
    T, K, E = case["tokens"], case["choices"], case["experts"]
    score = torch.randn(T, E, generator=g, device="cuda") + 1.5 * torch.randn(E, generator=g, device="cuda")
    top, ids = score.topk(K, dim=1)
    weights = torch.softmax(top, dim=1)
    out = torch.rand(T, K, generator=g, device="cuda") < case["empty"] / 2
    out[T - int(T * case["empty"] / 2):] = True
    return ids.masked_fill(out, -1), weights


def _prepare_rotation(case, g):
    """Frequencies, which axis turns which pair, and positions: of one axis, sequences one after another; of
    several, text whose axes agree followed by frames of an image grid."""
    T, pairs, axes = case["tokens"], case["rotary_dim"] // 2, case["axes"]
    freq = 10000.0 ** (-torch.arange(pairs, device="cuda", dtype=torch.float32) / pairs)
    if axes == 1:
        first = int(torch.randint(0, 512, (), generator=g, device="cuda"))
        return freq, None, ((torch.arange(T, device="cuda") + first) % 8192).to(torch.int32)[None]
    i = torch.arange(T, device="cuda")
    text = T // 4
    j = (i - text).clamp(min=0)
    width = int(torch.randint(20, 60, (), generator=g, device="cuda"))
    grid = torch.stack([j // (width * 24), j // width % 24, j % width])[:axes]
    positions = torch.where(i < text, i, text + grid).to(torch.int32)
    pair = torch.arange(pairs, device="cuda")
    pair_axes = (pair % axes if case["interleaved"] else pair * axes // pairs).to(torch.int32)
    return freq, pair_axes, positions.contiguous()


def prepare(case, seed):
    g = torch.Generator("cuda")
    g.manual_seed(seed)
    op, s = case["op"], {"case": case}
    if op in ("sort", "dispatch", "combine", "dispatch_backward", "combine_backward"):
        ids, weights = _route(case, g)
        if op == "sort":
            return {**s, "ids": ids.to(torch.int32 if case["ids"] == "i32" else torch.int64)}
        T, K, H, type_ = case["tokens"], case["choices"], case["hidden"], TYPES[case["type"]]
        s["slot"] = _sort(ids, case["experts"])[0]
        if op in ("dispatch", "combine_backward"):
            s["x"] = torch.randn(T, H, generator=g, device="cuda", dtype=type_)
        if op != "dispatch":
            s["rows"] = torch.randn(T * K, H, generator=g, device="cuda", dtype=type_)
        if op in ("combine", "combine_backward"):
            s["weights"] = weights.to(type_ if case["weights"] == "rows" else torch.float32)
        return s
    T, D, type_ = case["tokens"], case["dim"], TYPES[case["type"]]
    s["freq"], s["pair_axes"], s["positions"] = _prepare_rotation(case, g)
    if op == "rotary":
        H = case["heads"]
        # fused: a slice of the product that gives queries, keys and values together
        x = torch.randn(T, H + 2 if case["fused"] else H, D, generator=g, device="cuda", dtype=type_)
        return {**s, "x": x[:, :H]}
    B, Hq, Hk, page = case["sequences"], case["q_heads"], case["kv_heads"], case["page"]
    qkv = torch.randn(T, Hq + 2 * Hk, D, generator=g, device="cuda", dtype=type_)
    s["q"], s["k"], s["v"] = qkv[:, :Hq] if Hq else None, qkv[:, Hq:Hq + Hk], qkv[:, Hq + Hk:]
    if T == B:
        new = torch.ones(B, dtype=torch.int64, device="cuda")
        s["starts"] = None
    else:  # uneven parts of the tokens, some sequences without any
        cut = torch.randint(0, T + 1, (B - 1,), generator=g, device="cuda").sort()[0]
        starts = torch.cat([cut.new_zeros(1), cut, cut.new_full((1,), T)])
        new = starts[1:] - starts[:-1]
        s["starts"] = starts.to(torch.int32)
    lengths = torch.randint(0, case["cached"] + 1, (B,), generator=g, device="cuda")
    need = (lengths + new + page - 1) // page
    total = B * ((case["cached"] + page - 1) // page + 2) + T // page  # what the longest sequences need at most
    columns = int(need.max())
    # the pages that each sequence holds lie anywhere in the pool; the rest of its table is empty
    at = torch.cumsum(need, 0) - need
    column = torch.arange(columns, device="cuda")
    pool = torch.randperm(total, generator=g, device="cuda")
    table = torch.where(column < need[:, None], pool[(at[:, None] + column).clamp(max=total - 1)], -1)
    s["table"], s["lengths"] = table.to(torch.int32), lengths.to(torch.int32)
    if case["axes"] == 1:
        s["positions"] = None  # they follow from the lengths
    shape = (total, Hk, page, D) if case["head_major"] else (total, page, Hk, D)
    s["k_cache"] = torch.randn(shape, generator=g, device="cuda", dtype=type_)
    s["v_cache"] = torch.randn(shape, generator=g, device="cuda", dtype=type_)
    return s


# ---- the plain forms ---------------------------------------------------------------------------------------------

def _sort(ids, experts):
    flat = ids.reshape(-1).to(torch.int64)
    key = torch.where((flat >= 0) & (flat < experts), flat, experts)
    by, order = torch.sort(key, stable=True)
    slot = torch.empty_like(order)
    slot[order] = torch.arange(order.numel(), device=order.device)
    slot = torch.where(key < experts, slot, ~slot)
    source = torch.where(by < experts, order, ~order)
    offsets = torch.searchsorted(by, torch.arange(experts + 1, device=by.device))
    return slot.view(ids.shape).to(torch.int32), source.to(torch.int32), offsets.to(torch.int32)


def _turns(positions, freq, pair_axes):
    """cos and sin of every token's pairs, in 32 bits: [T, pairs] each."""
    p = positions.to(torch.float32)
    p = p[0][:, None] if pair_axes is None else p[pair_axes.long()].t()
    angle = p * freq
    return torch.cos(angle), torch.sin(angle)


def _rotate(x, cos, sin, interleaved):
    pairs = cos.shape[1]
    cos, sin, y = cos[:, None], sin[:, None], x.float()
    part = y[..., :2 * pairs]
    a, b = (part[..., 0::2], part[..., 1::2]) if interleaved else (part[..., :pairs], part[..., pairs:])
    a, b = a * cos - b * sin, b * cos + a * sin
    turned = torch.stack([a, b], -1).flatten(-2) if interleaved else torch.cat([a, b], -1)
    return torch.cat([turned, y[..., 2 * pairs:]], -1).to(x.dtype)


def _plain(s):
    case, op = s["case"], s["case"]["op"]
    if op == "sort":
        return _sort(s["ids"], case["experts"])
    if op in ("dispatch", "combine", "dispatch_backward", "combine_backward"):
        slot = s["slot"]
        routed, row = slot >= 0, torch.where(slot >= 0, slot, ~slot).long()
    if op == "dispatch":
        rows = s["x"].new_empty(slot.numel(), s["x"].shape[1])
        rows[row] = torch.where(routed[..., None], s["x"][:, None], 0)
        return rows
    if op == "dispatch_backward":
        return torch.where(routed[..., None], s["rows"][row].float(), 0).sum(1).to(s["rows"].dtype)
    if op in ("combine", "combine_backward"):
        w = torch.where(routed, s["weights"].float(), 0)
        picked = torch.where(routed[..., None], s["rows"][row].float(), 0)
        if op == "combine":
            return (w[..., None] * picked).sum(1).to(s["rows"].dtype)
        grad = s["x"].float()[:, None]
        grad_rows = torch.empty_like(s["rows"])
        grad_rows[row] = (w[..., None] * grad).to(grad_rows.dtype)
        return grad_rows, (picked * grad).sum(2).to(s["weights"].dtype)
    if op == "rotary":
        cos, sin = _turns(s["positions"], s["freq"], s["pair_axes"])
        return _rotate(s["x"], cos, -sin if case["inverse"] else sin, case["interleaved"])
    seq, place = _places(s)
    positions = place.to(torch.int32)[None] if s["positions"] is None else s["positions"]
    cos, sin = _turns(positions, s["freq"], s["pair_axes"])
    page, at = s["table"][seq, place // case["page"]].long(), place % case["page"]
    for cache, new in ((s["k_cache"], _rotate(s["k"], cos, sin, case["interleaved"])), (s["v_cache"], s["v"])):
        if case["head_major"]:
            cache[page, :, at] = new
        else:
            cache[page, at] = new
    out = [s["k_cache"], s["v_cache"]]
    return out + ([_rotate(s["q"], cos, sin, case["interleaved"])] if s["q"] is not None else [])


def _places(s):
    """Each new token's sequence and its place there."""
    T = s["k"].shape[0]
    t = torch.arange(T, device="cuda")
    if s["starts"] is None:
        return t, s["lengths"].long()
    seq = torch.searchsorted(s["starts"].long(), t, right=True) - 1
    return seq, s["lengths"].long()[seq] + t - s["starts"].long()[seq]


# ---- the framework's calls ---------------------------------------------------------------------------------------

def _own(s):
    import bmmc_index_transforms_gb300 as bm

    case, op = s["case"], s["case"]["op"]
    if op == "sort":
        return bm.expert_sort(s["ids"], case["experts"])
    if op == "dispatch":
        return bm.expert_dispatch(s["x"], s["slot"])
    if op == "dispatch_backward":
        return bm.expert_combine(s["rows"], s["slot"])
    if op == "combine":
        return bm.expert_combine(s["rows"], s["slot"], s["weights"])
    if op == "combine_backward":
        return bm.expert_combine_backward(s["x"], s["rows"], s["slot"], s["weights"])
    if op == "rotary":
        return bm.rotary(s["x"], s["positions"], s["freq"], s["pair_axes"], interleaved=case["interleaved"], inverse=case["inverse"])
    q = bm.paged_append(s["k"], s["v"], s["k_cache"], s["v_cache"], s["table"], s["lengths"], starts=s["starts"], q=s["q"],
                        positions=s["positions"], inv_freq=s["freq"], pair_axes=s["pair_axes"],
                        interleaved=case["interleaved"], head_major=case["head_major"])
    return [s["k_cache"], s["v_cache"]] + ([q] if q is not None else [])


def run(state):
    return _own(state) if own else _plain(state)


# ---- what a pass cannot do without -------------------------------------------------------------------------------

def work(case):
    op, T = case["op"], case["tokens"]
    if op == "sort":
        n = T * case["choices"]
        return {"bytes": n * (4 if case["ids"] == "i32" else 8) + 8 * n + 4 * (case["experts"] + 1), "flops": 0}
    es = SIZE[case["type"]]
    if op in ("dispatch", "combine", "dispatch_backward", "combine_backward"):
        n, H = T * case["choices"], case["hidden"]
        w = (4 if case.get("weights") == "f32" else es) if "weights" in case else 0
        moved = {"dispatch": T + n, "combine": n + T, "dispatch_backward": n + T, "combine_backward": T + 2 * n}[op]
        flops = {"dispatch": 0, "combine": 2 * n * H, "dispatch_backward": n * H, "combine_backward": 3 * n * H}[op]
        return {"bytes": moved * H * es + n * (4 + w * (2 if op == "combine_backward" else 1)), "flops": flops}
    pairs = case["rotary_dim"] // 2
    known = 4 * pairs * (2 if case["axes"] > 1 else 1)
    if op == "rotary":
        return {"bytes": 2 * T * case["heads"] * case["dim"] * es + 4 * T * case["axes"] + known, "flops": 6 * T * case["heads"] * pairs}
    heads, turned = case["q_heads"] + 2 * case["kv_heads"], case["q_heads"] + case["kv_heads"]
    known += 4 * T * (case["axes"] if case["axes"] > 1 else 0) + 8 * case["sequences"] + 4 * max(case["sequences"], T // case["page"])
    return {"bytes": 2 * T * heads * case["dim"] * es + known, "flops": 6 * T * turned * pairs}


# ---- the definitions in 64 bits ----------------------------------------------------------------------------------

def _turned64(x, positions, freq, pair_axes, interleaved, sign):
    """A pair is a complex number, a rotation a product with exp(i angle)."""
    P = freq.numel()
    which = torch.zeros(P, dtype=torch.long, device="cuda") if pair_axes is None else pair_axes.long()
    angle = sign * positions.double()[which].t() * freq.double()
    factor = torch.polar(torch.ones_like(angle), angle)[:, None]
    y = x.double().clone()
    first, second = (slice(0, 2 * P, 2), slice(1, 2 * P, 2)) if interleaved else (slice(0, P), slice(P, 2 * P))
    z = torch.complex(y[..., first], y[..., second]) * factor
    y[..., first], y[..., second] = z.real, z.imag
    return y


def exact(case, seed):
    op = case["op"]
    if op == "sort":
        return None  # whole numbers
    s = prepare(case, seed)
    if op == "rotary":
        return _turned64(s["x"], s["positions"], s["freq"], s["pair_axes"], case["interleaved"], -1 if case["inverse"] else 1)
    if op == "append":
        seq, place = _places(s)
        positions = place[None] if s["positions"] is None else s["positions"]
        turn = lambda x: _turned64(x, positions, s["freq"], s["pair_axes"], case["interleaved"], 1)  # noqa: E731
        where = s["table"].long()[seq, place // case["page"]] * case["page"] + place % case["page"]
        out = []
        for cache, new in ((s["k_cache"], turn(s["k"])), (s["v_cache"], s["v"].double())):
            y = cache.double()
            flat = (y.transpose(1, 2) if case["head_major"] else y).reshape(-1, case["kv_heads"], case["dim"]).index_copy(0, where, new)
            flat = flat.view(cache.shape[0], case["page"], case["kv_heads"], case["dim"])
            out.append(flat.transpose(1, 2).contiguous() if case["head_major"] else flat)
        return out + ([turn(s["q"])] if s["q"] is not None else [])
    T, K, H, slot = case["tokens"], case["choices"], case["hidden"], s["slot"].reshape(-1)
    choice = torch.nonzero(slot >= 0).flatten()  # the routed choices, their tokens and rows
    token, row = choice // K, slot[choice].long()
    if op == "dispatch":
        rows = torch.zeros(T * K, H, dtype=torch.float64, device="cuda")
        return rows.index_copy_(0, row, s["x"].double()[token])
    if op in ("combine", "dispatch_backward"):
        new = s["rows"].double()[row]
        if op == "combine":
            new *= s["weights"].double().reshape(-1)[choice, None]
        out = torch.zeros(T, H, dtype=torch.float64, device="cuda")
        return out.index_add_(0, token, new)
    grad, w = s["x"].double(), s["weights"].double().reshape(-1)
    grad_rows = torch.zeros(T * K, H, dtype=torch.float64, device="cuda")
    grad_w = torch.zeros(T * K, dtype=torch.float64, device="cuda")
    for a in range(0, choice.numel(), 16384):  # in parts, for memory
        c, t, r = choice[a:a + 16384], token[a:a + 16384], row[a:a + 16384]
        grad_rows[r] = w[c, None] * grad[t]
        grad_w[c] = torch.einsum("ch,ch->c", s["rows"][r].double(), grad[t])
    return grad_rows, grad_w.view(T, K)
