"""Operators that stand at the ends of a decoder with experts, around its moves of tokens, as cases to measure:

  lookup            embedding_lookup: the rows of a table that the tokens name, scaled
  lookup_backward   embedding_backward: the gradient by the table, the rows of equal tokens added up
  balance           expert_balance: a router's balance loss and the number of choices of each expert
  balance_backward  expert_balance_backward: its gradient by the router's logits
  append8           paged_append with scales: keys and values written to a paged cache in 8 bits, turned on the way
  read              paged_read: a cache's entries, in 8 bits or more, read back in the order of the sequences

A case is a dict of plain values; "op" is one of the names above."""
import math

import numpy as np
import torch

own = False  # False: the plain form below; True: the calls of bmmc_index_transforms_gb300

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn, "i8": torch.int8}
SIZE = {"f32": 4, "f16": 2, "bf16": 2, "e4m3": 1, "i8": 1}
MOST = {"e4m3": 448.0, "i8": 127.0}  # the largest value of a type in 8 bits
LEAST = 2.0 ** -126  # the smallest scale


def listed():
    return [
        # the tokens of one decoding step, a few slots of the batch empty: latency
        {"name": "lookup decode", "op": "lookup", "type": "bf16", "tokens": 64, "vocab": 32768, "hidden": 4096, "scale": 64.0, "empty": 0.1},
        # a training or prefill batch's tokens, as frequent as words are: bandwidth
        {"name": "lookup batch", "op": "lookup", "type": "bf16", "tokens": 16384, "vocab": 131072, "hidden": 4096, "scale": 1.0, "empty": 0.02},
        # a small training batch in half precision with odd sizes, its gradient kept in 32 bits
        {"name": "lookup backward odd", "op": "lookup_backward", "type": "f16", "out": "f32", "tokens": 2039, "vocab": 10007, "hidden": 1031, "scale": 32.0, "empty": 0.05},
        # a training batch over a large vocabulary: the largest of the list, most rows without a token
        {"name": "lookup backward batch", "op": "lookup_backward", "type": "bf16", "out": "bf16", "tokens": 32768, "vocab": 131072, "hidden": 4096, "scale": 1.0, "empty": 0.02},
        # a micro-batch of a small router: latency
        {"name": "balance small", "op": "balance", "type": "bf16", "tokens": 509, "choices": 2, "experts": 8, "ids": "i64", "empty": 0.05},
        # a training batch over many experts, logits in 32 bits as routers keep them
        {"name": "balance batch", "op": "balance", "type": "f32", "tokens": 65521, "choices": 8, "experts": 256, "ids": "i32", "empty": 0.02},
        # the same two's gradients, the small one with an odd number of experts
        {"name": "balance backward odd", "op": "balance_backward", "type": "f16", "tokens": 1021, "choices": 4, "experts": 61, "ids": "i64", "empty": 0.05},
        {"name": "balance backward batch", "op": "balance_backward", "type": "f32", "tokens": 65521, "choices": 8, "experts": 256, "ids": "i32", "empty": 0.02},
        # one token for each of 256 sequences: a decoding step's append to a cache in 8 bits, the queries turned with it
        {"name": "append8 decode", "op": "append8", "type": "bf16", "cache": "e4m3", "sequences": 256, "tokens": 256, "q_heads": 32, "kv_heads": 8, "dim": 128, "rotary_dim": 128, "interleaved": False, "page": 16, "cached": 500, "head_major": False},
        # prompts of uneven lengths, appended to what they had
        {"name": "append8 prompts", "op": "append8", "type": "bf16", "cache": "e4m3", "sequences": 13, "tokens": 16001, "q_heads": 32, "kv_heads": 8, "dim": 128, "rotary_dim": 128, "interleaved": False, "page": 64, "cached": 3000, "head_major": True},
        # a few short sequences read back from a cache of whole numbers: latency
        {"name": "read short", "op": "read", "type": "f16", "cache": "i8", "sequences": 5, "rows": 167, "kv_heads": 4, "dim": 96, "page": 16, "cached": 60, "window": False, "head_major": False},
        # the caches of a batch read back for a chunk of new tokens each
        {"name": "read batch", "op": "read", "type": "bf16", "cache": "e4m3", "sequences": 32, "rows": 65536, "kv_heads": 8, "dim": 128, "page": 64, "cached": 4096, "window": False, "head_major": True},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["lookup", "lookup_backward", "lookup_backward", "balance", "balance_backward", "append8", "append8", "read", "read"])
    type_ = rng.choice(["f32", "f16", "bf16", "bf16"])
    if op in ("lookup", "lookup_backward"):
        # a multiple of 8 mostly, as models have it; else any width
        hidden = _log(rng, 8, 1024) * 8 if rng.random() < 0.75 else _log(rng, 1, 4097)
        c = {"op": op, "type": type_, "hidden": hidden, "scale": rng.choice([1.0, 0.125, 45.25]), "empty": rng.choice([0.0, 0.05, 0.3])}
        if op == "lookup":
            c["vocab"] = _log(rng, 2, max(2, min(200003, (131072 * 4096 * 2) // (hidden * SIZE[type_]))))
            c["tokens"] = _log(rng, 1, max(1, min(65536, (65536 * 4096 * 2) // (hidden * SIZE[type_]))))
        else:
            c["out"] = rng.choice([type_, "f32"])
            c["vocab"] = _log(rng, 2, max(2, min(200003, (131072 * 4096 * 2) // (hidden * SIZE[c["out"]]))))
            c["tokens"] = _log(rng, 1, max(1, min(100003, (32768 * 4096 * 2) // (hidden * SIZE[type_]))))
        return c
    if op in ("balance", "balance_backward"):
        experts = _log(rng, 2, 512)
        return {"op": op, "type": type_, "tokens": _log(rng, 1, min(131072, 65536 * 256 // experts)), "choices": rng.randint(1, min(8, experts)), "experts": experts, "ids": rng.choice(["i32", "i64"]), "empty": rng.choice([0.0, 0.05, 0.5])}
    dim = rng.choice([32, 64, 80, 96, 128, 192, 256, 66, 10])
    kv_heads = _log(rng, 1, 16)
    sequences = _log(rng, 1, 512)
    c = {"op": op, "type": type_, "sequences": sequences, "kv_heads": kv_heads, "dim": dim, "page": rng.choice([1, 16, 64, 100]), "cached": _log(rng, 1, max(1, min(4096, 65536 // sequences))), "head_major": rng.random() < 0.5}
    if op == "read":
        # 8 bits, or the type itself: the entries are then only moved
        return {**c, "rows": max(1, c["sequences"] * c["cached"] // 2), "cache": rng.choice(["e4m3", "e4m3", "i8", type_]), "window": rng.random() < 0.3}
    # keys in whole numbers come turned already; those in floating point are turned on the way
    cache = rng.choice(["e4m3", "e4m3", "i8"])
    rotary_dim = 0 if cache == "i8" else dim if rng.random() < 0.6 else 2 * rng.randint(1, dim // 2)
    q_heads = 0 if cache == "i8" else kv_heads * rng.choice([0, 1, 4])
    tokens = sequences if rng.random() < 0.5 else max(sequences, _log(rng, 1, 16384))
    return {**c, "cache": cache, "tokens": tokens, "q_heads": q_heads, "rotary_dim": rotary_dim, "interleaved": rng.random() < 0.4}


# ---- inputs ------------------------------------------------------------------------------------------------------

def _prepare_tokens(case, g):
    """Token ids: the r-th most frequent about r times as rare as the first, the rows of the table in any order, the
    batch's last tokens padding, which names no row."""
    T, V = case["tokens"], case["vocab"]
    u = torch.rand(T, generator=g, device="cuda", dtype=torch.float64)
    rank = (torch.exp(u * math.log(V + 1)) - 1).long().clamp(0, V - 1)
    ids = torch.randperm(V, generator=g, device="cuda")[rank]
    ids[T - int(T * case["empty"]):] = -1
    return ids


def _prepare_cache(case, g, lengths, need):
    """A pool of pages that the sequences hold in any order, filled; the rest of a sequence's table is empty."""
    B, Hk, D, page = case["sequences"], case["kv_heads"], case["dim"], case["page"]
    type_ = TYPES[case["cache"]]
    total = B * ((case["cached"] + page - 1) // page + 2) + case.get("tokens", case.get("rows")) // page  # what the longest sequences need at most
    at = torch.cumsum(need, 0) - need
    columns = max(1, int(need.max()))
    column = torch.arange(columns, device="cuda")
    pool = torch.randperm(total, generator=g, device="cuda")
    table = torch.where(column < need[:, None], pool[(at[:, None] + column).clamp(max=total - 1)], -1)
    lead = (total, Hk, page) if case["head_major"] else (total, page, Hk)
    s = {"table": table.to(torch.int32), "lengths": lengths.to(torch.int32)}
    for name in ("k", "v"):
        x = torch.randn(*lead, D, generator=g, device="cuda", dtype=torch.float32)
        if case["cache"] in MOST:
            x = x * (MOST[case["cache"]] / 4)
            x = x.clamp(-MOST[case["cache"]], MOST[case["cache"]])
            s[name + "_scales"] = torch.rand(lead, generator=g, device="cuda", dtype=torch.float32) * 0.02 + 0.001
        else:
            s[name + "_scales"] = None
        s[name + "_cache"] = (x.round() if case["cache"] == "i8" else x).to(type_)
    return s


def prepare(case, seed):
    g = torch.Generator("cuda")
    g.manual_seed(seed)
    op, s = case["op"], {"case": case}
    if op in ("lookup", "lookup_backward"):
        T, V, H, type_ = case["tokens"], case["vocab"], case["hidden"], TYPES[case["type"]]
        s["ids"] = _prepare_tokens(case, g)
        if op == "lookup":
            s["table"] = torch.randn(V, H, generator=g, device="cuda", dtype=type_)
        else:
            s["grad"] = torch.randn(T, H, generator=g, device="cuda", dtype=type_)
        return s
    if op in ("balance", "balance_backward"):
        T, K, E = case["tokens"], case["choices"], case["experts"]
        # some experts more popular than others; the last tokens of the batch are empty and a few choices more left out
        logits = 1.5 * torch.randn(T, E, generator=g, device="cuda") + torch.randn(E, generator=g, device="cuda")
        s["logits"] = logits.to(TYPES[case["type"]])
        ids = s["logits"].float().topk(K, dim=1)[1]
        out = torch.rand(T, K, generator=g, device="cuda") < case["empty"] / 2
        out[T - int(T * case["empty"] / 2):] = True
        ids = ids.masked_fill(out, -1).to(torch.int32 if case["ids"] == "i32" else torch.int64)
        s["ids"] = ids
        if op == "balance_backward":
            s["counts"] = _count(ids, E)
            # the loss's coefficient, in half precision with the scale that keeps its gradients representable
            s["grad"] = (torch.rand((), generator=g, device="cuda") * 0.02 + 0.001) * (65536 if case["type"] == "f16" else 1)
        return s
    B, Hk, D, page = case["sequences"], case["kv_heads"], case["dim"], case["page"]
    if op == "read":
        # uneven sequences, read whole or (a window) their last part; a few rows behind them are nobody's
        part = torch.rand(B, generator=g, device="cuda", dtype=torch.float64) + 0.1
        count = (part / part.sum() * case["rows"]).long()
        firsts = torch.randint(0, case["cached"] + 1, (B,), generator=g, device="cuda") if case["window"] else torch.zeros_like(count)
        s |= _prepare_cache(case, g, firsts + count, (firsts + count + page - 1) // page)
        s["starts"] = torch.cat([count.new_zeros(1), torch.cumsum(count, 0)]).to(torch.int32)
        s["firsts"] = firsts.to(torch.int32) if case["window"] else None
        return s
    lengths = torch.randint(0, case["cached"] + 1, (B,), generator=g, device="cuda")
    T, Hq, type_ = case["tokens"], case["q_heads"], TYPES[case["type"]]
    # slices of the product that gives queries, keys and values together; some channels of the keys are large
    qkv = torch.randn(T, Hq + 2 * Hk, D, generator=g, device="cuda", dtype=type_)
    qkv[:, Hq:Hq + Hk, ::16] *= 6
    s["q"], s["k"], s["v"] = qkv[:, :Hq] if Hq else None, qkv[:, Hq:Hq + Hk], qkv[:, Hq + Hk:]
    if T == B:
        new, s["starts"] = torch.ones(B, dtype=torch.int64, device="cuda"), None
    else:  # uneven parts of the tokens, some sequences without any
        cut = torch.randint(0, T + 1, (B - 1,), generator=g, device="cuda").sort()[0]
        starts = torch.cat([cut.new_zeros(1), cut, cut.new_full((1,), T)])
        new, s["starts"] = starts[1:] - starts[:-1], starts.to(torch.int32)
    s |= _prepare_cache(case, g, lengths, (lengths + new + page - 1) // page)
    pairs = case["rotary_dim"] // 2
    s["freq"] = 10000.0 ** (-torch.arange(pairs, device="cuda", dtype=torch.float32) / pairs) if pairs else None
    return s


# ---- the plain forms ---------------------------------------------------------------------------------------------

def _count(ids, experts):
    """Each expert's routed choices and, behind them, the tokens that have any."""
    routed = (ids >= 0) & (ids < experts)
    key = torch.where(routed, ids.long(), experts).reshape(-1)
    each = torch.zeros(experts + 1, dtype=torch.int64, device=ids.device).index_add_(0, key, torch.ones_like(key))
    each[experts] = routed.any(1).sum()
    return each.to(torch.int32)


def _shares(s):
    """The tokens that count, the softmax of all logits, each expert's share of the choices."""
    ids, E = s["ids"], s["case"]["experts"]
    there = ((ids >= 0) & (ids < E)).any(1)
    x = s["logits"].float()
    e = torch.exp(x - x.amax(1, keepdim=True))
    counts = s["counts"] if "counts" in s else _count(ids, E)
    each = counts[:E].float()
    return there, e / e.sum(1, keepdim=True), counts, each / each.sum().clamp(min=1)


def _places(s, starts, firsts, rows):
    """Each row's sequence and its entry there."""
    t = torch.arange(rows, device="cuda")
    if starts is None:
        return t, firsts.long()
    seq = torch.searchsorted(starts.long()[1:], t, right=True).clamp(max=s["case"]["sequences"] - 1)
    at = t - starts.long()[seq]
    return seq, at if firsts is None else firsts.long()[seq] + at


def _turn(x, place, freq, interleaved):
    x = x.float()
    if freq is None:
        return x
    pairs = freq.numel()
    angle = (place.to(torch.float32)[:, None] * freq)[:, None]
    cos, sin, part = torch.cos(angle), torch.sin(angle), x[..., :2 * pairs]
    a, b = (part[..., 0::2], part[..., 1::2]) if interleaved else (part[..., :pairs], part[..., pairs:])
    a, b = a * cos - b * sin, b * cos + a * sin
    turned = torch.stack([a, b], -1).flatten(-2) if interleaved else torch.cat([a, b], -1)
    return torch.cat([turned, x[..., 2 * pairs:]], -1)


def _quantise(x, cache):
    """Values in 8 bits and the scale of each head, its largest value over the type's."""
    scale = (x.abs().amax(-1) / MOST[cache]).clamp(min=LEAST)
    y = (x * (1.0 / scale)[..., None]).clamp(-MOST[cache], MOST[cache])
    return (y.round() if cache == "i8" else y).to(TYPES[cache]), scale


def _plain(s):
    case, op = s["case"], s["case"]["op"]
    if op == "lookup":
        there = s["ids"] >= 0
        rows = s["table"][torch.where(there, s["ids"], 0)].float() * case["scale"]
        return torch.where(there[:, None], rows, 0).to(s["table"].dtype)
    if op == "lookup_backward":
        V, H = case["vocab"], case["hidden"]
        out = torch.zeros(V + 1, H, device="cuda")  # one row more, for padding
        out.index_add_(0, torch.where(s["ids"] >= 0, s["ids"], V), s["grad"].float())
        return (out[:V] * case["scale"]).to(TYPES[case["out"]])
    if op == "balance":
        there, p, counts, share = _shares(s)
        mean = (p * there[:, None]).sum(0) / there.sum().clamp(min=1)
        return case["experts"] * (share * mean).sum(), counts
    if op == "balance_backward":
        there, p, counts, share = _shares(s)
        g = p * (share - (p * share).sum(1, keepdim=True))
        g *= s["grad"] * case["experts"] / there.sum().clamp(min=1)
        return (g * there[:, None]).to(s["logits"].dtype)
    page = case["page"]
    if op == "read":
        seq, place = _places(s, s["starts"], s["firsts"], case["rows"])
        there = place < s["lengths"].long()[seq]
        place = torch.where(there, place, 0)
        entry, at = s["table"][seq, place // page].long().clamp(min=0), place % page
        out = []
        for name in ("k", "v"):
            cache, scales = s[name + "_cache"], s[name + "_scales"]
            x = (cache[entry, :, at] if case["head_major"] else cache[entry, at]).float()
            if scales is not None:
                x = x * (scales[entry, :, at] if case["head_major"] else scales[entry, at])[..., None]
            out.append(torch.where(there[:, None, None], x, 0).to(TYPES[case["type"]]))
        return out
    T = s["k"].shape[0]
    if s["starts"] is None:
        seq, place = torch.arange(T, device="cuda"), s["lengths"].long()
    else:
        seq, place = _places(s, s["starts"], s["lengths"], T)
    entry, at = s["table"][seq, place // page].long(), place % page
    new = {"k": _turn(s["k"], place, s["freq"], case["interleaved"]), "v": s["v"].float()}
    out = []
    for name in ("k", "v"):
        values, scales = _quantise(new[name], case["cache"])
        for to, what in ((s[name + "_cache"], values), (s[name + "_scales"], scales)):
            if what.dtype == torch.float8_e4m3fn:  # moved as bytes
                to, what = to.view(torch.uint8), what.view(torch.uint8)
            if case["head_major"]:
                to[entry, :, at] = what
            else:
                to[entry, at] = what
        out += [s[name + "_cache"], s[name + "_scales"]]
    return out + ([_turn(s["q"], place, s["freq"], case["interleaved"]).to(s["q"].dtype)] if s["q"] is not None else [])


# ---- the framework's calls ---------------------------------------------------------------------------------------

def _own(s):
    import bmmc_index_transforms_gb300 as bm

    case, op = s["case"], s["case"]["op"]
    if op == "lookup":
        return bm.embedding_lookup(s["table"], s["ids"], scale=case["scale"])
    if op == "lookup_backward":
        return bm.embedding_backward(s["grad"], s["ids"], case["vocab"], scale=case["scale"], dtype=TYPES[case["out"]])
    if op == "balance":
        return bm.expert_balance(s["logits"], s["ids"])
    if op == "balance_backward":
        return bm.expert_balance_backward(s["grad"], s["logits"], s["ids"], s["counts"])
    if op == "read":
        return list(bm.paged_read(s["k_cache"], s["v_cache"], s["table"], s["starts"], case["rows"], firsts=s["firsts"],
                                  k_scales=s["k_scales"], v_scales=s["v_scales"], dtype=TYPES[case["type"]],
                                  head_major=case["head_major"]))
    q = bm.paged_append(s["k"], s["v"], s["k_cache"], s["v_cache"], s["table"], s["lengths"], starts=s["starts"], q=s["q"],
                        inv_freq=s["freq"], interleaved=case["interleaved"], head_major=case["head_major"],
                        k_scales=s["k_scales"], v_scales=s["v_scales"])
    return [s["k_cache"], s["k_scales"], s["v_cache"], s["v_scales"]] + ([q] if q is not None else [])


def run(state):
    return _own(state) if own else _plain(state)


# ---- what a pass cannot do without -------------------------------------------------------------------------------

def _distinct(case):
    """Rows of the table that the tokens name, on average."""
    T, V = case["tokens"] - int(case["tokens"] * case["empty"]), case["vocab"]
    r = np.arange(V, dtype=np.float64)
    p = np.log((r + 2) / (r + 1)) / math.log(V + 1)
    return float((1 - (1 - p) ** T).sum())


def work(case):
    op = case["op"]
    if op in ("lookup", "lookup_backward"):
        T, H, es = case["tokens"], case["hidden"], SIZE[case["type"]]
        there = T - int(T * case["empty"])
        if op == "lookup":
            return {"bytes": (_distinct(case) + T) * H * es + 8 * T, "flops": there * H}
        return {"bytes": there * H * es + case["vocab"] * H * SIZE[case["out"]] + 8 * T, "flops": there * H}
    if op in ("balance", "balance_backward"):
        T, E = case["tokens"], case["experts"]
        there = T - int(T * case["empty"] / 2)
        ids = T * case["choices"] * (4 if case["ids"] == "i32" else 8)
        rows = there * E * SIZE[case["type"]]
        if op == "balance":
            return {"bytes": rows + ids + 4 * (E + 2), "flops": 4 * there * E}
        return {"bytes": rows + T * E * SIZE[case["type"]] + ids + 4 * (E + 2), "flops": 7 * there * E}
    B, Hk, D, es, cs = case["sequences"], case["kv_heads"], case["dim"], SIZE[case["type"]], SIZE[case["cache"]]
    scale = 4 if case["cache"] in MOST else 0
    if op == "read":
        R = case["rows"]
        return {"bytes": 2 * R * Hk * (D * (cs + es) + scale) + 8 * B + 4 * R / case["page"], "flops": 2 * R * Hk * D if scale else 0}
    T, Hq, pairs = case["tokens"], case["q_heads"], case["rotary_dim"] // 2
    known = 4 * pairs + 8 * B + 4 * max(B, T // case["page"])
    return {"bytes": T * (2 * Hq * D * es + 2 * Hk * (D * (es + cs) + scale)) + known, "flops": 6 * T * (Hq + Hk) * pairs + 6 * T * Hk * D}


# ---- the definitions in 64 bits ----------------------------------------------------------------------------------

def _turned64(x, place, freq, interleaved):
    """A pair is a complex number, a rotation a product with exp(i angle); the angle is defined as a product in 32 bits."""
    y = x.double().clone()
    if freq is None:
        return y
    P = freq.numel()
    angle = (place.float()[:, None] * freq).double()
    factor = torch.polar(torch.ones_like(angle), angle)[:, None]
    first, second = (slice(0, 2 * P, 2), slice(1, 2 * P, 2)) if interleaved else (slice(0, P), slice(P, 2 * P))
    z = torch.complex(y[..., first], y[..., second]) * factor
    y[..., first], y[..., second] = z.real, z.imag
    return y


def _nearest_e4m3(x):
    """The nearest value with 3 bits behind the leading one and exponents from -6 on, ties to even, up to 448."""
    _, e = torch.frexp(x)
    step = torch.exp2((e - 4).clamp(min=-9).double())
    return (torch.round(x / step) * step).clamp(-448, 448)


def exact(case, seed):
    op = case["op"]
    s = prepare(case, seed)
    if op == "lookup":
        out = torch.zeros(case["tokens"], case["hidden"], dtype=torch.float64, device="cuda")
        at = torch.nonzero(s["ids"] >= 0).flatten()
        out[at] = s["table"].index_select(0, s["ids"][at]).double() * case["scale"]
        return out
    if op == "lookup_backward":
        at = torch.nonzero(s["ids"] >= 0).flatten()
        ids, order = s["ids"][at].sort()
        out = torch.zeros(case["vocab"], case["hidden"], dtype=torch.float64, device="cuda")
        for a in range(0, at.numel(), 16384):  # in parts, for memory
            part = order[a:a + 16384]
            out.index_add_(0, ids[a:a + 16384], s["grad"][at[part]].double())
        return out * case["scale"]
    if op in ("balance", "balance_backward"):
        E = case["experts"]
        x = s["logits"].double().requires_grad_(op == "balance_backward")
        routed = (s["ids"] >= 0) & (s["ids"] < E)
        there = torch.nonzero(routed.any(1)).flatten()
        each = torch.bincount(s["ids"][routed].long(), minlength=E).double()
        n = max(1, there.numel())
        loss = E * ((each / max(1.0, float(each.sum()))) * (torch.softmax(x[there], dim=1).sum(0) / n)).sum()
        if op == "balance":
            return loss, None
        return torch.autograd.grad(loss, x)[0] * s["grad"].double()
    page, Hk, D = case["page"], case["kv_heads"], case["dim"]

    def by_entry(x):  # [pages * page, heads, ...]
        return (x.transpose(1, 2) if case["head_major"] else x).flatten(0, 1)

    if op == "read":
        seq, place = _places(s, s["starts"], s["firsts"], case["rows"])
        there = torch.nonzero(place < s["lengths"].long()[seq]).flatten()
        seq, place = seq[there], place[there]
        where = s["table"].long()[seq, place // page] * page + place % page
        out = []
        for name in ("k", "v"):
            x = by_entry(s[name + "_cache"].view(torch.uint8) if case["cache"] == "e4m3" else s[name + "_cache"])[where]
            x = (x.view(torch.float8_e4m3fn) if case["cache"] == "e4m3" else x).double()
            if s[name + "_scales"] is not None:
                x = x * by_entry(s[name + "_scales"])[where].double()[..., None]
            out.append(torch.zeros(case["rows"], Hk, D, dtype=torch.float64, device="cuda").index_copy_(0, there, x))
        return out
    T = case["tokens"]
    t = torch.arange(T, device="cuda")
    seq = t if s["starts"] is None else torch.bucketize(t, s["starts"].long()[1:], right=True)
    place = s["lengths"].long()[seq] + (0 if s["starts"] is None else t - s["starts"].long()[seq])
    where = s["table"].long()[seq, place // page] * page + place % page
    out = []
    for name, new in (("k", _turned64(s["k"], place, s["freq"], case["interleaved"])), ("v", s["v"].double())):
        scale = new.abs().amax(-1) / MOST[case["cache"]]
        values = None
        if case["cache"] == "e4m3":
            values = _nearest_e4m3(torch.where(scale[..., None] > 0, new / scale[..., None], 0))
        for x, what in ((s[name + "_cache"], values), (s[name + "_scales"], scale)):
            if what is None:  # whole numbers
                out.append(None)
                continue
            flat = by_entry(x.double()).index_copy(0, where, what)
            flat = flat.view(-1, page, *flat.shape[1:])
            out.append(flat.transpose(1, 2).contiguous() if case["head_major"] else flat)
    return out + ([_turned64(s["q"], place, s["freq"], case["interleaved"])] if s["q"] is not None else [])
