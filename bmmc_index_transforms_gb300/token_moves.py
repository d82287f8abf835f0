"""Moves of tokens by maps held on the device, on torch tensors: by expert
and back, and into the pages of a cache.

Argument marshalling for the entry points of the same names in
``include/bmmc.h``: tensors become pointers, sizes and strides, and outputs
that are not given are allocated.  Every element is moved by the library's
CUDA kernels, on the current stream or the one given; nothing waits for the
device, so the calls can be captured in a CUDA graph.
"""

from __future__ import annotations

import ctypes

from . import _capi

__all__ = ["expert_sort", "expert_dispatch", "expert_combine", "expert_combine_backward", "rotary", "paged_append"]

_types = {}  # torch dtype -> bmmc_dtype


def _setup():
    import torch

    if not _types:
        _types.update({torch.float32: _capi.F32, torch.float16: _capi.F16, torch.bfloat16: _capi.BF16})
    return torch


def _type(x, where: str, name: str) -> int:
    t = _types.get(x.dtype)
    if t is None:
        raise ValueError(f"{where}: {name} is {x.dtype}; float32, float16 and bfloat16 are supported")
    return t


def _on_device(torch, where: str, **tensors) -> None:
    """Every tensor on the current device, where the library launches."""
    cur = torch.cuda.current_device() if torch.cuda.is_available() else -1
    for name, x in tensors.items():
        if x is not None and (not x.is_cuda or x.get_device() != cur):
            raise ValueError(f"{where}: {name} is on {x.device}, but the current device is cuda:{cur}")


def _stream(torch, stream) -> int:
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream if isinstance(stream, int) else int(stream.cuda_stream)


def _check(status: int, where: str) -> None:
    if status != _capi.OK:
        from . import BmmcError

        raise BmmcError(status, where)


def _need(ok: bool, where: str, message: str) -> None:
    if not ok:
        raise ValueError(f"{where}: {message}")


def _matrix(x, where: str, name: str, rows=None, cols=None) -> None:
    """A 2-D tensor whose rows are dense (any row stride)."""
    _need(x.dim() == 2 and (x.shape[1] < 2 or x.stride(1) == 1), where, f"{name} must be 2-D with dense rows")
    _need((rows is None or x.shape[0] == rows) and (cols is None or x.shape[1] == cols), where,
          f"{name} has shape {tuple(x.shape)}, expected ({rows}, {cols})")


def _slot(slot, torch, where: str) -> None:
    _need(slot.dim() == 2 and slot.dtype == torch.int32 and slot.is_contiguous(), where,
          "slot must be a contiguous int32 tensor [tokens, choices]")


def expert_sort(experts, num_experts: int, stream=None):
    """(slot, source, offsets) of a router's choices ``experts`` [tokens,
    choices] (int32 or int64; ids outside [0, num_experts) are not routed).

    ``slot`` [tokens, choices]: the choice's row among all choices sorted by
    expert (stable), or ~row where it is not routed; ``source`` [tokens *
    choices]: the flat choice of each row, or its complement; ``offsets``
    [num_experts + 1]: expert e has rows offsets[e] .. offsets[e + 1] - 1."""
    torch = _setup()
    where = "expert_sort"
    _need(experts.dim() == 2 and experts.dtype in (torch.int32, torch.int64) and experts.is_contiguous(), where,
          "experts must be a contiguous int32 or int64 tensor [tokens, choices]")
    _on_device(torch, where, experts=experts)
    T, K = experts.shape
    L = _capi.lib()
    size = ctypes.c_size_t()
    _check(L.expert_sort_workspace(T, K, num_experts, size), where)
    n = T * K
    # one allocation: source, offsets, then the workspace
    rest = torch.empty(n + num_experts + 1 + size.value // 4, dtype=torch.int32, device=experts.device)
    slot = torch.empty((T, K), dtype=torch.int32, device=experts.device)
    at = rest.data_ptr()
    _check(L.expert_sort(experts.data_ptr(), experts.element_size(), T, K, num_experts, slot.data_ptr(), at, at + 4 * n,
                         at + 4 * (n + num_experts + 1), size.value, _stream(torch, stream)), where)
    return slot, rest[:n], rest[n:n + num_experts + 1]


def expert_dispatch(x, slot, num_rows=None, out=None, stream=None):
    """rows[slot[t, k]] = x[t] for every routed choice, zero in the rows of
    the others; [num_rows, hidden], num_rows = tokens * choices unless fewer
    are asked for (choices numbered num_rows and above are dropped)."""
    torch = _setup()
    where = "expert_dispatch"
    _slot(slot, torch, where)
    T, K = slot.shape
    _matrix(x, where, "x", rows=T)
    R = T * K if num_rows is None else int(num_rows)
    _need(0 <= R <= T * K, where, f"num_rows {R} is outside [0, {T * K}]")
    H = x.shape[1]
    if out is None:
        out = torch.empty((R, H), dtype=x.dtype, device=x.device)
    else:
        _matrix(out, where, "out", R, H)
        _need(out.dtype == x.dtype, where, "out must have the type of x")
    _on_device(torch, where, x=x, slot=slot, out=out)
    _check(_capi.lib().expert_dispatch(x.data_ptr(), x.stride(0), slot.data_ptr(), T, K, H, _type(x, where, "x"),
                                       out.data_ptr(), out.stride(0), R, _stream(torch, stream)), where)
    return out


def _weights(weights, slot, rows, where: str) -> int:
    _need(tuple(weights.shape) == tuple(slot.shape) and weights.is_contiguous(), where,
          "weights must be a contiguous tensor of slot's shape")
    t = _type(weights, where, "weights")
    _need(t == _capi.F32 or weights.dtype == rows.dtype, where, "weights must be float32 or of the rows' type")
    return t


def expert_combine(rows, slot, weights=None, out=None, stream=None):
    """out[t] = sum over the routed choices k of weights[t, k] *
    rows[slot[t, k]] (weights float32 or of the rows' type); without weights
    the plain sum, which is the gradient of expert_dispatch by x."""
    torch = _setup()
    where = "expert_combine"
    _slot(slot, torch, where)
    T, K = slot.shape
    _matrix(rows, where, "rows")
    R, H = rows.shape
    _need(R <= T * K, where, f"rows has {R} rows for {T * K} choices")
    wt = _capi.F32 if weights is None else _weights(weights, slot, rows, where)
    if out is None:
        out = torch.empty((T, H), dtype=rows.dtype, device=rows.device)
    else:
        _matrix(out, where, "out", T, H)
        _need(out.dtype == rows.dtype, where, "out must have the type of rows")
    _on_device(torch, where, rows=rows, slot=slot, weights=weights, out=out)
    _check(_capi.lib().expert_combine(rows.data_ptr(), rows.stride(0), R, slot.data_ptr(),
                                      None if weights is None else weights.data_ptr(), wt, T, K, H,
                                      _type(rows, where, "rows"), out.data_ptr(), out.stride(0),
                                      _stream(torch, stream)), where)
    return out


def expert_combine_backward(grad, rows, slot, weights, stream=None):
    """(grad_rows, grad_weights) of expert_combine(rows, slot, weights) from
    the gradient of its result."""
    torch = _setup()
    where = "expert_combine_backward"
    _slot(slot, torch, where)
    T, K = slot.shape
    _matrix(rows, where, "rows")
    R, H = rows.shape
    _need(R <= T * K, where, f"rows has {R} rows for {T * K} choices")
    _matrix(grad, where, "grad", T, H)
    _need(grad.dtype == rows.dtype, where, "grad must have the type of rows")
    wt = _weights(weights, slot, rows, where)
    _on_device(torch, where, grad=grad, rows=rows, slot=slot, weights=weights)
    grad_rows = torch.empty((R, H), dtype=rows.dtype, device=rows.device)
    grad_weights = torch.empty((T, K), dtype=weights.dtype, device=rows.device)
    _check(_capi.lib().expert_combine_backward(
        grad.data_ptr(), grad.stride(0), rows.data_ptr(), rows.stride(0), R, slot.data_ptr(), weights.data_ptr(), wt, T, K,
        H, _type(rows, where, "rows"), grad_rows.data_ptr(), H, grad_weights.data_ptr(), _stream(torch, stream)), where)
    return grad_rows, grad_weights


def _heads(x, where: str, name: str, like=None):
    """token_heads_t of a tensor [tokens, heads, dim] with dense heads."""
    _need(x.dim() == 3 and (x.shape[2] < 2 or x.stride(2) == 1), where,
          f"{name} must be [tokens, heads, dim] with dense heads")
    if like is not None:
        _need(x.dtype == like.dtype and x.shape[0] == like.shape[0], where,
              f"{name} must have the type and the tokens of the other heads")
    T, H, D = x.shape
    return x.data_ptr(), H, D, x.stride(0), x.stride(1)


_NO_HEADS = (0, 0, 0, 0, 0)


def _turns(torch, tokens, positions, inv_freq, pair_axes, flags, where: str):
    """rotary_turns_t"""
    if inv_freq is None:
        _need(positions is None and pair_axes is None, where, "positions and pair_axes need inv_freq")
        return 0, 0, 0, 0, 0, 0, 0, flags
    _need(inv_freq.dim() == 1 and inv_freq.dtype == torch.float32 and inv_freq.is_contiguous(), where,
          "inv_freq must be a contiguous float32 tensor [pairs]")
    pairs = inv_freq.shape[0]
    axes_ptr = 0
    if pair_axes is not None:
        _need(pair_axes.dtype == torch.int32 and tuple(pair_axes.shape) == (pairs,) and pair_axes.is_contiguous(),
              where, "pair_axes must be a contiguous int32 tensor [pairs]")
        axes_ptr = pair_axes.data_ptr()
    if positions is None:
        return inv_freq.data_ptr(), axes_ptr, 0, 0, 0, 0, pairs, flags
    d = positions.dim()
    _need(d in (1, 2) and positions.shape[-1] == tokens and positions.dtype in (torch.int32, torch.int64)
          and (tokens < 2 or positions.stride(-1) == 1), where,
          "positions must be an int32 or int64 tensor [tokens] or [axes, tokens] with dense rows")
    axes, stride = (1, 0) if d == 1 else (positions.shape[0], positions.stride(0))
    return (inv_freq.data_ptr(), axes_ptr, positions.data_ptr(), positions.element_size(), axes, stride, pairs, flags)


def rotary(x, positions, inv_freq, pair_axes=None, *, interleaved: bool = False, inverse: bool = False, out=None,
           stream=None):
    """Heads x [tokens, heads, dim] (any token and head strides) turned by
    their tokens' positions [tokens] or [axes, tokens]: pair i, the elements
    i and i + pairs of a head, or 2i and 2i + 1 if interleaved, by the angle
    position * inv_freq[i], with the position on axis pair_axes[i] (axis 0
    without pair_axes; no turn for an axis that is not there).  Elements from
    2 * pairs on are copied.  inverse turns back, which is the gradient.  out
    may be x."""
    torch = _setup()
    where = "rotary"
    X = _heads(x, where, "x")
    if out is None:
        out = torch.empty(x.shape, dtype=x.dtype, device=x.device)
    O = _heads(out, where, "out", x)
    _need(X[1:3] == O[1:3], where, "out must have the shape of x")
    _need(positions is not None and inv_freq is not None, where, "positions and inv_freq are needed")
    flags = (_capi.ROTARY_ADJACENT if interleaved else 0) | (_capi.ROTARY_INVERSE if inverse else 0)
    T = x.shape[0]
    turns = _turns(torch, T, positions, inv_freq, pair_axes, flags, where)
    _on_device(torch, where, x=x, out=out, positions=positions, inv_freq=inv_freq, pair_axes=pair_axes)
    _check(_capi.lib().rotary(_capi.ROTARY_ARGS.pack(T, _type(x, where, "x"), *X, *O, *turns), _stream(torch, stream)),
           where)
    return out


def paged_append(k, v, k_cache, v_cache, page_table, lengths, *, starts=None, q=None, q_out=None, positions=None,
                 inv_freq=None, pair_axes=None, interleaved: bool = False, head_major: bool = False, stream=None):
    """Append new keys and values [tokens, kv_heads, dim] to a paged cache,
    the keys turned on the way as by rotary (without inv_freq: as they are).

    The caches are [pages, page_size, kv_heads, dim], or [pages, kv_heads,
    page_size, dim] if head_major; any strides with dense heads.  Sequence b
    has lengths[b] entries cached and the new tokens starts[b] .. starts[b+1]
    - 1 (without starts, one token for each sequence); its entry e lies in
    page page_table[b, e // page_size].  Tokens without a page there (a
    negative entry, or beyond the table) or outside every sequence are not
    written.  Without positions a token's position is its entry's number.
    Returns the queries q [tokens, q_heads, dim] turned alike (in q_out, which
    may be q), or None without q.  lengths is left as it is."""
    torch = _setup()
    where = "paged_append"
    T = k.shape[0] if k.dim() else 0
    K, V = _heads(k, where, "k"), _heads(v, where, "v", k)
    _need(K[1] == V[1], where, "k and v must have the same heads")
    caches, geometry = [], None
    for name, c, X in (("k_cache", k_cache, K), ("v_cache", v_cache, V)):
        _need(c.dim() == 4 and c.dtype == k.dtype and (c.shape[3] < 2 or c.stride(3) == 1), where,
              f"{name} must be 4-D of k's type with dense heads")
        pages, page, heads, dim = c.shape
        s = c.stride()
        page_stride, slot_stride, head_stride = s[0], s[1], s[2]
        if head_major:
            page, heads, slot_stride, head_stride = heads, page, head_stride, slot_stride
        _need(heads == X[1] and dim == X[2] and geometry in (None, (pages, page)), where,
              f"{name} has shape {tuple(c.shape)}, which does not fit the new heads or the other cache")
        geometry = (pages, page)
        caches += [c.data_ptr(), page_stride, slot_stride, head_stride]
    Q = O = _NO_HEADS
    if q is not None:
        Q = _heads(q, where, "q", k)
        if q_out is None:
            q_out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
        O = _heads(q_out, where, "q_out", k)
        _need(Q[1:3] == O[1:3], where, "q_out must have the shape of q")
    else:
        _need(q_out is None, where, "q_out without q")
    _need(page_table.dim() == 2 and page_table.dtype == torch.int32
          and (page_table.shape[1] < 2 or page_table.stride(1) == 1), where,
          "page_table must be an int32 tensor [sequences, columns] with dense rows")
    B, columns = page_table.shape
    _need(lengths.dtype == torch.int32 and tuple(lengths.shape) == (B,) and lengths.is_contiguous(), where,
          "lengths must be a contiguous int32 tensor [sequences]")
    if starts is None:
        _need(T == B, where, f"{T} tokens for {B} sequences need starts")
    else:
        _need(starts.dtype == torch.int32 and tuple(starts.shape) == (B + 1,) and starts.is_contiguous(), where,
              "starts must be a contiguous int32 tensor [sequences + 1]")
    turns = _turns(torch, T, positions, inv_freq, pair_axes, _capi.ROTARY_ADJACENT if interleaved else 0, where)
    _on_device(torch, where, k=k, v=v, k_cache=k_cache, v_cache=v_cache, page_table=page_table, lengths=lengths,
               starts=starts, q=q, q_out=q_out, positions=positions, inv_freq=inv_freq, pair_axes=pair_axes)
    args = _capi.PAGED_APPEND_ARGS.pack(
        T, _type(k, where, "k"), *K, *V, *Q, *O, *turns, 0 if starts is None else starts.data_ptr(), lengths.data_ptr(), B,
        page_table.data_ptr(), page_table.stride(0), columns, *geometry, *caches)
    _check(_capi.lib().paged_append(args, _stream(torch, stream)), where)
    return q_out
