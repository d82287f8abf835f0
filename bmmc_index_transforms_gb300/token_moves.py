"""Moves of tokens by maps held on the device, on torch tensors: by expert
and back, and into the pages of a cache.

Argument marshalling for the entry points of the same names in
``include/bmmc.h``: tensors become pointers, sizes and strides, and outputs
that are not given are allocated.  Every element is moved by the library's
CUDA kernels, on the current stream or the one given; nothing waits for the
device, so the calls can be captured in a CUDA graph.

``stream`` is a torch stream or a raw handle.  The tensors a call makes, its
outputs and workspaces, are that stream's: they come from its memory and go
back to it, so another stream that uses them waits for it first (and, as with
any tensor of torch's, is recorded where they may be dropped meanwhile).  The
inputs have to be ready on it and to last until its work is done.

Results carry no autograd history: the gradients are calls of their own
(``examples/expert_decoder.py`` wraps them in autograd functions).

The calls of a decoding step take a few microseconds on the device, less than
a careless binding takes on the host: a check costs no more than its
comparison here, and what a refusal says is put together when it is raised.
"""

from __future__ import annotations

import ctypes

from . import _capi
from ._streams import empty_on

__all__ = ["expert_sort", "expert_dispatch", "expert_combine", "expert_combine_backward", "rotary", "paged_append"]

_torch = _empty = _library = _raw_stream = _current_device = _int32 = _int64 = _float32 = None
_types = {}       # torch dtype -> bmmc_dtype, with the flag of device pointers
_widths = {}      # integer torch dtype -> its bytes
_workspaces = {}  # (tokens, choices, experts) -> bytes that expert_sort asks for
_DEVICE = _capi.DEVICE_POINTERS
_F32 = _capi.F32 | _DEVICE


def _setup():
    """torch is imported by the first call that gets a tensor."""
    global _torch, _empty, _library, _raw_stream, _current_device, _int32, _int64, _float32
    import torch

    _types.update({torch.float32: _F32, torch.float16: _capi.F16 | _DEVICE, torch.bfloat16: _capi.BF16 | _DEVICE})
    _int32, _int64, _float32 = torch.int32, torch.int64, torch.float32
    _widths.update({_int32: 4, _int64: 8})
    _empty, _current_device = torch.empty, torch.cuda.current_device
    # the handle itself, where torch gives it without a Stream object around it
    _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    if _raw_stream is None:
        _raw_stream = lambda device: torch.cuda.current_stream(device).cuda_stream  # noqa: E731
    _library, _torch = _capi.lib(), torch


def _no(where: str, message: str):
    raise ValueError(f"{where}: {message}")


def _stream(device: int, stream, where: str, *tensors) -> int:
    """The stream to launch on, given the first tensor's device; every tensor
    has to be on the current device, where the library launches (and which it
    is told: it does not ask for the pointers again)."""
    if device < 0 or device != _current_device():
        _no(where, f"a tensor is on {'the host' if device < 0 else f'cuda:{device}'}, not on the current device")
    for x in tensors:
        if x is not None and x.get_device() != device:
            _no(where, f"a tensor is on {x.device}, but the current device is cuda:{device}")
    if stream is None:
        return _raw_stream(device)
    return stream if isinstance(stream, int) else int(stream.cuda_stream)


def _empty_there(stream, st: int):
    """torch.empty for a call that was given a stream, whose handle is st."""
    return _empty if st == _raw_stream(_current_device()) else empty_on(stream)


def _check(status: int, where: str) -> None:
    if status:
        from . import BmmcError

        raise BmmcError(status, where)


def _no_type(x, where: str, name: str):
    _no(where, f"{name} is {x.dtype}; float32, float16 and bfloat16 are supported")


def _matrix(x, where: str, name: str):
    """Rows, columns and row stride of a 2-D tensor whose rows are dense."""
    if x.dim() != 2:
        _no(where, f"{name} must be 2-D with dense rows")
    (rows, cols), (stride, inner) = x.shape, x.stride()
    if inner != 1 and cols > 1:
        _no(where, f"{name} must be 2-D with dense rows")
    return rows, cols, stride


def _slot(slot, where: str):
    if slot.dtype is not _int32 or slot.dim() != 2 or not slot.is_contiguous():
        _no(where, "slot must be a contiguous int32 tensor [tokens, choices]")
    return slot.shape


def _output(out, rows: int, cols: int, like, where: str) -> int:
    """The row stride of `out`, which has to be a [rows, cols] tensor of
    like's type."""
    r, c, stride = _matrix(out, where, "out")
    if r != rows or c != cols or out.dtype != like.dtype:
        _no(where, f"out has shape {tuple(out.shape)} and type {out.dtype}, expected shape ({rows}, {cols}) and "
                   f"type {like.dtype}")
    return stride


def expert_sort(experts, num_experts: int, stream=None):
    """(slot, source, offsets) of a router's choices ``experts`` [tokens,
    choices] (int32 or int64; ids outside [0, num_experts) are not routed).

    ``slot`` [tokens, choices]: the choice's row among all choices sorted by
    expert (stable), or ~row where it is not routed; ``source`` [tokens *
    choices]: the flat choice of each row, or its complement; ``offsets``
    [num_experts + 1]: expert e has rows offsets[e] .. offsets[e + 1] - 1."""
    if _torch is None:
        _setup()
    where = "expert_sort"
    width = _widths.get(experts.dtype)
    if width is None or experts.dim() != 2 or not experts.is_contiguous():
        _no(where, "experts must be a contiguous int32 or int64 tensor [tokens, choices]")
    st = _stream(experts.get_device(), stream, where)
    T, K = experts.shape
    need = _workspaces.get((T, K, num_experts))
    if need is None:
        size = ctypes.c_size_t()
        _check(_library.expert_sort_workspace(T, K, num_experts, size), where)
        if len(_workspaces) > 1000:
            _workspaces.clear()
        need = _workspaces[T, K, num_experts] = size.value
    device = experts.device
    empty = _empty if stream is None else _empty_there(stream, st)
    slot = empty((T, K), dtype=_int32, device=device)
    source = empty(T * K, dtype=_int32, device=device)
    offsets = empty(num_experts + 1, dtype=_int32, device=device)
    work_ptr = None
    if need:
        work = empty(need // 4, dtype=_int32, device=device)
        work_ptr = work.data_ptr()
    status = _library.expert_sort(experts.data_ptr(), width | _DEVICE, T, K, num_experts, slot.data_ptr(),
                                  source.data_ptr(), offsets.data_ptr(), work_ptr, need, st)
    if status:
        _check(status, where)
    return slot, source, offsets


def expert_dispatch(x, slot, num_rows=None, out=None, stream=None):
    """rows[slot[t, k]] = x[t] for every routed choice, zero in the rows of
    the others; [num_rows, hidden], num_rows = tokens * choices unless fewer
    are asked for (choices numbered num_rows and above are dropped)."""
    if _torch is None:
        _setup()
    where = "expert_dispatch"
    T, K = _slot(slot, where)
    tokens, H, x_stride = _matrix(x, where, "x")
    if tokens != T:
        _no(where, f"x has shape {tuple(x.shape)} for {T} tokens")
    R = T * K if num_rows is None else int(num_rows)
    if not 0 <= R <= T * K:
        _no(where, f"num_rows {R} is outside [0, {T * K}]")
    t = _types.get(x.dtype)
    if t is None:
        _no_type(x, where, "x")
    if out is None:
        st = _stream(x.get_device(), stream, where, slot)
        empty = _empty if stream is None else _empty_there(stream, st)
        out, stride = empty((R, H), dtype=x.dtype, device=x.device), H
    else:
        st = _stream(x.get_device(), stream, where, slot, out)
        stride = _output(out, R, H, x, where)
    status = _library.expert_dispatch(x.data_ptr(), x_stride, slot.data_ptr(), T, K, H, t, out.data_ptr(), stride, R, st)
    if status:
        _check(status, where)
    return out


def _weights(weights, slot, rows, where: str) -> int:
    if weights.shape != slot.shape or not weights.is_contiguous():
        _no(where, "weights must be a contiguous tensor of slot's shape")
    if weights.dtype is not _float32 and weights.dtype != rows.dtype:
        _no(where, "weights must be float32 or of the rows' type")
    return _types[weights.dtype] & ~_DEVICE


def expert_combine(rows, slot, weights=None, out=None, stream=None):
    """out[t] = sum over the routed choices k of weights[t, k] *
    rows[slot[t, k]] (weights float32 or of the rows' type); without weights
    the plain sum, which is the gradient of expert_dispatch by x."""
    if _torch is None:
        _setup()
    where = "expert_combine"
    T, K = _slot(slot, where)
    R, H, row_stride = _matrix(rows, where, "rows")
    if R > T * K:
        _no(where, f"rows has {R} rows for {T * K} choices")
    t = _types.get(rows.dtype)
    if t is None:
        _no_type(rows, where, "rows")
    wt, wp = 0, None
    if weights is not None:
        wt, wp = _weights(weights, slot, rows, where), weights.data_ptr()
    st = _stream(rows.get_device(), stream, where, slot, weights, out)
    if out is None:
        empty = _empty if stream is None else _empty_there(stream, st)
        out, stride = empty((T, H), dtype=rows.dtype, device=rows.device), H
    else:
        stride = _output(out, T, H, rows, where)
    status = _library.expert_combine(rows.data_ptr(), row_stride, R, slot.data_ptr(), wp, wt, T, K, H, t, out.data_ptr(),
                                     stride, st)
    if status:
        _check(status, where)
    return out


def expert_combine_backward(grad, rows, slot, weights, stream=None):
    """(grad_rows, grad_weights) of expert_combine(rows, slot, weights) from
    the gradient of its result."""
    if _torch is None:
        _setup()
    where = "expert_combine_backward"
    T, K = _slot(slot, where)
    R, H, row_stride = _matrix(rows, where, "rows")
    if R > T * K:
        _no(where, f"rows has {R} rows for {T * K} choices")
    tokens, cols, grad_stride = _matrix(grad, where, "grad")
    if tokens != T or cols != H or grad.dtype != rows.dtype:
        _no(where, f"grad must have the shape ({T}, {H}) and the type of rows")
    t = _types.get(rows.dtype)
    if t is None:
        _no_type(rows, where, "rows")
    wt = _weights(weights, slot, rows, where)
    st = _stream(rows.get_device(), stream, where, grad, slot, weights)
    device = rows.device
    empty = _empty if stream is None else _empty_there(stream, st)
    grad_rows = empty((R, H), dtype=rows.dtype, device=device)
    grad_weights = empty((T, K), dtype=weights.dtype, device=device)
    status = _library.expert_combine_backward(grad.data_ptr(), grad_stride, rows.data_ptr(), row_stride, R,
                                              slot.data_ptr(), weights.data_ptr(), wt, T, K, H, t, grad_rows.data_ptr(), H,
                                              grad_weights.data_ptr(), st)
    if status:
        _check(status, where)
    return grad_rows, grad_weights


def _heads(x, where: str, name: str):
    """token_heads_t of a tensor [tokens, heads, dim] with dense heads, and
    its tokens."""
    if x.dim() != 3:
        _no(where, f"{name} must be [tokens, heads, dim] with dense heads")
    (tokens, heads, dim), (token_stride, head_stride, inner) = x.shape, x.stride()
    if inner != 1 and dim > 1:
        _no(where, f"{name} must be [tokens, heads, dim] with dense heads")
    return (x.data_ptr(), heads, dim, token_stride, head_stride), tokens


_NO_HEADS = (0, 0, 0, 0, 0)


def _alike(x, tokens: int, dtype, where: str, name: str):
    h, n = _heads(x, where, name)
    if n != tokens or x.dtype != dtype:
        _no(where, f"{name} must have the type and the tokens of the other heads")
    return h


def _turned_output(x, X, out, tokens: int, stream, st: int, where: str, name: str):
    """`out`, checked, or a new tensor; and its heads."""
    heads, dim = X[1], X[2]
    if out is None:
        empty = _empty if stream is None else _empty_there(stream, st)
        out = empty((tokens, heads, dim), dtype=x.dtype, device=x.device)
        return out, (out.data_ptr(), heads, dim, heads * dim, dim)
    O = _alike(out, tokens, x.dtype, where, name)
    if O[1:3] != X[1:3]:
        _no(where, f"{name} must have the shape ({tokens}, {heads}, {dim})")
    return out, O


def _turns(tokens: int, positions, inv_freq, pair_axes, flags: int, where: str):
    """rotary_turns_t"""
    if inv_freq is None:
        if positions is not None or pair_axes is not None:
            _no(where, "positions and pair_axes need inv_freq")
        return 0, 0, 0, 0, 0, 0, 0, flags
    if inv_freq.dtype is not _float32 or inv_freq.dim() != 1 or not inv_freq.is_contiguous():
        _no(where, "inv_freq must be a contiguous float32 tensor [pairs]")
    pairs = inv_freq.shape[0]
    axes_ptr = 0
    if pair_axes is not None:
        if pair_axes.dtype is not _int32 or pair_axes.shape != inv_freq.shape or not pair_axes.is_contiguous():
            _no(where, "pair_axes must be a contiguous int32 tensor [pairs]")
        axes_ptr = pair_axes.data_ptr()
    if positions is None:
        return inv_freq.data_ptr(), axes_ptr, 0, 0, 0, 0, pairs, flags
    width = _widths.get(positions.dtype)
    shape, strides = positions.shape, positions.stride()
    if width is None or len(shape) not in (1, 2) or shape[-1] != tokens or (tokens > 1 and strides[-1] != 1):
        _no(where, "positions must be an int32 or int64 tensor [tokens] or [axes, tokens] with dense rows")
    axes, stride = (1, 0) if len(shape) == 1 else (shape[0], strides[0])
    return inv_freq.data_ptr(), axes_ptr, positions.data_ptr(), width, axes, stride, pairs, flags


def rotary(x, positions, inv_freq, pair_axes=None, *, interleaved: bool = False, inverse: bool = False, out=None,
           stream=None):
    """Heads x [tokens, heads, dim] (any token and head strides) turned by
    their tokens' positions [tokens] or [axes, tokens]: pair i, the elements
    i and i + pairs of a head, or 2i and 2i + 1 if interleaved, by the angle
    position * inv_freq[i], with the position on axis pair_axes[i] (axis 0
    without pair_axes; no turn for an axis that is not there).  Elements from
    2 * pairs on are copied.  inverse turns back, which is the gradient.  out
    may be x."""
    if _torch is None:
        _setup()
    where = "rotary"
    X, T = _heads(x, where, "x")
    t = _types.get(x.dtype)
    if t is None:
        _no_type(x, where, "x")
    if positions is None or inv_freq is None:
        _no(where, "positions and inv_freq are needed")
    flags = (_capi.ROTARY_ADJACENT if interleaved else 0) | (_capi.ROTARY_INVERSE if inverse else 0)
    turns = _turns(T, positions, inv_freq, pair_axes, flags, where)
    st = _stream(x.get_device(), stream, where, positions, inv_freq, pair_axes, out)
    out, O = _turned_output(x, X, out, T, stream, st, where, "out")
    status = _library.rotary(_capi.ROTARY_ARGS.pack(T, t, *X, *O, *turns), st)
    if status:
        _check(status, where)
    return out


def _cache(c, X, dtype, head_major: bool, where: str, name: str):
    """(pages, page_size) and paged_cache_t of a cache."""
    if c.dim() != 4 or c.dtype != dtype:
        _no(where, f"{name} must be 4-D of k's type with dense heads")
    (pages, page, heads, dim), (page_stride, slot_stride, head_stride, inner) = c.shape, c.stride()
    if inner != 1 and dim > 1:
        _no(where, f"{name} must be 4-D of k's type with dense heads")
    if head_major:
        page, heads, slot_stride, head_stride = heads, page, head_stride, slot_stride
    if heads != X[1] or dim != X[2]:
        _no(where, f"{name} has shape {tuple(c.shape)}, which does not fit the new heads")
    return (pages, page), (c.data_ptr(), page_stride, slot_stride, head_stride)


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
    if _torch is None:
        _setup()
    where = "paged_append"
    K, T = _heads(k, where, "k")
    dtype = k.dtype
    t = _types.get(dtype)
    if t is None:
        _no_type(k, where, "k")
    V = _alike(v, T, dtype, where, "v")
    if K[1] != V[1]:
        _no(where, "k and v must have the same heads")
    geometry, k_at = _cache(k_cache, K, dtype, head_major, where, "k_cache")
    other, v_at = _cache(v_cache, V, dtype, head_major, where, "v_cache")
    if geometry != other:
        _no(where, f"v_cache has shape {tuple(v_cache.shape)}, which does not fit k_cache's pages")
    B, columns, table_stride = _matrix(page_table, where, "page_table")
    if page_table.dtype is not _int32:
        _no(where, "page_table must be an int32 tensor [sequences, columns]")
    if lengths.dtype is not _int32 or lengths.shape != (B,) or not lengths.is_contiguous():
        _no(where, "lengths must be a contiguous int32 tensor [sequences]")
    starts_ptr = 0
    if starts is None:
        if T != B:
            _no(where, f"{T} tokens for {B} sequences need starts")
    elif starts.dtype is not _int32 or starts.shape != (B + 1,) or not starts.is_contiguous():
        _no(where, "starts must be a contiguous int32 tensor [sequences + 1]")
    else:
        starts_ptr = starts.data_ptr()
    turns = _turns(T, positions, inv_freq, pair_axes, _capi.ROTARY_ADJACENT if interleaved else 0, where)
    st = _stream(k.get_device(), stream, where, v, k_cache, v_cache, page_table, lengths, starts, q, q_out, positions,
                 inv_freq, pair_axes)
    Q = O = _NO_HEADS
    if q is not None:
        Q = _alike(q, T, dtype, where, "q")
        q_out, O = _turned_output(q, Q, q_out, T, stream, st, where, "q_out")
    elif q_out is not None:
        _no(where, "q_out without q")
    status = _library.paged_append(_capi.PAGED_APPEND_ARGS.pack(
        T, t, *K, *V, *Q, *O, *turns, starts_ptr, lengths.data_ptr(), B, page_table.data_ptr(), table_stride, columns,
        *geometry, *k_at, *v_at), st)
    if status:
        _check(status, where)
    return q_out
