"""Run one permutation configuration a few times, for profilers.

    python -m bmmc_index_transforms_gb300.profile_case --kind random --n 26 --reps 3
    python -m bmmc_index_transforms_gb300.profile_case --kind lmad_slice_2d --shape 8192,8193 --reps 2

Kinds: random (seed), worst (seed, low 10 bits mapped to high bits), bitrev,
complement (A = I, c on the high bits: contiguous tiles on both sides),
window (seed, a random BMMC on the low --window bits and the identity above:
tiles scattered only inside aligned windows of 2^window elements),
transpose (square, n even), dims5 (the 5-D (4,2,0,3,1) permutation of a
[32,64,64,64,32]-shaped array scaled to n bits), copy (the copy kernel on the
same bytes), two_factor (seed, two passes through caller scratch).
General LMAD copies (--shape, --elem): lmad_slice_2d, lmad_slice_3d,
lmad_reversed_rows (the Futhark copy post's "Impact" functions on a
row-major array of that shape), lmad_transpose (the shape's axes
reversed, made contiguous) and lmad_permute (the shape's axes in the order
--perm, out dimension k = in dimension perm[k], made contiguous; --blocked
auto / force / never chooses for the blocked copy).
Moves of tokens (--tokens, --type; --choices, --experts, --hidden or --heads,
--kv-heads, --dim): token_sort, token_dispatch, token_combine,
token_combine_backward, token_rotary (positions on three axes), token_append
(8 sequences, pages of 64 entries, queries turned with the keys),
token_append8 and token_read8 (the same with e4m3 pages), token_lookup and
token_lookup_backward (--vocab; ids as frequent as words), token_balance,
token_balance_backward.
Prints the plan and the CUDA-event time of each repetition.
"""

from __future__ import annotations

import argparse
import math
import sys

import torch

import bmmc_index_transforms_gb300 as bm
from bmmc_index_transforms_gb300 import maps, synth


def _accept(n, elem):
    def f(rows):
        try:
            bm.bmmc_plan_destroy(bm.bmmc_plan(n, rows, 0, elem))
            return True
        except bm.BmmcError as e:
            if e.status == 2:
                return False
            raise
    return f


def main(argv=None):
    ap = argparse.ArgumentParser()
    ap.add_argument("--kind", default="random",
                    choices=["random", "worst", "bitrev", "transpose", "dims5", "copy", "two_factor",
                             "complement", "window", "lmad_slice_2d", "lmad_slice_3d", "lmad_reversed_rows",
                             "lmad_transpose", "lmad_permute", "token_sort", "token_dispatch", "token_combine",
                             "token_combine_backward", "token_rotary", "token_append", "token_lookup",
                             "token_lookup_backward", "token_balance", "token_balance_backward", "token_append8",
                             "token_read8"])
    ap.add_argument("--n", type=int, default=26)
    ap.add_argument("--elem", type=int, default=4)
    ap.add_argument("--seed", type=int, default=0)
    ap.add_argument("--reps", type=int, default=3)
    ap.add_argument("--t-in", type=int, default=0)
    ap.add_argument("--t-out", type=int, default=0)
    ap.add_argument("--tile-bits", type=int, default=0)
    ap.add_argument("--shape", default="8192,8193")
    ap.add_argument("--window", type=int, default=22, help="window: log2 elements of a window")
    ap.add_argument("--perm", default="", help="lmad_permute: axis order of the destination")
    ap.add_argument("--blocked", default="auto", choices=["auto", "force", "never"])
    ap.add_argument("--type", default="bf16", choices=["f32", "f16", "bf16"])
    for name, value in (("tokens", 4096), ("vocab", 131072), ("choices", 8), ("experts", 64), ("hidden", 4096), ("heads", 32),
                        ("kv-heads", 8), ("dim", 128)):
        ap.add_argument(f"--{name}", type=int, default=value)
    a = ap.parse_args(argv)
    if a.kind.startswith("token_"):
        return token_case(a)
    if a.kind.startswith("lmad_"):
        return lmad_case(a)
    n, elem = a.n, a.elem
    nbytes = (1 << n) * elem
    d_in = torch.arange(nbytes // 4, dtype=torch.int32, device="cuda")
    d_out = torch.empty_like(d_in)
    mode = 1 if a.kind == "two_factor" else 0
    if a.kind in ("random", "two_factor"):
        rows, c, _ = synth.draw_bmmc(a.seed, n, _accept(n, elem))
    elif a.kind == "worst":
        rows, c, _ = synth.draw_bmmc(a.seed, n, _accept(n, elem), low_to_high=min(10, n // 2))
    elif a.kind == "window":
        m = min(a.window, n)
        low, cl, _ = synth.draw_bmmc(a.seed, m, _accept(m, elem))
        rows, c = list(low) + maps.identity_rows(n)[m:], cl
    elif a.kind == "complement":
        # A = I, c on the bits above the tile: every tile is contiguous on both sides
        rows, c = maps.identity_rows(n), ((1 << n) - 1) & ~((1 << 16) - 1)
    elif a.kind == "bitrev":
        rows, c = maps.bitrev_rows(n), 0
    elif a.kind == "transpose":
        rows, c = maps.rotate_rows(n, n // 2), 0
    elif a.kind == "dims5":
        # split n bits like [32,64,64,64,32] (5,6,6,6,5 bits) scaled to n
        base = [5, 6, 6, 6, 5]
        while sum(base) > n:
            base[base.index(max(base))] -= 1
        while sum(base) < n:
            base[base.index(min(base))] += 1
        rows, c = maps.axes_rows(base, synth.FIVE_D_AXES), 0
    else:
        rows, c = None, 0
    stream = torch.cuda.current_stream()
    if rows is None:
        fn = lambda: bm.bmmc_copy(d_in, d_out, nbytes, stream)  # noqa: E731
        print(f"copy of {nbytes} bytes")
        plan = None
    else:
        plan = bm.Plan(rows, c, elem, mode=mode, t_in=a.t_in, t_out=a.t_out, tile_bits=a.tile_bits)
        print("plan:", plan.info)
        if mode == 1:
            scratch = torch.empty_like(d_in)
            fn = lambda: plan.permute_scratch(d_in, d_out, scratch, stream)  # noqa: E731
        else:
            fn = lambda: plan.permute(d_in, d_out, stream)  # noqa: E731
    for r in range(a.reps):
        s, e = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        s.record(stream)
        fn()
        e.record(stream)
        torch.cuda.synchronize()
        ms = s.elapsed_time(e)
        print(f"rep {r}: {ms:.4f} ms, {2 * nbytes / ms / 1e6:.1f} GB/s effective")
    if plan:
        plan.close()
    return 0


def lmad_view(a) -> dict:
    """The LMAD copy of an lmad_* kind: sizes, offsets and strides in
    elements, as lmad_copy takes them."""
    shape = [int(v) for v in a.shape.split(",")]
    if a.kind in ("lmad_transpose", "lmad_permute"):
        perm = ([int(v) for v in a.perm.split(",")] if a.kind == "lmad_permute"
                else list(range(len(shape)))[::-1])
        if sorted(perm) != list(range(len(shape))):
            raise SystemExit("--perm must order the axes of --shape")
        out_rm = synth.row_major_strides([shape[p] for p in perm])
        out_strides = [0] * len(shape)
        for pos, p in enumerate(perm):
            out_strides[p] = out_rm[pos]
        total = 1
        for v in shape:
            total *= v
        return dict(sizes=shape, in_offset=0, in_strides=synth.row_major_strides(shape), in_elems=total,
                    out_offset=0, out_strides=out_strides, out_elems=total)
    return synth.page_lmad_workload(a.kind[len("lmad_"):], shape)


def token_call(a):
    """The call of a token_* kind, and the bytes that it cannot do without."""
    g = torch.Generator("cuda").manual_seed(a.seed)
    dtype = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}[a.type]
    T, K, H, es = a.tokens, a.choices, a.hidden, 4 if a.type == "f32" else 2
    new = lambda *s: torch.randn(*s, generator=g, device="cuda", dtype=dtype)  # noqa: E731
    if a.kind in ("token_lookup", "token_lookup_backward"):
        u = torch.rand(T, generator=g, device="cuda", dtype=torch.float64)
        ids = (torch.exp(u * math.log(a.vocab + 1)) - 1).long().clamp(max=a.vocab - 1)
        if a.kind == "token_lookup":
            table = new(a.vocab, H)
            return lambda: bm.embedding_lookup(table, ids), (T + int(ids.unique().numel())) * H * es
        grad = new(T, H)
        return lambda: bm.embedding_backward(grad, ids, a.vocab), (T + a.vocab) * H * es
    if a.kind in ("token_balance", "token_balance_backward"):
        logits = new(T, a.experts)
        ids = logits.float().topk(K, dim=1)[1].int()
        if a.kind == "token_balance":
            return lambda: bm.expert_balance(logits, ids), T * (a.experts * es + K * 4)
        counts, by = bm.expert_balance(logits, ids)[1], torch.ones((), device="cuda")
        return lambda: bm.expert_balance_backward(by, logits, ids, counts), T * (2 * a.experts * es + K * 4)
    if a.kind in ("token_rotary", "token_append", "token_append8", "token_read8"):
        pairs = a.dim // 2
        freq = 10000.0 ** (-torch.arange(pairs, device="cuda") / pairs)
        axes = (torch.arange(pairs, device="cuda") * 3 // pairs).int()
        positions = torch.randint(0, 4096, (3, T), generator=g, device="cuda").int()
        if a.kind == "token_rotary":
            x = new(T, a.heads, a.dim)
            return lambda: bm.rotary(x, positions, freq, axes), 2 * x.numel() * es
        qkv = new(T, a.heads + 2 * a.kv_heads, a.dim)
        q, k, v = qkv.split([a.heads, a.kv_heads, a.kv_heads], dim=1)
        starts = (torch.arange(9, device="cuda") * T // 8).int()
        columns = (T // 8 + 1000) // 64 + 2
        table = torch.randperm(8 * columns, generator=g, device="cuda").int().view(8, columns)
        lengths = torch.randint(0, 1000, (8,), generator=g, device="cuda").int()
        if a.kind in ("token_append8", "token_read8"):
            caches = [torch.zeros(8 * columns, 64, a.kv_heads, a.dim, device="cuda", dtype=torch.float8_e4m3fn) for _ in range(2)]
            k_scales, v_scales = (torch.ones(8 * columns, 64, a.kv_heads, device="cuda") for _ in range(2))
            scales = dict(k_scales=k_scales, v_scales=v_scales)
            moved = 2 * T * a.kv_heads * (a.dim * (es + 1) + 4)
            if a.kind == "token_read8":
                return lambda: bm.paged_read(*caches, table, starts, T, dtype=dtype, **scales), moved
            return lambda: bm.paged_append(k, v, *caches, table, lengths, starts=starts, q=q, inv_freq=freq,
                                           **scales), moved + 2 * q.numel() * es
        caches = [new(8 * columns, 64, a.kv_heads, a.dim) for _ in range(2)]
        return lambda: bm.paged_append(k, v, *caches, table, lengths, starts=starts, q=q, positions=positions,
                                       inv_freq=freq, pair_axes=axes), 2 * qkv.numel() * es
    ids = torch.rand(T, a.experts, generator=g, device="cuda").topk(K, dim=1)[1]
    slot = bm.expert_sort(ids, a.experts)[0]
    if a.kind == "token_sort":
        return lambda: bm.expert_sort(ids, a.experts), T * K * 16
    if a.kind == "token_dispatch":
        x = new(T, H)
        return lambda: bm.expert_dispatch(x, slot), (T + T * K) * H * es
    rows, w = new(T * K, H), torch.rand(T, K, generator=g, device="cuda")
    if a.kind == "token_combine":
        return lambda: bm.expert_combine(rows, slot, w), (T + T * K) * H * es
    x = new(T, H)
    return lambda: bm.expert_combine_backward(x, rows, slot, w), (T + 2 * T * K) * H * es


def token_case(a):
    call, nbytes = token_call(a)
    stream = torch.cuda.current_stream()
    for r in range(a.reps):
        s, t = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        s.record(stream)
        call()
        t.record(stream)
        torch.cuda.synchronize()
        ms = s.elapsed_time(t)
        print(f"rep {r}: {ms:.4f} ms, {nbytes / ms / 1e6:.1f} GB/s effective")
    return 0


def lmad_case(a):
    e = a.elem
    w = lmad_view(a)
    src = torch.empty(w["in_elems"] * e, dtype=torch.uint8, device="cuda")
    dst = torch.empty(w["out_elems"] * e, dtype=torch.uint8, device="cuda")
    args = (w["sizes"], w["in_offset"], w["in_strides"], w["out_offset"], w["out_strides"], e)
    print("analysis:", bm.lmad_copy_query(*args, src, dst, blocked=a.blocked))
    stream = torch.cuda.current_stream()
    for r in range(a.reps):
        s, t = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        s.record(stream)
        bm.lmad_copy(*args, src, dst, stream, blocked=a.blocked)
        t.record(stream)
        torch.cuda.synchronize()
        ms = s.elapsed_time(t)
        print(f"rep {r}: {ms:.4f} ms, {2 * w['out_elems'] * e / ms / 1e6:.1f} GB/s effective")
    return 0


if __name__ == "__main__":
    sys.exit(main())
