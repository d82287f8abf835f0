// What the kernels that turn heads and find their tokens' places in a paged
// cache share (rotary.cu, paged_cache8.cu).  Each source includes bounds.cuh,
// with its own BMMC_CHK_FILE tag, before this header.
#pragma once

#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "../../include/bmmc.h"
#include "token_moves.hpp"
#include "token_words.cuh"

namespace bmmc {

constexpr int kMaxTokensPerBlock = 64;
constexpr int kAhead = 2;               // turns whose inputs a thread has in flight

// Heads of one kind (queries, keys, values): where they lie and where they
// go.  Strides in bytes.  place: 0 = the token's own place (dst_token apart),
// 1 / 2 = the token's place in the key / value cache.
struct Heads {
    const char* src;
    char* dst;
    int64_t src_token, src_head, dst_token, dst_head;
    int heads, turned, place;
    int turning, items;  // words of a head that are turned (pairs of words in halves), and all
    int across, magic;   // threads side by side on a head's words, and 65536 / across rounded up
    int words, batch;    // staged rows: words of a head, heads of a warp at a time
    unsigned words_magic;  // 2^32 / words rounded up (words > 1)
    unsigned ahead;      // bytes of a token's heads to fetch ahead; 0: they do not lie in one run of 16-byte words
};

struct MoveParams {
    Heads part[3];
    int parts;
    int64_t tokens;
    int group_log2;  // threads of a token
    bool adjacent;   // staged rows: pairs side by side
    bool device;     // the heads are the device's own memory and may be fetched ahead
    // rotation
    const void* positions;  // NULL: the token's place in its sequence
    int position_bytes, axes, pairs;
    unsigned pairs_magic;  // 2^32 / pairs rounded up (pairs > 1)
    int64_t axis_stride;
    const float* freq;
    const int* pair_axes;  // NULL: axis 0
    float sign;
    // places in the cache; page_size 0: there is none
    const int *starts, *lengths, *table;  // lengths NULL: zeros
    int64_t sequences, table_stride, table_columns, pages;
    int page_size;
    int64_t page_stride[2], slot_stride[2];  // of the key and the value cache, bytes
};

// The last sequence whose start is <= t, -1 if there is none: by a whole
// warp, 32 starts at a time, and by one thread.  Any starts, in order or not,
// give an index in range.
__device__ inline int64_t find_sequence_warp(const int* starts, int64_t sequences, int64_t t, int lane) {
    int64_t lo = 0, n = sequences;  // the answer lies in [lo, lo + n) or is lo - 1
    while (n > 0) {
        const int64_t step = (n + 31) / 32;
        const int64_t i = lo + lane * step;
        const bool before = lane * step < n && BMMC_RD_OK(starts + i, 4) && starts[i] <= t;
        const int c = __popc(__ballot_sync(~0u, before));
        if (c == 0) return lo - 1;
        const int64_t at = lo + (c - 1) * step;  // starts[at] <= t
        if (step == 1) return at;
        n = min(step, lo + n - at) - 1;
        lo = at + 1;
    }
    return lo - 1;
}

__device__ inline int64_t find_sequence(const int* starts, int64_t sequences, int64_t t) {
    int64_t lo = 0, hi = sequences;  // starts[lo - 1] <= t, starts[hi] > t
    while (lo < hi) {
        const int64_t mid = (lo + hi) >> 1;
        if (BMMC_RD_OK(starts + mid, 4) && starts[mid] <= t) lo = mid + 1;
        else hi = mid;
    }
    return lo - 1;
}

// Token t's position in its sequence b and its byte offsets in the caches.
struct Place {
    int64_t at;       // 0 outside every sequence
    int64_t byte[2];  // -1: no page
    int page, slot;   // -1: no page
};

__device__ inline Place place_of(const MoveParams& p, int64_t t, int64_t b) {
    Place r{0, {-1, -1}, -1, -1};
    int64_t first = t;
    if (p.starts) {
        if (b < 0 || !BMMC_RD_OK(p.starts + b, 8)) return r;
        first = p.starts[b];
    } else if (t >= p.sequences) {
        return r;
    }
    if (p.lengths && !BMMC_RD_OK(p.lengths + b, 4)) return r;
    const int length = p.lengths ? p.lengths[b] : 0, next = p.starts ? p.starts[b + 1] : 0;  // on their way together
    if (p.starts && t >= next) return r;
    r.at = (int64_t)length + (t - first);
    if (r.at < 0 || r.at >= (int64_t)1 << 32) return r;  // (more only by starts below zero)
    const unsigned at = (unsigned)r.at, column = at / p.page_size;
    if (column >= p.table_columns) return r;
    if (!BMMC_RD_OK(p.table + b * p.table_stride + column, 4)) return r;
    const int page = p.table[b * p.table_stride + column];
    if (page < 0 || page >= p.pages) return r;
    r.page = page;
    r.slot = (int)(at - column * p.page_size);
    for (int c = 0; c < 2; ++c) r.byte[c] = page * p.page_stride[c] + (int64_t)r.slot * p.slot_stride[c];
    return r;
}

// Written out, so that every variant rounds alike.
__device__ __forceinline__ float turned_first(float x, float y, float2 r) { return fmaf(x, r.x, -__fmul_rn(y, r.y)); }
__device__ __forceinline__ float turned_second(float x, float y, float2 r) { return fmaf(y, r.x, __fmul_rn(x, r.y)); }

// The start of a block that takes tokens t0 .. t0 + nt - 1 and some of the
// parts: the tokens' places in the caches and positions, and the cosines and
// sines of their pairs, into shared memory (with slots, the places' pages and
// entries too); the whole block takes part.
__device__ __forceinline__ void begin_block(const MoveParams& p, int64_t t0, int nt, int first_part, int last_part,
                                            Slots<float2> turns, Slots<int64_t> places, Slots<float> place_numbers,
                                            Slots<int> slots = Slots<int>(nullptr, 0)) {
    const int tid = threadIdx.x, threads = blockDim.x;
    const bool turning = p.pairs && p.part[first_part].turned;
    // A thread's first turns (what they need but for a position that follows
    // from the place), and all the heads (to L2), are on their way while the
    // places are worked out.
    float freq[kAhead] = {}, position[kAhead] = {};
    bool by_place[kAhead] = {};
    const auto start_turn = [&](int i, float& f, float& at, bool& from_place) {
        const int k = quotient(i, p.pairs, p.pairs_magic), pair = i - k * p.pairs;
        const int axis = p.pair_axes && BMMC_RD_OK(p.pair_axes + pair, 4) ? p.pair_axes[pair] : 0;
        f = BMMC_RD_OK(p.freq + pair, 4) ? p.freq[pair] : 0.0f;
        at = 0.0f;  // an axis that is not there does not turn
        from_place = !p.positions && axis == 0;
        if (p.positions && axis >= 0 && axis < p.axes) {
            const int64_t j = axis * p.axis_stride + t0 + k;
            if (BMMC_RD_OK(static_cast<const char*>(p.positions) + j * p.position_bytes, p.position_bytes))
                at = p.position_bytes == 4 ? (float)static_cast<const int32_t*>(p.positions)[j]
                                           : (float)static_cast<const int64_t*>(p.positions)[j];
        }
    };
#pragma unroll
    for (int u = 0; u < kAhead; ++u)
        if (turning && tid + u * threads < nt * p.pairs) start_turn(tid + u * threads, freq[u], position[u], by_place[u]);
    if (tid < nt * (last_part - first_part)) {
        const Heads& h = p.part[first_part + tid / nt];
        if (h.ahead)
            asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(
                             __cvta_generic_to_global(h.src + (t0 + tid % nt) * h.src_token)),
                         "r"(h.ahead)
                         : "memory");
    }
    const auto keep_place = [&](int i, const Place& r) {
        places.set(i, r.byte[0]);
        places.set(kMaxTokensPerBlock + i, r.byte[1]);
        place_numbers.set(i, (float)r.at);
        if (slots.p) slots.set(i, r.page), slots.set(kMaxTokensPerBlock + i, r.slot);
    };
    if (p.page_size) {
        if (p.starts && nt <= 8) {
            for (int i = tid >> 5; i < nt; i += threads >> 5) {
                const Place r = place_of(p, t0 + i, find_sequence_warp(p.starts, p.sequences, t0 + i, tid & 31));
                if ((tid & 31) == 0) keep_place(i, r);
            }
        } else if (tid < nt) {
            const int64_t t = t0 + tid;
            const Place r = place_of(p, t, p.starts ? find_sequence(p.starts, p.sequences, t) : t);
            keep_place(tid, r);
        }
        if (!p.positions) __syncthreads();
    }
    if (turning) {
        const auto end_turn = [&](int i, float f, float at, bool from_place) {
            if (from_place) at = place_numbers.get(quotient(i, p.pairs, p.pairs_magic));
            float s, c;
            sincosf(at * f, &s, &c);
            turns.set(i, make_float2(c, p.sign * s));
        };
#pragma unroll
        for (int u = 0; u < kAhead; ++u)
            if (tid + u * threads < nt * p.pairs) end_turn(tid + u * threads, freq[u], position[u], by_place[u]);
        for (int i = tid + kAhead * threads; i < nt * p.pairs; i += threads) {
            float f, at;
            bool from_place;
            start_turn(i, f, at, from_place);
            end_turn(i, f, at, from_place);
        }
    }
    __syncthreads();
}

inline bmmc_status check_heads(const token_heads_t& x, int64_t tokens, int es) {
    if (!x.data || x.heads < 1 || x.dim < 1 || x.dim > ROTARY_MAX_DIM || x.heads > (1 << 24) / x.dim ||
        bad_stride(x.token_stride, tokens) || bad_stride(x.head_stride, x.heads))
        return BMMC_ERR_INVALID_ARG;
    return (uintptr_t)x.data % es ? BMMC_ERR_MISALIGNED : BMMC_OK;
}

// The array as rows along its longer stride.
inline Rows rows_of(const token_heads_t& x, int64_t tokens, int es) {
    const bool by_token = x.heads < 2 || x.token_stride >= x.head_stride;
    const int64_t n = by_token ? tokens : x.heads, s = by_token ? x.token_stride : x.head_stride;
    const int64_t m = by_token ? x.heads : tokens, u = by_token ? x.head_stride : x.token_stride;
    return Rows{x.data, n, s * es, ((m - 1) * u + x.dim) * es};
}

inline bool same_place(const token_heads_t& a, const token_heads_t& b, int64_t tokens) {
    return a.data == b.data && (tokens < 2 || a.token_stride == b.token_stride) &&
           (a.heads < 2 || a.head_stride == b.head_stride);
}

inline bool writable(const token_heads_t& x, int64_t tokens) {
    const int64_t sizes[2] = {tokens, x.heads}, strides[2] = {x.token_stride, x.head_stride};
    return one_to_one(x.dim, sizes, strides);
}

// Whether key and value cache, of elements of es bytes, lie between each other: by page, entry or head.
inline bool caches_between(const paged_append_args_t& a, int es) {
    const paged_cache_t &k = a.k_cache, &v = a.v_cache;
    const int64_t sizes[3] = {a.pages, a.page_size, a.k.heads};
    const int64_t strides[3] = {k.page_stride * es, k.slot_stride * es, k.head_stride * es};
    const int64_t others[3] = {v.page_stride * es, v.slot_stride * es, v.head_stride * es};
    for (int i = 0; i < 3; ++i)
        if (sizes[i] > 1 && strides[i] != others[i]) return false;
    return lie_between(a.k.dim * es, a.v.dim * es, sizes, strides, (int64_t)((uintptr_t)v.data - (uintptr_t)k.data));
}

inline uint64_t address_bits(const token_heads_t& x, int es) {
    return (uint64_t)(uintptr_t)x.data | (uint64_t)(x.token_stride * es) | (uint64_t)(x.head_stride * es) |
           (uint64_t)(x.dim * es);
}

// The rotation's arguments, checked and put into p.
inline bmmc_status set_turns(MoveParams& p, const rotary_turns_t& r, bool need_positions) {
    p.pairs = 0;
    if (r.flags & ~(int64_t)(ROTARY_ADJACENT | ROTARY_INVERSE)) return BMMC_ERR_INVALID_ARG;
    if (!r.inv_freq) return r.pairs || r.positions || r.pair_axes ? BMMC_ERR_INVALID_ARG : BMMC_OK;
    if (r.pairs < 1 || r.pairs > ROTARY_MAX_DIM / 2 || (need_positions && !r.positions)) return BMMC_ERR_INVALID_ARG;
    if ((uintptr_t)r.inv_freq % 4 || (uintptr_t)r.pair_axes % 4) return BMMC_ERR_MISALIGNED;
    if (r.positions) {
        if (r.position_bytes != 4 && r.position_bytes != 8) return BMMC_ERR_UNSUPPORTED_ELEM;
        if (r.axes < 1 || r.axes > ROTARY_MAX_AXES || bad_stride(r.axis_stride, r.axes)) return BMMC_ERR_INVALID_ARG;
        if ((uintptr_t)r.positions % r.position_bytes) return BMMC_ERR_MISALIGNED;
        p.position_bytes = (int)r.position_bytes;
        p.axes = (int)r.axes;
        p.axis_stride = r.axis_stride;
    }
    p.positions = r.positions;
    p.pairs = (int)r.pairs;
    p.pairs_magic = magic_of((int)r.pairs);
    p.freq = r.inv_freq;
    p.pair_axes = r.pair_axes;
    p.sign = r.flags & ROTARY_INVERSE ? -1.0f : 1.0f;
    return BMMC_OK;
}

// What the turns read.
inline Rows turn_rows(const rotary_turns_t& r, int64_t tokens, int what) {
    if (what == 0) return Rows{r.inv_freq, 1, 0, r.pairs * 4};
    if (what == 1) return Rows{r.pair_axes, 1, 0, r.pairs * 4};
    return Rows{r.positions, r.axes, r.axis_stride * r.position_bytes, tokens * r.position_bytes};
}

// Whether an output may share bytes with what the turns read.
inline bool meets_turns(const Rows& out, const rotary_turns_t& r, int64_t tokens) {
    for (int what = 0; what < 3; ++what)
        if (may_overlap(turn_rows(r, tokens, what), out)) return true;
    return false;
}

// The bits that a word's size has to divide on account of the pairs.
inline uint64_t pair_bits(const rotary_turns_t& r, int es) {
    return (uint64_t)(r.flags & ROTARY_ADJACENT ? 2 * r.pairs : r.pairs) * es;
}

inline Heads heads_of(const token_heads_t& x, int es, int turned) {
    Heads h{};
    h.src = static_cast<const char*>(x.data);
    h.src_token = x.token_stride * es;
    h.src_head = x.head_stride * es;
    h.heads = (int)x.heads;
    h.turned = turned;
    return h;
}

// A cache of `pages` pages of entries of heads * dim elements of es bytes.
inline bmmc_status check_cache(const paged_cache_t& m, int64_t pages, int64_t page_size, int64_t heads, int64_t dim, int es) {
    if ((!m.data && pages) || bad_stride(m.page_stride, pages) || bad_stride(m.slot_stride, page_size) ||
        bad_stride(m.head_stride, heads))
        return BMMC_ERR_INVALID_ARG;
    if ((uintptr_t)m.data % es) return BMMC_ERR_MISALIGNED;
    const int64_t sizes[3] = {pages, page_size, heads};
    const int64_t strides[3] = {m.page_stride, m.slot_stride, m.head_stride};
    return one_to_one(dim, sizes, strides) ? BMMC_OK : BMMC_ERR_INVALID_ARG;
}

inline Rows cache_rows(const paged_cache_t& m, int64_t pages, int64_t page_size, int64_t heads, int64_t dim, int es) {
    return Rows{m.data, pages, m.page_stride * es,
                ((page_size - 1) * m.slot_stride + (heads - 1) * m.head_stride + dim) * es};
}


// A call of paged_append: its arguments checked, the kernel's parameters, and
// the arrays it reads and writes.
struct AppendCall {
    MoveParams moves{};
    Rows k, v, q{}, written[3], maps[3];
    int dims[3];
    uint64_t in_bits = 0, cache_bits = 0, q_bits = 0;  // addresses and strides in bytes, or'ed
};

// The last check: whether the GPU reaches the arrays.
inline bmmc_status append_reachable(const paged_append_args_t& a, bool device) {
    return all_reachable(device, {a.k.data, a.v.data, a.q.data, a.q_out.data, a.k_cache.data, a.v_cache.data, a.starts, a.lengths,
                                  a.table, a.turns.inv_freq, a.turns.pair_axes, a.turns.positions});
}

// es: bytes of an element of the new heads, cache_es: of the caches.
inline bmmc_status read_append(const paged_append_args_t& a, int es, int cache_es, bool device, AppendCall& c) {
    MoveParams& p = c.moves;
    p.device = device;
    const bool with_q = a.q.data || a.q_out.data;
    bmmc_status s = check_heads(a.k, a.tokens, es);
    if (s == BMMC_OK) s = check_heads(a.v, a.tokens, es);
    if (s == BMMC_OK && with_q) s = check_heads(a.q, a.tokens, es);
    if (s == BMMC_OK && with_q) s = check_heads(a.q_out, a.tokens, es);
    if (s != BMMC_OK) return s;
    const int64_t turned = 2 * a.turns.pairs;
    if (a.k.heads != a.v.heads || turned > a.k.dim || (a.turns.flags & ROTARY_INVERSE)) return BMMC_ERR_INVALID_ARG;
    if (with_q && (a.q.heads != a.q_out.heads || a.q.dim != a.q_out.dim || turned > a.q.dim ||
                   !writable(a.q_out, a.tokens)))
        return BMMC_ERR_INVALID_ARG;
    if (a.sequences < 0 || a.sequences > kMaxTokens || (a.sequences && !a.lengths) ||
        (a.sequences && a.table_columns && !a.table) || a.table_columns < 0 || a.table_columns > kMaxTokens ||
        bad_stride(a.table_stride, a.sequences) || a.pages < 0 || a.pages > kMaxTokens ||
        a.page_size < 1 || a.page_size > kMaxTokens || (!a.starts && a.sequences != a.tokens))
        return BMMC_ERR_INVALID_ARG;
    if ((uintptr_t)a.starts % 4 || (uintptr_t)a.lengths % 4 || (uintptr_t)a.table % 4) return BMMC_ERR_MISALIGNED;
    const paged_cache_t* cache[2] = {&a.k_cache, &a.v_cache};
    const token_heads_t* from[2] = {&a.k, &a.v};
    for (int i = 0; i < 2; ++i) {
        if ((s = check_cache(*cache[i], a.pages, a.page_size, from[i]->heads, from[i]->dim, cache_es)) != BMMC_OK) return s;
        c.written[i] = cache_rows(*cache[i], a.pages, a.page_size, from[i]->heads, from[i]->dim, cache_es);
        p.page_stride[i] = cache[i]->page_stride * cache_es;
        p.slot_stride[i] = cache[i]->slot_stride * cache_es;
        c.cache_bits |= (uint64_t)(uintptr_t)cache[i]->data | (uint64_t)p.page_stride[i] | (uint64_t)p.slot_stride[i] |
                        (uint64_t)(cache[i]->head_stride * cache_es);
    }
    c.k = rows_of(a.k, a.tokens, es), c.v = rows_of(a.v, a.tokens, es);
    if (may_overlap(c.written[0], c.written[1]) && !caches_between(a, cache_es)) return BMMC_ERR_ALIAS;
    for (int i = 0; i < 2; ++i)
        if (may_overlap(c.written[i], c.k) || may_overlap(c.written[i], c.v)) return BMMC_ERR_ALIAS;
    if (with_q) {
        const Rows q = rows_of(a.q, a.tokens, es), to = rows_of(a.q_out, a.tokens, es);
        if (may_overlap(to, c.k) || may_overlap(to, c.v) || may_overlap(to, c.written[0]) || may_overlap(to, c.written[1]) ||
            may_overlap(q, c.written[0]) || may_overlap(q, c.written[1]) ||
            (!same_place(a.q, a.q_out, a.tokens) && may_overlap(q, to)))
            return BMMC_ERR_ALIAS;
        c.q = q, c.written[2] = to;
    } else {
        c.written[2] = Rows{nullptr, 0, 0, 0};
    }
    if ((s = set_turns(p, a.turns, false)) != BMMC_OK) return s;
    c.maps[0] = Rows{a.starts, 1, 0, (a.sequences + 1) * 4};
    c.maps[1] = Rows{a.lengths, 1, 0, a.sequences * 4};
    c.maps[2] = Rows{a.table, a.sequences, a.table_stride * 4, a.table_columns * 4};
    for (const Rows& w : c.written) {
        if (meets_turns(w, a.turns, a.tokens)) return BMMC_ERR_ALIAS;
        for (const Rows& m : c.maps)
            if (may_overlap(m, w)) return BMMC_ERR_ALIAS;
    }
    for (int i = 0; i < 2; ++i) {
        Heads& h = p.part[p.parts++];
        h = heads_of(*from[i], es, i == 0);
        h.dst = static_cast<char*>(cache[i]->data);
        h.dst_head = cache[i]->head_stride * cache_es;
        h.place = i + 1;
        c.in_bits |= address_bits(*from[i], es);
    }
    if (with_q) {
        Heads& h = p.part[p.parts++];
        h = heads_of(a.q, es, 1);
        h.dst = static_cast<char*>(a.q_out.data);
        h.dst_token = a.q_out.token_stride * es;
        h.dst_head = a.q_out.head_stride * es;
        c.q_bits = address_bits(a.q, es) | address_bits(a.q_out, es);
    }
    p.tokens = a.tokens;
    p.starts = a.starts;
    p.lengths = a.lengths;
    p.table = a.table;
    p.sequences = a.sequences;
    p.table_stride = a.table_stride;
    p.table_columns = a.table_columns;
    p.pages = a.pages;
    p.page_size = (int)a.page_size;
    c.dims[0] = (int)a.k.dim, c.dims[1] = (int)a.v.dim, c.dims[2] = (int)a.q.dim;
    return BMMC_OK;
}

}  // namespace bmmc
