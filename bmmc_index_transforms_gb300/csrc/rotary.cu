// Rotary positions with several axes, and the append of keys and values to a
// paged cache with the rotation applied on the way: rotary and paged_append
// (declared in include/bmmc.h).
//
// Pair i of a head is turned by the angle position[axis(i)] * freq[i]:
//   (a, b) -> (a cos - b sin, b cos + a sin),
// an orthogonal map, so its gradient is the turn by the opposite angle.
// The angle is the product rounded to 32 bits, which is the angle that a
// model sees whose positions are turned in 32 bits.
#include <cuda_runtime.h>

#include <cstdint>
#include <type_traits>

#include "../../include/bmmc.h"
#include "token_moves.hpp"
#include "token_words.cuh"

using namespace bmmc;

namespace {

constexpr int kThreads = 256;
constexpr int kMaxTokensPerBlock = 8;

// Heads of one kind (queries, keys, values): where they lie and where they
// go.  Strides in bytes.  place: 0 = the token's own place (dst_token apart),
// 1 / 2 = the token's place in the key / value cache.
struct Heads {
    const char* src;
    char* dst;
    int64_t src_token, src_head, dst_token, dst_head;
    int heads, dim, turned, place;
};

struct MoveParams {
    Heads part[3];
    int parts;
    int64_t tokens;
    int per_block;  // tokens of one block
    // rotation
    const void* positions;  // NULL: the token's place in its sequence
    int position_bytes, axes, pairs;
    int64_t axis_stride;
    const float* freq;
    const int* pair_axes;  // NULL: axis 0
    float sign;
    // places in the cache
    const int *starts, *lengths, *table;
    int64_t sequences, table_stride, table_columns, pages;
    int page_size;
    int64_t page_stride[2], slot_stride[2];  // of the key and the value cache, bytes
};

// The last sequence whose start is <= t, by a whole warp, 32 starts at a
// time; -1 if there is none.  Any starts, in order or not, give an index in
// range.
__device__ int64_t find_sequence(const int* starts, int64_t sequences, int64_t t, int lane) {
    int64_t lo = 0, n = sequences;  // the answer lies in [lo, lo + n) or is lo - 1
    while (n > 0) {
        const int64_t step = (n + 31) / 32;
        const int64_t i = lo + lane * step;
        const bool before = lane * step < n && starts[i] <= t;
        const int c = __popc(__ballot_sync(~0u, before));
        if (c == 0) return lo - 1;
        const int64_t at = lo + (c - 1) * step;  // starts[at] <= t
        if (step == 1) return at;
        n = min(step, lo + n - at) - 1;
        lo = at + 1;
    }
    return lo - 1;
}

// Written out, so that every variant rounds alike.
__device__ __forceinline__ float turned_first(float x, float y, float2 r) { return fmaf(x, r.x, -__fmul_rn(y, r.y)); }
__device__ __forceinline__ float turned_second(float x, float y, float2 r) { return fmaf(y, r.x, __fmul_rn(x, r.y)); }

template <class T, int W, bool ADJACENT>
__global__ void __launch_bounds__(kThreads) move_heads_kernel(const __grid_constant__ MoveParams p) {
    extern __shared__ float2 s_turn[];  // [per_block][pairs] cos, sin
    __shared__ int64_t s_place[2][kMaxTokensPerBlock];  // byte offsets in the caches, -1 = none
    __shared__ float s_position[kMaxTokensPerBlock];
    const int64_t t0 = (int64_t)blockIdx.x * p.per_block;
    const int nt = (int)min((int64_t)p.per_block, p.tokens - t0);
    const int tid = threadIdx.x, lane = tid & 31;
    if (p.page_size) {
        for (int i = tid >> 5; i < nt; i += kThreads / 32) {
            const int64_t t = t0 + i;
            int64_t b = t, first = t;
            if (p.starts) {
                b = find_sequence(p.starts, p.sequences, t, lane);
                if (b >= 0) {
                    first = p.starts[b];
                    if (t >= p.starts[b + 1]) b = -1;
                }
            } else if (t >= p.sequences) {
                b = -1;
            }
            int64_t at = 0, page = -1;
            if (b >= 0) {
                at = (int64_t)p.lengths[b] + (t - first);
                const int64_t column = at / p.page_size;
                if (at >= 0 && column < p.table_columns) page = p.table[b * p.table_stride + column];
            }
            if (lane == 0) {
                const bool in = page >= 0 && page < p.pages;
                const int64_t row = at % p.page_size;
                for (int c = 0; c < 2; ++c)
                    s_place[c][i] = in ? page * p.page_stride[c] + row * p.slot_stride[c] : -1;
                s_position[i] = (float)at;
            }
        }
        __syncthreads();
    }
    if (p.pairs) {
        for (int i = tid; i < nt * p.pairs; i += kThreads) {
            const int k = i / p.pairs, pair = i - k * p.pairs;
            const int axis = p.pair_axes ? p.pair_axes[pair] : 0;
            float at = 0.0f;  // an axis that is not there does not turn
            if (!p.positions) {
                if (axis == 0) at = s_position[k];
            } else if (axis >= 0 && axis < p.axes) {
                const int64_t j = axis * p.axis_stride + t0 + k;
                at = p.position_bytes == 4 ? (float)static_cast<const int32_t*>(p.positions)[j]
                                           : (float)static_cast<const int64_t*>(p.positions)[j];
            }
            float s, c;
            sincosf(at * p.freq[pair], &s, &c);
            s_turn[i] = make_float2(c, p.sign * s);
        }
        __syncthreads();
    }
    for (int q = 0; q < p.parts; ++q) {
        const Heads h = p.part[q];
        const int pairs = h.turned ? p.pairs : 0;
        // items of a head: first those that turn (W pairs in halves, or W / 2
        // pairs side by side, at least one), then W elements each that are copied
        const int turning = !ADJACENT ? pairs / W : W > 1 ? 2 * pairs / W : pairs;
        const int per_head = turning + (h.dim - 2 * pairs) / W;
        for (int idx = tid; idx < nt * h.heads * per_head; idx += kThreads) {
            const int k = idx / (h.heads * per_head), in = idx - k * (h.heads * per_head);
            const int head = in / per_head, j = in - head * per_head;
            int64_t to = (t0 + k) * h.dst_token;
            if (h.place) {
                to = s_place[h.place - 1][k];
                if (to < 0) continue;
            }
            const char* src = h.src + (t0 + k) * h.src_token + head * h.src_head;
            char* dst = h.dst + to + head * h.dst_head;
            Pack<T, W> a, b;
            if (j >= turning) {
                const int64_t at = (int64_t)(2 * pairs + (j - turning) * W) * sizeof(T);
                a.load(src + at);
                a.store(dst + at);
            } else if (ADJACENT && W > 1) {
                const int64_t at = (int64_t)j * sizeof(a);
                a.load(src + at);
#pragma unroll
                for (int i = 0; i + 1 < W; i += 2) {
                    const float2 r = s_turn[k * p.pairs + (j * W + i) / 2];
                    const float x = a.get(i), y = a.get(i + 1);
                    a.set(i, turned_first(x, y, r));
                    a.set(i + 1, turned_second(x, y, r));
                }
                a.store(dst + at);
            } else {
                const int64_t at = (int64_t)(ADJACENT ? 2 * j : j * W) * sizeof(T);
                const int64_t half = (int64_t)(ADJACENT ? 1 : pairs) * sizeof(T);
                a.load(src + at);
                b.load(src + at + half);
#pragma unroll
                for (int i = 0; i < W; ++i) {
                    const float2 r = s_turn[k * p.pairs + j * W + i];
                    const float x = a.get(i), y = b.get(i);
                    a.set(i, turned_first(x, y, r));
                    b.set(i, turned_second(x, y, r));
                }
                a.store(dst + at);
                b.store(dst + at + half);
            }
        }
    }
}

// Tokens of one block: enough items for every thread, while there are blocks
// enough for the machine.
int tokens_per_block(const MoveParams& p, int W) {
    int64_t items = 0;
    for (int q = 0; q < p.parts; ++q) items += (int64_t)p.part[q].heads * p.part[q].dim / (2 * W);
    int n = 1;
    while (n < kMaxTokensPerBlock && n * items < 2 * kThreads && p.tokens / (2 * n) >= 152 * 4 &&
           2 * n * p.pairs * sizeof(float2) <= 32 * 1024)
        n *= 2;
    return n;
}

template <class T, int W>
bmmc_status launch_width(MoveParams& p, bool adjacent, cudaStream_t st) {
    p.per_block = tokens_per_block(p, W);
    const unsigned grid = (unsigned)((p.tokens + p.per_block - 1) / p.per_block);
    const size_t smem = (size_t)p.per_block * p.pairs * sizeof(float2);
    if (adjacent) move_heads_kernel<T, W, true><<<grid, kThreads, smem, st>>>(p);
    else move_heads_kernel<T, W, false><<<grid, kThreads, smem, st>>>(p);
    return launched();
}

template <class T>
bmmc_status launch_type(MoveParams& p, bool adjacent, int bytes, cudaStream_t st) {
    constexpr int es = sizeof(T);
    switch (bytes) {
        case 16: return launch_width<T, 16 / es>(p, adjacent, st);
        case 8: return launch_width<T, 8 / es>(p, adjacent, st);
        case 4: return launch_width<T, 4 / es>(p, adjacent, st);
    }
    return launch_width<T, 1>(p, adjacent, st);
}

bmmc_status launch(MoveParams& p, int type, bool adjacent, int bytes, cudaStream_t st) {
    switch (type) {
        case BMMC_F32: return launch_type<float>(p, adjacent, bytes, st);
        case BMMC_F16: return launch_type<__half>(p, adjacent, bytes, st);
    }
    return launch_type<__nv_bfloat16>(p, adjacent, bytes, st);
}

bool bad_stride(int64_t s) { return s < 0 || s > kMaxStride; }

bmmc_status check_heads(const token_heads_t& x, int es) {
    if (!x.data || x.heads < 1 || x.dim < 1 || x.dim > ROTARY_MAX_DIM || x.heads > (1 << 24) / x.dim ||
        bad_stride(x.token_stride) || bad_stride(x.head_stride))
        return BMMC_ERR_INVALID_ARG;
    return (uintptr_t)x.data % es ? BMMC_ERR_MISALIGNED : BMMC_OK;
}

// The array as rows along its longer stride.
Rows rows_of(const token_heads_t& x, int64_t tokens, int es) {
    const bool by_token = x.heads < 2 || x.token_stride >= x.head_stride;
    const int64_t n = by_token ? tokens : x.heads, s = by_token ? x.token_stride : x.head_stride;
    const int64_t m = by_token ? x.heads : tokens, u = by_token ? x.head_stride : x.token_stride;
    return Rows{x.data, n, s * es, ((m - 1) * u + x.dim) * es};
}

bool same_place(const token_heads_t& a, const token_heads_t& b, int64_t tokens) {
    return a.data == b.data && (tokens < 2 || a.token_stride == b.token_stride) &&
           (a.heads < 2 || a.head_stride == b.head_stride);
}

bool writable(const token_heads_t& x, int64_t tokens) {
    const int64_t sizes[2] = {tokens, x.heads}, strides[2] = {x.token_stride, x.head_stride};
    return one_to_one(x.dim, sizes, strides);
}

uint64_t address_bits(const token_heads_t& x, int es) {
    return (uint64_t)(uintptr_t)x.data | (uint64_t)(x.token_stride * es) | (uint64_t)(x.head_stride * es) |
           (uint64_t)(x.dim * es);
}

// The rotation's arguments, checked and put into p; tokens > 0.
bmmc_status set_turns(MoveParams& p, const rotary_turns_t& r, int64_t tokens, bool need_positions) {
    p.pairs = 0;
    if (r.flags & ~(int64_t)(ROTARY_ADJACENT | ROTARY_INVERSE)) return BMMC_ERR_INVALID_ARG;
    if (!r.inv_freq) return r.pairs || r.positions || r.pair_axes ? BMMC_ERR_INVALID_ARG : BMMC_OK;
    if (r.pairs < 1 || r.pairs > ROTARY_MAX_DIM / 2 || (need_positions && !r.positions)) return BMMC_ERR_INVALID_ARG;
    if ((uintptr_t)r.inv_freq % 4 || (uintptr_t)r.pair_axes % 4) return BMMC_ERR_MISALIGNED;
    if (r.positions) {
        if (r.position_bytes != 4 && r.position_bytes != 8) return BMMC_ERR_UNSUPPORTED_ELEM;
        if (r.axes < 1 || r.axes > r.pairs || bad_stride(r.axis_stride)) return BMMC_ERR_INVALID_ARG;
        if ((uintptr_t)r.positions % r.position_bytes) return BMMC_ERR_MISALIGNED;
        p.position_bytes = (int)r.position_bytes;
        p.axes = (int)r.axes;
        p.axis_stride = r.axis_stride;
    }
    p.positions = r.positions;
    p.pairs = (int)r.pairs;
    p.freq = r.inv_freq;
    p.pair_axes = r.pair_axes;
    p.sign = r.flags & ROTARY_INVERSE ? -1.0f : 1.0f;
    return all_reachable({r.inv_freq, r.pair_axes, r.positions});
}

// The bits that a word's size has to divide on account of the pairs.
uint64_t pair_bits(const rotary_turns_t& r, int es) {
    return (uint64_t)(r.flags & ROTARY_ADJACENT ? 2 * r.pairs : r.pairs) * es;
}

Heads heads_of(const token_heads_t& x, int es, int turned) {
    Heads h{};
    h.src = static_cast<const char*>(x.data);
    h.src_token = x.token_stride * es;
    h.src_head = x.head_stride * es;
    h.heads = (int)x.heads;
    h.dim = (int)x.dim;
    h.turned = turned;
    return h;
}

}  // namespace

extern "C" {

bmmc_status rotary(const rotary_args_t* a, void* stream) {
    if (!a || a->tokens < 0 || a->tokens > kMaxTokens) return BMMC_ERR_INVALID_ARG;
    const int es = dtype_bytes((int)a->type);
    if (!es) return BMMC_ERR_UNSUPPORTED_ELEM;
    if (!a->tokens) return BMMC_OK;
    bmmc_status s = check_heads(a->x, es);
    if (s == BMMC_OK) s = check_heads(a->out, es);
    if (s != BMMC_OK) return s;
    if (a->x.heads != a->out.heads || a->x.dim != a->out.dim || !a->turns.inv_freq || 2 * a->turns.pairs > a->x.dim ||
        !writable(a->out, a->tokens))
        return BMMC_ERR_INVALID_ARG;
    if (!same_place(a->x, a->out, a->tokens) && may_overlap(rows_of(a->x, a->tokens, es), rows_of(a->out, a->tokens, es)))
        return BMMC_ERR_ALIAS;
    MoveParams p{};
    if ((s = set_turns(p, a->turns, a->tokens, true)) != BMMC_OK) return s;
    if ((s = all_reachable({a->x.data, a->out.data})) != BMMC_OK) return s;
    p.parts = 1;
    p.part[0] = heads_of(a->x, es, 1);
    p.part[0].dst = static_cast<char*>(a->out.data);
    p.part[0].dst_token = a->out.token_stride * es;
    p.part[0].dst_head = a->out.head_stride * es;
    p.tokens = a->tokens;
    const int wb = word_bytes(es, {address_bits(a->x, es), address_bits(a->out, es), pair_bits(a->turns, es)});
    return launch(p, (int)a->type, a->turns.flags & ROTARY_ADJACENT, wb, static_cast<cudaStream_t>(stream));
}

bmmc_status paged_append(const paged_append_args_t* a, void* stream) {
    if (!a || a->tokens < 0 || a->tokens > kMaxTokens) return BMMC_ERR_INVALID_ARG;
    const int es = dtype_bytes((int)a->type);
    if (!es) return BMMC_ERR_UNSUPPORTED_ELEM;
    if (!a->tokens) return BMMC_OK;
    const bool with_q = a->q.data || a->q_out.data;
    bmmc_status s = check_heads(a->k, es);
    if (s == BMMC_OK) s = check_heads(a->v, es);
    if (s == BMMC_OK && with_q) s = check_heads(a->q, es);
    if (s == BMMC_OK && with_q) s = check_heads(a->q_out, es);
    if (s != BMMC_OK) return s;
    const int64_t turned = 2 * a->turns.pairs;
    if (a->k.heads != a->v.heads || turned > a->k.dim || (a->turns.flags & ROTARY_INVERSE)) return BMMC_ERR_INVALID_ARG;
    if (with_q && (a->q.heads != a->q_out.heads || a->q.dim != a->q_out.dim || turned > a->q.dim ||
                   !writable(a->q_out, a->tokens)))
        return BMMC_ERR_INVALID_ARG;
    if (a->sequences < 0 || a->sequences > kMaxTokens || (a->sequences && !a->lengths) ||
        (a->sequences && a->table_columns && !a->table) || a->table_columns < 0 || a->table_columns > kMaxTokens || bad_stride(a->table_stride) || a->pages < 0 || a->pages > kMaxTokens ||
        a->page_size < 1 || a->page_size > kMaxTokens || (!a->starts && a->sequences != a->tokens))
        return BMMC_ERR_INVALID_ARG;
    if ((uintptr_t)a->starts % 4 || (uintptr_t)a->lengths % 4 || (uintptr_t)a->table % 4) return BMMC_ERR_MISALIGNED;
    const paged_cache_t* cache[2] = {&a->k_cache, &a->v_cache};
    const token_heads_t* from[2] = {&a->k, &a->v};
    Rows cache_rows[2];
    MoveParams p{};
    uint64_t bits = 0;
    for (int c = 0; c < 2; ++c) {
        const paged_cache_t& m = *cache[c];
        if ((!m.data && a->pages) || bad_stride(m.page_stride) || bad_stride(m.slot_stride) || bad_stride(m.head_stride))
            return BMMC_ERR_INVALID_ARG;
        if ((uintptr_t)m.data % es) return BMMC_ERR_MISALIGNED;
        const int64_t sizes[3] = {a->pages, a->page_size, from[c]->heads};
        const int64_t strides[3] = {m.page_stride, m.slot_stride, m.head_stride};
        if (!one_to_one(from[c]->dim, sizes, strides)) return BMMC_ERR_INVALID_ARG;
        cache_rows[c] = Rows{m.data, a->pages, m.page_stride * es,
                             ((a->page_size - 1) * m.slot_stride + (from[c]->heads - 1) * m.head_stride + from[c]->dim) * es};
        p.page_stride[c] = m.page_stride * es;
        p.slot_stride[c] = m.slot_stride * es;
        bits |= (uint64_t)(uintptr_t)m.data | (uint64_t)p.page_stride[c] | (uint64_t)p.slot_stride[c] |
                (uint64_t)(m.head_stride * es);
    }
    const Rows k = rows_of(a->k, a->tokens, es), v = rows_of(a->v, a->tokens, es);
    if (may_overlap(cache_rows[0], cache_rows[1])) return BMMC_ERR_ALIAS;
    for (const Rows& c : cache_rows)
        if (may_overlap(c, k) || may_overlap(c, v)) return BMMC_ERR_ALIAS;
    if (with_q) {
        const Rows q = rows_of(a->q, a->tokens, es), to = rows_of(a->q_out, a->tokens, es);
        if (may_overlap(to, k) || may_overlap(to, v) || may_overlap(to, cache_rows[0]) || may_overlap(to, cache_rows[1]) ||
            may_overlap(q, cache_rows[0]) || may_overlap(q, cache_rows[1]) ||
            (!same_place(a->q, a->q_out, a->tokens) && may_overlap(q, to)))
            return BMMC_ERR_ALIAS;
    }
    if ((s = set_turns(p, a->turns, a->tokens, false)) != BMMC_OK) return s;
    if ((s = all_reachable({a->k.data, a->v.data, a->q.data, a->q_out.data, a->k_cache.data, a->v_cache.data, a->starts,
                            a->lengths, a->table})) != BMMC_OK)
        return s;
    for (int c = 0; c < 2; ++c) {
        Heads& h = p.part[p.parts++];
        h = heads_of(*from[c], es, c == 0);
        h.dst = static_cast<char*>(cache[c]->data);
        h.dst_head = cache[c]->head_stride * es;
        h.place = c + 1;
        bits |= address_bits(*from[c], es);
    }
    if (with_q) {
        Heads& h = p.part[p.parts++];
        h = heads_of(a->q, es, 1);
        h.dst = static_cast<char*>(a->q_out.data);
        h.dst_token = a->q_out.token_stride * es;
        h.dst_head = a->q_out.head_stride * es;
        bits |= address_bits(a->q, es) | address_bits(a->q_out, es);
    }
    p.tokens = a->tokens;
    p.starts = a->starts;
    p.lengths = a->lengths;
    p.table = a->table;
    p.sequences = a->sequences;
    p.table_stride = a->table_stride;
    p.table_columns = a->table_columns;
    p.pages = a->pages;
    p.page_size = (int)a->page_size;
    const int wb = word_bytes(es, {bits, pair_bits(a->turns, es)});
    return launch(p, (int)a->type, a->turns.flags & ROTARY_ADJACENT, wb, static_cast<cudaStream_t>(stream));
}

}  // extern "C"
