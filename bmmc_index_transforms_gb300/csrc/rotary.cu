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

#include <algorithm>
#include <cstdint>
#include <type_traits>

#include "../../include/bmmc.h"
#define BMMC_CHK_FILE 7  // site tag of this file in bounds-checked builds
#include "bounds.cuh"
#include "paged_places.cuh"
#include "token_moves.hpp"
#include "token_words.cuh"

using namespace bmmc;

namespace {

constexpr int kThreads = 128;           // threads of a block, at most (one token may take 256)
constexpr int kMostThreads = 256;
constexpr int kHeadsAtOnce = 2;         // heads whose words a thread has in flight

// A block takes some tokens, a group of threads each.  Its threads find the
// tokens' places and put the cosines and sines of their pairs into shared
// memory, once for all heads; then a thread keeps those of its word of a head
// in registers and walks over the heads, two at a time.
//
// Bound by HBM where there are tokens enough: 32768 tokens x 32 heads x 128 bf16
// 79.7 us = 6740 GB/s; 16001 tokens' queries, keys and values (32 + 8 + 8 heads)
// into pages 64.2 us (floor 58.9; 64001 tokens 228.5, at the copy rate): what is left
// is the start of a block, whose loads of starts, lengths and table follow one
// another, which is why positions, frequencies and, to L2, the heads are sent
// for first (without that 76 us).  12 heads of 96 f32 with adjacent pairs, 10007
// tokens: 16.7 us (13.8).  Shapes tried there: one head at a time 71.5 us, four
// 71-95; 6 blocks of 256 threads on an SM instead of 4, whose registers then spill,
// 88; blocks of 256 threads 70.8, of 128 68.1.  256 single tokens: 4.3 us, the
// chain lengths - table - sine - store and a launch.
//
// One head a token has a sine and a cosine for every pair of elements: 65536 x 1
// x 64 15.1 us for 2.5 us of bytes, 4 heads 19.3 for 9.9.  Not bound by their
// instructions: the issue slots are 51 % in use, and for each issue 2.3 warps
// wait for a load, 2.2 for shared memory or a special function, 2.0 for a result
// and 1.9 at the barrier.  A thread has two turns on their way at a time (kAhead),
// the rest of its eight follow one after another.
template <class T, int W, bool ADJACENT>
__global__ void __launch_bounds__(kMostThreads, 4)
    move_heads_kernel(const __grid_constant__ MoveParams p BMMC_SPANS_PARAM) {
    extern __shared__ float2 s_turn[];  // [tokens of the block][pairs] cos, sin
    __shared__ int64_t s_place[2][kMaxTokensPerBlock];  // byte offsets in the caches, -1 = none
    __shared__ float s_position[kMaxTokensPerBlock];
    BMMC_SPANS_ENTER(s_turn, chk::dyn_smem_bytes(), s_place, sizeof(s_place), s_position, sizeof(s_position));
    const int tid = threadIdx.x, per_block = blockDim.x >> p.group_log2;
    const Slots<float2> turns(s_turn, per_block * p.pairs);
    const Slots<int64_t> places(&s_place[0][0], 2 * kMaxTokensPerBlock);
    const Slots<float> place_numbers(s_position, kMaxTokensPerBlock);
    const int64_t t0 = (int64_t)blockIdx.x * per_block;
    const int nt = (int)min((int64_t)per_block, p.tokens - t0);
    // a block of a small call takes one part only
    const int first_part = gridDim.y > 1 ? blockIdx.y : 0, last_part = gridDim.y > 1 ? first_part + 1 : p.parts;
    begin_block(p, t0, nt, first_part, last_part, turns, places, place_numbers);
    const int k = tid >> p.group_log2, in = tid & ((1 << p.group_log2) - 1);
    if (k >= nt) return;
    for (int q = first_part; q < last_part; ++q) {
        const Heads& h = p.part[q];
        const int down = (in * h.magic) >> 16, step = (1 << p.group_log2) / h.across;
        if (down >= step) continue;
        int64_t to = (t0 + k) * h.dst_token;
        if (h.place) {
            to = places.get((h.place - 1) * kMaxTokensPerBlock + k);
            if (to < 0) continue;
        }
        const char* const src = h.src + (t0 + k) * h.src_token;
        char* const dst = h.dst + to;
        const Slots<float2> turn = turns.part(k * p.pairs, p.pairs);
        for (int j = in - down * h.across; j < h.items; j += h.across) {
            const bool turned = j < h.turning;
            // where the word lies, and its other half
            int64_t at, half = 0;
            if (ADJACENT) {
                at = W > 1 ? (int64_t)j * W : turned ? 2 * j : j + h.turning;
                half = 1;
            } else {
                at = turned ? (int64_t)j * W : (int64_t)(j + h.turning) * W;
                half = p.pairs;
            }
            at *= sizeof(T), half *= sizeof(T);
            constexpr bool kTwo = !ADJACENT || W == 1;  // an item has two words
            constexpr int kTurns = kTwo ? W : W / 2;
            float2 r[kTurns];
            if (turned)
#pragma unroll
                for (int i = 0; i < kTurns; ++i)
                    r[i] = turn.get(j * kTurns + i);
            for (int head = down; head < h.heads; head += kHeadsAtOnce * step) {
                Pack<T, W> a[kHeadsAtOnce], b[kHeadsAtOnce];
#pragma unroll
                for (int u = 0; u < kHeadsAtOnce; ++u)
                    if (u == 0 || head + u * step < h.heads) {
                        const char* from = src + (head + u * step) * h.src_head + at;
                        if (BMMC_RD_OK(from, sizeof(a[u]))) a[u].load(from);
                        if (kTwo && turned && BMMC_RD_OK(from + half, sizeof(b[u]))) b[u].load(from + half);
                    }
#pragma unroll
                for (int u = 0; u < kHeadsAtOnce; ++u)
                    if (u == 0 || head + u * step < h.heads) {
                        char* out = dst + (head + u * step) * h.dst_head + at;
                        if (turned) {
                            float x[W], y[W];
                            if constexpr (kTwo) {
#pragma unroll
                                for (int i = 0; i < W; ++i) {
                                    x[i] = turned_first(a[u].get(i), b[u].get(i), r[i]);
                                    y[i] = turned_second(a[u].get(i), b[u].get(i), r[i]);
                                }
                                b[u].set(y);
                                if (BMMC_WR_OK(out + half, sizeof(b[u]))) b[u].store(out + half);
                            } else {
#pragma unroll
                                for (int i = 0; i < W; i += 2) {
                                    x[i] = turned_first(a[u].get(i), a[u].get(i + 1), r[i / 2]);
                                    x[i + 1] = turned_second(a[u].get(i), a[u].get(i + 1), r[i / 2]);
                                }
                            }
                            a[u].set(x);
                        }
                        if (BMMC_WR_OK(out, sizeof(a[u]))) a[u].store(out);
                    }
            }
        }
    }
}

constexpr int kRowThreads = 128;
constexpr int kRowBytes = 2048;  // of a warp's rows in shared memory
constexpr int kRowBatch = 32;    // most rows of a warp at a time

// The same for heads whose pairs do not lie in the words that their rows allow
// (an odd number of pairs in halves of a 16-bit type): a warp brings some rows
// (heads of tokens) into shared memory in words, turns their pairs there by
// element, and writes them back in words.
//
// 16384 tokens x 16 heads of 128 bf16 (floor 20.1 us): 37 pairs in halves 33.5 us,
// by element from memory 108; 36 pairs 30.6, in words of 8 bytes 40.5; 16001
// tokens appended with 37 pairs 92 us, by element 290.  Rows of 4-byte words (heads
// of 66) are no faster this way (49 and 47 us) and keep the other.  2 KB of rows a
// warp in flight; with 1 KB the append takes 98, with 8 tokens a block instead of 4
// 108.
template <class T, class Word>
__global__ void __launch_bounds__(kRowThreads)
    move_rows_kernel(const __grid_constant__ MoveParams p BMMC_SPANS_PARAM) {
    constexpr int kWarps = kRowThreads / 32;
    extern __shared__ float2 s_turn[];  // [tokens of the block][pairs] cos, sin
    __shared__ int64_t s_place[2][kMaxTokensPerBlock];
    __shared__ float s_position[kMaxTokensPerBlock];
    __shared__ struct {
        __align__(16) char data[kRowBytes];
        const char* src[kRowBatch];
        char* dst[kRowBatch];  // NULL: not written
        int turns[kRowBatch];  // where its token's turns start
    } s_rows[kWarps];
    BMMC_SPANS_ENTER(s_turn, chk::dyn_smem_bytes(), s_place, sizeof(s_place), s_position, sizeof(s_position), s_rows,
                     sizeof(s_rows));
    const int tid = threadIdx.x, lane = tid & 31, per_block = blockDim.x >> p.group_log2;
    const Slots<float2> turns(s_turn, per_block * p.pairs);
    const Slots<int64_t> places(&s_place[0][0], 2 * kMaxTokensPerBlock);
    const Slots<float> place_numbers(s_position, kMaxTokensPerBlock);
    const int64_t t0 = (int64_t)blockIdx.x * per_block;
    const int nt = (int)min((int64_t)per_block, p.tokens - t0);
    const int first_part = gridDim.y > 1 ? blockIdx.y : 0, last_part = gridDim.y > 1 ? first_part + 1 : p.parts;
    begin_block(p, t0, nt, first_part, last_part, turns, places, place_numbers);
    auto& mine = s_rows[tid >> 5];
    const Slots<Word> words(reinterpret_cast<Word*>(mine.data), kRowBytes / (int)sizeof(Word));
    const Slots<T> elements(reinterpret_cast<T*>(mine.data), kRowBytes / (int)sizeof(T));
    const Slots<const char*> src(mine.src, kRowBatch);
    const Slots<char*> dst(mine.dst, kRowBatch);
    const Slots<int> turns_of(mine.turns, kRowBatch);
    for (int q = first_part; q < last_part; ++q) {
        const Heads& h = p.part[q];
        const int row_elements = h.words * (int)(sizeof(Word) / sizeof(T));
        for (int r0 = (tid >> 5) * h.batch; r0 < nt * h.heads; r0 += kWarps * h.batch) {
            const int rows = min(h.batch, nt * h.heads - r0);
            if (lane < rows) {
                const int k = (r0 + lane) / h.heads, head = r0 + lane - k * h.heads;
                const int64_t to = h.place ? places.get((h.place - 1) * kMaxTokensPerBlock + k) : (t0 + k) * h.dst_token;
                src.set(lane, h.src + (t0 + k) * h.src_token + head * h.src_head);
                dst.set(lane, to < 0 ? nullptr : h.dst + to + head * h.dst_head);
                turns_of.set(lane, k * p.pairs);
            }
            __syncwarp();
#pragma unroll 4
            for (int x = lane; x < rows * h.words; x += 32) {
                const int row = quotient(x, h.words, h.words_magic);
                const char* const from = src.get(row) + (x - row * h.words) * sizeof(Word);
                if (BMMC_RD_OK(from, sizeof(Word))) words.set(x, *reinterpret_cast<const Word*>(from));
            }
            __syncwarp();
            if (h.turned) {
#pragma unroll 2
                for (int x = lane; x < rows * p.pairs; x += 32) {
                    const int row = quotient(x, p.pairs, p.pairs_magic), i = x - row * p.pairs;
                    const int a = row * row_elements + (p.adjacent ? 2 * i : i), b = a + (p.adjacent ? 1 : p.pairs);
                    const float2 r = turns.get(turns_of.get(row) + i);
                    const float u = to_f32(elements.get(a)), v = to_f32(elements.get(b));
                    elements.set(a, from_f32<T>(turned_first(u, v, r)));
                    elements.set(b, from_f32<T>(turned_second(u, v, r)));
                }
                __syncwarp();
            }
#pragma unroll 4
            for (int x = lane; x < rows * h.words; x += 32) {
                const int row = quotient(x, h.words, h.words_magic);
                char* const row_to = dst.get(row);
                char* const to = row_to + (x - row * h.words) * sizeof(Word);
                if (row_to && BMMC_WR_OK(to, sizeof(Word))) *reinterpret_cast<Word*>(to) = words.get(x);
            }
            __syncwarp();
        }
    }
}

// Threads of a token: as many as the words of its largest part in a small
// call (so that all its loads are in flight at once), a quarter of them in one
// that fills the machine (each thread uses its cosines and sines for several
// heads: append of 16001 tokens 70.8 us, with half 94, with an eighth 73.9).
// *split: the parts go to blocks of their own, where all of these still run
// at once.  Returns the block's threads.
int deal_out(MoveParams& p, const int (&dims)[3], int W, int es, bool adjacent, bool* split) {
    int64_t most = std::max(1, p.pairs / kAhead);  // (at least as many as find their turns at once)
    for (int q = 0; q < p.parts; ++q) {
        Heads& h = p.part[q];
        const int pairs = h.turned ? p.pairs : 0;
        h.turning = !adjacent ? pairs / W : W > 1 ? 2 * pairs / W : pairs;
        h.items = h.turning + (dims[q] - 2 * pairs) / W;
        most = std::max(most, (int64_t)h.heads * h.items);
    }
    int full = 2, group;
    while (full < 8 && (1 << full) < most) ++full;
    const bool small = (p.tokens << full) <= kSms * 1024;
    group = small ? std::min(full, 7) : most > 1024 ? full : std::max(2, full - 2);
    int threads = small ? std::max(64, 1 << group) : std::max(kThreads, 1 << group);
    while ((threads >> group) > kMaxTokensPerBlock) ++group;
    while ((threads >> group) > 1 && (threads >> group) * p.pairs * sizeof(float2) > 32 * 1024) ++group;
    p.group_log2 = group;
    for (int q = 0; q < p.parts; ++q) {
        Heads& h = p.part[q];
        h.across = std::min(h.items, 1 << group);
        h.magic = (65536 + h.across - 1) / h.across;
        const bool dense = p.device && W * es == 16 && (h.heads < 2 || h.src_head == (int64_t)dims[q] * es);
        h.ahead = dense ? std::min((unsigned)(h.heads * dims[q] * es), 65536u) : 0u;
    }
    *split = p.parts > 1 && p.tokens / (threads >> group) * p.parts * threads <= kSms * 1024;
    return threads;
}

// Staged rows: words of `bytes`; tokens of a block by the size of the call.
template <class T, class Word>
bmmc_status launch_rows(MoveParams& p, const int (&dims)[3], bool adjacent, const chk::Spans& spans, cudaStream_t st) {
    (void)spans;
    p.adjacent = adjacent;
    int per_block = p.tokens >= kSms * 32 ? 4 : 1;
    while (per_block > 1 && per_block * p.pairs * sizeof(float2) > 32 * 1024) per_block >>= 1;
    p.group_log2 = per_block == 4 ? 5 : per_block == 2 ? 6 : 7;
    for (int q = 0; q < p.parts; ++q) {
        Heads& h = p.part[q];
        const int row_bytes = dims[q] * (int)sizeof(T);
        h.words = row_bytes / (int)sizeof(Word);
        h.words_magic = magic_of(h.words);
        // no more rows a warp than its share
        h.batch = std::min({kRowBytes / row_bytes, kRowBatch, (per_block * h.heads + 3) / 4});
        const bool dense = p.device && sizeof(Word) == 16 && (h.heads < 2 || h.src_head == (int64_t)row_bytes);
        h.ahead = dense ? std::min((unsigned)(h.heads * row_bytes), 65536u) : 0u;
    }
    const bool split = p.parts > 1 && p.tokens * p.parts <= kSms * 8;
    const dim3 grid((unsigned)((p.tokens + per_block - 1) / per_block), split ? p.parts : 1);
    return launch(move_rows_kernel<T, Word>, grid, dim3(kRowThreads), (size_t)per_block * p.pairs * sizeof(float2), st,
                  nullptr, p BMMC_SPANS_ARG(spans));
}

template <class T, int W>
bmmc_status launch_width(MoveParams& p, const int (&dims)[3], bool adjacent, const chk::Spans& spans, cudaStream_t st) {
    (void)spans;
    bool split;
    const int threads = deal_out(p, dims, W, sizeof(T), adjacent, &split);
    const int per_block = threads >> p.group_log2;
    const dim3 grid((unsigned)((p.tokens + per_block - 1) / per_block), split ? p.parts : 1);
    const size_t smem = (size_t)per_block * p.pairs * sizeof(float2);
    const auto kernel = adjacent ? move_heads_kernel<T, W, true> : move_heads_kernel<T, W, false>;
    return launch(kernel, grid, dim3(threads), smem, st, nullptr, p BMMC_SPANS_ARG(spans));
}

template <class T>
bmmc_status launch_type(MoveParams& p, const int (&dims)[3], bool adjacent, int bytes, int row_word,
                        const chk::Spans& spans, cudaStream_t st) {
    constexpr int es = sizeof(T);
    bool staged = row_word >= 8 && row_word > bytes;
    for (int q = 0; q < p.parts; ++q) staged = staged && dims[q] * es <= kRowBytes;
    if (staged)
        return row_word == 16 ? launch_rows<T, uint4>(p, dims, adjacent, spans, st)
                              : launch_rows<T, uint2>(p, dims, adjacent, spans, st);
    switch (bytes) {
        case 16: return launch_width<T, 16 / es>(p, dims, adjacent, spans, st);
        case 8: return launch_width<T, 8 / es>(p, dims, adjacent, spans, st);
        case 4: return launch_width<T, 4 / es>(p, dims, adjacent, spans, st);
    }
    return launch_width<T, 1>(p, dims, adjacent, spans, st);
}

bmmc_status launch_moves(MoveParams& p, const int (&dims)[3], int type, bool adjacent, int bytes, int row_word,
                         const chk::Spans& spans, cudaStream_t st) {
    switch (type) {
        case BMMC_F32: return launch_type<float>(p, dims, adjacent, bytes, row_word, spans, st);
        case BMMC_F16: return launch_type<__half>(p, dims, adjacent, bytes, row_word, spans, st);
    }
    return launch_type<__nv_bfloat16>(p, dims, adjacent, bytes, row_word, spans, st);
}

}  // namespace

extern "C" {

bmmc_status rotary(const rotary_args_t* a, void* stream) {
    if (!a || a->tokens < 0 || a->tokens > kMaxTokens) return BMMC_ERR_INVALID_ARG;
    int type = a->type < 0 || a->type > 0xfff ? -1 : (int)a->type;
    const bool device = device_pointers(type);
    const int es = dtype_bytes(type);
    if (!es) return BMMC_ERR_UNSUPPORTED_ELEM;
    if (!a->tokens) return BMMC_OK;
    bmmc_status s = check_heads(a->x, a->tokens, es);
    if (s == BMMC_OK) s = check_heads(a->out, a->tokens, es);
    if (s != BMMC_OK) return s;
    if (a->x.heads != a->out.heads || a->x.dim != a->out.dim || !a->turns.inv_freq || 2 * a->turns.pairs > a->x.dim ||
        !writable(a->out, a->tokens))
        return BMMC_ERR_INVALID_ARG;
    if (!same_place(a->x, a->out, a->tokens) && may_overlap(rows_of(a->x, a->tokens, es), rows_of(a->out, a->tokens, es)))
        return BMMC_ERR_ALIAS;
    MoveParams p{};
    if ((s = set_turns(p, a->turns, true)) != BMMC_OK) return s;
    if (meets_turns(rows_of(a->out, a->tokens, es), a->turns, a->tokens)) return BMMC_ERR_ALIAS;
    if ((s = all_reachable(device, {a->x.data, a->out.data, a->turns.inv_freq, a->turns.pair_axes, a->turns.positions})) !=
        BMMC_OK)
        return s;
    p.device = device;
    p.parts = 1;
    p.part[0] = heads_of(a->x, es, 1);
    p.part[0].dst = static_cast<char*>(a->out.data);
    p.part[0].dst_token = a->out.token_stride * es;
    p.part[0].dst_head = a->out.head_stride * es;
    p.tokens = a->tokens;
    const int dims[3] = {(int)a->x.dim};
    const chk::Spans spans = spans_of({rows_of(a->x, a->tokens, es), turn_rows(a->turns, a->tokens, 0),
                                       turn_rows(a->turns, a->tokens, 1), turn_rows(a->turns, a->tokens, 2)},
                                      {rows_of(a->out, a->tokens, es)});
    const uint64_t bits = address_bits(a->x, es) | address_bits(a->out, es);
    const int wb = word_bytes(es, {bits, pair_bits(a->turns, es)});
    return launch_moves(p, dims, type, a->turns.flags & ROTARY_ADJACENT, wb, word_bytes(es, {bits}), spans,
                        static_cast<cudaStream_t>(stream));
}

bmmc_status paged_append(const paged_append_args_t* a, void* stream) {
    if (!a || a->tokens < 0 || a->tokens > kMaxTokens) return BMMC_ERR_INVALID_ARG;
    int type = a->type < 0 || a->type > 0xfff ? -1 : (int)a->type;
    const bool device = device_pointers(type);
    const int es = dtype_bytes(type);
    if (!es) return BMMC_ERR_UNSUPPORTED_ELEM;
    if (!a->tokens) return BMMC_OK;
    AppendCall c;
    bmmc_status s = read_append(*a, es, es, device, c);
    if (s == BMMC_OK) s = append_reachable(*a, device);
    if (s != BMMC_OK) return s;
    const uint64_t bits = c.in_bits | c.cache_bits | c.q_bits;
    const chk::Spans spans = spans_of({c.k, c.v, c.q, turn_rows(a->turns, a->tokens, 0), turn_rows(a->turns, a->tokens, 1),
                                       turn_rows(a->turns, a->tokens, 2), c.maps[0], c.maps[1], c.maps[2]},
                                      {c.written[0], c.written[1], c.written[2]});
    const int wb = word_bytes(es, {bits, pair_bits(a->turns, es)});
    return launch_moves(c.moves, c.dims, type, a->turns.flags & ROTARY_ADJACENT, wb, word_bytes(es, {bits}), spans,
                        static_cast<cudaStream_t>(stream));
}

}  // extern "C"

namespace bmmc {
cudaError_t bounds_record_rotary(unsigned long long out[chk::kRecordWords], bool clear) {
    return chk::read_record(out, clear);
}
}  // namespace bmmc
