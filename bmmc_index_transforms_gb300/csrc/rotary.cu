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
#include "token_moves.hpp"
#include "token_words.cuh"

using namespace bmmc;

namespace {

constexpr int kThreads = 128;           // threads of a block, at most (one token may take 256)
constexpr int kMostThreads = 256;
constexpr int kMaxTokensPerBlock = 64;
constexpr int kHeadsAtOnce = 2;         // heads whose words a thread has in flight
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
    const int *starts, *lengths, *table;
    int64_t sequences, table_stride, table_columns, pages;
    int page_size;
    int64_t page_stride[2], slot_stride[2];  // of the key and the value cache, bytes
};

// The last sequence whose start is <= t, -1 if there is none: by a whole
// warp, 32 starts at a time, and by one thread.  Any starts, in order or not,
// give an index in range.
__device__ int64_t find_sequence_warp(const int* starts, int64_t sequences, int64_t t, int lane) {
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

__device__ int64_t find_sequence(const int* starts, int64_t sequences, int64_t t) {
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
};

__device__ Place place_of(const MoveParams& p, int64_t t, int64_t b) {
    Place r{0, {-1, -1}};
    int64_t first = t;
    if (p.starts) {
        if (b < 0 || !BMMC_RD_OK(p.starts + b, 8)) return r;
        first = p.starts[b];
    } else if (t >= p.sequences) {
        return r;
    }
    if (!BMMC_RD_OK(p.lengths + b, 4)) return r;
    const int length = p.lengths[b], next = p.starts ? p.starts[b + 1] : 0;  // on their way together
    if (p.starts && t >= next) return r;
    r.at = (int64_t)length + (t - first);
    if (r.at < 0 || r.at >= (int64_t)1 << 32) return r;  // (more only by starts below zero)
    const unsigned at = (unsigned)r.at, column = at / p.page_size;
    if (column >= p.table_columns) return r;
    if (!BMMC_RD_OK(p.table + b * p.table_stride + column, 4)) return r;
    const int page = p.table[b * p.table_stride + column];
    if (page < 0 || page >= p.pages) return r;
    for (int c = 0; c < 2; ++c)
        r.byte[c] = page * p.page_stride[c] + (int64_t)(at - column * p.page_size) * p.slot_stride[c];
    return r;
}

// Written out, so that every variant rounds alike.
__device__ __forceinline__ float turned_first(float x, float y, float2 r) { return fmaf(x, r.x, -__fmul_rn(y, r.y)); }
__device__ __forceinline__ float turned_second(float x, float y, float2 r) { return fmaf(y, r.x, __fmul_rn(x, r.y)); }

// The start of a block that takes tokens t0 .. t0 + nt - 1 and some of the
// parts: the tokens' places in the caches and positions, and the cosines and
// sines of their pairs, into shared memory; the whole block takes part.
__device__ __forceinline__ void begin_block(const MoveParams& p, int64_t t0, int nt, int first_part, int last_part,
                                            Slots<float2> turns, Slots<int64_t> places, Slots<float> place_numbers) {
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

bmmc_status check_heads(const token_heads_t& x, int64_t tokens, int es) {
    if (!x.data || x.heads < 1 || x.dim < 1 || x.dim > ROTARY_MAX_DIM || x.heads > (1 << 24) / x.dim ||
        bad_stride(x.token_stride, tokens) || bad_stride(x.head_stride, x.heads))
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

// Whether key and value cache lie between each other: by page, entry or head.
bool caches_between(const paged_append_args_t& a, int es) {
    const paged_cache_t &k = a.k_cache, &v = a.v_cache;
    const int64_t sizes[3] = {a.pages, a.page_size, a.k.heads};
    const int64_t strides[3] = {k.page_stride * es, k.slot_stride * es, k.head_stride * es};
    const int64_t others[3] = {v.page_stride * es, v.slot_stride * es, v.head_stride * es};
    for (int i = 0; i < 3; ++i)
        if (sizes[i] > 1 && strides[i] != others[i]) return false;
    return lie_between(a.k.dim * es, a.v.dim * es, sizes, strides, (int64_t)((uintptr_t)v.data - (uintptr_t)k.data));
}

uint64_t address_bits(const token_heads_t& x, int es) {
    return (uint64_t)(uintptr_t)x.data | (uint64_t)(x.token_stride * es) | (uint64_t)(x.head_stride * es) |
           (uint64_t)(x.dim * es);
}

// The rotation's arguments, checked and put into p.
bmmc_status set_turns(MoveParams& p, const rotary_turns_t& r, bool need_positions) {
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
Rows turn_rows(const rotary_turns_t& r, int64_t tokens, int what) {
    if (what == 0) return Rows{r.inv_freq, 1, 0, r.pairs * 4};
    if (what == 1) return Rows{r.pair_axes, 1, 0, r.pairs * 4};
    return Rows{r.positions, r.axes, r.axis_stride * r.position_bytes, tokens * r.position_bytes};
}

// Whether an output may share bytes with what the turns read.
bool meets_turns(const Rows& out, const rotary_turns_t& r, int64_t tokens) {
    for (int what = 0; what < 3; ++what)
        if (may_overlap(turn_rows(r, tokens, what), out)) return true;
    return false;
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
    h.turned = turned;
    return h;
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
    const bool with_q = a->q.data || a->q_out.data;
    bmmc_status s = check_heads(a->k, a->tokens, es);
    if (s == BMMC_OK) s = check_heads(a->v, a->tokens, es);
    if (s == BMMC_OK && with_q) s = check_heads(a->q, a->tokens, es);
    if (s == BMMC_OK && with_q) s = check_heads(a->q_out, a->tokens, es);
    if (s != BMMC_OK) return s;
    const int64_t turned = 2 * a->turns.pairs;
    if (a->k.heads != a->v.heads || turned > a->k.dim || (a->turns.flags & ROTARY_INVERSE)) return BMMC_ERR_INVALID_ARG;
    if (with_q && (a->q.heads != a->q_out.heads || a->q.dim != a->q_out.dim || turned > a->q.dim ||
                   !writable(a->q_out, a->tokens)))
        return BMMC_ERR_INVALID_ARG;
    if (a->sequences < 0 || a->sequences > kMaxTokens || (a->sequences && !a->lengths) ||
        (a->sequences && a->table_columns && !a->table) || a->table_columns < 0 || a->table_columns > kMaxTokens ||
        bad_stride(a->table_stride, a->sequences) || a->pages < 0 || a->pages > kMaxTokens ||
        a->page_size < 1 || a->page_size > kMaxTokens || (!a->starts && a->sequences != a->tokens))
        return BMMC_ERR_INVALID_ARG;
    if ((uintptr_t)a->starts % 4 || (uintptr_t)a->lengths % 4 || (uintptr_t)a->table % 4) return BMMC_ERR_MISALIGNED;
    const paged_cache_t* cache[2] = {&a->k_cache, &a->v_cache};
    const token_heads_t* from[2] = {&a->k, &a->v};
    Rows cache_rows[2];
    MoveParams p{};
    p.device = device;
    uint64_t bits = 0;
    for (int c = 0; c < 2; ++c) {
        const paged_cache_t& m = *cache[c];
        if ((!m.data && a->pages) || bad_stride(m.page_stride, a->pages) || bad_stride(m.slot_stride, a->page_size) ||
            bad_stride(m.head_stride, from[c]->heads))
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
    if (may_overlap(cache_rows[0], cache_rows[1]) && !caches_between(*a, es)) return BMMC_ERR_ALIAS;
    for (const Rows& c : cache_rows)
        if (may_overlap(c, k) || may_overlap(c, v)) return BMMC_ERR_ALIAS;
    if (with_q) {
        const Rows q = rows_of(a->q, a->tokens, es), to = rows_of(a->q_out, a->tokens, es);
        if (may_overlap(to, k) || may_overlap(to, v) || may_overlap(to, cache_rows[0]) || may_overlap(to, cache_rows[1]) ||
            may_overlap(q, cache_rows[0]) || may_overlap(q, cache_rows[1]) ||
            (!same_place(a->q, a->q_out, a->tokens) && may_overlap(q, to)))
            return BMMC_ERR_ALIAS;
    }
    if ((s = set_turns(p, a->turns, false)) != BMMC_OK) return s;
    const Rows none{nullptr, 0, 0, 0};
    const Rows written[3] = {cache_rows[0], cache_rows[1], with_q ? rows_of(a->q_out, a->tokens, es) : none};
    const Rows maps[3] = {Rows{a->starts, 1, 0, (a->sequences + 1) * 4}, Rows{a->lengths, 1, 0, a->sequences * 4},
                          Rows{a->table, a->sequences, a->table_stride * 4, a->table_columns * 4}};
    for (const Rows& w : written) {
        if (meets_turns(w, a->turns, a->tokens)) return BMMC_ERR_ALIAS;
        for (const Rows& m : maps)
            if (may_overlap(m, w)) return BMMC_ERR_ALIAS;
    }
    if ((s = all_reachable(device, {a->k.data, a->v.data, a->q.data, a->q_out.data, a->k_cache.data, a->v_cache.data, a->starts,
                            a->lengths, a->table, a->turns.inv_freq, a->turns.pair_axes, a->turns.positions})) != BMMC_OK)
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
    const int dims[3] = {(int)a->k.dim, (int)a->v.dim, (int)a->q.dim};
    const chk::Spans spans =
        spans_of({k, v, with_q ? rows_of(a->q, a->tokens, es) : none, turn_rows(a->turns, a->tokens, 0),
                  turn_rows(a->turns, a->tokens, 1), turn_rows(a->turns, a->tokens, 2), maps[0], maps[1], maps[2]},
                 {written[0], written[1], written[2]});
    const int wb = word_bytes(es, {bits, pair_bits(a->turns, es)});
    return launch_moves(p, dims, type, a->turns.flags & ROTARY_ADJACENT, wb, word_bytes(es, {bits}), spans,
                        static_cast<cudaStream_t>(stream));
}

}  // extern "C"

namespace bmmc {
cudaError_t bounds_record_rotary(unsigned long long out[chk::kRecordWords], bool clear) {
    return chk::read_record(out, clear);
}
}  // namespace bmmc
