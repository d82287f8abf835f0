// Rows of a table named by tokens, and the gradient by the table:
// embedding_lookup and embedding_backward (declared in include/bmmc.h).
//
//   lookup:   out[t] = scale * table[id[t]]
//   gradient: out[v] = scale * sum over the tokens t with id[t] = v of grad[t]
//
// The lookup is a gather of rows, its gradient the gather's transpose.  Equal
// tokens are brought together by a stable sort of the tokens by id; the rows
// of a run are then added up in the order of the tokens.
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>
#include <type_traits>

#include "../../include/bmmc.h"
#define BMMC_CHK_FILE 8  // site tag of this file in bounds-checked builds
#include "bounds.cuh"
#include "token_moves.hpp"
#include "token_words.cuh"

using namespace bmmc;

namespace {

#ifdef BMMC_BOUNDS_CHECK
__device__ __forceinline__ uint32_t chk_dynamic_bytes() { return chk::dyn_smem_bytes(); }
#endif

// A token's id; -1 where it names no row.
template <class Id>
__device__ __forceinline__ int64_t row_named(Id id, int64_t vocab) {
    return id >= 0 && (int64_t)id < vocab ? (int64_t)id : -1;
}

// ---- lookup ------------------------------------------------------------------

// Pure movement but for one product: a word a thread.
template <class T, int W, bool ACROSS, class Id>
__global__ void __launch_bounds__(256) lookup_kernel(const char* __restrict__ table, int64_t table_stride, int64_t vocab,
                                                     const Id* __restrict__ ids, int64_t tokens, int length, float scale,
                                                     char* __restrict__ out, int64_t out_stride BMMC_SPANS_PARAM) {
    BMMC_SPANS_ENTER_GLOBAL();
    const int64_t t = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
    const int w = blockIdx.y * blockDim.x + threadIdx.x;
    if (t >= tokens) return;
    char* const to = out + t * out_stride;
    const Walk<T, W, ACROSS> walk(length, to);
    if (!walk.in(w)) return;
    const int64_t row = BMMC_RD_OK(ids + t, sizeof(Id)) ? row_named(ids[t], vocab) : -1;
    typename Walk<T, W, ACROSS>::Fetch f;
    walk.fetch(f, row >= 0, table + (row < 0 ? 0 : row) * table_stride, w);
    Pack<T, W> y = walk.get(f);
    float v[W];
#pragma unroll
    for (int i = 0; i < W; ++i) v[i] = row < 0 ? 0.0f : y.get(i) * scale;
    y.set(v);
    walk.store(y, to, w);
}

// ---- the sort of the tokens --------------------------------------------------

constexpr int kSortThreads = 1024;
constexpr int kSortRounds = 4;  // keys of a thread and tile
constexpr int kMaxDigit = 10;   // bits of the keys that a pass sorts by
constexpr int kMaxSortBlocks = kSms;

// A token's key: its id, or `vocab` where it names no row.
template <class Id>
__device__ __forceinline__ uint32_t key_of(const Id* ids, int64_t i, int64_t vocab) {
    const int64_t row = BMMC_RD_OK(ids + i, sizeof(Id)) ? row_named(ids[i], vocab) : -1;
    return (uint32_t)(row < 0 ? vocab : row);
}

// What a pass sorts: the tokens by their ids (FIRST), or what the pass before
// it has sorted.
template <class Id, bool FIRST>
struct Sorted {
    const Id* ids;
    const uint32_t *keys, *order;
    int64_t vocab;
    __device__ __forceinline__ uint32_t key(int64_t i) const {
        if constexpr (FIRST) return key_of(ids, i, vocab);
        else return BMMC_RD_OK(keys + i, 4) ? keys[i] : 0;
    }
    __device__ __forceinline__ uint32_t token(int64_t i) const {
        if constexpr (FIRST) return (uint32_t)i;
        else return BMMC_RD_OK(order + i, 4) ? order[i] : 0;
    }
};

// counts[block][digit] of each block's part.
template <class Id, bool FIRST>
__global__ void __launch_bounds__(kSortThreads) digit_count_kernel(Sorted<Id, FIRST> in, int64_t n, int shift, int digit,
                                                                   int64_t per_block, int* __restrict__ counts
                                                                       BMMC_SPANS_PARAM) {
    __shared__ int s_hist[1 << kMaxDigit];
    BMMC_SPANS_ENTER(s_hist, sizeof(s_hist));
    const int bins = 1 << digit;
    const Slots<int> hist(s_hist, bins);
    for (int d = threadIdx.x; d < bins; d += blockDim.x) hist.set(d, 0);
    __syncthreads();
    const int64_t lo = (int64_t)blockIdx.x * per_block, hi = min(n, lo + per_block);
    for (int64_t i = lo + threadIdx.x; i < hi; i += blockDim.x) hist.add((in.key(i) >> shift) & (bins - 1), 1);
    __syncthreads();
    for (int d = threadIdx.x; d < bins; d += blockDim.x)
        if (BMMC_WR_OK(counts + (int64_t)blockIdx.x * bins + d, 4)) counts[(int64_t)blockIdx.x * bins + d] = hist.get(d);
}

// Exclusive prefix sum of v[0..n) in shared memory, in place, by the whole block
// of 32 warps.  tmp: 32 ints.
__device__ void exclusive_scan(Slots<int> v, int n, Slots<int> tmp) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int carry = 0;
    for (int at = 0; at < n; at += blockDim.x) {
        const int i = at + threadIdx.x, x = i < n ? v.get(i) : 0;
        int s = x;
        for (int d = 1; d < 32; d <<= 1) {
            const int y = __shfl_up_sync(~0u, s, d);
            if (lane >= d) s += y;
        }
        if (lane == 31) tmp.set(warp, s);
        __syncthreads();
        if (warp == 0) {
            int w = tmp.get(lane);
            for (int d = 1; d < 32; d <<= 1) {
                const int y = __shfl_up_sync(~0u, w, d);
                if (lane >= d) w += y;
            }
            tmp.set(lane, w);
        }
        __syncthreads();
        if (i < n) v.set(i, carry + (warp ? tmp.get(warp - 1) : 0) + s - x);
        carry += tmp.get(31);
        __syncthreads();
    }
}

// The lanes with the same digit, from one ballot for each of its bits.
__device__ __forceinline__ unsigned same_digit(int d, int bits) {
    unsigned same = ~0u;
    for (int b = 0; b < bits; ++b) {
        const bool one = (d >> b) & 1;
        const unsigned ones = __ballot_sync(~0u, one);
        same &= one ? ones : ~ones;
    }
    return same;
}

// One pass of the sort, stable: every block puts its part in place, a tile at
// a time.  A key's rank among the equal digits of its warp comes from ballots
// and the warp's running counts; sums over the warps and the counts of the
// blocks ahead complete its place.
template <class Id, bool FIRST>
__global__ void __launch_bounds__(kSortThreads) digit_place_kernel(Sorted<Id, FIRST> in, int64_t n, int shift, int digit,
                                                                   int64_t per_block, const int* __restrict__ counts,
                                                                   uint32_t* __restrict__ keys,
                                                                   uint32_t* __restrict__ order BMMC_SPANS_PARAM) {
    constexpr int kWarps = kSortThreads / 32;
    extern __shared__ int s_mem[];
    BMMC_SPANS_ENTER(s_mem, chk_dynamic_bytes());
    const int bins = 1 << digit;
    const Slots<int> mem(s_mem, bins + 32 + kWarps * bins / 2);
    const Slots<int> base = mem.part(0, bins), tmp = mem.part(bins, 32);  // where the next key of each digit goes
    const Slots<unsigned short> hist(reinterpret_cast<unsigned short*>(s_mem + bins + 32), kWarps * bins);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    // all blocks' counts of a digit, then, by the scan, where its keys start; plus those of the blocks ahead
    int ahead = 0;
    for (int d = threadIdx.x; d < bins; d += blockDim.x) {
        int all = 0;
        ahead = 0;
#pragma unroll 8
        for (int b = 0; b < (int)gridDim.x; ++b) {
            const int c = BMMC_RD_OK(counts + (int64_t)b * bins + d, 4) ? counts[(int64_t)b * bins + d] : 0;
            all += c;
            if (b < (int)blockIdx.x) ahead += c;
        }
        base.set(d, all);
    }
    __syncthreads();
    exclusive_scan(base, bins, tmp);
    if ((int)threadIdx.x < bins) base.set(threadIdx.x, base.get(threadIdx.x) + ahead);  // (a digit a thread at most)
    const Slots<unsigned short> mine = hist.part(warp * bins, bins);
    const int64_t lo = (int64_t)blockIdx.x * per_block, hi = min(n, lo + per_block);
    for (int64_t at = lo; at < hi; at += kSortThreads * kSortRounds) {
        uint32_t key[kSortRounds], token[kSortRounds];
        int rank[kSortRounds];
#pragma unroll
        for (int r = 0; r < kSortRounds; ++r) {
            const int64_t i = at + (warp * kSortRounds + r) * 32 + lane;
            key[r] = i < hi ? in.key(i) : 0;
            token[r] = i < hi ? in.token(i) : 0;
        }
        for (int d = lane; d < bins; d += 32) mine.set(d, 0);
        __syncwarp();
#pragma unroll
        for (int r = 0; r < kSortRounds; ++r) {
            const bool there = at + (warp * kSortRounds + r) * 32 + lane < hi;
            const int d = (key[r] >> shift) & (bins - 1);
            const unsigned same = same_digit(d, digit) & __ballot_sync(~0u, there);
            const int before = there ? mine.get(d) : 0;
            rank[r] = before + __popc(same & ((1u << lane) - 1));
            __syncwarp();
            if (there && lane == __ffs(same) - 1) mine.set(d, (unsigned short)(before + __popc(same)));
            __syncwarp();
        }
        __syncthreads();
        int in_tile = 0;
        if ((int)threadIdx.x < bins) {
            for (int w = 0; w < kWarps; ++w) {
                const int c = hist.get(w * bins + threadIdx.x);
                hist.set(w * bins + threadIdx.x, (unsigned short)in_tile);
                in_tile += c;
            }
        }
        __syncthreads();
#pragma unroll
        for (int r = 0; r < kSortRounds; ++r) {
            if (at + (warp * kSortRounds + r) * 32 + lane >= hi) continue;
            const int d = (key[r] >> shift) & (bins - 1);
            const int to = base.get(d) + mine.get(d) + rank[r];
            if ((unsigned)to >= (unsigned)n) continue;  // (ids that change meanwhile)
            if (BMMC_WR_OK(keys + to, 4)) keys[to] = key[r];
            if (BMMC_WR_OK(order + to, 4)) order[to] = token[r];
        }
        __syncthreads();
        if ((int)threadIdx.x < bins) base.set(threadIdx.x, base.get(threadIdx.x) + in_tile);
    }
}

// ---- the sums ------------------------------------------------------------------

// A chunk is kChunk places of the sorted tokens.  A run of equal ids that
// reaches over two chunks at most is added up by the block of the chunk in
// which it starts.  One that reaches over three or more is long: each of its
// chunks adds up its part (in partial: part 0 of a chunk belongs to a run that
// goes on from the chunk before, part 1 to one that starts in it), and the join
// kernel adds the parts.
constexpr int kChunk = 32;
constexpr int kSumThreads = 256;
constexpr int kSumAhead = 8;  // rows whose words a thread has in flight

struct Runs {
    const uint32_t* keys;
    int64_t n;
    __device__ __forceinline__ int64_t key(int64_t i) const {
        return i >= 0 && i < n && BMMC_RD_OK(keys + i, 4) ? (int64_t)keys[i] : -1;
    }
};

// v (added to what is there) to W elements of a row, `left` of which it has.
template <class O, int W, bool WORDS>
__device__ __forceinline__ void put(float (&v)[W], O* p, int left, bool accumulate) {
    constexpr int P = 16 / sizeof(O) < W ? 16 / sizeof(O) : W;
    if constexpr (WORDS) {
#pragma unroll
        for (int a = 0; a < W; a += P) {
            Pack<O, P> y;
            float u[P];
            if (accumulate && BMMC_RD_OK(p + a, sizeof(y))) y.load(p + a);
#pragma unroll
            for (int i = 0; i < P; ++i) u[i] = accumulate ? v[a + i] + y.get(i) : v[a + i];
            y.set(u);
            if (BMMC_WR_OK(p + a, sizeof(y))) y.store(p + a);
        }
    } else {
#pragma unroll
        for (int i = 0; i < W; ++i)
            if (i < left && BMMC_WR_OK(p + i, sizeof(O)))
                p[i] = from_f32<O>(accumulate && BMMC_RD_OK(p + i, sizeof(O)) ? v[i] + to_f32(p[i]) : v[i]);
    }
}

template <class T, class O, int W, bool WORDS>
__global__ void __launch_bounds__(kSumThreads) sum_rows_kernel(
    const char* __restrict__ grad, int64_t grad_stride, const uint32_t* __restrict__ keys,
    const uint32_t* __restrict__ order, int64_t n, int64_t vocab, int length, float scale, int accumulate,
    char* __restrict__ out, int64_t out_stride, float* __restrict__ partial, int partial_stride BMMC_SPANS_PARAM) {
    __shared__ int s_key[2 * kChunk + 1], s_token[2 * kChunk];
    BMMC_SPANS_ENTER(s_key, sizeof(s_key), s_token, sizeof(s_token));
    const Slots<int> ids(s_key, 2 * kChunk + 1), tokens(s_token, 2 * kChunk);
    const Runs runs{keys, n};
    const int64_t lo = (int64_t)blockIdx.x * kChunk;
    for (int i = threadIdx.x; i <= 2 * kChunk; i += blockDim.x) {
        ids.set(i, (int)runs.key(lo + i));
        if (i < 2 * kChunk)
            tokens.set(i, lo + i < n && BMMC_RD_OK(order + lo + i, 4) ? (int)order[lo + i] : 0);
    }
    const int64_t before = runs.key(lo - 1), far_before = runs.key(lo - kChunk - 1);
    __syncthreads();
    const int here = (int)min((int64_t)kChunk, n - lo), w = blockIdx.y * blockDim.x + threadIdx.x;
    if (w * W >= length) return;
    const Walk<T, W, !WORDS> walk(length, nullptr);
    // the run that goes on from the chunk before: its owner's, or a part of a long one
    int begin = 0, end = here, first_part = -1;
    const int first = ids.get(0), last = ids.get(here - 1);
    if (first == before) {
        while (begin < here && ids.get(begin) == first) ++begin;
        const bool goes_on = begin == here && ids.get(here) == first;
        if (far_before == first || goes_on) first_part = begin, begin = 0;
    }
    // the run that goes on behind this chunk, where it starts in this one
    bool last_part = false;
    if ((begin < here && first_part < here) && ids.get(here) == last) {
        if (runs.key(lo + 2 * kChunk) == last && here == kChunk) last_part = true;
        else
            while (end < 2 * kChunk && ids.get(end) == last) ++end;
    }
    float sum[W] = {};
    int id = ids.get(begin < here ? begin : 0);
    const auto put_out = [&](bool part, int which) {
        if (id < 0 || id >= vocab) return;
        if (part) {
            float* const to = partial + ((int64_t)blockIdx.x * 2 + which) * partial_stride + w * W;
#pragma unroll
            for (int i = 0; i < W; ++i)
                if (BMMC_WR_OK(to + i, 4)) to[i] = sum[i];
        } else {
#pragma unroll
            for (int i = 0; i < W; ++i) sum[i] *= scale;
            put<O, W, WORDS>(sum, reinterpret_cast<O*>(out + (int64_t)id * out_stride) + w * W, length - w * W, accumulate);
        }
#pragma unroll
        for (int i = 0; i < W; ++i) sum[i] = 0.0f;
    };
    for (int at = begin; at < end; at += kSumAhead) {
        typename Walk<T, W, !WORDS>::Fetch f[kSumAhead];
#pragma unroll
        for (int u = 0; u < kSumAhead; ++u) {
            const bool want = at + u < end && ids.get(at + u) < vocab;
            walk.fetch(f[u], want, grad + (int64_t)(want ? tokens.get(at + u) : 0) * grad_stride, w);
        }
#pragma unroll
        for (int u = 0; u < kSumAhead; ++u) {
            if (at + u >= end) break;
            const int next = ids.get(at + u);
            if (next != id) {
                put_out(at + u == first_part, 0);
                id = next;
            }
            const Pack<T, W> y = walk.get(f[u]);
#pragma unroll
            for (int i = 0; i < W; ++i) sum[i] += y.get(i);
        }
    }
    if (begin < end) put_out(last_part || end == first_part, last_part ? 1 : 0);
}

// Joins the parts of the long runs: a block looks at kOwners chunks for runs
// that start there, and takes 128 columns of each: its warps add every eighth
// part, then the eight sums are added in order.
constexpr int kOwners = 16;

template <class O>
__global__ void __launch_bounds__(256) join_parts_kernel(const uint32_t* __restrict__ keys, int64_t n, int64_t vocab,
                                                         int length, float scale, int accumulate, char* __restrict__ out,
                                                         int64_t out_stride, const float* __restrict__ partial,
                                                         int partial_stride BMMC_SPANS_PARAM) {
    __shared__ float s_sum[8][128];
    BMMC_SPANS_ENTER(s_sum, sizeof(s_sum));
    const Slots<float> sums(&s_sum[0][0], 8 * 128);
    const Runs runs{keys, n};
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    for (int c = 0; c < kOwners; ++c) {
        const int64_t chunk = (int64_t)blockIdx.x * kOwners + c, lo = chunk * kChunk, hi = lo + kChunk;
        const int64_t id = runs.key(hi - 1);
        if (hi + kChunk >= n || runs.key(hi) != id || runs.key(hi + kChunk) != id || id >= vocab) continue;
        if (runs.key(lo - 1) == id) continue;  // it goes on from the chunk before
        for (int first = blockIdx.y * 128; first < length; first += gridDim.y * 128) {
            float4 sum = make_float4(0, 0, 0, 0);
            const int col = first + lane * 4;
            for (int64_t k = warp; k == 0 || runs.key(lo + k * kChunk) == id; k += 8) {
                const float* const from = partial + ((chunk + k) * 2 + (k == 0)) * partial_stride + col;
                const float4 v = col < partial_stride && BMMC_RD_OK(from, 16) ? *reinterpret_cast<const float4*>(from)
                                                                               : make_float4(0, 0, 0, 0);
                sum.x += v.x, sum.y += v.y, sum.z += v.z, sum.w += v.w;
            }
            const float v4[4] = {sum.x, sum.y, sum.z, sum.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) sums.set(warp * 128 + lane * 4 + i, v4[i]);
            __syncthreads();
            const int at = first + threadIdx.x;
            if (threadIdx.x < 128 && at < length) {
                float v[1] = {0.0f};
                for (int g = 0; g < 8; ++g) v[0] += sums.get(g * 128 + threadIdx.x);
                v[0] *= scale;
                put<O, 1, false>(v, reinterpret_cast<O*>(out + id * out_stride) + at, 1, accumulate);
            }
            __syncthreads();
        }
    }
}

// Rows of zeros.
template <class T>
__global__ void __launch_bounds__(256) clear_rows_kernel(char* __restrict__ out, int64_t out_stride, int64_t rows, int length
                                                             BMMC_SPANS_PARAM) {
    BMMC_SPANS_ENTER_GLOBAL();
    constexpr int W = 16 / sizeof(T);
    const int64_t t = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
    const int w = blockIdx.y * blockDim.x + threadIdx.x;
    if (t >= rows) return;
    char* const to = out + t * out_stride;
    const Walk<T, W, true> walk(length, to);
    Pack<T, W> zero;
    zero.word = uint4{};
    if (walk.in(w)) walk.store(zero, to, w);
}

// ---- host ----------------------------------------------------------------------

struct SortShape {
    int passes, digit, blocks;
    int64_t per_block;
};

SortShape sort_shape(int64_t n, int64_t vocab) {
    SortShape s;
    int bits = 1;  // of the keys 0 .. vocab
    while (bits < 32 && (vocab >> bits)) ++bits;
    s.passes = (bits + kMaxDigit - 1) / kMaxDigit;
    s.digit = (bits + s.passes - 1) / s.passes;
    const int64_t tile = kSortThreads * kSortRounds, tiles = (n + tile - 1) / tile;
    const int64_t per = (tiles + kMaxSortBlocks - 1) / kMaxSortBlocks;
    s.per_block = (per ? per : 1) * tile;
    s.blocks = (int)((n + s.per_block - 1) / s.per_block);
    return s;
}

int64_t up16(int64_t bytes) { return (bytes + 15) & ~(int64_t)15; }

// The workspace: two arrays of keys and two of tokens, the blocks' counts, and
// two sums a chunk.
struct Workspace {
    int64_t array, counts, partial;  // bytes
    int partial_stride;              // floats
    int64_t bytes() const { return 4 * array + counts + partial; }
};

Workspace workspace_of(int64_t n, int64_t vocab, int64_t hidden) {
    const SortShape s = sort_shape(n, vocab);
    Workspace w;
    w.array = up16(n * 4);
    w.counts = up16((int64_t)s.blocks * (4 << s.digit));
    w.partial_stride = (int)((hidden + 7) & ~(int64_t)7);
    const int64_t chunks = (n + kChunk - 1) / kChunk;
    w.partial = chunks < 3 ? 0 : chunks * 2 * w.partial_stride * 4;  // a long run has three
    return w;
}

bmmc_status check_ids(int id_bytes, int64_t tokens, int64_t vocab, int64_t hidden) {
    if (id_bytes != 4 && id_bytes != 8) return BMMC_ERR_UNSUPPORTED_ELEM;
    if (tokens < 0 || tokens > kMaxTokens || vocab < 0 || vocab >= kMaxTokens || hidden < 1 || hidden > (1 << 24))
        return BMMC_ERR_INVALID_ARG;
    return BMMC_OK;
}

template <class Id>
bmmc_status sort_tokens(const SortShape& s, const Id* ids, int64_t n, int64_t vocab, uint32_t* (&keys)[2],
                        uint32_t* (&order)[2], int* counts, const chk::Spans& spans, cudaStream_t st) {
    (void)spans;
    const size_t smem = ((1 << s.digit) + 32) * 4 + (size_t)(kSortThreads / 32) * (2 << s.digit);
    for (int pass = 0; pass < s.passes; ++pass) {
        const int shift = pass * s.digit, from = (pass & 1) ^ 1, to = pass & 1;
        bmmc_status status;
        const auto run = [&](auto in, auto count, auto place) {
            if (smem > 48 * 1024 && cudaFuncSetAttribute(place, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) != cudaSuccess) {
                cudaGetLastError();
                return BMMC_ERR_CUDA;
            }
            status = launch(count, dim3(s.blocks), dim3(kSortThreads), 0, st, nullptr, in, n, shift, s.digit, s.per_block,
                            counts BMMC_SPANS_ARG(spans));
            if (status != BMMC_OK) return status;
            return launch(place, dim3(s.blocks), dim3(kSortThreads), smem, st, nullptr, in, n, shift, s.digit, s.per_block,
                          (const int*)counts, keys[to], order[to] BMMC_SPANS_ARG(spans));
        };
        if (pass == 0)
            status = run(Sorted<Id, true>{ids, nullptr, nullptr, vocab}, digit_count_kernel<Id, true>, digit_place_kernel<Id, true>);
        else
            status = run(Sorted<Id, false>{nullptr, keys[from], order[from], vocab}, digit_count_kernel<Id, false>,
                         digit_place_kernel<Id, false>);
        if (status != BMMC_OK) return status;
    }
    return BMMC_OK;
}

}  // namespace

extern "C" {

bmmc_status embedding_lookup(const void* table, int64_t table_stride, int64_t vocab, const void* ids, int id_bytes,
                             int64_t tokens, int64_t hidden, int type, float scale, void* out, int64_t out_stride,
                             void* stream) {
    const bool device = device_pointers(type);
    const int es = dtype_bytes(type);
    if (!es) return BMMC_ERR_UNSUPPORTED_ELEM;
    bmmc_status s = check_ids(id_bytes, tokens, vocab, hidden);
    if (s != BMMC_OK) return s;
    if (bad_stride(table_stride, vocab) || bad_output_stride(out_stride, hidden, tokens)) return BMMC_ERR_INVALID_ARG;
    if (!tokens) return BMMC_OK;
    if ((!table && vocab) || !ids || !out) return BMMC_ERR_INVALID_ARG;
    if (misaligned(table, es) || misaligned(out, es) || misaligned(ids, id_bytes)) return BMMC_ERR_MISALIGNED;
    const Rows from{table, vocab, table_stride * es, hidden * es}, names{ids, 1, 0, tokens * id_bytes};
    const Rows to{out, tokens, out_stride * es, hidden * es};
    if (may_overlap(from, to) || may_overlap(names, to)) return BMMC_ERR_ALIAS;
    if ((s = all_reachable(device, {table, ids, out})) != BMMC_OK) return s;
    const Way way = way_of(hidden, es, {(uint64_t)(uintptr_t)table, (uint64_t)(uintptr_t)out, (uint64_t)(table_stride * es),
                                        (uint64_t)(out_stride * es), (uint64_t)(hidden * es)});
    const chk::Spans spans = spans_of({from, names}, {to});
    (void)spans;
    by_type(type, way, [&](auto e, auto width, auto across) {
        using T = decltype(e);
        constexpr int W = decltype(width)::value;
        constexpr bool A = decltype(across)::value;
        const Cover c = cover(tokens, way.words, tokens * way.words <= kFewWords ? 128 : 256);
        const auto go = [&](auto id) {
            using Id = decltype(id);
            s = launch(lookup_kernel<T, W, A, Id>, c.grid, c.block, 0, static_cast<cudaStream_t>(stream), nullptr,
                       static_cast<const char*>(table), table_stride * es, vocab, static_cast<const Id*>(ids), tokens,
                       (int)hidden, scale, static_cast<char*>(out), out_stride * es BMMC_SPANS_ARG(spans));
        };
        id_bytes == 4 ? go(int32_t{}) : go(int64_t{});
    });
    return s;
}

bmmc_status embedding_backward_workspace(int64_t tokens, int64_t vocab, int64_t hidden, size_t* bytes) {
    if (!bytes) return BMMC_ERR_INVALID_ARG;
    *bytes = 0;
    const bmmc_status s = check_ids(4, tokens, vocab, hidden);
    if (s != BMMC_OK) return s;
    if (tokens && vocab) *bytes = (size_t)workspace_of(tokens, vocab, hidden).bytes();
    return BMMC_OK;
}

bmmc_status embedding_backward(const void* grad, int64_t grad_stride, const void* ids, int id_bytes, int64_t tokens,
                               int64_t hidden, int type, float scale, int accumulate, void* out, int64_t out_stride,
                               int64_t vocab, int out_type, void* workspace, size_t workspace_bytes, void* stream) {
    const bool device = device_pointers(type);
    const int es = dtype_bytes(type), os = dtype_bytes(out_type);
    if (!es || (out_type != type && out_type != BMMC_F32)) return BMMC_ERR_UNSUPPORTED_ELEM;
    bmmc_status s = check_ids(id_bytes, tokens, vocab, hidden);
    if (s != BMMC_OK) return s;
    if (bad_stride(grad_stride, tokens) || bad_output_stride(out_stride, hidden, vocab)) return BMMC_ERR_INVALID_ARG;
    if (!vocab || (!tokens && accumulate)) return BMMC_OK;
    if (!out || (tokens && (!grad || !ids))) return BMMC_ERR_INVALID_ARG;
    const Workspace w = workspace_of(tokens, vocab, hidden);
    const int64_t need = tokens ? w.bytes() : 0;
    if (need && (!workspace || workspace_bytes < (size_t)need)) return BMMC_ERR_NO_SCRATCH;
    if (misaligned(grad, es) || misaligned(out, os) || misaligned(ids, id_bytes) || (need && misaligned(workspace, 16)))
        return BMMC_ERR_MISALIGNED;
    const Rows from{grad, tokens, grad_stride * es, hidden * es}, names{ids, 1, 0, tokens * id_bytes};
    const Rows to{out, vocab, out_stride * os, hidden * os}, scratch{need ? workspace : nullptr, 1, 0, need};
    if (may_overlap(from, to) || may_overlap(names, to) || may_overlap(scratch, to) || may_overlap(from, scratch) ||
        may_overlap(names, scratch))
        return BMMC_ERR_ALIAS;
    if ((s = all_reachable(device, {grad, ids, out, need ? workspace : nullptr})) != BMMC_OK) return s;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const chk::Spans spans = spans_of({from, names, scratch, to}, {to, scratch});
    (void)spans;
    if (!accumulate) {
        const int words = (int)((hidden + 2 * (16 / os - 1)) / (16 / os));
        const Cover c = cover(vocab, words, 256);
        s = os == 4 ? launch(clear_rows_kernel<uint32_t>, c.grid, c.block, 0, st, nullptr, static_cast<char*>(out),
                             out_stride * os, vocab, (int)hidden BMMC_SPANS_ARG(spans))
                    : launch(clear_rows_kernel<uint16_t>, c.grid, c.block, 0, st, nullptr, static_cast<char*>(out),
                             out_stride * os, vocab, (int)hidden BMMC_SPANS_ARG(spans));
        if (s != BMMC_OK || !tokens) return s;
    }
    char* const at = static_cast<char*>(workspace);
    uint32_t* keys[2] = {reinterpret_cast<uint32_t*>(at), reinterpret_cast<uint32_t*>(at + w.array)};
    uint32_t* order[2] = {reinterpret_cast<uint32_t*>(at + 2 * w.array), reinterpret_cast<uint32_t*>(at + 3 * w.array)};
    int* const counts = reinterpret_cast<int*>(at + 4 * w.array);
    float* const partial = reinterpret_cast<float*>(at + 4 * w.array + w.counts);
    const SortShape shape = sort_shape(tokens, vocab);
    s = id_bytes == 4 ? sort_tokens(shape, static_cast<const int32_t*>(ids), tokens, vocab, keys, order, counts, spans, st)
                      : sort_tokens(shape, static_cast<const int64_t*>(ids), tokens, vocab, keys, order, counts, spans, st);
    if (s != BMMC_OK) return s;
    const uint32_t *key = keys[(shape.passes - 1) & 1], *token = order[(shape.passes - 1) & 1];
    const int64_t chunks = (tokens + kChunk - 1) / kChunk;
    const bool words = word_bytes(2, {(uint64_t)(uintptr_t)grad, (uint64_t)(uintptr_t)out, (uint64_t)(grad_stride * es),
                                      (uint64_t)(out_stride * os), (uint64_t)(hidden * es), (uint64_t)(hidden * os)}) == 16;
    const auto sum = [&](auto kernel, int W) {
        const int row = (int)((hidden + W - 1) / W), x = row < kSumThreads ? (row + 31) / 32 * 32 : kSumThreads;
        return launch(kernel, dim3((unsigned)chunks, (unsigned)((row + x - 1) / x)), dim3(x), 0, st, nullptr,
                      static_cast<const char*>(grad), grad_stride * es, key, token, tokens, vocab, (int)hidden, scale,
                      accumulate, static_cast<char*>(out), out_stride * os, partial, w.partial_stride BMMC_SPANS_ARG(spans));
    };
    const auto typed = [&](auto t, auto o) {
        using T = decltype(t);
        using O = decltype(o);
        constexpr int W = 16 / sizeof(T);
        return words ? sum(sum_rows_kernel<T, O, W, true>, W) : sum(sum_rows_kernel<T, O, W, false>, W);
    };
    if (type == BMMC_F32) s = typed(float{}, float{});
    else if (type == BMMC_F16) s = out_type == BMMC_F32 ? typed(__half{}, float{}) : typed(__half{}, __half{});
    else s = out_type == BMMC_F32 ? typed(__nv_bfloat16{}, float{}) : typed(__nv_bfloat16{}, __nv_bfloat16{});
    if (s != BMMC_OK || chunks < 3) return s;
    const dim3 grid((unsigned)((chunks + kOwners - 1) / kOwners), (unsigned)std::min<int64_t>((hidden + 127) / 128, kMostParts));
    const auto join = [&](auto kernel) {
        return launch(kernel, grid, dim3(256), 0, st, nullptr, key, tokens, vocab, (int)hidden, scale, accumulate,
                      static_cast<char*>(out), out_stride * os, (const float*)partial, w.partial_stride BMMC_SPANS_ARG(spans));
    };
    if (out_type == BMMC_F32) return join(join_parts_kernel<float>);
    return out_type == BMMC_F16 ? join(join_parts_kernel<__half>) : join(join_parts_kernel<__nv_bfloat16>);
}

}  // extern "C"

namespace bmmc {
cudaError_t bounds_record_embedding(unsigned long long out[chk::kRecordWords], bool clear) {
    return chk::read_record(out, clear);
}
}  // namespace bmmc
