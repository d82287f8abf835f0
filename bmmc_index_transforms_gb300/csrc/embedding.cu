// Rows of a table named by tokens, and the gradient by the table:
// embedding_lookup and embedding_backward (declared in include/bmmc.h).
//
//   lookup:   out[t] = scale * table[id[t]]
//   gradient: out[v] = scale * sum over the tokens t with id[t] = v of grad[t]
//
// The lookup is a gather of rows, its gradient the gather's transpose.  Equal
// tokens are brought together by a stable sort of the tokens by id; the rows
// of a run are then added up in the order of the tokens.
#include <cooperative_groups.h>
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

// Pure movement but for one product: K words of one token a thread, all on their
// way once the id is known.  16384 tokens of 4096 bf16, as frequent as words, of a
// table of 131072: 31.1 us, 90 % of the copy rate over the rows that differ (with one
// word a thread 40.9); rows of 4092 34.8, of 4095, cut out of two words each, 46.
// 65536 rows of 1000 29.2 us, of 520 17.5, of 513 24.7, of 200 7.2 (25.2, 13.2, 13.0, 5.1 of
// bytes; a word a thread in whole warps a row took 39.6, 35.2, 35.7 and 10.3).  64 tokens
// 1.5 us, a launch; there a word a thread has the shorter way.
template <class T, int W, bool ACROSS, int K, class Id>
__global__ void __launch_bounds__(256) lookup_kernel(const char* __restrict__ table, int64_t table_stride, int64_t vocab,
                                                     const Id* __restrict__ ids, int64_t tokens, int length, float scale,
                                                     char* __restrict__ out, int64_t out_stride BMMC_SPANS_PARAM) {
    BMMC_SPANS_ENTER_GLOBAL();
    const int64_t t = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
    if (t >= tokens) return;
    char* const to = out + t * out_stride;
    const Walk<T, W, ACROSS> walk(length, to);
    const int64_t row = BMMC_RD_OK(ids + t, sizeof(Id)) ? row_named(ids[t], vocab) : -1;
    const char* const from = table + (row < 0 ? 0 : row) * table_stride;
    const int w0 = blockIdx.y * blockDim.x * K + threadIdx.x;
    typename Walk<T, W, ACROSS>::Fetch f[K];
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const int w = w0 + k * blockDim.x;
        walk.fetch(f[k], row >= 0 && walk.in(w), from, w);
    }
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const int w = w0 + k * blockDim.x;
        if (!walk.in(w)) break;
        Pack<T, W> y = walk.get(f[k]);
        float v[W];
#pragma unroll
        for (int i = 0; i < W; ++i) v[i] = row < 0 ? 0.0f : y.get(i) * scale;
        y.set(v);
        walk.store(y, to, w);
    }
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

// The kernels of a gradient are launched early, one behind another: each waits for
// the one before it as a whole before it reads or writes anything.  While it waits,
// what it is going to read (counts, keys, order, partial sums) is still being
// written: those are no __restrict__ const parameters, which the compiler may read
// ahead of the wait or by loads that are not told of the writes.  Ordinary loads
// stay behind the wait, which shows them what was written; __ldcg in their place took
// the gradient of 2039 x 1031 23.3 us instead of 22.4, of 32768 rows of 4096 220.8 instead
// of 219.4.

// What a pass sorts: the tokens by their ids (FIRST), or what the pass before
// it has sorted.
template <class Id, bool FIRST>
struct Sorted {
    static constexpr bool kFirst = FIRST;
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
    cudaTriggerProgrammaticLaunchCompletion();
    for (int d = threadIdx.x; d < bins; d += blockDim.x) hist.set(d, 0);
    __syncthreads();
    cudaGridDependencySynchronize();
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
                                                                   int64_t per_block, const int* counts,
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
    cudaTriggerProgrammaticLaunchCompletion();
    cudaGridDependencySynchronize();
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

// The whole sort as one cluster of blocks, R keys a thread: keys and tokens stay
// in registers, and each pass hands them to their places in the shared memory
// of the cluster's blocks.
//
// 32768 ids below 131072, two passes of 9 bits: 19 us alone (with keys and tokens
// handed over in two words 21; four blocks of eight keys a thread 35), beside the
// clearing of a large table nothing.  What bounds it: a quarter of the issue slots'
// cycles wait for the cluster's barriers, the rest for shared memory and the
// ballots of the ranks.
constexpr int kSortCluster = 8;

template <class Id, int R>
__global__ void __launch_bounds__(kSortThreads) sort_cluster_kernel(const Id* __restrict__ ids, int n, int64_t vocab, int passes,
                                                                    int digit, uint32_t* __restrict__ keys,
                                                                    uint32_t* __restrict__ order BMMC_SPANS_PARAM) {
    constexpr int kWarps = kSortThreads / 32, kTile = kSortThreads * R;
    extern __shared__ int s_mem[];
    BMMC_SPANS_ENTER(s_mem, chk_dynamic_bytes());
    const auto cluster = cooperative_groups::this_cluster();
    const int bins = 1 << digit, blocks = (int)gridDim.x, rank_in = (int)blockIdx.x;
    const Slots<int> mem(s_mem, 2 * bins + 32 + kWarps * bins / 2 + 2 * kTile);
    const Slots<int> base = mem.part(0, bins), mine_of = mem.part(bins, bins), tmp = mem.part(2 * bins, 32);
    const Slots<unsigned short> hist(reinterpret_cast<unsigned short*>(s_mem + 2 * bins + 32), kWarps * bins);
    const Slots<uint2> placed(reinterpret_cast<uint2*>(s_mem + 2 * bins + 32 + kWarps * bins / 2), kTile);  // keys and tokens
    cudaTriggerProgrammaticLaunchCompletion();  // the rows may be cleared meanwhile
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, first = warp * R * 32 + lane;
    const Slots<unsigned short> mine = hist.part(warp * bins, bins);
    const int here = min(kTile, n - rank_in * kTile);
    uint32_t key[R], token[R];
    int rank[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const int i = first + r * 32;
        token[r] = rank_in * kTile + i;
        key[r] = i < here ? key_of(ids, token[r], vocab) : 0;
    }
    for (int pass = 0; pass < passes; ++pass) {
        const int shift = pass * digit;
        for (int d = lane; d < bins; d += 32) mine.set(d, 0);
        __syncwarp();
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const bool there = first + r * 32 < here;
            const int d = (key[r] >> shift) & (bins - 1);
            const unsigned same = same_digit(d, digit) & __ballot_sync(~0u, there);
            const int before = there ? mine.get(d) : 0;
            rank[r] = before + __popc(same & ((1u << lane) - 1));
            __syncwarp();
            if (there && lane == __ffs(same) - 1) mine.set(d, (unsigned short)(before + __popc(same)));
            __syncwarp();
        }
        __syncthreads();
        for (int d = threadIdx.x; d < bins; d += kSortThreads) {
            int in_tile = 0;
#pragma unroll 8
            for (int w = 0; w < kWarps; ++w) {
                const int c = hist.get(w * bins + d);
                hist.set(w * bins + d, (unsigned short)in_tile);
                in_tile += c;
            }
            mine_of.set(d, in_tile);
        }
        cluster.sync();  // the counts are there, and all keys are in registers
        int ahead = 0;
        for (int d = threadIdx.x; d < bins; d += kSortThreads) {  // (a digit a thread at most)
            int all = 0;
            for (int b = 0; b < blocks; ++b) {
                const int c = mine_of.ok(d) ? *cluster.map_shared_rank(mine_of.p + d, b) : 0;
                all += c;
                if (b < rank_in) ahead += c;
            }
            base.set(d, all);
        }
        __syncthreads();
        exclusive_scan(base, bins, tmp);
        if ((int)threadIdx.x < bins) base.set(threadIdx.x, base.get(threadIdx.x) + ahead);
        __syncthreads();
#pragma unroll
        for (int r = 0; r < R; ++r) {
            if (first + r * 32 >= here) continue;
            const int d = (key[r] >> shift) & (bins - 1);
            const int to = base.get(d) + mine.get(d) + rank[r], b = to / kTile, at = to - b * kTile;
            if (placed.ok(at) && b < blocks) *cluster.map_shared_rank(placed.p + at, b) = make_uint2(key[r], token[r]);
        }
        cluster.sync();  // everything is in its place, and no block's counts are read any more
        if (pass + 1 == passes) break;
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int i = first + r * 32;
            if (i >= here) continue;
            const uint2 y = placed.get(i);
            key[r] = y.x, token[r] = y.y;
        }
    }
    for (int i = threadIdx.x; i < here; i += kSortThreads) {
        const int64_t to = (int64_t)rank_in * kTile + i;
        const uint2 y = placed.get(i);
        if (BMMC_WR_OK(keys + to, 4)) keys[to] = y.x;
        if (BMMC_WR_OK(order + to, 4)) order[to] = y.y;
    }
}

// ---- the sums ------------------------------------------------------------------

// A chunk is some places (kChunk at most) of the sorted tokens.  A run of equal ids that
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

// Where sums go.
struct SumTo {
    char* out;
    int64_t stride;  // bytes
    int64_t vocab;
    float scale;
    int length, accumulate;
    float* partial;
    int partial_stride;
};

// v (added to what is there) to element p.
template <class O>
__device__ __forceinline__ void put_one(O* p, float v, bool accumulate) {
    if (!BMMC_WR_OK(p, sizeof(O))) return;
    *p = from_f32<O>(accumulate && BMMC_RD_OK(p, sizeof(O)) ? v + to_f32(*p) : v);
}

// The same to W elements, in words.
template <class O, int W>
__device__ __forceinline__ void put_words(const float (&v)[W], O* p, bool accumulate) {
    constexpr int P = 16 / sizeof(O) < W ? 16 / sizeof(O) : W;
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
}

// Bound by HBM: 32768 rows of 4096 bf16 66 us under the profiler, 338 MB, 75 % of the
// copy rate; what is missing is the end of a chunk (its last run may be as long
// again) and the blocks' start.  Chunks of 16 instead of 32: the whole gradient 273
// us instead of 266; 128 threads a block 265; four rows ahead instead of eight 265.
// In small calls chunks of 8, so that more blocks have some.
//
// A block adds the runs of a chunk, a thread a word of their rows.  Rows that
// are not made of words of 16 bytes (WORDS false) are cut out of two words each;
// their sums are exchanged in shared memory, so that a warp writes neighbouring
// elements (32768 rows of 4095 bf16 into 32768: 168 us, of 4096 116).
template <class T, class O, int W, bool WORDS>
__global__ void __launch_bounds__(kSumThreads) sum_rows_kernel(const char* __restrict__ grad, int64_t grad_stride,
                                                               const uint32_t* keys, const uint32_t* order, int64_t n,
                                                               int chunk, const SumTo o BMMC_SPANS_PARAM) {
    __shared__ int s_key[2 * kChunk + 1], s_token[2 * kChunk];
    __shared__ float s_sum[WORDS ? 1 : kSumThreads * W];
    BMMC_SPANS_ENTER(s_key, sizeof(s_key), s_token, sizeof(s_token), s_sum, sizeof(s_sum));
    const Slots<int> ids(s_key, 2 * kChunk + 1);
    const Slots<int> tokens(s_token, 2 * kChunk);
    const Slots<float> sums(s_sum, WORDS ? 1 : kSumThreads * W);
    cudaTriggerProgrammaticLaunchCompletion();  // the join waits for the sums by itself
    cudaGridDependencySynchronize();
    const Runs runs{keys, n};
    const int64_t lo = (int64_t)blockIdx.x * chunk;
    for (int i = threadIdx.x; i <= 2 * chunk; i += blockDim.x) {
        ids.set(i, (int)runs.key(lo + i));
        if (i < 2 * chunk) tokens.set(i, lo + i < n && BMMC_RD_OK(order + lo + i, 4) ? (int)order[lo + i] : 0);
    }
    const int64_t before = runs.key(lo - 1), far_before = runs.key(lo - chunk - 1);
    __syncthreads();
    const int here = (int)min((int64_t)chunk, n - lo), w = blockIdx.y * blockDim.x + threadIdx.x;
    if ((w - (WORDS ? 0 : (int)(threadIdx.x & 31))) * W >= o.length) return;  // (the lanes of an exchange stay together)
    const Walk<T, W, !WORDS> walk(o.length, nullptr);
    const bool mine = w * W < o.length;
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
    if (begin < here && first_part < here && ids.get(here) == last) {
        if (here == chunk && ids.get(2 * chunk) == last) last_part = true;
        else
            while (end < 2 * chunk && ids.get(end) == last) ++end;
    }
    float sum[W] = {};
    int id = ids.get(begin < here ? begin : 0);
    const auto put_out = [&](bool part, int which) {
        if (id >= 0 && id < o.vocab) {
            if (part) {
                float* const to = o.partial + ((int64_t)blockIdx.x * 2 + which) * o.partial_stride + w * W;
                if (mine) put_words<float, W>(sum, to, false);
            } else {
                O* const row = reinterpret_cast<O*>(o.out + (int64_t)id * o.stride);
#pragma unroll
                for (int i = 0; i < W; ++i) sum[i] *= o.scale;
                if constexpr (WORDS) {
                    put_words<O, W>(sum, row + w * W, o.accumulate);
                } else {
                    const int lane = threadIdx.x & 31, warp = threadIdx.x - lane, at = (w - lane) * W;
                    __syncwarp();
#pragma unroll
                    for (int i = 0; i < W; ++i) sums.set(threadIdx.x * W + (i ^ (lane / (32 / W) & (W - 1))), sum[i]);
                    __syncwarp();
#pragma unroll
                    for (int i = 0; i < W; ++i) {
                        const int e = i * 32 + lane, l = e / W;  // element e of the warp's, which lane l has
                        if (at + e < o.length)
                            put_one(row + at + e, sums.get((warp + l) * W + (e % W ^ (l / (32 / W) & (W - 1)))), o.accumulate);
                    }
                }
            }
        }
#pragma unroll
        for (int i = 0; i < W; ++i) sum[i] = 0.0f;
    };
    for (int at = begin; at < end; at += kSumAhead) {
        typename Walk<T, W, !WORDS>::Fetch f[kSumAhead];
#pragma unroll
        for (int u = 0; u < kSumAhead; ++u) {
            const bool want = at + u < end && ids.get(at + u) < o.vocab;
            walk.fetch(f[u], want && mine, grad + (int64_t)(want ? tokens.get(at + u) : 0) * grad_stride, w);
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

// Joins the parts of the long runs: a block looks at 32 chunks for runs that
// start there, and takes 128 columns of each: its warps add every eighth part,
// then the eight sums are added in order.  However long a run, a block for 128 columns
// has it alone: the gradient of 100003 rows of 1280 bf16 into 131072 takes 138 us with ids
// as frequent as words, 227 where one id is half of them, and 287 where all are one;
// of 1048576 rows 774, 1675 and 2660.
template <class O>
__global__ void __launch_bounds__(256) join_parts_kernel(const uint32_t* keys, int64_t n, int chunk,
                                                         const SumTo o BMMC_SPANS_PARAM) {
    __shared__ float s_sum[8 * 128];
    BMMC_SPANS_ENTER(s_sum, sizeof(s_sum));
    const Slots<float> sums(s_sum, 8 * 128);
    const Runs runs{keys, n};
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    cudaGridDependencySynchronize();
    const int64_t c0 = (int64_t)blockIdx.x * 32;
    const int64_t lo_of = (c0 + lane) * chunk, hi_of = lo_of + chunk, id_of = runs.key(hi_of - 1);
    const bool starts = id_of >= 0 && id_of < o.vocab && runs.key(hi_of) == id_of && runs.key(hi_of + chunk) == id_of &&
                        runs.key(lo_of - 1) != id_of;
    for (unsigned owners = __ballot_sync(~0u, starts); owners; owners &= owners - 1) {
        const int64_t c = c0 + __ffs(owners) - 1, id = runs.key((c + 1) * chunk - 1);
        int64_t parts = 1;  // chunks of the run
        for (bool all = true; all;) {
            const unsigned more = __ballot_sync(~0u, runs.key((c + parts + lane) * chunk) == id);
            all = more == ~0u;
            parts += all ? 32 : __ffs(~more) - 1;
        }
        const float* const from = o.partial + (c * 2) * o.partial_stride;  // part 1 of the first chunk, part 0 of the others
        for (int first = blockIdx.y * 128; first < o.length; first += gridDim.y * 128) {
            float4 sum = make_float4(0, 0, 0, 0);
            const int col = first + lane * 4;
#pragma unroll 4
            for (int64_t k = warp; k < parts; k += 8) {
                const float* const p = from + (k * 2 + (k == 0)) * o.partial_stride + col;
                const float4 v = col < o.partial_stride && BMMC_RD_OK(p, 16) ? __ldcg(reinterpret_cast<const float4*>(p))
                                                                            : make_float4(0, 0, 0, 0);
                sum.x += v.x, sum.y += v.y, sum.z += v.z, sum.w += v.w;
            }
            const float v4[4] = {sum.x, sum.y, sum.z, sum.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) sums.set(warp * 128 + lane * 4 + i, v4[i]);
            __syncthreads();
            const int at = first + threadIdx.x;
            if (threadIdx.x < 128 && at < o.length) {
                float v = 0.0f;
                for (int g = 0; g < 8; ++g) v += sums.get(g * 128 + threadIdx.x);
                put_one(reinterpret_cast<O*>(o.out + id * o.stride) + at, v * o.scale, o.accumulate);
            }
            __syncthreads();
        }
    }
}

// Rows of zeros.  Rows without gaps are one long one, whose words of 16 bytes are
// dealt out to short blocks; rows with gaps have a warp each.  The grid starts
// beside the sort; its last block waits for that, so that what comes next on the
// stream may count on both.  131072 rows of 4096 bf16 139 us, 7.7 TB/s of stores; the
// whole gradient took 220 us this way, 246 with a wave of blocks that stay (four on an SM: 270)
// and 250 with bulk copies of zeros from shared memory.
constexpr int kClearWords = 4;  // of a thread

template <class T>
__global__ void __launch_bounds__(256) clear_rows_kernel(char* __restrict__ out, int64_t out_stride, int64_t rows,
                                                         int64_t row_bytes BMMC_SPANS_PARAM) {
    BMMC_SPANS_ENTER_GLOBAL();
    cudaTriggerProgrammaticLaunchCompletion();
    const auto head_of = [&](const char* row) { return min((int64_t)(-reinterpret_cast<uintptr_t>(row) & 15u), row_bytes); };
    // the elements ahead of the first word and behind the last one
    const auto ends = [&](char* row, int at, int step) {
        const int64_t head = head_of(row), tail = head + (row_bytes - head) / 16 * 16;
        for (int64_t i = at; i < (head + row_bytes - tail) / (int64_t)sizeof(T); i += step) {
            T* const e = reinterpret_cast<T*>(row + (i * (int64_t)sizeof(T) < head ? 0 : tail - head)) + i;
            if (BMMC_WR_OK(e, sizeof(T))) *e = T{};
        }
    };
    if (rows == 1) {
        const int64_t words = (row_bytes - head_of(out)) / 16;
        uint4* const w = reinterpret_cast<uint4*>(out + head_of(out));
        const int64_t i0 = (int64_t)blockIdx.x * blockDim.x * kClearWords + threadIdx.x;
#pragma unroll
        for (int k = 0; k < kClearWords; ++k) {
            const int64_t i = i0 + k * blockDim.x;
            if (i < words && BMMC_WR_OK(w + i, 16)) w[i] = uint4{};
        }
        if (blockIdx.x == 0) ends(out, threadIdx.x, blockDim.x);
    } else {
        const int lane = threadIdx.x & 31;
        const int64_t r = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) >> 5;
        if (r < rows) {
            char* const row = out + r * out_stride;
            uint4* const w = reinterpret_cast<uint4*>(row + head_of(row));
            for (int64_t i = lane; i < (row_bytes - head_of(row)) / 16; i += 32)
                if (BMMC_WR_OK(w + i, 16)) w[i] = uint4{};
            ends(row, lane, 32);
        }
    }
    if (blockIdx.x + 1 == gridDim.x) cudaGridDependencySynchronize();
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

// Keys a thread takes where the sort is one block, or else one cluster; 0: it is
// neither.  Eight blocks of four keys a thread end at 32768 tokens, which take 19 us
// (as four blocks of eight keys a thread 35); 100003 in launches of their own take 28.
// Eight blocks of eight keys, up to 65536, were not timed.
int cluster_rounds(int64_t n) {
    for (int r : {1, 2})
        if (n <= (int64_t)kSortThreads * r) return r;
    for (int r : {1, 2, 4})
        if (n <= (int64_t)kSortCluster * kSortThreads * r) return r;
    return 0;
}

// Places of a chunk: fewer where there are few tokens, so that more blocks have
// some.
int chunk_of(int64_t n, int64_t hidden) { return n * ((hidden + 1023) / 1024) <= kSms * 256 ? 8 : kChunk; }

// The workspace: the sorted keys and tokens (both twice where the sort is not one
// cluster, with the blocks' counts), and two sums a chunk.
struct Workspace {
    int64_t array, counts, partial;  // bytes
    int arrays, chunk, partial_stride;  // partial_stride: floats
    int64_t bytes() const { return arrays * array + counts + partial; }
};

Workspace workspace_of(int64_t n, int64_t vocab, int64_t hidden) {
    Workspace w;
    const bool cluster = cluster_rounds(n);
    w.array = up16(n * 4);
    w.arrays = cluster ? 2 : 4;
    const SortShape s = sort_shape(n, vocab);
    w.counts = cluster ? 0 : up16((int64_t)s.blocks * (4 << s.digit));
    w.partial_stride = (int)((hidden + 7) & ~(int64_t)7);
    w.chunk = chunk_of(n, hidden);
    const int64_t chunks = (n + w.chunk - 1) / w.chunk;
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
        cudaLaunchAttribute early{};
        early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
        early.val.programmaticStreamSerializationAllowed = 1;
        const auto run = [&](auto in) {
            using In = decltype(in);
            constexpr auto place = digit_place_kernel<Id, In::kFirst>;
            bmmc_status status = allow_smem<place>(smem);
            if (status != BMMC_OK) return status;
            // (the first one waits for the work before the call, as any launch does)
            status = launch(digit_count_kernel<Id, In::kFirst>, dim3(s.blocks), dim3(kSortThreads), 0, st, pass ? &early : nullptr,
                            in, n, shift, s.digit, s.per_block, counts BMMC_SPANS_ARG(spans));
            if (status != BMMC_OK) return status;
            return launch(place, dim3(s.blocks), dim3(kSortThreads), smem, st, &early, in, n, shift, s.digit, s.per_block,
                          (const int*)counts, keys[to], order[to] BMMC_SPANS_ARG(spans));
        };
        const bmmc_status status = pass == 0 ? run(Sorted<Id, true>{ids, nullptr, nullptr, vocab})
                                             : run(Sorted<Id, false>{nullptr, keys[from], order[from], vocab});
        if (status != BMMC_OK) return status;
    }
    return BMMC_OK;
}

// The sort as one cluster.
template <class Id, int R>
bmmc_status sort_together(const SortShape& s, const Id* ids, int64_t n, int64_t vocab, uint32_t* keys, uint32_t* order,
                          const chk::Spans& spans, cudaStream_t st) {
    (void)spans;
    const int tile = kSortThreads * R, blocks = (int)((n + tile - 1) / tile);
    const size_t smem = ((2 << s.digit) + 32 + (kSortThreads / 64 << s.digit) + 2 * tile) * 4;
    constexpr auto kernel = sort_cluster_kernel<Id, R>;
    const bmmc_status allowed = allow_smem<kernel>(smem);
    if (allowed != BMMC_OK) return allowed;
    cudaLaunchAttribute together{};
    together.id = cudaLaunchAttributeClusterDimension;
    together.val.clusterDim.x = blocks;
    together.val.clusterDim.y = together.val.clusterDim.z = 1;
    return launch(kernel, dim3(blocks), dim3(kSortThreads), smem, st, &together, ids, (int)n, vocab, s.passes, s.digit, keys,
                  order BMMC_SPANS_ARG(spans));
}

}  // namespace

extern "C" {

// Words of a row from which on a thread of a large lookup takes four (65536 rows
// of 25 words: 7.2 us, one a thread 8.4; of 9 words no difference).
constexpr int kFourWords = 16;

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
        const auto go = [&](auto id, auto each) {
            using Id = decltype(id);
            constexpr int K = decltype(each)::value;
            const int each_words = (way.words + K - 1) / K;
            Cover c = cover(tokens, each_words, 128);
            if (tokens * way.words > kFewWords && each_words < 96) {  // short rows: side by side, without idle lanes
                c.block = dim3(each_words, 256 / each_words);
                c.grid = dim3((unsigned)((tokens + c.block.y - 1) / c.block.y));
            }
            s = launch(lookup_kernel<T, W, A, K, Id>, c.grid, c.block, 0, static_cast<cudaStream_t>(stream), nullptr,
                       static_cast<const char*>(table), table_stride * es, vocab, static_cast<const Id*>(ids), tokens,
                       (int)hidden, scale, static_cast<char*>(out), out_stride * es BMMC_SPANS_ARG(spans));
        };
        const auto with = [&](auto id) {
            if (tokens * way.words > kFewWords && way.words >= kFourWords) go(id, std::integral_constant<int, 4>{});
            else go(id, std::integral_constant<int, 1>{});
        };
        id_bytes == 4 ? with(int32_t{}) : with(int64_t{});
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
    cudaLaunchAttribute early{};
    early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    early.val.programmaticStreamSerializationAllowed = 1;
    const auto clear = [&](cudaLaunchAttribute* attribute) {
        const bool flat = vocab == 1 || out_stride == hidden;
        const int64_t rows = flat ? 1 : vocab, bytes = (flat ? vocab : 1) * hidden * os;
        const int64_t blocks = flat ? bytes / (256 * kClearWords * 16) + 1 : (vocab + 7) / 8;
        const auto go = [&](auto kernel) {
            return launch(kernel, dim3((unsigned)blocks), dim3(256), 0, st, attribute, static_cast<char*>(out), out_stride * os,
                          rows, bytes BMMC_SPANS_ARG(spans));
        };
        return os == 4 ? go(clear_rows_kernel<uint32_t>) : go(clear_rows_kernel<uint16_t>);
    };
    if (!tokens) return clear(nullptr);
    char* const at = static_cast<char*>(workspace);
    const auto array = [&](int i) { return reinterpret_cast<uint32_t*>(at + i * w.array); };
    int* const counts = reinterpret_cast<int*>(at + w.arrays * w.array);
    float* const partial = reinterpret_cast<float*>(at + w.arrays * w.array + w.counts);
    const SortShape shape = sort_shape(tokens, vocab);
    const uint32_t *key = array(0), *token = array(1);
    const auto sorted = [&](const auto* names) {
        using Id = std::remove_cv_t<std::remove_pointer_t<decltype(names)>>;
        switch (cluster_rounds(tokens)) {
            case 1: return sort_together<Id, 1>(shape, names, tokens, vocab, array(0), array(1), spans, st);
            case 4: return sort_together<Id, 4>(shape, names, tokens, vocab, array(0), array(1), spans, st);
            case 2: return sort_together<Id, 2>(shape, names, tokens, vocab, array(0), array(1), spans, st);
        }
        uint32_t *keys[2] = {array(0), array(2)}, *order[2] = {array(1), array(3)};
        key = keys[(shape.passes - 1) & 1], token = order[(shape.passes - 1) & 1];
        return sort_tokens(shape, names, tokens, vocab, keys, order, counts, spans, st);
    };
    s = id_bytes == 4 ? sorted(static_cast<const int32_t*>(ids)) : sorted(static_cast<const int64_t*>(ids));
    if (s == BMMC_OK && !accumulate) s = clear(&early);  // beside the sort, or the last of its kernels
    if (s != BMMC_OK) return s;
    const int64_t chunks = (tokens + w.chunk - 1) / w.chunk;
    const bool words = word_bytes(2, {(uint64_t)(uintptr_t)grad, (uint64_t)(uintptr_t)out, (uint64_t)(grad_stride * es),
                                      (uint64_t)(out_stride * os), (uint64_t)(hidden * es), (uint64_t)(hidden * os)}) == 16;
    const SumTo o{static_cast<char*>(out), out_stride * os, vocab, scale, (int)hidden, accumulate, partial, w.partial_stride};
    const auto sum = [&](auto kernel, int W) {
        const int row = (int)((hidden + W - 1) / W), parts = (row + kSumThreads - 1) / kSumThreads;
        const int x = ((row + parts - 1) / parts + 31) / 32 * 32;
        return launch(kernel, dim3((unsigned)chunks, (unsigned)((row + x - 1) / x)), dim3(x), 0, st, &early,
                      static_cast<const char*>(grad), grad_stride * es, key, token, tokens, w.chunk, o BMMC_SPANS_ARG(spans));
    };
    const auto typed = [&](auto t, auto to) {
        using T = decltype(t);
        using O = decltype(to);
        constexpr int W = 16 / sizeof(T);
        return words ? sum(sum_rows_kernel<T, O, W, true>, W) : sum(sum_rows_kernel<T, O, W, false>, W);
    };
    if (type == BMMC_F32) s = typed(float{}, float{});
    else if (type == BMMC_F16) s = out_type == BMMC_F32 ? typed(__half{}, float{}) : typed(__half{}, __half{});
    else s = out_type == BMMC_F32 ? typed(__nv_bfloat16{}, float{}) : typed(__nv_bfloat16{}, __nv_bfloat16{});
    if (s != BMMC_OK || chunks < 3) return s;
    const dim3 grid((unsigned)((chunks + 31) / 32), (unsigned)std::min<int64_t>((hidden + 127) / 128, kMostParts));
    const auto join = [&](auto kernel) {
        return launch(kernel, grid, dim3(256), 0, st, &early, key, tokens, w.chunk, o BMMC_SPANS_ARG(spans));
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
