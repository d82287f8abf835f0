// A router's balance loss with the number of choices of each expert, and its
// gradient: expert_balance and expert_balance_backward (declared in
// include/bmmc.h).
//
// With p[t] the softmax of token t's logits, c[e] the routed choices of expert
// e, C their sum, n the tokens that have one and f[e] = c[e] / C:
//   loss = E * sum over e of f[e] * (sum over those tokens of p[t][e]) / n,
//   d loss / d logit[t][e] = E / n * p[t][e] * (f[e] - sum over j of f[j] * p[t][j]),
// as the counts do not depend on the logits.
#include <cooperative_groups.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "../../include/bmmc.h"
#define BMMC_CHK_FILE 9  // site tag of this file in bounds-checked builds
#include "bounds.cuh"
#include "token_moves.hpp"
#include "token_words.cuh"

using namespace bmmc;

namespace {

#ifdef BMMC_BOUNDS_CHECK
__device__ __forceinline__ uint32_t chk_dynamic_bytes() { return chk::dyn_smem_bytes(); }
#endif

constexpr int kMaxExperts = 4096;
constexpr int kHeldExperts = 1024;  // up to here a row's logits are held in registers
constexpr int kHeldThreads = 1024;
// Threads of a block by the logits of a lane, whose registers they are.
constexpr int held_threads(int each) { return each == 8 ? 1024 : each == 16 ? 512 : 256; }
constexpr int kCluster = 8;
constexpr int kOneCluster = 4;       // rows a thread of one cluster takes, at most

// How rows are dealt out: `lanes` lanes (a power of two) hold one row, N
// logits each.
struct Router {
    const char* logits;
    int64_t stride;  // bytes
    const char* ids;
    int64_t tokens;
    int id_bytes, choices, experts, lanes;
};

// A lane's logits of a row, in words of 16 bytes (WORDS: the rows are made of
// those) or one by one.  Logits past the last expert are -inf.
template <class T, int N, bool WORDS>
struct Logits {
    static constexpr int W = WORDS ? 16 / sizeof(T) : 1, kPacks = N / W;
    Pack<T, W> pack[kPacks];
    // the first expert of pack j
    static __device__ __forceinline__ int expert(int j, int lanes, int in) { return (j * lanes + in) * W; }
    __device__ __forceinline__ void load(const char* row, int experts, int lanes, int in) {
#pragma unroll
        for (int j = 0; j < kPacks; ++j) {
            const int e = expert(j, lanes, in);
            if (e < experts && BMMC_RD_OK(row + e * sizeof(T), W * sizeof(T))) pack[j].load(row + e * sizeof(T));
            else
#pragma unroll
                for (int i = 0; i < W; ++i) pack[j].e[i] = from_f32<T>(-INFINITY);
        }
    }
    __device__ __forceinline__ float get(int i) const { return pack[i / W].get(i % W); }
};

// Over the lanes of a row; FULL: all 32 of the warp.  (The largest of a warp's
// numbers is one instruction, and one that is NaN does not count.)
template <bool FULL>
__device__ __forceinline__ float group_max(float v, int lanes) {
    if constexpr (FULL) {
        // (volatile: all of the lanes meet in it, wherever the compiler puts what surrounds it)
        asm volatile("redux.sync.max.f32 %0, %0, 0xffffffff;" : "+f"(v));
    } else {
        for (int d = lanes >> 1; d; d >>= 1) v = fmaxf(v, __shfl_xor_sync(~0u, v, d));
    }
    return v;
}
template <bool FULL>
__device__ __forceinline__ float group_sum(float v, int lanes) {
    if constexpr (FULL) {
#pragma unroll
        for (int d = 16; d; d >>= 1) v += __shfl_xor_sync(~0u, v, d);
    } else {
        for (int d = lanes >> 1; d; d >>= 1) v += __shfl_xor_sync(~0u, v, d);
    }
    return v;
}

// exp(d), d <= 0, by the instruction for powers of two, 2^e with e the rounded
// d * log2(e), times 1 + r where r = d - e * ln(2) is what the rounding left out
// (below 2^-17, so that its square does not count).  Without it the result is off by
// |d| * 2^-24 of itself, which the rounding of a difference of logits is worth only
// where these have 32 bits: differences of 16-bit logits are mostly exact.  With it, by
// the instruction's 2 ulp, a rounding and |d| * 2^-28 for ln(2) in 32 bits; below
// 2^-126 it is zero.  Far differences (-inf, whose r would be NaN) are cut off at -200,
// where it is zero anyway; NaN stays.  65521 x 256 22.2 us without r, 22.8 with it, 131072 x
// 128 of 16 bits 19.6 and 20.8; expf in its place is as exact, takes 22.1 and 26.5, and
// the gradients 30.7 and 26.3 instead of 25.4 and 24.7.
__device__ __forceinline__ float power(float d) {
    float y;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(d), "f"(-200.0f));
    const float e = d * 1.44269504088896341f;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(e));
    return fmaf(y, fmaf(e, -0.693147180559945309f, d), y);
}

// One over the sum of a row's powers: the instruction's value, within 1 ulp, and one
// step of Newton's iteration, which leaves the rounding; zero for a row whose
// logits are all -inf.
__device__ __forceinline__ float over_sum(float sum) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(sum));
    y = fmaf(y, fmaf(-sum, y, 1.0f), y);
    return sum == 0.0f ? 0.0f : y;
}

// v[i] = exp(logit - largest), and one over their sum.  A row whose logits are
// all -inf has shares of zero: nothing is subtracted from it.
template <bool FULL, class L, int N>
__device__ __forceinline__ float softmax_of(const L& row, float (&v)[N], int lanes) {
    float m = -INFINITY, sum = 0.0f;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        v[i] = row.get(i);
        m = fmaxf(m, v[i]);
    }
    m = group_max<FULL>(m, lanes);
    if (m == -INFINITY) m = 0.0f;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        v[i] = power(v[i] - m);
        sum += v[i];
    }
    sum = group_sum<FULL>(sum, lanes);
    return over_sum(sum);
}

// Which of the `n` tokens from t0 on have a routed choice, a thread a token, as
// bits; with COUNT each expert's choices are counted.  Apart from the walk over
// the rows, whose warps spend 30 instructions less on each that way.
template <class Id, bool COUNT>
__device__ __forceinline__ bool look_at(const Router& r, int64_t t, Slots<int> hist) {
    bool any = false;
    const Id* const ids = reinterpret_cast<const Id*>(r.ids) + t * r.choices;
#pragma unroll 4
    for (int k = 0; k < r.choices; ++k) {
        const Id id = BMMC_RD_OK(ids + k, sizeof(Id)) ? ids[k] : (Id)-1;
        const bool is = id >= 0 && id < (Id)r.experts;
        if (COUNT && is) hist.add((int)id, 1);
        any |= is;
    }
    return any;
}

template <bool COUNT>
__device__ __forceinline__ void look_at_choices(const Router& r, int64_t t0, int n, Slots<unsigned> there, Slots<int> hist) {
    bool any = false;
    if ((int)threadIdx.x < n)
        any = r.id_bytes == 4 ? look_at<int32_t, COUNT>(r, t0 + threadIdx.x, hist) : look_at<int64_t, COUNT>(r, t0 + threadIdx.x, hist);
    const unsigned all = __ballot_sync(~0u, any);
    if ((threadIdx.x & 31) == 0) there.set(threadIdx.x >> 5, all);
    if (COUNT && (threadIdx.x & 31) == 0 && all) hist.add(r.experts, __popc(all));
}

__device__ __forceinline__ bool is_there(Slots<unsigned> there, int i) { return there.get(i >> 5) >> (i & 31) & 1; }

// A warp's walk over the rows of a tile, `rows` at a time.
struct Walker {
    int i, first, step, n;  // the lane's row in the tile, the warp's first one
    int64_t hop;            // bytes to the next
    const char* row;
    int in;                 // the lane's number in the row
    __device__ __forceinline__ Walker(const Router& r, int64_t t0, int n_) : n(n_) {
        const int lane = threadIdx.x & 31, rows = 32 / r.lanes;
        in = lane & (r.lanes - 1);
        step = (blockDim.x >> 5) * rows;
        first = (threadIdx.x >> 5) * rows;
        i = first + lane / r.lanes;
        row = r.logits + (t0 + i) * r.stride;
        hop = step * r.stride;
    }
    __device__ __forceinline__ bool more() const { return first < n; }
    __device__ __forceinline__ bool here() const { return i < n; }
    __device__ __forceinline__ void next() { i += step, first += step, row += hop; }
};

// The loss from the experts' sums of shares and counts, by a block: each thread
// has its part of the sum of count * sum, of the counts, and of the tokens
// (one thread has these).
__device__ __forceinline__ void finish_loss(float dot, int choices, int tokens, int experts, float* loss, Slots<float> dots,
                                            Slots<int> all, Slots<int> there) {
    for (int d = 16; d; d >>= 1) dot += __shfl_xor_sync(~0u, dot, d);
    choices = __reduce_add_sync(~0u, choices);
    tokens = __reduce_add_sync(~0u, tokens);
    if ((threadIdx.x & 31) == 0) {
        const int warp = threadIdx.x >> 5;
        dots.set(warp, dot), all.set(warp, choices), there.set(warp, tokens);
    }
    __syncthreads();
    if (threadIdx.x) return;
    dot = 0.0f, choices = 0, tokens = 0;
    for (int w = 0; w < (int)blockDim.x >> 5; ++w) dot += dots.get(w), choices += all.get(w), tokens += there.get(w);
    if (BMMC_WR_OK(loss, 4)) *loss = tokens ? dot / (float)choices * ((float)experts / (float)tokens) : 0.0f;
}

// Each block's sums of the shares of its tokens, and its counts.  In a small
// call the blocks are one cluster, whose first joins them; in others each leaves
// a row of `sums` and `counts` (loss NULL).
//
// The bytes could be moved in 10.1 us at 65521 tokens of 256 experts in 32 bits;
// the two launches take 22.7.  A row is about 150 instructions of a warp (72 for
// its 256 logits, the rest exchanges, loads and the walk), 8.5 us of issue slots
// in all; the rest is latency: a block's start and its choices, the chain load -
// largest - powers - sum - shares of 14 rows a warp, the block's own sum over its
// warps, and the join (4 us).  One block of 32 warps an SM was taken for the join's
// sake (before the powers carried their remainder 22.3 us; blocks of 512 threads 23.8,
// of 256 27.6; two rows ahead instead of one 22.7, and with 512 experts 35.9 instead of
// 38.4).  A row read three times from memory by a warp, its sums in shared memory, took
// 130 us.  131072 tokens of 61 experts of 16 bits 15.2 us, of 8 7.5; 509 tokens of 8, one
// block, 3.6.
template <class T, int N, bool WORDS, bool FULL>
__global__ void __launch_bounds__(held_threads(N)) balance_held_kernel(const Router r, int64_t per_block,
                                                                       float* __restrict__ sums, int* __restrict__ counts,
                                                                       float* __restrict__ loss BMMC_SPANS_PARAM) {
    extern __shared__ int s_mem[];
    __shared__ float s_dot[32];
    __shared__ int s_all[32], s_there[32];
    __shared__ unsigned s_routed[32];
    BMMC_SPANS_ENTER(s_mem, chk_dynamic_bytes(), s_dot, sizeof(s_dot), s_all, sizeof(s_all), s_there, sizeof(s_there), s_routed,
                     sizeof(s_routed));
    const int E = r.experts, warps = blockDim.x >> 5, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const Slots<int> mem(s_mem, (warps + 1) * E + 1), hist = mem.part(0, E + 1);  // counts; [E]: tokens
    const Slots<float> all(reinterpret_cast<float*>(s_mem + E + 1), warps * E);    // each warp's sums
    cudaTriggerProgrammaticLaunchCompletion();
    const Slots<float> dots(s_dot, 32);
    const Slots<int> alls(s_all, 32);
    const Slots<int> theres(s_there, 32);
    const Slots<unsigned> routed(s_routed, 32);
    using L = Logits<T, N, WORDS>;
    for (int e = threadIdx.x; e <= E; e += blockDim.x) hist.set(e, 0);
    float acc[N] = {};
    const int64_t lo = (int64_t)blockIdx.x * per_block, hi = min(r.tokens, lo + per_block);
    for (int64_t t0 = lo; t0 < hi; t0 += blockDim.x) {
        Walker w(r, t0, (int)min((int64_t)blockDim.x, hi - t0));
        L next;
        next.load(w.row, w.here() ? E : 0, r.lanes, w.in);
        __syncthreads();
        look_at_choices<true>(r, t0, w.n, routed, hist);
        __syncthreads();
        while (w.more()) {
            const L row = next;
            const bool counts_in = w.here() && is_there(routed, w.i);
            w.next();
            next.load(w.row, w.here() ? E : 0, r.lanes, w.in);
            float v[N];
            const float over = softmax_of<FULL>(row, v, r.lanes);
            if (counts_in) {
#pragma unroll
                for (int i = 0; i < N; ++i) acc[i] = fmaf(v[i], over, acc[i]);
            }
        }
    }
    __syncthreads();
    const int in = lane & (r.lanes - 1);
    for (int d = r.lanes; d < 32; d <<= 1)
#pragma unroll
        for (int i = 0; i < N; ++i) acc[i] += __shfl_xor_sync(~0u, acc[i], d);
    if (lane < r.lanes) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int e = L::expert(i / L::W, r.lanes, in) + i % L::W;
            if (e < E) all.set(warp * E + e, acc[i]);
        }
    }
    __syncthreads();
    for (int e = threadIdx.x; e <= E; e += blockDim.x) {
        float sum = 0.0f;
        if (e < E) {
#pragma unroll 8
            for (int k = 0; k < warps; ++k) sum += all.get(k * E + e);
        }
        if (loss) {
            if (e < E) all.set(e, sum);
            continue;
        }
        const int64_t at = (int64_t)blockIdx.x * (E + 1) + e;
        if (BMMC_WR_OK(sums + at, 4)) sums[at] = sum;
        if (BMMC_WR_OK(counts + at, 4)) counts[at] = hist.get(e);
    }
    if (!loss) return;
    const auto cluster = cooperative_groups::this_cluster();
    if (gridDim.x > 1) cluster.sync();
    else __syncthreads();
    float dot = 0.0f;
    int choices = 0, there = 0;
    if (cluster.block_rank() == 0) {
        for (int e = threadIdx.x; e <= E; e += blockDim.x) {
            float sum = 0.0f;
            int count = 0;
            for (int b = 0; b < (int)gridDim.x; ++b) {
                if (e < E && all.ok(e)) sum += *cluster.map_shared_rank(all.p + e, b);
                if (hist.ok(e)) count += *cluster.map_shared_rank(hist.p + e, b);
            }
            if (BMMC_WR_OK(counts + e, 4)) counts[e] = count;
            if (e == E) there = count;
            else if (count) dot += sum * (float)count, choices += count;  // (an expert without choices has no part, whatever its sum)
        }
    }
    if (gridDim.x > 1) cluster.sync();  // no block leaves while its sums are read
    if (cluster.block_rank() == 0)
        finish_loss(dot, choices, there, E, loss, dots, alls, theres);
}

// More experts: by a warp a row, whose logits are read three times, the sums
// in shared memory.
constexpr int kThreads = 256, kWarps = kThreads / 32;

template <class T>
__device__ __forceinline__ float logit(const char* row, int e) {
    const T* const p = reinterpret_cast<const T*>(row) + e;
    return BMMC_RD_OK(p, sizeof(T)) ? to_f32(*p) : 0.0f;
}

// Whether a token has a routed choice, by a warp; with COUNT each expert's are
// counted.
template <bool COUNT>
__device__ __forceinline__ bool look_at_row(const Router& r, int64_t t, int lane, Slots<int> hist) {
    bool any = false;
    for (int k = lane; k < r.choices; k += 32) {
        const char* const at = r.ids + (t * r.choices + k) * r.id_bytes;
        if (!BMMC_RD_OK(at, r.id_bytes)) continue;
        const int64_t id = r.id_bytes == 4 ? (int64_t)*reinterpret_cast<const int32_t*>(at) : *reinterpret_cast<const int64_t*>(at);
        const bool is = id >= 0 && id < r.experts;
        if (COUNT && is) hist.add((int)id, 1);
        any |= is;
    }
    return __any_sync(~0u, any);
}

// What a row's softmax subtracts and multiplies by, by a warp.
template <class T>
__device__ __forceinline__ float long_softmax_of(const char* row, int experts, int lane, float* over) {
    float m = -INFINITY, sum = 0.0f;
    for (int e = lane; e < experts; e += 32) m = fmaxf(m, logit<T>(row, e));
    m = group_max<true>(m, 32);
    if (m == -INFINITY) m = 0.0f;
    for (int e = lane; e < experts; e += 32) sum += power(logit<T>(row, e) - m);
    sum = group_sum<true>(sum, 32);
    *over = over_sum(sum);
    return m;
}

template <class T>
__global__ void __launch_bounds__(kThreads) balance_long_kernel(const Router r, float* __restrict__ sums,
                                                                int* __restrict__ counts BMMC_SPANS_PARAM) {
    extern __shared__ int s_mem[];
    BMMC_SPANS_ENTER(s_mem, chk_dynamic_bytes());
    const int E = r.experts, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const Slots<int> mem(s_mem, (kWarps + 1) * E + 1), hist = mem.part(0, E + 1);
    const Slots<float> all(reinterpret_cast<float*>(s_mem + E + 1), kWarps * E);
    const Slots<float> mine = all.part(warp * E, E);
    cudaTriggerProgrammaticLaunchCompletion();
    for (int e = threadIdx.x; e <= E; e += kThreads) hist.set(e, 0);
    for (int e = lane; e < E; e += 32) mine.set(e, 0.0f);
    __syncthreads();
    for (int64_t t = (int64_t)blockIdx.x * kWarps + warp; t < r.tokens; t += (int64_t)gridDim.x * kWarps) {
        if (!look_at_row<true>(r, t, lane, hist)) continue;
        if (lane == 0) hist.add(E, 1);
        const char* const row = r.logits + t * r.stride;
        float over;
        const float m = long_softmax_of<T>(row, E, lane, &over);
        for (int e = lane; e < E; e += 32) mine.set(e, mine.get(e) + power(logit<T>(row, e) - m) * over);
    }
    __syncthreads();
    for (int e = threadIdx.x; e <= E; e += kThreads) {
        float sum = 0.0f;
        if (e < E)
            for (int w = 0; w < kWarps; ++w) sum += all.get(w * E + e);
        const int64_t at = (int64_t)blockIdx.x * (E + 1) + e;
        if (BMMC_WR_OK(sums + at, 4)) sums[at] = sum;
        if (BMMC_WR_OK(counts + at, 4)) counts[at] = hist.get(e);
    }
}

// The rows of sums and counts joined by one cluster: its blocks take every
// eighth row, in each of them a few threads an expert, and the first block adds
// what they have, in order.  The rows are still being written when this kernel
// starts: they are read by __ldcg, behind the wait.
__global__ void __launch_bounds__(1024) balance_join_kernel(const float* sums, const int* counts,
                                                            int rows, int experts, int parts, float* __restrict__ loss,
                                                            int* __restrict__ out_counts BMMC_SPANS_PARAM) {
    extern __shared__ int s_mem[];  // [parts][experts + 1] of each
    __shared__ float s_dot[32];
    __shared__ int s_all[32], s_there[32];
    BMMC_SPANS_ENTER(s_mem, chk_dynamic_bytes(), s_dot, sizeof(s_dot), s_all, sizeof(s_all), s_there, sizeof(s_there));
    const int width = experts + 1;
    const Slots<float> dots(s_dot, 32);
    const Slots<int> alls(s_all, 32);
    const Slots<int> theres(s_there, 32);
    const Slots<float> part_sums(reinterpret_cast<float*>(s_mem), parts * width);
    const Slots<int> part_counts(s_mem + parts * width, parts * width);
    const auto cluster = cooperative_groups::this_cluster();
    const int rank = (int)cluster.block_rank(), blocks = kCluster;
    cudaGridDependencySynchronize();
    for (int i = threadIdx.x; i < parts * width; i += 1024) {
        const int part = i / width, e = i - part * width;
        float sum = 0.0f;
        int count = 0;
#pragma unroll 4
        for (int b = part * blocks + rank; b < rows; b += parts * blocks) {
            const int64_t at = (int64_t)b * width + e;
            sum += BMMC_RD_OK(sums + at, 4) ? __ldcg(sums + at) : 0.0f;
            count += BMMC_RD_OK(counts + at, 4) ? __ldcg(counts + at) : 0;
        }
        part_sums.set(i, sum), part_counts.set(i, count);
    }
    __syncthreads();
    for (int e = threadIdx.x; e < width; e += 1024) {
        float sum = 0.0f;
        int count = 0;
        for (int k = 0; k < parts; ++k) sum += part_sums.get(k * width + e), count += part_counts.get(k * width + e);
        part_sums.set(e, sum), part_counts.set(e, count);
    }
    cluster.sync();
    float dot = 0.0f;
    int all = 0, there = 0;
    if (rank == 0) {
        for (int e = threadIdx.x; e < width; e += 1024) {
            float sum = 0.0f;
            int count = 0;
#pragma unroll
            for (int b = 0; b < kCluster; ++b) {
                if (part_sums.ok(e)) sum += *cluster.map_shared_rank(part_sums.p + e, b);
                if (part_counts.ok(e)) count += *cluster.map_shared_rank(part_counts.p + e, b);
            }
            if (BMMC_WR_OK(out_counts + e, 4)) out_counts[e] = count;
            if (e == experts) there = count;
            else if (count) dot += sum * (float)count, all += count;  // (an expert without choices has no part, whatever its sum)
        }
    }
    cluster.sync();  // no block leaves while its sums are read
    if (rank == 0)
        finish_loss(dot, all, there, experts, loss, dots, alls, theres);
}

// The counts' sum, by a block: all of its threads take part.
__device__ __forceinline__ int sum_of_counts(const int* counts, int experts, Slots<int> tmp) {
    int all = 0;
    for (int e = threadIdx.x; e < experts; e += blockDim.x) all += BMMC_RD_OK(counts + e, 4) ? counts[e] : 0;
    all = __reduce_add_sync(~0u, all);
    if ((threadIdx.x & 31) == 0) tmp.set(threadIdx.x >> 5, all);
    __syncthreads();
    all = 0;
    for (int w = 0; w < (int)blockDim.x >> 5; ++w) all += tmp.get(w);
    return all;
}

__device__ __forceinline__ float count_at(const int* counts, int e) { return BMMC_RD_OK(counts + e, 4) ? (float)counts[e] : 0.0f; }

// grad * E / n; 0 where no token has a routed choice.
__device__ __forceinline__ float factor_of(const float* grad, const int* counts, int experts) {
    const int n = BMMC_RD_OK(counts + experts, 4) ? counts[experts] : 0;
    return n ? (BMMC_RD_OK(grad, 4) ? *grad : 0.0f) * ((float)experts / (float)n) : 0.0f;
}

// As above, with the shares' weighted sum between and the gradient written: 65521
// tokens of 256 experts in 32 bits 25.4 us for 20.0 us of bytes (a wave of five
// blocks of 256 threads an SM; 1214 shorter blocks, which each start by reading the
// counts, took 0.2 us more).  131072 of 128 experts of 16 bits 24.6 (10.5): twice the
// logits for the bytes, and the exchanges of half a warp.
template <class T, int N, bool WORDS, bool FULL>
__global__ void __launch_bounds__(256) balance_backward_held_kernel(const float* __restrict__ grad, const Router r,
                                                                    int64_t per_block,
                                                                    const int* __restrict__ counts, char* __restrict__ out,
                                                                    int64_t out_stride BMMC_SPANS_PARAM) {
    __shared__ int s_all[8];
    __shared__ unsigned s_routed[8];
    BMMC_SPANS_ENTER(s_all, sizeof(s_all), s_routed, sizeof(s_routed));
    const Slots<unsigned> routed(s_routed, 8);
    const Slots<int> alls(s_all, 8);
    using L = Logits<T, N, WORDS>;
    const int E = r.experts;
    const int64_t lo = (int64_t)blockIdx.x * per_block, hi = min(r.tokens, lo + per_block);
    const int all = sum_of_counts(counts, E, alls);
    const float factor = factor_of(grad, counts, E), each = all ? 1.0f / (float)all : 0.0f;
    const int in = threadIdx.x & (r.lanes - 1);
    float f[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int e = L::expert(i / L::W, r.lanes, in) + i % L::W;
        f[i] = e < E ? count_at(counts, e) * each : 0.0f;
    }
    for (int64_t t0 = lo; t0 < hi; t0 += blockDim.x) {
        Walker w(r, t0, (int)min((int64_t)blockDim.x, hi - t0));
        L next;
        next.load(w.row, w.here() ? E : 0, r.lanes, w.in);
        __syncthreads();
        look_at_choices<false>(r, t0, w.n, routed, Slots<int>(nullptr, 0));
        __syncthreads();
        char* to = out + (t0 + w.i) * out_stride;
        const int64_t out_hop = w.step * out_stride;
        for (; w.more(); to += out_hop) {
            const L row = next;
            const bool here = w.here(), counts_in = here && is_there(routed, w.i);
            w.next();
            next.load(w.row, w.here() ? E : 0, r.lanes, w.in);
            float v[N], dot = 0.0f;
            const float over = softmax_of<FULL>(row, v, r.lanes);
#pragma unroll
            for (int i = 0; i < N; ++i) dot = fmaf(v[i], f[i], dot);
            dot = group_sum<FULL>(dot, r.lanes) * over;
            if (!here) continue;
            const float by = factor * over;
#pragma unroll
            for (int j = 0; j < L::kPacks; ++j) {
                const int e = L::expert(j, r.lanes, w.in);
                Pack<T, L::W> y;
                float g[L::W];
#pragma unroll
                for (int i = 0; i < L::W; ++i) g[i] = counts_in ? v[j * L::W + i] * by * (f[j * L::W + i] - dot) : 0.0f;
                y.set(g);
                if (e < E && BMMC_WR_OK(to + e * sizeof(T), sizeof(y))) y.store(to + e * sizeof(T));
            }
        }
    }
}

template <class T>
__global__ void __launch_bounds__(kThreads) balance_backward_long_kernel(const float* __restrict__ grad, const Router r,
                                                                         const int* __restrict__ counts,
                                                                         char* __restrict__ out, int64_t out_stride
                                                                             BMMC_SPANS_PARAM) {
    extern __shared__ int s_mem[];
    __shared__ int s_all[kWarps];
    BMMC_SPANS_ENTER(s_mem, chk_dynamic_bytes(), s_all, sizeof(s_all));
    const int E = r.experts, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const Slots<float> share(reinterpret_cast<float*>(s_mem), E);
    const Slots<int> alls(s_all, kWarps);
    const int all = sum_of_counts(counts, E, alls);
    const float factor = factor_of(grad, counts, E), each = all ? 1.0f / (float)all : 0.0f;
    for (int e = threadIdx.x; e < E; e += kThreads) share.set(e, count_at(counts, e) * each);
    __syncthreads();
    for (int64_t t = (int64_t)blockIdx.x * kWarps + warp; t < r.tokens; t += (int64_t)gridDim.x * kWarps) {
        T* const to = reinterpret_cast<T*>(out + t * out_stride);
        const char* const row = r.logits + t * r.stride;
        if (!look_at_row<false>(r, t, lane, Slots<int>(nullptr, 0))) {
            for (int e = lane; e < E; e += 32)
                if (BMMC_WR_OK(to + e, sizeof(T))) to[e] = from_f32<T>(0.0f);
            continue;
        }
        float over, dot = 0.0f;
        const float m = long_softmax_of<T>(row, E, lane, &over);
        for (int e = lane; e < E; e += 32) dot += power(logit<T>(row, e) - m) * share.get(e);
        dot = group_sum<true>(dot, 32) * over;
        for (int e = lane; e < E; e += 32)
            if (BMMC_WR_OK(to + e, sizeof(T)))
                to[e] = from_f32<T>(factor * over * power(logit<T>(row, e) - m) * (share.get(e) - dot));
    }
}

// ---- host ----------------------------------------------------------------------

// Lanes of a row whose logits are held, and logits of a lane.
struct Held {
    int lanes, each;
};

Held held(int experts) {
    Held h{1, 8};
    while (h.lanes < 32 && h.lanes * 8 < experts) h.lanes <<= 1;
    while (h.lanes * h.each < experts) h.each <<= 1;
    return h;
}

// Blocks of a call; where they are not one cluster, each leaves a row of sums.
struct Shape {
    int blocks, threads;
    bool together;
    int parts;  // threads of the join that share an expert
};

Shape shape_of(int64_t tokens, int experts) {
    Shape s{1, kThreads, false, std::min(16, std::max(1, 1024 / (experts + 1)))};
    if (experts > kHeldExperts) {
        const int64_t b = (tokens + kWarps - 1) / kWarps;
        s.blocks = (int)std::min<int64_t>(b < 1 ? 1 : b, 2 * kSms);
        return s;
    }
    const Held h = held(experts);
    s.threads = held_threads(h.each);
    const int64_t per = (int64_t)s.threads / h.lanes, b = (tokens + per - 1) / per;  // blocks of a row a thread
    s.together = b <= kOneCluster * kCluster;
    s.blocks = 1;
    if (b <= 1) s.threads = std::max(32, (int)(tokens * h.lanes + 31) / 32 * 32);
    else if (s.together)
        while (s.blocks < kCluster && s.blocks < b) s.blocks <<= 1;
    else
        s.blocks = (int)std::min<int64_t>(b, kSms * (kHeldThreads / s.threads));
    return s;
}

bmmc_status check_router(int64_t tokens, int choices, int experts, int id_bytes) {
    if (id_bytes != 4 && id_bytes != 8) return BMMC_ERR_UNSUPPORTED_ELEM;
    if (tokens < 0 || choices < 1 || choices > EXPERT_MAX_CHOICES || tokens > kMaxTokens / choices || experts < 1 ||
        experts > kMaxExperts)
        return BMMC_ERR_INVALID_ARG;
    return BMMC_OK;
}

// Calls f(T{}) for the logits' type.
template <class F>
bmmc_status by_logits(int type, F&& f) {
    if (type == BMMC_F32) return f(float{});
    return type == BMMC_F16 ? f(__half{}) : f(__nv_bfloat16{});
}

// Calls f(T{}, logits of a lane, whether rows are made of words, whether a warp
// has one row).
template <class F>
bmmc_status by_held(int type, const Held& h, bool words, F&& f) {
    return by_logits(type, [&](auto t) {
        const auto with = [&](auto n, auto full) {
            return words ? f(t, n, std::true_type{}, full) : f(t, n, std::false_type{}, full);
        };
        if (h.lanes < 32) return with(std::integral_constant<int, 8>{}, std::false_type{});
        if (h.each == 8) return with(std::integral_constant<int, 8>{}, std::true_type{});
        return h.each == 16 ? with(std::integral_constant<int, 16>{}, std::true_type{})
                            : with(std::integral_constant<int, 32>{}, std::true_type{});
    });
}

}  // namespace

extern "C" {

bmmc_status expert_balance_workspace(int64_t tokens, int choices, int experts, size_t* bytes) {
    if (!bytes) return BMMC_ERR_INVALID_ARG;
    *bytes = 0;
    const bmmc_status s = check_router(tokens, choices, experts, 4);
    if (s != BMMC_OK) return s;
    const Shape shape = shape_of(tokens, experts);
    *bytes = shape.together ? 0 : (size_t)shape.blocks * (experts + 1) * 8;
    return s;
}

bmmc_status expert_balance(const void* logits, int64_t stride, int type, const void* ids, int id_bytes, int64_t tokens,
                           int choices, int experts, float* loss, int32_t* counts, void* workspace, size_t workspace_bytes,
                           void* stream) {
    const bool device = device_pointers(type);
    const int es = dtype_bytes(type);
    if (!es) return BMMC_ERR_UNSUPPORTED_ELEM;
    bmmc_status s = check_router(tokens, choices, experts, id_bytes);
    if (s != BMMC_OK) return s;
    if (bad_stride(stride, tokens)) return BMMC_ERR_INVALID_ARG;
    if (!loss || !counts || (tokens && (!logits || !ids))) return BMMC_ERR_INVALID_ARG;
    size_t need = 0;
    expert_balance_workspace(tokens, choices, experts, &need);
    if (need && (!workspace || workspace_bytes < need)) return BMMC_ERR_NO_SCRATCH;
    if (misaligned(logits, es) || misaligned(ids, id_bytes) || misaligned(loss, 4) || misaligned(counts, 4) ||
        (need && misaligned(workspace, 16)))
        return BMMC_ERR_MISALIGNED;
    const Rows in[2] = {{logits, tokens, stride * es, experts * (int64_t)es}, {ids, 1, 0, tokens * choices * id_bytes}};
    const Rows out[3] = {{loss, 1, 0, 4}, {counts, 1, 0, (experts + 1) * 4ll}, {need ? workspace : nullptr, 1, 0, (int64_t)need}};
    for (int i = 0; i < 3; ++i) {
        if (may_overlap(in[0], out[i]) || may_overlap(in[1], out[i])) return BMMC_ERR_ALIAS;
        for (int j = 0; j < i; ++j)
            if (may_overlap(out[i], out[j])) return BMMC_ERR_ALIAS;
    }
    if ((s = all_reachable(device, {logits, ids, loss, counts, need ? workspace : nullptr})) != BMMC_OK) return s;
    const chk::Spans spans = spans_of({in[0], in[1], out[2]}, {out[0], out[1], out[2]});
    (void)spans;
    const Shape shape = shape_of(tokens, experts);
    Router r{static_cast<const char*>(logits), stride * es, static_cast<const char*>(ids), tokens, id_bytes, choices, experts, 32};
    float* const sums = static_cast<float*>(need ? workspace : nullptr);
    int* const parts = need ? static_cast<int*>(workspace) + (size_t)shape.blocks * (experts + 1) : counts;
    const size_t smem = ((shape.threads / 32 + 1) * (size_t)experts + 1) * 4;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    cudaLaunchAttribute together{};
    together.id = cudaLaunchAttributeClusterDimension;
    together.val.clusterDim.x = shape.together ? shape.blocks : kCluster;
    together.val.clusterDim.y = together.val.clusterDim.z = 1;
    if (experts > kHeldExperts) {
        s = by_logits(type, [&](auto t) {
            constexpr auto kernel = balance_long_kernel<decltype(t)>;
            const bmmc_status allowed = allow_smem<kernel>(smem);
            if (allowed != BMMC_OK) return allowed;
            return launch(kernel, dim3(shape.blocks), dim3(shape.threads), smem, st, nullptr, r, sums, parts BMMC_SPANS_ARG(spans));
        });
    } else {
        const Held h = held(experts);
        r.lanes = h.lanes;
        const bool words = word_bytes(2, {(uint64_t)(uintptr_t)logits, (uint64_t)r.stride, (uint64_t)(experts * es)}) == 16;
        const int64_t per_block = (tokens + shape.blocks - 1) / shape.blocks;
        s = by_held(type, h, words, [&](auto t, auto n, auto w, auto full) {
            constexpr auto kernel = balance_held_kernel<decltype(t), decltype(n)::value, decltype(w)::value, decltype(full)::value>;
            const bmmc_status allowed = allow_smem<kernel>(smem);
            if (allowed != BMMC_OK) return allowed;
            return launch(kernel, dim3(shape.blocks), dim3(shape.threads), smem, st, shape.together ? &together : nullptr, r, per_block,
                          sums, parts, shape.together ? loss : (float*)nullptr BMMC_SPANS_ARG(spans));
        });
    }
    if (s != BMMC_OK || shape.together) return s;
    cudaLaunchAttribute attributes[2] = {together, {}};
    attributes[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attributes[1].val.programmaticStreamSerializationAllowed = 1;
    return launch_with(balance_join_kernel, dim3(kCluster), dim3(1024), (size_t)shape.parts * (experts + 1) * 8, st, attributes, 2,
                       (const float*)sums, (const int*)parts, shape.blocks, experts, shape.parts, loss,
                       counts BMMC_SPANS_ARG(spans));
}

bmmc_status expert_balance_backward(const float* grad, const void* logits, int64_t stride, int type, const void* ids,
                                    int id_bytes, int64_t tokens, int choices, int experts, const int32_t* counts,
                                    void* grad_logits, int64_t grad_stride, void* stream) {
    const bool device = device_pointers(type);
    const int es = dtype_bytes(type);
    if (!es) return BMMC_ERR_UNSUPPORTED_ELEM;
    bmmc_status s = check_router(tokens, choices, experts, id_bytes);
    if (s != BMMC_OK) return s;
    if (bad_stride(stride, tokens) || bad_output_stride(grad_stride, experts, tokens)) return BMMC_ERR_INVALID_ARG;
    if (!tokens) return BMMC_OK;
    if (!grad || !logits || !ids || !counts || !grad_logits) return BMMC_ERR_INVALID_ARG;
    if (misaligned(logits, es) || misaligned(grad_logits, es) || misaligned(ids, id_bytes) || misaligned(grad, 4) ||
        misaligned(counts, 4))
        return BMMC_ERR_MISALIGNED;
    const Rows in[4] = {{logits, tokens, stride * es, experts * (int64_t)es}, {ids, 1, 0, tokens * choices * id_bytes},
                        {grad, 1, 0, 4}, {counts, 1, 0, (experts + 1) * 4ll}};
    const Rows out{grad_logits, tokens, grad_stride * es, experts * (int64_t)es};
    for (const Rows& r : in)
        if (may_overlap(r, out)) return BMMC_ERR_ALIAS;
    if ((s = all_reachable(device, {grad, logits, ids, counts, grad_logits})) != BMMC_OK) return s;
    const chk::Spans spans = spans_of({in[0], in[1], in[2], in[3]}, {out});
    (void)spans;
    Router r{static_cast<const char*>(logits), stride * es, static_cast<const char*>(ids), tokens, id_bytes, choices, experts, 32};
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    char* const to = static_cast<char*>(grad_logits);
    const Held h = held(experts);
    const bool is_held = experts <= kHeldExperts;
    if (is_held) r.lanes = h.lanes;
    const int64_t per = (int64_t)kThreads / r.lanes, b = std::min<int64_t>((tokens + per - 1) / per, kSms * 5);  // a wave of them
    const int64_t per_block = (tokens + b - 1) / b;
    const dim3 grid((unsigned)((tokens + per_block - 1) / per_block));
    if (!is_held)
        return by_logits(type, [&](auto t) {
            return launch(balance_backward_long_kernel<decltype(t)>, grid, dim3(kThreads), (size_t)experts * 4, st, nullptr, grad,
                          r, (const int*)counts, to, grad_stride * es BMMC_SPANS_ARG(spans));
        });
    const bool words = word_bytes(2, {(uint64_t)(uintptr_t)logits, (uint64_t)r.stride, (uint64_t)(experts * es),
                                      (uint64_t)(uintptr_t)grad_logits, (uint64_t)(grad_stride * es)}) == 16;
    return by_held(type, h, words, [&](auto t, auto n, auto w, auto full) {
        const auto kernel = balance_backward_held_kernel<decltype(t), decltype(n)::value, decltype(w)::value, decltype(full)::value>;
        return launch(kernel, grid, dim3(kThreads), 0, st, nullptr, grad, r, per_block, (const int*)counts, to,
                      grad_stride * es BMMC_SPANS_ARG(spans));
    });
}

}  // extern "C"

namespace bmmc {
cudaError_t bounds_record_balance(unsigned long long out[chk::kRecordWords], bool clear) {
    return chk::read_record(out, clear);
}
}  // namespace bmmc
