// Tokens sorted by expert and back: expert_sort, expert_dispatch,
// expert_combine and expert_combine_backward (declared in include/bmmc.h).
//
// A router gives each of T tokens K choices e[t,k].  The sort numbers the
// T*K choices by expert (stable: by t*K + k inside one expert), which is a
// permutation of T*K known only on the device: slot is the map, source its
// inverse.  Choices that are not routed (an id outside [0, E)) are sorted
// behind all others and marked by the complement of the number, so that the
// map stays a permutation and every row of the sorted array has one writer.
#include <cuda_runtime.h>

#include <cstdint>
#include <type_traits>

#include "../../include/bmmc.h"
#include "token_moves.hpp"
#include "token_words.cuh"

using namespace bmmc;

namespace {

// ---- sort ------------------------------------------------------------------

constexpr int kMaxExperts = 4096;
constexpr int kSortRounds = 4;       // ids per lane and tile
constexpr int kMaxSortBlocks = 152;  // blocks of a sort that one block does not cover: one for each SM

template <class Id>
__device__ __forceinline__ int key_of(Id id, int experts) {
    return id >= 0 && id < (Id)experts ? (int)id : experts;
}

// Exclusive prefix sum of v[0..n) in shared memory, in place, by all threads
// of the block.  tmp: 32 ints.
__device__ void block_exclusive_scan(int* v, int n, int* tmp) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    int carry = 0;
    for (int at = 0; at < n; at += blockDim.x) {
        const int i = at + threadIdx.x;
        const int x = i < n ? v[i] : 0;
        int s = x;
        for (int d = 1; d < 32; d <<= 1) {
            const int y = __shfl_up_sync(~0u, s, d);
            if (lane >= d) s += y;
        }
        if (lane == 31) tmp[warp] = s;
        __syncthreads();
        if (warp == 0) {
            int w = lane < warps ? tmp[lane] : 0;
            for (int d = 1; d < 32; d <<= 1) {
                const int y = __shfl_up_sync(~0u, w, d);
                if (lane >= d) w += y;
            }
            tmp[lane] = w;
        }
        __syncthreads();
        if (i < n) v[i] = carry + (warp ? tmp[warp - 1] : 0) + s - x;
        carry += tmp[31];
        __syncthreads();
    }
}

// counts[b][e] = choices of block b's part with key e (e = E: not routed);
// the blocks' rows are `pitch` apart, a multiple of 4, zero past the keys.
template <class Id>
__global__ void __launch_bounds__(1024) sort_count_kernel(const Id* __restrict__ ids, int64_t n, int experts,
                                                          int64_t per_block, int pitch, int* __restrict__ counts) {
    extern __shared__ int s_hist[];
    cudaTriggerProgrammaticLaunchCompletion();  // the place kernel may rank its first tile meanwhile
    for (int e = threadIdx.x; e < pitch; e += blockDim.x) s_hist[e] = 0;
    __syncthreads();
    const int64_t lo = (int64_t)blockIdx.x * per_block, hi = min(n, lo + per_block);
    for (int64_t at = lo + threadIdx.x; at < hi; at += (int64_t)blockDim.x * kSortRounds) {
        int key[kSortRounds];
#pragma unroll
        for (int r = 0; r < kSortRounds; ++r) {
            const int64_t i = at + (int64_t)r * blockDim.x;
            key[r] = i < hi ? key_of(ids[i], experts) : -1;
        }
#pragma unroll
        for (int r = 0; r < kSortRounds; ++r)
            if (key[r] >= 0) atomicAdd(&s_hist[key[r]], 1);
    }
    __syncthreads();
    for (int e = threadIdx.x; e < pitch; e += blockDim.x) counts[(int64_t)blockIdx.x * pitch + e] = s_hist[e];
}

// base[e] += the counts of key e over all blocks, before[e] += those over the
// blocks ahead of this one (both zero in shared memory at the start): four
// keys a load, the blocks dealt out to groups of threads.
__device__ __forceinline__ void sum_counts(const int* counts, int pitch, int* base, int* before) {
    const int quads = pitch >> 2, groups = max(1, (int)blockDim.x / quads);
    for (int item = threadIdx.x; item < groups * quads; item += blockDim.x) {
        const int q = item % quads, group = item / quads;
        int4 all = make_int4(0, 0, 0, 0), ahead = all;
#pragma unroll 8
        for (int b = group; b < (int)gridDim.x; b += groups) {
            const int4 c = __ldcg(reinterpret_cast<const int4*>(counts) + (int64_t)b * quads + q);
            all.x += c.x, all.y += c.y, all.z += c.z, all.w += c.w;
            if (b < (int)blockIdx.x) ahead.x += c.x, ahead.y += c.y, ahead.z += c.z, ahead.w += c.w;
        }
        const int a4[4] = {all.x, all.y, all.z, all.w}, b4[4] = {ahead.x, ahead.y, ahead.z, ahead.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            atomicAdd(&base[4 * q + i], a4[i]);
            atomicAdd(&before[4 * q + i], b4[i]);
        }
    }
}

// Each block numbers its part, a tile of blockDim.x * R choices at a time.
// Inside a warp a choice's rank among equal keys comes from a match of the
// 32 keys of a round plus the warp's running count of that key; a column sum
// over the warps and the block's start for the key complete its place.  The
// starts come from the counts of all blocks, or (counts == NULL: one block
// and one tile) from the tile itself.  Integer sums: the result does not
// depend on timing.  The first tile is ranked before the counts are waited
// for, so that this work runs beside the count kernel.
template <class Id, int R>
__global__ void __launch_bounds__(1024) sort_place_kernel(const Id* __restrict__ ids, int64_t n, int experts,
                                                          int64_t per_block, int pitch, const int* counts,
                                                          int* __restrict__ slot, int* __restrict__ source,
                                                          int* __restrict__ offsets) {
    extern __shared__ int s_mem[];
    const int keys = experts + 1, warps = blockDim.x >> 5;
    int* base = s_mem;          // [pitch] where the block's next choice of each key goes
    int* total = base + pitch;  // [pitch] choices of the tile
    int* tmp = total + pitch;   // [32]
    int* hist = tmp + 32;       // [warps][keys] counts of the tile, then starts inside it
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int* mine = hist + warp * keys;
    const int64_t lo = (int64_t)blockIdx.x * per_block, hi = min(n, lo + per_block);
    int64_t at = lo;
    do {
        int key[R], rank[R];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int64_t i = at + ((int64_t)warp * R + r) * 32 + lane;
            key[r] = i < hi ? key_of(ids[i], experts) : -1;
        }
        for (int e = lane; e < keys; e += 32) mine[e] = 0;
        __syncwarp();
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const unsigned same = __match_any_sync(~0u, key[r]);
            const int before = key[r] < 0 ? 0 : mine[key[r]];
            rank[r] = before + __popc(same & ((1u << lane) - 1));
            __syncwarp();
            if (key[r] >= 0 && lane == __ffs(same) - 1) mine[key[r]] = before + __popc(same);
            __syncwarp();
        }
        if (counts && at == lo) {
            for (int e = threadIdx.x; e < pitch; e += blockDim.x) base[e] = total[e] = 0;
            __syncthreads();
            cudaGridDependencySynchronize();
            sum_counts(counts, pitch, base, total);
            __syncthreads();
            block_exclusive_scan(base, keys, tmp);
            for (int e = threadIdx.x; e < keys; e += blockDim.x) {
                if (blockIdx.x == 0) offsets[e] = base[e];
                base[e] += total[e];
            }
        }
        __syncthreads();
        for (int e = threadIdx.x; e < keys; e += blockDim.x) {
            int run = 0;
            for (int w = 0; w < warps; ++w) {
                const int c = hist[w * keys + e];
                hist[w * keys + e] = run;
                run += c;
            }
            total[e] = run;
            if (!counts) base[e] = run;
        }
        __syncthreads();
        if (!counts) {
            block_exclusive_scan(base, keys, tmp);
            for (int e = threadIdx.x; e < keys; e += blockDim.x) offsets[e] = base[e];
        }
#pragma unroll
        for (int r = 0; r < R; ++r) {
            if (key[r] < 0) continue;
            const int64_t i = at + ((int64_t)warp * R + r) * 32 + lane;
            const int to = base[key[r]] + mine[key[r]] + rank[r];
            const bool routed = key[r] < experts;
            slot[i] = routed ? to : ~to;
            if ((unsigned)to < (unsigned)n) source[to] = routed ? (int)i : ~(int)i;  // also if ids changed meanwhile
        }
        at += (int64_t)blockDim.x * R;
        if (at >= hi) break;
        __syncthreads();
        for (int e = threadIdx.x; e < keys; e += blockDim.x) base[e] += total[e];
    } while (true);
}

struct SortShape {
    int warps, blocks, rounds, pitch;
    int64_t per_block;
    size_t smem;  // of the place kernel
};

constexpr size_t kSortSmem = 200 * 1024;

// One block where one tile covers all choices (of one round a warp where that
// is enough), else at most kMaxSortBlocks blocks of whole tiles.  A block has
// as many warps as their counts of every key leave room for.
SortShape sort_shape(int64_t n, int experts) {
    SortShape s;
    s.pitch = (experts + 4) & ~3;
    const auto smem = [&](int warps) { return ((size_t)warps * (experts + 1) + 2 * s.pitch + 32) * sizeof(int); };
    s.warps = 32;
    while (smem(s.warps) > kSortSmem) s.warps >>= 1;
    s.rounds = n <= s.warps * 32 ? 1 : kSortRounds;
    const int64_t tile = (int64_t)s.warps * 32 * s.rounds;
    const int64_t tiles = n <= tile ? 1 : (n + tile - 1) / tile;
    const int64_t per = (tiles + kMaxSortBlocks - 1) / kMaxSortBlocks;
    s.per_block = per * tile;
    s.blocks = (int)((tiles + per - 1) / per);
    if (s.blocks == 1) s.warps = n < 32 ? 1 : (int)((n + 32 * s.rounds - 1) / (32 * s.rounds));
    s.smem = smem(s.warps);
    return s;
}

template <class Id, int R>
bmmc_status launch_sort(const SortShape& s, const void* ids_, int64_t n, int experts, int32_t* slot, int32_t* source,
                        int32_t* offsets, int* counts, cudaStream_t st) {
    const Id* ids = static_cast<const Id*>(ids_);
    const auto place = sort_place_kernel<Id, R>;
    if (s.smem > 48 * 1024 &&
        cudaFuncSetAttribute(place, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSortSmem) != cudaSuccess) {
        cudaGetLastError();
        return BMMC_ERR_CUDA;
    }
    const int* none = nullptr;
    if (s.blocks == 1) {
        place<<<1, s.warps * 32, s.smem, st>>>(ids, n, experts, s.per_block, s.pitch, none, slot, source, offsets);
        return launched();
    }
    sort_count_kernel<Id><<<s.blocks, 1024, s.pitch * sizeof(int), st>>>(ids, n, experts, s.per_block, s.pitch, counts);
    if (launched() != BMMC_OK) return BMMC_ERR_CUDA;
    cudaLaunchAttribute early[1];
    early[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    early[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(s.blocks);
    cfg.blockDim = dim3(s.warps * 32);
    cfg.dynamicSmemBytes = s.smem;
    cfg.stream = st;
    cfg.attrs = early;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, place, ids, n, experts, s.per_block, s.pitch, (const int*)counts, slot, source,
                           offsets) != cudaSuccess) {
        cudaGetLastError();
        return BMMC_ERR_CUDA;
    }
    return BMMC_OK;
}

// ---- dispatch ----------------------------------------------------------------

// How the words of the tokens' rows are dealt out: blocks of x * y threads
// take y tokens and x * U words of each, U words a thread, x apart; gridDim.y
// parts make up a row.
struct Cover {
    dim3 grid, block;
};

Cover cover(int64_t tokens, int words, int U, int most) {
    const int need = (words + U - 1) / U;  // threads of a row
    const int parts = (need + most - 1) / most;
    const int x = ((need + parts - 1) / parts + 31) / 32 * 32;
    const int y = x >= most ? 1 : most / x;
    Cover c;
    c.block = dim3(x, y);
    c.grid = dim3((unsigned)((tokens + y - 1) / y), (unsigned)((words + x * U - 1) / (x * U)));
    return c;
}

// Fewer words than this many: one word a thread, so that the call is spread
// over the machine and every load is in flight at once.
constexpr int64_t kFewWords = 152 * 2048;

// Pure movement: each word of a token's row is read once and written to the
// rows of its choices.
template <class Word, int U>
__global__ void __launch_bounds__(256) dispatch_kernel(const char* __restrict__ x, int64_t x_stride,
                                                       const int* __restrict__ slot, int64_t tokens, int choices,
                                                       int64_t n_rows, int words, char* __restrict__ rows,
                                                       int64_t row_stride) {
    const int64_t t = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
    const int w = blockIdx.y * blockDim.x * U + threadIdx.x;
    if (t >= tokens || w >= words) return;
    const Word* from = reinterpret_cast<const Word*>(x + t * x_stride);
    Word v[U];
#pragma unroll
    for (int u = 0; u < U; ++u)
        if (w + u * (int)blockDim.x < words) v[u] = from[w + u * blockDim.x];
    slot += t * choices;
#pragma unroll 4
    for (int k = 0; k < choices; ++k) {
        const int s = __ldg(slot + k);
        const int64_t row = s < 0 ? ~s : s;
        if (row >= n_rows) continue;
        Word* to = reinterpret_cast<Word*>(rows + row * row_stride);
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (w + u * (int)blockDim.x < words) to[w + u * blockDim.x] = s < 0 ? Word{} : v[u];
    }
}

// ---- combine -----------------------------------------------------------------

// A weight of the rows' type or of 32 bits.
template <class T>
__device__ __forceinline__ float weight_at(const void* weights, int in_f32, int64_t i) {
    return in_f32 ? static_cast<const float*>(weights)[i] : to_f32(static_cast<const T*>(weights)[i]);
}

// Each thread holds the sums of U words in 32 bits, adds the choices in order,
// KB of them loaded at a time, and rounds once.
template <class T, int W, int U, int KB>
__global__ void __launch_bounds__(256) combine_kernel(const char* __restrict__ rows, int64_t row_stride, int64_t n_rows,
                                                      const int* __restrict__ slot, const void* __restrict__ weights,
                                                      int weights_f32, int64_t tokens, int choices, int words,
                                                      char* __restrict__ out, int64_t out_stride) {
    const int64_t t = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
    const int w = blockIdx.y * blockDim.x * U + threadIdx.x;
    if (t >= tokens || w >= words) return;
    float sum[U][W];
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
        for (int i = 0; i < W; ++i) sum[u][i] = 0.0f;
    for (int k0 = 0; k0 < choices; k0 += KB) {
        int s[KB];
        float f[KB];
        Pack<T, W> y[KB][U];
#pragma unroll
        for (int j = 0; j < KB; ++j) {
            s[j] = k0 + j < choices ? slot[t * choices + k0 + j] : -1;
            if (s[j] >= n_rows) s[j] = -1;
        }
#pragma unroll
        for (int j = 0; j < KB; ++j) {
            f[j] = 1.0f;
            if (weights && s[j] >= 0) f[j] = weight_at<T>(weights, weights_f32, t * choices + k0 + j);
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (s[j] >= 0 && w + u * (int)blockDim.x < words)
                    y[j][u].load(rows + s[j] * row_stride + (int64_t)(w + u * (int)blockDim.x) * sizeof(y[j][u]));
        }
#pragma unroll
        for (int j = 0; j < KB; ++j)
            if (s[j] >= 0)
#pragma unroll
                for (int u = 0; u < U; ++u)
#pragma unroll
                    for (int i = 0; i < W; ++i) sum[u][i] = fmaf(f[j], y[j][u].get(i), sum[u][i]);
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
        if (w + u * (int)blockDim.x < words) {
            Pack<T, W> o;
            o.set(sum[u]);
            o.store(out + t * out_stride + (int64_t)(w + u * (int)blockDim.x) * sizeof(o));
        }
}

// grad_rows[slot] = w * grad and grad_weights = <rows[slot], grad>, a choice
// after the other; the products are summed in 32 bits, by lanes and then
// across them in a fixed order.
template <class T, int W>
__global__ void __launch_bounds__(256) combine_backward_kernel(
    const char* __restrict__ grad, int64_t grad_stride, const char* __restrict__ rows, int64_t row_stride,
    int64_t n_rows, const int* __restrict__ slot, const void* __restrict__ weights, int weights_f32, int64_t tokens,
    int choices, int words, char* __restrict__ grad_rows, int64_t grad_row_stride, void* __restrict__ grad_weights) {
    __shared__ float s_part[8];
    const int64_t t = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
    const bool live = t < tokens;
    const int lane = threadIdx.x & 31, per = blockDim.x >> 5;
    const int warp = threadIdx.y * per + (threadIdx.x >> 5);
    for (int k = 0; k < choices; ++k) {
        float dot = 0.0f;
        if (live) {
            const int s = slot[t * choices + k];
            const int64_t row = s < 0 ? ~s : s;
            const float f = s < 0 ? 0.0f : weight_at<T>(weights, weights_f32, t * choices + k);
            if (row < n_rows)
                for (int w = threadIdx.x; w < words; w += blockDim.x) {
                    Pack<T, W> g, y, o;
                    float v[W];
                    g.load(grad + t * grad_stride + (int64_t)w * sizeof(g));
                    if (s >= 0) {
                        y.load(rows + row * row_stride + (int64_t)w * sizeof(y));
#pragma unroll
                        for (int i = 0; i < W; ++i) {
                            dot = fmaf(g.get(i), y.get(i), dot);
                            v[i] = f * g.get(i);
                        }
                    } else {
#pragma unroll
                        for (int i = 0; i < W; ++i) v[i] = 0.0f;
                    }
                    o.set(v);
                    o.store(grad_rows + row * grad_row_stride + (int64_t)w * sizeof(o));
                }
        }
        for (int d = 16; d; d >>= 1) dot += __shfl_xor_sync(~0u, dot, d);
        if (lane == 0) s_part[warp] = dot;
        __syncthreads();
        if (live && threadIdx.x == 0) {
            float sum = 0.0f;
            for (int i = 0; i < per; ++i) sum += s_part[warp + i];
            if (weights_f32) static_cast<float*>(grad_weights)[t * choices + k] = sum;
            else static_cast<T*>(grad_weights)[t * choices + k] = from_f32<T>(sum);
        }
        __syncthreads();
    }
}

// Calls f(T{}, elements per word) for the type and the word's width.
template <class F>
void by_type(int type, int bytes, F&& f) {
    auto width = [&](auto t) {
        constexpr int es = sizeof(t);
        switch (bytes) {
            case 16: f(t, std::integral_constant<int, 16 / es>{}); break;
            case 8: f(t, std::integral_constant<int, 8 / es>{}); break;
            case 4: f(t, std::integral_constant<int, 4 / es>{}); break;
            default: f(t, std::integral_constant<int, 1>{}); break;
        }
    };
    switch (type) {
        case BMMC_F32: width(float{}); break;
        case BMMC_F16: width(__half{}); break;
        default: width(__nv_bfloat16{}); break;
    }
}

bmmc_status check_moves(int64_t tokens, int choices, int64_t hidden, int64_t n_rows, int type, int* es) {
    if (!(*es = dtype_bytes(type))) return BMMC_ERR_UNSUPPORTED_ELEM;
    if (tokens < 0 || choices < 1 || choices > EXPERT_MAX_CHOICES || tokens > kMaxTokens / choices || hidden < 1 ||
        hidden > (1 << 24) || n_rows < 0 || n_rows > tokens * choices)
        return BMMC_ERR_INVALID_ARG;
    return BMMC_OK;
}

bool bad_stride(int64_t stride, int64_t hidden, int64_t rows) {
    return stride > kMaxStride || (rows > 1 && stride < hidden) || stride < 0;
}

bool misaligned(const void* p, size_t bytes) { return (uintptr_t)p & (bytes - 1); }

}  // namespace

extern "C" {

bmmc_status expert_sort_workspace(int64_t tokens, int choices, int experts, size_t* bytes) {
    if (!bytes) return BMMC_ERR_INVALID_ARG;
    *bytes = 0;
    if (tokens < 0 || choices < 1 || choices > EXPERT_MAX_CHOICES || tokens > kMaxTokens / choices || experts < 1 ||
        experts > kMaxExperts)
        return BMMC_ERR_INVALID_ARG;
    const SortShape s = sort_shape(tokens * choices, experts);
    *bytes = s.blocks > 1 ? (size_t)s.blocks * s.pitch * sizeof(int) : 0;
    return BMMC_OK;
}

bmmc_status expert_sort(const void* ids, int id_bytes, int64_t tokens, int choices, int experts, int32_t* slot,
                        int32_t* source, int32_t* offsets, void* workspace, size_t workspace_bytes, void* stream) {
    size_t need = 0;
    bmmc_status s = expert_sort_workspace(tokens, choices, experts, &need);
    if (s != BMMC_OK) return s;
    const bool checked = pointers_checked(id_bytes);
    if (id_bytes != 4 && id_bytes != 8) return BMMC_ERR_UNSUPPORTED_ELEM;
    const int64_t n = tokens * choices;
    if (!offsets || (n && (!ids || !slot || !source))) return BMMC_ERR_INVALID_ARG;
    if (need && (!workspace || workspace_bytes < need)) return BMMC_ERR_NO_SCRATCH;
    if (misaligned(ids, id_bytes) || misaligned(slot, 4) || misaligned(source, 4) || misaligned(offsets, 4) ||
        (need && misaligned(workspace, 16)))
        return BMMC_ERR_MISALIGNED;
    const Rows in{ids, 1, 0, n * id_bytes};
    const Rows o[4] = {{slot, 1, 0, n * 4}, {source, 1, 0, n * 4}, {offsets, 1, 0, (experts + 1) * 4ll},
                       {need ? workspace : nullptr, 1, 0, (int64_t)need}};
    for (int i = 0; i < 4; ++i) {
        if (may_overlap(in, o[i])) return BMMC_ERR_ALIAS;
        for (int j = 0; j < i; ++j)
            if (may_overlap(o[i], o[j])) return BMMC_ERR_ALIAS;
    }
    if ((s = all_reachable(checked, {ids, slot, source, offsets, need ? workspace : nullptr})) != BMMC_OK) return s;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    int* counts = static_cast<int*>(need ? workspace : nullptr);
    const SortShape shape = sort_shape(n, experts);
    const auto go = [&](auto launch) { return launch(shape, ids, n, experts, slot, source, offsets, counts, st); };
    if (id_bytes == 4) return shape.rounds == 1 ? go(launch_sort<int32_t, 1>) : go(launch_sort<int32_t, kSortRounds>);
    return shape.rounds == 1 ? go(launch_sort<int64_t, 1>) : go(launch_sort<int64_t, kSortRounds>);
}

bmmc_status expert_dispatch(const void* x, int64_t x_stride, const int32_t* slot, int64_t tokens, int choices,
                            int64_t hidden, int type, void* rows, int64_t row_stride, int64_t n_rows, void* stream) {
    int es = 0;
    const bool checked = pointers_checked(type);
    bmmc_status s = check_moves(tokens, choices, hidden, n_rows, type, &es);
    if (s != BMMC_OK) return s;
    if (bad_stride(x_stride, 0, tokens) || bad_stride(row_stride, hidden, n_rows)) return BMMC_ERR_INVALID_ARG;
    if (!n_rows) return BMMC_OK;
    if (!x || !slot || !rows) return BMMC_ERR_INVALID_ARG;
    if (misaligned(x, es) || misaligned(rows, es) || misaligned(slot, 4)) return BMMC_ERR_MISALIGNED;
    const Rows in{x, tokens, x_stride * es, hidden * es}, out{rows, n_rows, row_stride * es, hidden * es};
    if (may_overlap(in, out) || may_overlap({slot, 1, 0, tokens * choices * 4}, out)) return BMMC_ERR_ALIAS;
    if ((s = all_reachable(checked, {x, slot, rows})) != BMMC_OK) return s;
    const int wb = word_bytes(es, {(uint64_t)(uintptr_t)x, (uint64_t)(uintptr_t)rows, (uint64_t)(x_stride * es),
                                   (uint64_t)(row_stride * es), (uint64_t)(hidden * es)});
    const int words = (int)(hidden * es / wb);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const char* from = static_cast<const char*>(x);
    char* to = static_cast<char*>(rows);
    auto go = [&](auto word) {
        using Word = decltype(word);
        const bool few = tokens * words <= kFewWords;
        const Cover c = few ? cover(tokens, words, 1, 128) : cover(tokens, words, 2, 256);
        const auto kernel = few ? dispatch_kernel<Word, 1> : dispatch_kernel<Word, 2>;
        kernel<<<c.grid, c.block, 0, st>>>(from, x_stride * es, slot, tokens, choices, n_rows, words, to, row_stride * es);
    };
    switch (wb) {
        case 16: go(uint4{}); break;
        case 8: go(uint2{}); break;
        case 4: go(uint32_t{}); break;
        default: go(uint16_t{}); break;
    }
    return launched();
}

bmmc_status expert_combine(const void* rows, int64_t row_stride, int64_t n_rows, const int32_t* slot,
                           const void* weights, int weight_type, int64_t tokens, int choices, int64_t hidden, int type,
                           void* out, int64_t out_stride, void* stream) {
    int es = 0;
    const bool checked = pointers_checked(type);
    bmmc_status s = check_moves(tokens, choices, hidden, n_rows, type, &es);
    if (s != BMMC_OK) return s;
    if (weights && weight_type != BMMC_F32 && weight_type != type) return BMMC_ERR_UNSUPPORTED_ELEM;
    if (bad_stride(row_stride, 0, n_rows) || bad_stride(out_stride, hidden, tokens)) return BMMC_ERR_INVALID_ARG;
    if (!tokens) return BMMC_OK;
    if ((!rows && n_rows) || !slot || !out) return BMMC_ERR_INVALID_ARG;
    const int ws = weights ? dtype_bytes(weight_type) : 4;
    if (misaligned(rows, es) || misaligned(out, es) || misaligned(slot, 4) || misaligned(weights, ws))
        return BMMC_ERR_MISALIGNED;
    const Rows to{out, tokens, out_stride * es, hidden * es};
    if (may_overlap({rows, n_rows, row_stride * es, hidden * es}, to) ||
        may_overlap({slot, 1, 0, tokens * choices * 4}, to) || may_overlap({weights, 1, 0, tokens * choices * ws}, to))
        return BMMC_ERR_ALIAS;
    if ((s = all_reachable(checked, {rows, slot, weights, out})) != BMMC_OK) return s;
    const int wb = word_bytes(es, {(uint64_t)(uintptr_t)rows, (uint64_t)(uintptr_t)out, (uint64_t)(row_stride * es),
                                   (uint64_t)(out_stride * es), (uint64_t)(hidden * es)});
    const int words = (int)(hidden * es / wb);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    by_type(type, wb, [&](auto e, auto width) {
        using T = decltype(e);
        constexpr int W = decltype(width)::value;
        constexpr int U = W * sizeof(T) > 4 ? 2 : 4;  // short words: more of them in flight
        const bool few = tokens * words <= kFewWords, two = choices <= 2;
        const Cover c = cover(tokens, words, few ? 1 : two ? 2 * U : U, few ? 128 : 256);
        const auto kernel = few ? combine_kernel<T, W, 1, 8> : two ? combine_kernel<T, W, 2 * U, 2> : combine_kernel<T, W, U, 4>;
        kernel<<<c.grid, c.block, 0, st>>>(static_cast<const char*>(rows), row_stride * es, n_rows, slot, weights,
                                          weight_type == BMMC_F32, tokens, choices, words, static_cast<char*>(out),
                                          out_stride * es);
    });
    return launched();
}

bmmc_status expert_combine_backward(const void* grad, int64_t grad_stride, const void* rows, int64_t row_stride,
                                    int64_t n_rows, const int32_t* slot, const void* weights, int weight_type,
                                    int64_t tokens, int choices, int64_t hidden, int type, void* grad_rows,
                                    int64_t grad_row_stride, void* grad_weights, void* stream) {
    int es = 0;
    const bool checked = pointers_checked(type);
    bmmc_status s = check_moves(tokens, choices, hidden, n_rows, type, &es);
    if (s != BMMC_OK) return s;
    if (weight_type != BMMC_F32 && weight_type != type) return BMMC_ERR_UNSUPPORTED_ELEM;
    if (bad_stride(grad_stride, 0, tokens) || bad_stride(row_stride, 0, n_rows) ||
        bad_stride(grad_row_stride, hidden, n_rows))
        return BMMC_ERR_INVALID_ARG;
    if (!tokens) return BMMC_OK;
    if (!grad || !slot || !weights || !grad_weights || (n_rows && (!rows || !grad_rows))) return BMMC_ERR_INVALID_ARG;
    const int ws = dtype_bytes(weight_type);
    if (misaligned(grad, es) || misaligned(rows, es) || misaligned(grad_rows, es) || misaligned(slot, 4) ||
        misaligned(weights, ws) || misaligned(grad_weights, ws))
        return BMMC_ERR_MISALIGNED;
    const int64_t n = tokens * choices;
    const Rows in[4] = {{grad, tokens, grad_stride * es, hidden * es}, {rows, n_rows, row_stride * es, hidden * es},
                        {slot, 1, 0, n * 4}, {weights, 1, 0, n * ws}};
    const Rows gr{grad_rows, n_rows, grad_row_stride * es, hidden * es}, gw{grad_weights, 1, 0, n * ws};
    for (const Rows& r : in)
        if (may_overlap(r, gr) || may_overlap(r, gw)) return BMMC_ERR_ALIAS;
    if (may_overlap(gr, gw)) return BMMC_ERR_ALIAS;
    if ((s = all_reachable(checked, {grad, rows, slot, weights, grad_rows, grad_weights})) != BMMC_OK) return s;
    const int wb = word_bytes(es, {(uint64_t)(uintptr_t)grad, (uint64_t)(uintptr_t)rows, (uint64_t)(uintptr_t)grad_rows,
                                   (uint64_t)(grad_stride * es), (uint64_t)(row_stride * es),
                                   (uint64_t)(grad_row_stride * es), (uint64_t)(hidden * es)});
    const int words = (int)(hidden * es / wb);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    int x = 32;
    while (x < words && x < 256) x <<= 1;
    const dim3 block(x, 256 / x);
    const unsigned blocks = (unsigned)((tokens + block.y - 1) / block.y);
    by_type(type, wb, [&](auto e, auto width) {
        combine_backward_kernel<decltype(e), decltype(width)::value><<<blocks, block, 0, st>>>(
            static_cast<const char*>(grad), grad_stride * es, static_cast<const char*>(rows), row_stride * es, n_rows,
            slot, weights, weight_type == BMMC_F32, tokens, choices, words, static_cast<char*>(grad_rows),
            grad_row_stride * es, grad_weights);
    });
    return launched();
}

}  // extern "C"
