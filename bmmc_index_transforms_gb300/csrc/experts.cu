// Tokens sorted by expert and back: expert_sort, expert_dispatch,
// expert_combine and expert_combine_backward (declared in include/bmmc.h).
//
// A router gives each of T tokens K choices e[t,k].  The sort numbers the
// T*K choices by expert (stable: by t*K + k inside one expert), which is a
// permutation of T*K known only on the device: slot is the map, source its
// inverse.  Choices that are not routed (an id outside [0, E)) are sorted
// behind all others and marked by the complement of the number, so that the
// map stays a permutation and every row of the sorted array has one writer.
#include <cooperative_groups.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>
#include <type_traits>

#include "../../include/bmmc.h"
#define BMMC_CHK_FILE 6  // site tag of this file in bounds-checked builds
#include "bounds.cuh"
#include "token_moves.hpp"
#include "token_words.cuh"

using namespace bmmc;

namespace {

// ---- sort ------------------------------------------------------------------

constexpr int kMaxExperts = 4096;
constexpr int kSortRounds = 4;       // ids per lane and tile
constexpr int kSortCluster = 8;      // blocks that are launched as one cluster
constexpr int kMaxSortBlocks = kSms;  // blocks of a sort that one block does not cover: one for each SM

#ifdef BMMC_BOUNDS_CHECK
__device__ __forceinline__ uint32_t chk_dynamic_bytes() { return chk::dyn_smem_bytes(); }
#endif

template <class Id>
__device__ __forceinline__ int key_of(Id id, int experts) {
    return id >= 0 && id < (Id)experts ? (int)id : experts;
}

// Exclusive prefix sum of v[0..n) in shared memory, in place, by all threads
// of the block.  tmp: 32 ints.
__device__ void block_exclusive_scan(Slots<int> v, int n, Slots<int> tmp) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    int carry = 0;
    for (int at = 0; at < n; at += blockDim.x) {
        const int i = at + threadIdx.x;
        const int x = i < n ? v.get(i) : 0;
        int s = x;
        for (int d = 1; d < 32; d <<= 1) {
            const int y = __shfl_up_sync(~0u, s, d);
            if (lane >= d) s += y;
        }
        if (lane == 31) tmp.set(warp, s);
        __syncthreads();
        if (warp == 0) {
            int w = lane < warps ? tmp.get(lane) : 0;
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

// counts[b][e] = choices of block b's part with key e (e = E: not routed);
// the blocks' rows are `pitch` apart, a multiple of 4, zero past the keys.
template <class Id>
__global__ void __launch_bounds__(1024) sort_count_kernel(const Id* __restrict__ ids, int64_t n, int experts,
                                                          int64_t per_block, int pitch, int* __restrict__ counts
                                                              BMMC_SPANS_PARAM) {
    extern __shared__ int s_hist[];
    BMMC_SPANS_ENTER(s_hist, chk_dynamic_bytes());
    const Slots<int> hist(s_hist, pitch);
    cudaTriggerProgrammaticLaunchCompletion();  // the place kernel may rank its first tile meanwhile
    for (int e = threadIdx.x; e < pitch; e += blockDim.x) hist.set(e, 0);
    __syncthreads();
    const int64_t lo = (int64_t)blockIdx.x * per_block, hi = min(n, lo + per_block);
    for (int64_t at = lo + threadIdx.x; at < hi; at += (int64_t)blockDim.x * kSortRounds) {
        int key[kSortRounds];
#pragma unroll
        for (int r = 0; r < kSortRounds; ++r) {
            const int64_t i = at + (int64_t)r * blockDim.x;
            key[r] = i < hi && BMMC_RD_OK(ids + i, sizeof(Id)) ? key_of(ids[i], experts) : -1;
        }
#pragma unroll
        for (int r = 0; r < kSortRounds; ++r)
            if (key[r] >= 0) hist.add(key[r], 1);
    }
    __syncthreads();
    for (int e = threadIdx.x; e < pitch; e += blockDim.x)
        if (BMMC_WR_OK(counts + (int64_t)blockIdx.x * pitch + e, 4)) counts[(int64_t)blockIdx.x * pitch + e] = hist.get(e);
}

// base[e] += the counts of key e over all blocks, before[e] += those over the
// blocks ahead of this one (both zero in shared memory at the start): four
// keys a load, the blocks dealt out to groups of threads.
__device__ __forceinline__ void sum_counts(const int* counts, int pitch, Slots<int> base, Slots<int> before) {
    const int quads = pitch >> 2, groups = max(1, (int)blockDim.x / quads);
    for (int item = threadIdx.x; item < groups * quads; item += blockDim.x) {
        const int q = item % quads, group = item / quads;
        int4 all = make_int4(0, 0, 0, 0), ahead = all;
#pragma unroll 8
        for (int b = group; b < (int)gridDim.x; b += groups) {
            const int4* const from = reinterpret_cast<const int4*>(counts) + (int64_t)b * quads + q;
            const int4 c = BMMC_RD_OK(from, 16) ? __ldcg(from) : make_int4(0, 0, 0, 0);
            all.x += c.x, all.y += c.y, all.z += c.z, all.w += c.w;
            if (b < (int)blockIdx.x) ahead.x += c.x, ahead.y += c.y, ahead.z += c.z, ahead.w += c.w;
        }
        const int a4[4] = {all.x, all.y, all.z, all.w}, b4[4] = {ahead.x, ahead.y, ahead.z, ahead.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            base.add(4 * q + i, a4[i]);
            before.add(4 * q + i, b4[i]);
        }
    }
}

// The lanes with the same key, from one ballot for each bit of the keys
// (`bits` of them).  With the match instruction in its place, and source
// written where it goes instead of in runs, 524168 ids took 11.9 us, not 11.0.
__device__ __forceinline__ unsigned same_key(int key, int bits) {
    unsigned same = ~0u;
    for (int b = 0; b < bits; ++b) {
        const bool one = (key >> b) & 1;
        const unsigned ones = __ballot_sync(~0u, one);
        same &= one ? ones : ~ones;
    }
    return same;
}

// What bounds it: not bytes (65521 x 8 ids of 32 bits, 256 experts, take 11.0 us
// on the device and could be moved in 0.9) but latency: two launches, the
// ids' first load and the barriers between a tile's steps leave 6.8 us of it
// when all other work is skipped.  One block per SM of 32 warps was taken for
// that reason; 64 blocks of twice the ids, which summed the blocks' counts one
// key a load, took 18 us.  384 ids are one block and one launch: 2.5 us; 4096 ids
// 6.8 us (7.4 with source written where it goes), 32768 as one cluster, without a
// second launch or a workspace, 8.8; 32800 in two launches 9.6.
//
// Each block numbers its part, a tile of blockDim.x * R choices at a time.
// Inside a warp a choice's rank among equal keys comes from the lanes of a
// round with its key plus the warp's running count of that key; a column sum
// over the warps and the block's start for the key complete its place.  The
// starts come from the counts of all blocks; or (counts == NULL: one tile a
// block) from the tile itself where there is one block, and from the tiles of
// the blocks of one cluster, which read each other's shared memory.  Integer sums: the result does not
// depend on timing.  The first tile is ranked before the counts are waited
// for, so that this work runs beside the count kernel; a tile of several
// rounds is put in order in shared memory, so that source is written in runs.
template <class Id, int R>
__global__ void __launch_bounds__(1024) sort_place_kernel(const Id* __restrict__ ids, int64_t n, int experts,
                                                          int64_t per_block, int pitch, int bits, const int* counts,
                                                          int* __restrict__ slot, int* __restrict__ source,
                                                          int* __restrict__ offsets BMMC_SPANS_PARAM) {
    extern __shared__ int s_mem[];
    BMMC_SPANS_ENTER(s_mem, chk_dynamic_bytes());
    const int keys = experts + 1, warps = blockDim.x >> 5, none = (1 << bits) - 1;
    const bool many = gridDim.x > 1;
    constexpr bool kOrder = R > 1;  // a tile large enough to put source in order before it is written
    const int tile = blockDim.x * R;
    const Slots<int> mem(s_mem, 4 * pitch + 32 + warps * keys + (kOrder ? tile : 0));
    const Slots<int> base = mem.part(0, pitch);           // where the block's next choice of each key goes
    const Slots<int> total = mem.part(pitch, pitch);      // choices of the tile
    const Slots<int> start = mem.part(2 * pitch, pitch);  // the tile's first choice of each key, in order (several blocks)
    const Slots<int> ahead = mem.part(3 * pitch, pitch);  // choices of the blocks before this one (a cluster)
    const Slots<int> tmp = mem.part(4 * pitch, 32);
    const Slots<int> hist = mem.part(4 * pitch + 32, warps * keys);  // [warps][keys] counts of the tile, then starts inside the key
    const Slots<int> order = mem.part(4 * pitch + 32 + warps * keys, kOrder ? tile : 0);  // the tile in order,
    const Slots<unsigned short> order_key(reinterpret_cast<unsigned short*>(order.p + tile), kOrder ? tile : 0);  // and its keys
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const Slots<int> mine = hist.part(warp * keys, keys);
    const int64_t lo = (int64_t)blockIdx.x * per_block, hi = min(n, lo + per_block);
    const Slots<int> first = many ? start : base;
    int64_t at = lo;
    do {
        int key[R], rank[R];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int64_t i = at + ((int64_t)warp * R + r) * 32 + lane;
            key[r] = i < hi && BMMC_RD_OK(ids + i, sizeof(Id)) ? key_of(ids[i], experts) : none;  // none: a key past all others
        }
        for (int e = lane; e < keys; e += 32) mine.set(e, 0);
        __syncwarp();
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const unsigned same = same_key(key[r], bits);
            const bool there = key[r] < keys;
            const int before = there ? mine.get(key[r]) : 0;
            rank[r] = before + __popc(same & ((1u << lane) - 1));
            __syncwarp();
            if (there && lane == __ffs(same) - 1) mine.set(key[r], before + __popc(same));
            __syncwarp();
        }
        if (counts && at == lo) {
            for (int e = threadIdx.x; e < pitch; e += blockDim.x) base.set(e, 0), total.set(e, 0);
            __syncthreads();
            cudaGridDependencySynchronize();
            sum_counts(counts, pitch, base, total);
            __syncthreads();
            block_exclusive_scan(base, keys, tmp);
            for (int e = threadIdx.x; e < keys; e += blockDim.x) {
                const int from = base.get(e);
                if (blockIdx.x == 0 && BMMC_WR_OK(offsets + e, 4)) offsets[e] = from;
                base.set(e, from + total.get(e));
            }
        }
        __syncthreads();
        for (int e = threadIdx.x; e < keys; e += blockDim.x) {
            int run = 0;
#pragma unroll 4
            for (int w = 0; w < warps; ++w) {
                const int c = hist.get(w * keys + e);
                hist.set(w * keys + e, run);
                run += c;
            }
            total.set(e, run);
            first.set(e, run);
        }
        if (many && !counts) {  // the tiles' counts, from the blocks of the cluster
            const auto cluster = cooperative_groups::this_cluster();
            cluster.sync();
            for (int e = threadIdx.x; e < keys; e += blockDim.x) {
                int all = 0, before = 0;
                for (int b = 0; b < (int)gridDim.x; ++b) {
                    const int c = total.ok(e) ? *cluster.map_shared_rank(total.p + e, b) : 0;
                    all += c;
                    if (b < (int)blockIdx.x) before += c;
                }
                base.set(e, all);
                ahead.set(e, before);
            }
            cluster.sync();  // no block leaves while its counts are read
            block_exclusive_scan(base, keys, tmp);
            for (int e = threadIdx.x; e < keys; e += blockDim.x) {
                const int from = base.get(e);
                if (blockIdx.x == 0 && BMMC_WR_OK(offsets + e, 4)) offsets[e] = from;
                base.set(e, from + ahead.get(e));
            }
        }
        __syncthreads();
        block_exclusive_scan(first, keys, tmp);
        if (!many)
            for (int e = threadIdx.x; e < keys; e += blockDim.x)
                if (BMMC_WR_OK(offsets + e, 4)) offsets[e] = base.get(e);
#pragma unroll
        for (int r = 0; r < R; ++r) {
            if (key[r] >= keys) continue;
            const int in_tile = ((warp * R) + r) * 32 + lane, in_key = mine.get(key[r]) + rank[r];
            const int64_t i = at + in_tile;
            const int to = base.get(key[r]) + in_key;
            const bool routed = key[r] < experts;
            if (BMMC_WR_OK(slot + i, 4)) slot[i] = routed ? to : ~to;
            if (kOrder) {
                const int j = first.get(key[r]) + in_key;
                order.set(j, in_tile);
                order_key.set(j, (unsigned short)key[r]);
            } else if (BMMC_WR_OK(source + to, 4)) {
                source[to] = routed ? (int)i : ~(int)i;
            }
        }
        if (!kOrder) return;
        __syncthreads();
        const int here = (int)min((int64_t)blockDim.x * R, hi - at);
        for (int j = threadIdx.x; j < here; j += blockDim.x) {
            const int k = order_key.get(j), i = (int)at + order.get(j), to = many ? base.get(k) + j - start.get(k) : j;
            if ((unsigned)to < (unsigned)n && BMMC_WR_OK(source + to, 4)) source[to] = k < experts ? i : ~i;  // also if ids changed meanwhile
        }
        at += (int64_t)blockDim.x * R;
        if (at >= hi) return;
        __syncthreads();
        for (int e = threadIdx.x; e < keys; e += blockDim.x) base.set(e, base.get(e) + total.get(e));
    } while (true);
}

struct SortShape {
    int warps, blocks, rounds, pitch, bits;
    int64_t per_block;
    size_t smem;  // of the place kernel
};

constexpr size_t kSortSmem = 200 * 1024;

// One block where one tile covers all choices (of one round a warp where that
// is enough), a cluster of blocks of one tile each, else at most
// kMaxSortBlocks blocks of whole tiles.  A block has
// as many warps as their counts of every key leave room for.
SortShape sort_shape(int64_t n, int experts) {
    SortShape s;
    s.pitch = (experts + 4) & ~3;
    s.bits = 1;  // of the keys 0 .. experts and one past them
    while ((1 << s.bits) < experts + 2) ++s.bits;
    const auto smem = [&](int warps) {
        return ((size_t)warps * (experts + 1) + 4 * s.pitch + 32) * sizeof(int) + (size_t)warps * 32 * kSortRounds * 6;
    };
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
                        int32_t* offsets, int* counts, const chk::Spans& spans, cudaStream_t st) {
    (void)spans;
    const Id* ids = static_cast<const Id*>(ids_);
    const auto place = sort_place_kernel<Id, R>;
    if (s.smem > 48 * 1024) {
        static std::atomic<uint64_t> allowed{0};  // devices that were told, bit by bit (others are told every time)
        int dev = 0;
        if (cudaGetDevice(&dev) != cudaSuccess) {
            cudaGetLastError();
            return BMMC_ERR_CUDA;
        }
        if (dev >= 64 || !(allowed.load(std::memory_order_relaxed) >> dev & 1)) {
            if (cudaFuncSetAttribute(place, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSortSmem) != cudaSuccess) {
                cudaGetLastError();
                return BMMC_ERR_CUDA;
            }
            if (dev < 64) allowed.fetch_or((uint64_t)1 << dev, std::memory_order_relaxed);
        }
    }
    const int* none = nullptr;
    if (s.blocks <= kSortCluster) {
        cudaLaunchAttribute together{};
        together.id = cudaLaunchAttributeClusterDimension;
        together.val.clusterDim.x = s.blocks;
        together.val.clusterDim.y = together.val.clusterDim.z = 1;
        return launch(place, dim3(s.blocks), dim3(s.warps * 32), s.smem, st, s.blocks > 1 ? &together : nullptr, ids, n,
                      experts, s.per_block, s.pitch, s.bits, none, slot, source, offsets BMMC_SPANS_ARG(spans));
    }
    const bmmc_status counted = launch(sort_count_kernel<Id>, dim3(s.blocks), dim3(1024), s.pitch * sizeof(int), st, nullptr,
                                       ids, n, experts, s.per_block, s.pitch, counts BMMC_SPANS_ARG(spans));
    if (counted != BMMC_OK) return counted;
    cudaLaunchAttribute early{};
    early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    early.val.programmaticStreamSerializationAllowed = 1;
    return launch(place, dim3(s.blocks), dim3(s.warps * 32), s.smem, st, &early, ids, n, experts, s.per_block, s.pitch,
                  s.bits, (const int*)counts, slot, source, offsets BMMC_SPANS_ARG(spans));
}

// ---- rows staged in shared memory ------------------------------------------

constexpr int kStagedThreads = 128;
constexpr int kStagedChoices = 8;
constexpr int kStagedWords = 1100;  // of a block, 17.6 KB: a dozen blocks on an SM have 200 KB in flight

// Word j of the aligned words that hold a row's bytes from `start` on, copied
// asynchronously; zero where it holds none of the row's `bytes` (or row NULL).
__device__ __forceinline__ void stage_word(Slots<uint4> words, int to, const char* row, int64_t start, int bytes, int j) {
    const char* const p =
        reinterpret_cast<const char*>((reinterpret_cast<uintptr_t>(row) + start) & ~(uintptr_t)15) + (int64_t)j * 16;
    if (!words.ok(to)) return;
    if (row && p + 16 > row && p < row + bytes && BMMC_RD_WORD_OK(p, 16))
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"((unsigned)__cvta_generic_to_shared(words.p + to)), "l"(p)
                     : "memory");
    else
        words.set(to, uint4{});
}

// The block's words are there.
__device__ __forceinline__ void staged() {
    asm volatile("cp.async.wait_all;" ::: "memory");
    __syncthreads();
}

// 16 bytes of a row, `start` bytes behind its start, from the staged words j
// and j + 1 that hold them.
template <class T, int W>
__device__ __forceinline__ Pack<T, W> staged_pack(Slots<uint4> words, int j, const char* row, int64_t start) {
    Pack<T, W> y;
    y.word = cut(words.get(j), words.get(j + 1), (unsigned)(reinterpret_cast<uintptr_t>(row) + start) & 15u);
    return y;
}

// Where a part's staged words start for rows that lie differently: the aligned
// word 16 bytes before byte `at` of the row; part + 3 words reach over the part
// of every row.
__device__ __forceinline__ int64_t stage_from(int64_t at) { return at - 16; }

// 16 bytes from byte `start` of a row on, out of words staged from byte `from`.
template <class T, int W>
__device__ __forceinline__ Pack<T, W> staged_pack_at(Slots<uint4> words, const char* row, int64_t from, int64_t start) {
    const int at = (int)((reinterpret_cast<uintptr_t>(row) + start) -
                         ((reinterpret_cast<uintptr_t>(row) + from) & ~(uintptr_t)15));
    Pack<T, W> y;
    y.word = cut(words.get(at >> 4), words.get((at >> 4) + 1), at & 15);
    return y;
}

// How a row's packs are cut into parts of at most `most`, and the threads of a
// block that walk over one, with few of them idle in the last round.
struct Parts {
    int count, words, threads;
};

template <class T>
Parts parts_of(int64_t hidden, int most) {
    constexpr int W = 16 / sizeof(T);
    const int packs = (int)((hidden + 2 * (W - 1)) / W);
    Parts p;
    p.count = (packs + most - 1) / most;
    p.words = (packs + p.count - 1) / p.count;
    const int rounds = (p.words + kStagedThreads - 1) / kStagedThreads;
    p.threads = ((p.words + rounds - 1) / rounds + 31) / 32 * 32;
    return p;
}

// ---- dispatch ----------------------------------------------------------------

// Pure movement: a token's row is read once and written to the rows of its
// choices, one word a thread.  Bound by HBM: 16384 tokens of 4096 bf16 to 8
// rows each, 1.21 GB, 180.8 us = 6685 GB/s, a plain copy's rate; to 2 rows
// each 59.9 us (6720 GB/s).  32 tokens of 2048 to 4 rows: 1.7 us, a launch.
template <class Word>
__global__ void __launch_bounds__(256, 8) dispatch_kernel(const char* __restrict__ x, int64_t x_stride,
                                                          const int* __restrict__ slot, int64_t tokens, int choices,
                                                          int64_t n_rows, int words, char* __restrict__ rows,
                                                          int64_t row_stride BMMC_SPANS_PARAM) {
    BMMC_SPANS_ENTER_GLOBAL();
    const int64_t t = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
    const int w = blockIdx.y * blockDim.x + threadIdx.x;
    if (t >= tokens || w >= words) return;
    const Word* const from = reinterpret_cast<const Word*>(x + t * x_stride) + w;
    const Word v = BMMC_RD_OK(from, sizeof(Word)) ? __ldg(from) : Word{};
    slot += t * choices;
#pragma unroll 4
    for (int k = 0; k < choices; ++k) {
        const int s = BMMC_RD_OK(slot + k, 4) ? __ldg(slot + k) : 0;
        const int64_t row = s < 0 ? ~s : s;
        Word* const to = reinterpret_cast<Word*>(rows + row * row_stride) + w;
        if (row < n_rows && BMMC_WR_OK(to, sizeof(Word))) *to = s < 0 ? Word{} : v;
    }
}

// The same for rows at any element-aligned address.  Thread w holds the row's
// aligned words w - 1 and w, whatever row they go to: of a row that lies
// `to` bytes behind its granule (the source `from` bytes behind its own), the
// words w - 1 and w cover granule w - 1 where from >= to, else granule w.
// The loads do not wait for slot.  16384 x 2 rows of 4095 bf16: 81.7 us (long rows
// are faster staged, below); a form that read each choice's words once slot was
// known took 136-181.
template <class T>
__global__ void __launch_bounds__(256, 6) dispatch_across_kernel(const char* __restrict__ x, int64_t x_stride,
                                                                 const int* __restrict__ slot, int64_t tokens,
                                                                 int choices, int64_t n_rows, int length,
                                                                 char* __restrict__ rows, int64_t row_stride
                                                                     BMMC_SPANS_PARAM) {
    BMMC_SPANS_ENTER_GLOBAL();
    constexpr int W = 16 / sizeof(T);
    const int64_t t = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
    const int w = blockIdx.y * blockDim.x + threadIdx.x;
    if (t >= tokens) return;
    const char* const row_x = x + t * x_stride;
    const int from = (int)((unsigned)reinterpret_cast<uintptr_t>(row_x) & 15u);
    const int bytes = length * (int)sizeof(T);
    uint4 a, b;  // bytes [w * 16 - 16 - from, + 32) of the row
    const char* const word = row_x + (int64_t)w * 16 - from;
    load_if(w > 0 && w * 16 - 16 - from < bytes && BMMC_RD_WORD_OK(word - 16, 16), a, word - 16);
    load_if(w * 16 - from < bytes && BMMC_RD_WORD_OK(word, 16), b, word);
    slot += t * choices;
#pragma unroll 2
    for (int k = 0; k < choices; ++k) {
        const int s = BMMC_RD_OK(slot + k, 4) ? __ldg(slot + k) : 0;
        const int64_t row = s < 0 ? ~s : s;
        if (row >= n_rows) continue;
        char* const out = rows + row * row_stride;
        const Walk<T, W, true> walk(length, out);
        const int to = (int)((unsigned)reinterpret_cast<uintptr_t>(out) & 15u);
        const int g = from >= to ? w - 1 : w;
        if (g < 0 || !walk.in(g)) continue;
        Pack<T, W> o;
        o.word = s < 0 ? uint4{} : cut(a, b, (from - to) & 15);
        walk.store(o, out, g);
    }
}

// The same, staged: a block brings a part of a token's row into shared memory,
// each word once, and cuts every choice's packs there.  16384 x 2 rows of 4095
// bf16 63.4 us (from registers 83.0, floor 60.3), of 4092 62.0 (85.6 in words of 8
// bytes), 4096 x 8 52.4 (56.9); short rows lie idle too long: 65536 x 2 of 1025 91
// (87), of 513 70 (53).
template <class T>
__global__ void __launch_bounds__(kStagedThreads)
    dispatch_staged_kernel(const char* __restrict__ x, int64_t x_stride, const int* __restrict__ slot, int choices,
                           int64_t n_rows, int length, int part, char* __restrict__ rows,
                           int64_t row_stride BMMC_SPANS_PARAM) {
    constexpr int W = 16 / sizeof(T);
    extern __shared__ uint4 s_words[];  // [part + 3]
    BMMC_SPANS_ENTER(s_words, chk::dyn_smem_bytes());
    const Slots<uint4> words(s_words, part + 3);
    const int64_t t = blockIdx.x;
    const char* const row_x = x + t * x_stride;
    const int first = blockIdx.y * part;
    const int64_t from = stage_from((int64_t)first * 16);
    for (int j = threadIdx.x; j < part + 3; j += blockDim.x)
        stage_word(words, j, row_x, from, length * (int)sizeof(T), j);
    staged();
    slot += t * choices;
    for (int k = 0; k < choices; ++k) {
        const int s = BMMC_RD_OK(slot + k, 4) ? __ldg(slot + k) : 0;
        const int64_t row = s < 0 ? ~s : s;
        if (row >= n_rows) continue;
        char* const to = rows + row * row_stride;
        const Walk<T, W, true> walk(length, to);
        const int packs = min(part, walk.packs() - first);
        for (int j = threadIdx.x; j < packs; j += blockDim.x) {
            Pack<T, W> o;
            if (s < 0) o.word = {};
            else o = staged_pack_at<T, W>(words, row_x, from, (int64_t)walk.at(first + j) * (int)sizeof(T));
            walk.store(o, to, first + j);
        }
    }
}

// ---- combine -----------------------------------------------------------------

// A weight of the rows' type or of 32 bits.
template <class T>
__device__ __forceinline__ float weight_at(const void* weights, int in_f32, int64_t i) {
    const int bytes = in_f32 ? 4 : (int)sizeof(T);
    (void)bytes;
    if (!BMMC_RD_OK(static_cast<const char*>(weights) + i * bytes, bytes)) return 0.0f;
    return in_f32 ? static_cast<const float*>(weights)[i] : to_f32(static_cast<const T*>(weights)[i]);
}

// Each thread holds the sums of a word in 32 bits, adds the choices in order,
// KB of them loaded at a time, and rounds once.  A choice that is not there
// adds zero times zero.
//
// Bound by HBM once enough loads are in flight, and by how soon slot is there
// before.  Measured on bf16 rows of 4096, blocks of 128: 16384 x 2 choices
// (floor 60.3 us) KB = 2 with 8 x 256 threads on an SM 63.5, with the registers
// it would like 75, KB = 1 70.6; 4096 x 8 (45.2) KB = 8 with 4 x 256 46.1,
// without a bound on its registers and blocks of 256 55.9.  Rows that lie across
// words: two loads for one, and the cut; 4096 x 8 rows of 4095 60.7 us,
// 40961 x 2 rows of 1031 f32 93.3 (both faster staged, below).  The bound on the
// registers makes the 16-bit types spill one of them there (4 bytes).  32 tokens x
// 8 rows of 4096: 2.1 us.
template <class T, int W, int KB, bool ACROSS>
__global__ void __launch_bounds__(256, KB > 2 ? 4 : ACROSS && sizeof(T) == 2 ? 6 : 8)
    combine_kernel(const char* __restrict__ rows, int64_t row_stride, int64_t n_rows, const int* __restrict__ slot,
                   const void* __restrict__ weights, int weights_f32, int64_t tokens, int choices, int length,
                   char* __restrict__ out, int64_t out_stride BMMC_SPANS_PARAM) {
    BMMC_SPANS_ENTER_GLOBAL();
    const int64_t t = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
    const int w = blockIdx.y * blockDim.x + threadIdx.x;
    if (t >= tokens) return;
    char* const to = out + t * out_stride;
    using Way = Walk<T, W, ACROSS>;
    const Way walk(length, to);
    if (!walk.in(w)) return;
    float sum[W];
#pragma unroll
    for (int i = 0; i < W; ++i) sum[i] = 0.0f;
    for (int k0 = 0; k0 < choices; k0 += KB) {
        int s[KB];
        float f[KB];
        typename Way::Fetch y[KB];
#pragma unroll
        for (int j = 0; j < KB; ++j) {
            const bool there = k0 + j < choices;
            const int64_t at = t * choices + k0 + j;
            s[j] = there && BMMC_RD_OK(slot + at, 4) ? slot[at] : -1;
            f[j] = there && weights ? weight_at<T>(weights, weights_f32, at) : 1.0f;
        }
#pragma unroll
        for (int j = 0; j < KB; ++j) {
            const bool want = s[j] >= 0 && s[j] < n_rows;
            walk.fetch(y[j], want, rows + s[j] * row_stride, w);
            if (!want) f[j] = 0.0f;
        }
#pragma unroll
        for (int j = 0; j < KB; ++j) {
            const Pack<T, W> v = walk.get(y[j]);
#pragma unroll
            for (int i = 0; i < W; ++i) sum[i] = fmaf(f[j], v.get(i), sum[i]);
        }
    }
    Pack<T, W> o;
    o.set(sum);
    walk.store(o, to, w);
}

// The same, staged: a block brings a part of the rows of one token's choices
// into shared memory and adds the packs there.
//
// What the asynchronous copies have in flight takes no registers, which rows
// across words and few choices need.  40961 x 2 rows of 1031 f32, one in twenty
// choices left out, 74.7 us (from registers 93.3; with all of them 78.9, 94 % of
// the copy rate); 16384 x 2 rows of 4095 bf16 66.8 (89), of
// 4096 62.1 (64.3), 40960 x 2 of 1024 f32 73.0 (79.2); 8192 x 4 rows of 4095 61.7,
// 4096 x 8 58.5 (60.7).  But 4096 x 8 rows of 4096 57 (46.1): with many choices that
// lie in words there is enough in flight without, as there is for short rows:
// 65536 x 2 rows of 1024 bf16 78.5 (63.4), of 701 70.8 (61.7), of 1025 92.4 (102.4).
// Where the rule draws its lines, calls of about 450 MB, staged (from registers):
// in words of 16 bytes three choices of 4096 bf16 89.4 us (93.7), of 1024 93.0
// (92.7), of 4096 f32 87.9 (81.4); four 86.7 (79.3), f32 84.2 (73.8); eight 82.2
// (67.0).  In words of 8 bytes four choices of 4092 bf16 88.1 (94.9), of 4094 f32
// 81.6 (81.1); five 89.3 (100.0), f32 79.7 (92.3); six 88.9 (88.2), f32 79.4 (83.4);
// eight 83.8 (75.3), f32 74.3 (72.4): five and some of six would gain by it.
// Parts of 800 words, or of 1100 with two choices: 640 words 67.5 us at 16384 x 2
// x 4095, 2200 77.4 at 4096 x 8.
template <class T>
__global__ void __launch_bounds__(kStagedThreads)
    combine_staged_kernel(const char* __restrict__ rows, int64_t row_stride, int64_t n_rows,
                          const int* __restrict__ slot, const void* __restrict__ weights, int weights_f32, int choices,
                          int length, int part, unsigned part_magic, char* __restrict__ out,
                          int64_t out_stride BMMC_SPANS_PARAM) {
    constexpr int W = 16 / sizeof(T);
    extern __shared__ uint4 s_words[];  // [choices][part + 1]
    __shared__ const char* s_row[kStagedChoices];  // NULL: not there
    __shared__ float s_weight[kStagedChoices];
    BMMC_SPANS_ENTER(s_words, chk::dyn_smem_bytes(), s_row, sizeof(s_row), s_weight, sizeof(s_weight));
    const Slots<uint4> words(s_words, choices * (part + 1));
    const Slots<const char*> row(s_row, kStagedChoices);
    const Slots<float> weight(s_weight, kStagedChoices);
    const int64_t t = blockIdx.x;
    const int tid = threadIdx.x;
    char* const to = out + t * out_stride;
    const Walk<T, W, true> walk(length, to);
    const int first = blockIdx.y * part, packs = min(part, walk.packs() - first);
    if (packs <= 0) return;
    if (tid < choices) {
        const int64_t at = t * choices + tid;
        const int s = BMMC_RD_OK(slot + at, 4) ? slot[at] : -1;
        const float f = weights ? weight_at<T>(weights, weights_f32, at) : 1.0f;
        const bool there = s >= 0 && s < n_rows;
        row.set(tid, there ? rows + s * row_stride : nullptr);
        weight.set(tid, there ? f : 0.0f);
    }
    __syncthreads();
    const int64_t start = (int64_t)walk.at(first) * (int)sizeof(T);  // of the part in a row, bytes
    for (int x = tid; x < choices * (part + 1); x += blockDim.x) {
        const int k = quotient(x, part + 1, part_magic), j = x - k * (part + 1);
        if (j <= packs) stage_word(words, x, row.get(k), start, length * (int)sizeof(T), j);
    }
    staged();
    for (int j = tid; j < packs; j += blockDim.x) {
        float sum[W];
#pragma unroll
        for (int i = 0; i < W; ++i) sum[i] = 0.0f;
        for (int k = 0; k < choices; ++k) {
            const Pack<T, W> y = staged_pack<T, W>(words.part(k * (part + 1), part + 1), j, row.get(k), start);
            const float f = weight.get(k);
#pragma unroll
            for (int i = 0; i < W; ++i) sum[i] = fmaf(f, y.get(i), sum[i]);
        }
        Pack<T, W> o;
        o.set(sum);
        walk.store(o, to, first + j);
    }
}

// The sums of v[0..N) over groups of `lanes` lanes (a power of two), in a
// fixed order; every lane gets all of them.
template <int N>
__device__ __forceinline__ void sum_lanes(float (&v)[N], int lanes) {
    for (int d = lanes >> 1; d; d >>= 1)
#pragma unroll
        for (int j = 0; j < N; ++j) v[j] += __shfl_xor_sync(~0u, v[j], d);
}

// grad_rows[slot] = w * grad and grad_weights = <rows[slot], grad>, KB choices
// at a time; the products are summed in 32 bits, by lanes and then across
// them in a fixed order.  x threads (a power of two, or whole warps) walk a
// token's row.
//
// Bound by HBM: grad_rows is written and rows are read once, grad once for KB
// choices.  16384 x 8 rows of 4096 bf16, 2.28 GB: KB = 4 with 4 x 256 threads on
// an SM 337.5 us = 6760 GB/s; KB = 8 (106 registers) 405, a choice after the
// other with a barrier each 357.  16384 x 2: KB = 2 with 6 x 256 threads, 128 of them
// on a token's row, 98.7 us = 6800 GB/s; with the registers it would like 131.6.
// Rows that lie across words take two loads and two cuts a word, and the 16-bit
// types spill one register (4 bytes) for the six blocks.
template <class T, int W, int KB, bool ACROSS>
__global__ void __launch_bounds__(256, KB <= 2 ? 6 : 4) combine_backward_kernel(
    const char* __restrict__ grad, int64_t grad_stride, const char* __restrict__ rows, int64_t row_stride,
    int64_t n_rows, const int* __restrict__ slot, const void* __restrict__ weights, int weights_f32, int64_t tokens,
    int choices, int length, char* __restrict__ grad_rows, int64_t grad_row_stride, void* __restrict__ grad_weights
        BMMC_SPANS_PARAM) {
    __shared__ float s_part[8][KB];
    BMMC_SPANS_ENTER(s_part, sizeof(s_part));
    const Slots<float> part(&s_part[0][0], 8 * KB);  // [warps][choices]
    const int64_t t = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
    const bool live = t < tokens;
    const int x = blockDim.x, tid = threadIdx.y * x + threadIdx.x, lane = tid & 31, warp = tid >> 5;
    using Way = Walk<T, W, ACROSS>;
    constexpr int JB = ACROSS ? 1 : KB;  // choices whose words are in flight at once
    const char* const g_row = grad + t * grad_stride;
    for (int k0 = 0; k0 < choices; k0 += KB) {
        float dot[KB];
        int s[KB];
        float f[KB];
#pragma unroll
        for (int j = 0; j < KB; ++j) {
            const bool there = live && k0 + j < choices;
            const int64_t at = t * choices + k0 + j;
            dot[j] = 0.0f;
            s[j] = there && BMMC_RD_OK(slot + at, 4) ? slot[at] : -1 - (int)n_rows;
            f[j] = there ? weight_at<T>(weights, weights_f32, at) : 0.0f;
            if (s[j] < 0) f[j] = 0.0f;
        }
#pragma unroll
        for (int j0 = 0; j0 < KB; j0 += JB) {
            for (int w = threadIdx.x; w * W < length + (ACROSS ? W - 1 : 0); w += x) {
                typename Way::Fetch fg[ACROSS ? JB : 1], fy[JB];
                if (!ACROSS) Way(length, nullptr).fetch(fg[0], live, g_row, w);
#pragma unroll
                for (int j = 0; j < JB; ++j) {
                    const int slot_j = s[j0 + j];
                    const int64_t row = slot_j < 0 ? ~slot_j : slot_j;
                    const Way walk(length, grad_rows + row * grad_row_stride);
                    const bool want = slot_j >= 0 && row < n_rows && walk.in(w);
                    if (ACROSS) walk.fetch(fg[j], want, g_row, w);
                    walk.fetch(fy[j], want, rows + row * row_stride, w);
                }
#pragma unroll
                for (int j = 0; j < JB; ++j) {
                    const int slot_j = s[j0 + j];
                    const int64_t row = slot_j < 0 ? ~slot_j : slot_j;
                    char* const to = grad_rows + row * grad_row_stride;
                    const Way walk(length, to);
                    if (row >= n_rows || !walk.in(w)) continue;
                    Pack<T, W> o;
                    o.word = {};
                    if (slot_j >= 0) {
                        Pack<T, W> g = walk.get(fg[ACROSS ? j : 0]), y = walk.get(fy[j]);
                        walk.trim(g, w);
                        walk.trim(y, w);
                        float v[W];
#pragma unroll
                        for (int i = 0; i < W; ++i) {
                            dot[j0 + j] = fmaf(g.get(i), y.get(i), dot[j0 + j]);
                            v[i] = f[j0 + j] * g.get(i);
                        }
                        o.set(v);
                    }
                    walk.store(o, to, w);
                }
            }
        }
        sum_lanes(dot, x < 32 ? x : 32);
        if (x > 32) {
            if (k0) __syncthreads();
            if (lane == 0)
#pragma unroll
                for (int j = 0; j < KB; ++j)
                    part.set(warp * KB + j, dot[j]);
            __syncthreads();
            const int first = threadIdx.y * (x >> 5);
#pragma unroll
            for (int j = 0; j < KB; ++j) {
                dot[j] = 0.0f;
                for (int i = 0; i < x >> 5; ++i) dot[j] += part.get((first + i) * KB + j);
            }
        }
        if (live && threadIdx.x == 0)
#pragma unroll
            for (int j = 0; j < KB; ++j)
                if (k0 + j < choices) {
                    const int64_t at = t * choices + k0 + j;
                    const int bytes = weights_f32 ? 4 : (int)sizeof(T);
                    (void)bytes;
                    if (!BMMC_WR_OK(static_cast<char*>(grad_weights) + at * bytes, bytes)) continue;
                    if (weights_f32) static_cast<float*>(grad_weights)[at] = dot[j];
                    else static_cast<T*>(grad_weights)[at] = from_f32<T>(dot[j]);
                }
    }
}

// The same for rows that lie across words, staged: a block takes a token, brings
// part after part of grad and of its choices' rows into shared memory, each word
// once, and cuts the packs there.  40961 x 2 rows of 1031 f32 142.8 us (from
// registers 180.3, floor 126.6), 16384 x 2 of 4095 bf16 123.8 (132.9), 65536 x 2 of
// 1025 183 (206), 16384 x 8 of 513 108 (150), 4096 x 8 of 4095 146 (144), but
// 65536 x 2 of 257 106 (93).  Rows in words of 8 bytes are faster from registers
// (4096 x 8 of 4092 113, staged 142).  Bound by its instructions: at 16384 x 8 of
// 513, 107 us for 42 us of bytes, the issue slots are 82 % in use, by 105 M warp
// instructions, and warps that could issue wait their turn (3.3 of the 13.7 that
// stand by for each issue) more than they wait for loads (0.6).
template <class T>
__global__ void __launch_bounds__(kStagedThreads)
    combine_backward_staged_kernel(const char* __restrict__ grad, int64_t grad_stride, const char* __restrict__ rows,
                                   int64_t row_stride, int64_t n_rows, const int* __restrict__ slot,
                                   const void* __restrict__ weights, int weights_f32, int choices, int length, int part,
                                   unsigned part_magic, char* __restrict__ grad_rows, int64_t grad_row_stride,
                                   void* __restrict__ grad_weights BMMC_SPANS_PARAM) {
    constexpr int W = 16 / sizeof(T);
    extern __shared__ uint4 s_words[];  // [choices + 1][part + 3]: grad, then the choices' rows
    __shared__ const char* s_row[kStagedChoices + 1];  // NULL: not there
    __shared__ char* s_to[kStagedChoices];             // NULL: not written
    __shared__ float s_weight[kStagedChoices];
    __shared__ float s_dot[kStagedThreads / 32][kStagedChoices];
    BMMC_SPANS_ENTER(s_words, chk::dyn_smem_bytes(), s_row, sizeof(s_row), s_to, sizeof(s_to), s_weight, sizeof(s_weight),
                     s_dot, sizeof(s_dot));
    const int64_t t = blockIdx.x;
    const int tid = threadIdx.x, pitch = part + 3;
    const Slots<uint4> words(s_words, (choices + 1) * pitch);
    const Slots<const char*> row_of(s_row, kStagedChoices + 1);
    const Slots<char*> to_of(s_to, kStagedChoices);
    const Slots<float> weight(s_weight, kStagedChoices);
    const Slots<float> dots(&s_dot[0][0], kStagedThreads / 32 * kStagedChoices);  // [warps][choices]
    if (tid < choices) {
        const int64_t at = t * choices + tid;
        const int s = BMMC_RD_OK(slot + at, 4) ? slot[at] : 0;
        const int64_t row = s < 0 ? ~s : s;
        const float f = weight_at<T>(weights, weights_f32, at);
        const bool there = s >= 0 && row < n_rows;
        row_of.set(tid + 1, there ? rows + row * row_stride : nullptr);
        to_of.set(tid, row < n_rows ? grad_rows + row * grad_row_stride : nullptr);
        weight.set(tid, there ? f : 0.0f);
    }
    if (tid == 0) row_of.set(0, grad + t * grad_stride);
    float dot[kStagedChoices];
#pragma unroll
    for (int k = 0; k < kStagedChoices; ++k) dot[k] = 0.0f;
    for (int first = 0; first * W < length + W - 1; first += part) {
        __syncthreads();  // the rows are known; the last part's words are used
        const int64_t from = stage_from((int64_t)first * 16);
        for (int x = tid; x < (choices + 1) * pitch; x += blockDim.x) {
            const int k = quotient(x, pitch, part_magic);
            stage_word(words, x, row_of.get(k), from, length * (int)sizeof(T), x - k * pitch);
        }
        staged();
#pragma unroll
        for (int k = 0; k < kStagedChoices; ++k) {
            if (k >= choices) continue;
            char* const to = to_of.get(k);
            if (!to) continue;
            const char* const row = row_of.get(k + 1);
            const Walk<T, W, true> walk(length, to);
            const int packs = min(part, walk.packs() - first);
            const float f = weight.get(k);
            for (int j = tid; j < packs; j += blockDim.x) {
                Pack<T, W> o;
                o.word = {};
                if (row) {
                    const int64_t start = (int64_t)walk.at(first + j) * (int)sizeof(T);
                    Pack<T, W> g = staged_pack_at<T, W>(words.part(0, pitch), row_of.get(0), from, start);
                    Pack<T, W> y = staged_pack_at<T, W>(words.part((k + 1) * pitch, pitch), row, from, start);
                    walk.trim(g, first + j);
                    walk.trim(y, first + j);
                    float v[W];
#pragma unroll
                    for (int i = 0; i < W; ++i) {
                        dot[k] = fmaf(g.get(i), y.get(i), dot[k]);
                        v[i] = f * g.get(i);
                    }
                    o.set(v);
                }
                walk.store(o, to, first + j);
            }
        }
    }
    sum_lanes(dot, 32);
    if ((tid & 31) == 0)
#pragma unroll
        for (int k = 0; k < kStagedChoices; ++k) dots.set((tid >> 5) * kStagedChoices + k, dot[k]);
    __syncthreads();
    if (tid < choices) {
        float sum = 0.0f;
        for (int i = 0; i < (int)blockDim.x >> 5; ++i) sum += dots.get(i * kStagedChoices + tid);
        const int64_t at = t * choices + tid;
        const int bytes = weights_f32 ? 4 : (int)sizeof(T);
        (void)bytes;
        if (!BMMC_WR_OK(static_cast<char*>(grad_weights) + at * bytes, bytes)) return;
        if (weights_f32) static_cast<float*>(grad_weights)[at] = sum;
        else static_cast<T*>(grad_weights)[at] = from_f32<T>(sum);
    }
}

bmmc_status check_moves(int64_t tokens, int choices, int64_t hidden, int64_t n_rows, int type, int* es) {
    if (!(*es = dtype_bytes(type))) return BMMC_ERR_UNSUPPORTED_ELEM;
    if (tokens < 0 || choices < 1 || choices > EXPERT_MAX_CHOICES || tokens > kMaxTokens / choices || hidden < 1 ||
        hidden > (1 << 24) || n_rows < 0 || n_rows > tokens * choices)
        return BMMC_ERR_INVALID_ARG;
    return BMMC_OK;
}

}  // namespace

extern "C" {

bmmc_status expert_sort_workspace(int64_t tokens, int choices, int experts, size_t* bytes) {
    if (!bytes) return BMMC_ERR_INVALID_ARG;
    *bytes = 0;
    if (tokens < 0 || choices < 1 || choices > EXPERT_MAX_CHOICES || tokens > kMaxTokens / choices || experts < 1 ||
        experts > kMaxExperts)
        return BMMC_ERR_INVALID_ARG;
    const SortShape s = sort_shape(tokens * choices, experts);
    *bytes = s.blocks > kSortCluster ? (size_t)s.blocks * s.pitch * sizeof(int) : 0;
    return BMMC_OK;
}

bmmc_status expert_sort(const void* ids, int id_bytes, int64_t tokens, int choices, int experts, int32_t* slot,
                        int32_t* source, int32_t* offsets, void* workspace, size_t workspace_bytes, void* stream) {
    size_t need = 0;
    bmmc_status s = expert_sort_workspace(tokens, choices, experts, &need);
    if (s != BMMC_OK) return s;
    const bool device = device_pointers(id_bytes);
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
    if ((s = all_reachable(device, {ids, slot, source, offsets, need ? workspace : nullptr})) != BMMC_OK) return s;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    int* counts = static_cast<int*>(need ? workspace : nullptr);
    const SortShape shape = sort_shape(n, experts);
    const chk::Spans spans = spans_of({in, o[3]}, {o[0], o[1], o[2], o[3]});
    const auto go = [&](auto launch) { return launch(shape, ids, n, experts, slot, source, offsets, counts, spans, st); };
    if (id_bytes == 4) return shape.rounds == 1 ? go(launch_sort<int32_t, 1>) : go(launch_sort<int32_t, kSortRounds>);
    return shape.rounds == 1 ? go(launch_sort<int64_t, 1>) : go(launch_sort<int64_t, kSortRounds>);
}

bmmc_status expert_dispatch(const void* x, int64_t x_stride, const int32_t* slot, int64_t tokens, int choices,
                            int64_t hidden, int type, void* rows, int64_t row_stride, int64_t n_rows, void* stream) {
    int es = 0;
    const bool device = device_pointers(type);
    bmmc_status s = check_moves(tokens, choices, hidden, n_rows, type, &es);
    if (s != BMMC_OK) return s;
    if (bad_stride(x_stride, tokens) || bad_output_stride(row_stride, hidden, n_rows)) return BMMC_ERR_INVALID_ARG;
    if (!n_rows) return BMMC_OK;
    if (!x || !slot || !rows) return BMMC_ERR_INVALID_ARG;
    if (misaligned(x, es) || misaligned(rows, es) || misaligned(slot, 4)) return BMMC_ERR_MISALIGNED;
    const Rows in{x, tokens, x_stride * es, hidden * es}, out{rows, n_rows, row_stride * es, hidden * es};
    if (may_overlap(in, out) || may_overlap({slot, 1, 0, tokens * choices * 4}, out)) return BMMC_ERR_ALIAS;
    if ((s = all_reachable(device, {x, slot, rows})) != BMMC_OK) return s;
    const Way way = way_of(hidden, es, {(uint64_t)(uintptr_t)x, (uint64_t)(uintptr_t)rows, (uint64_t)(x_stride * es),
                                   (uint64_t)(row_stride * es), (uint64_t)(hidden * es)});
    const int words = way.words;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const char* from = static_cast<const char*>(x);
    char* to = static_cast<char*>(rows);
    const int most = tokens * words <= kFewWords ? 128 : 256;
    const chk::Spans spans = spans_of({in, {slot, 1, 0, tokens * choices * 4}}, {out});
    (void)spans;
    const bool staged = way.bytes < 16 && tokens * words > kFewWords && hidden * es >= 4096;
    const auto copy = [&](auto word) {
        const Cover c = cover(tokens, words, most);
        return launch(dispatch_kernel<decltype(word)>, c.grid, c.block, 0, st, nullptr, from, x_stride * es, slot, tokens,
                      choices, n_rows, words, to, row_stride * es BMMC_SPANS_ARG(spans));
    };
    const auto across = [&](auto e) {
        using T = decltype(e);
        if (staged) {
            const Parts p = parts_of<T>(hidden, kStagedWords);
            return launch(dispatch_staged_kernel<T>, dim3((unsigned)tokens, p.count), dim3(p.threads),
                          (size_t)(p.words + 3) * 16, st, nullptr, from, x_stride * es, slot, choices, n_rows, (int)hidden,
                          p.words, to, row_stride * es BMMC_SPANS_ARG(spans));
        }
        const Cover c = cover(tokens, words + 1, most);  // one more: thread 0 holds no word w - 1
        return launch(dispatch_across_kernel<T>, c.grid, c.block, 0, st, nullptr, from, x_stride * es, slot,
                      tokens, choices, n_rows, (int)hidden, to, row_stride * es BMMC_SPANS_ARG(spans));
    };
    if (way.bytes == 16) return copy(uint4{});
    if (way.bytes == 8 && !staged) return copy(uint2{});
    return es == 4 ? across(uint32_t{}) : across(uint16_t{});
}

bmmc_status expert_combine(const void* rows, int64_t row_stride, int64_t n_rows, const int32_t* slot,
                           const void* weights, int weight_type, int64_t tokens, int choices, int64_t hidden, int type,
                           void* out, int64_t out_stride, void* stream) {
    int es = 0;
    const bool device = device_pointers(type);
    bmmc_status s = check_moves(tokens, choices, hidden, n_rows, type, &es);
    if (s != BMMC_OK) return s;
    if (weights && weight_type != BMMC_F32 && weight_type != type) return BMMC_ERR_UNSUPPORTED_ELEM;
    if (bad_stride(row_stride, n_rows) || bad_output_stride(out_stride, hidden, tokens)) return BMMC_ERR_INVALID_ARG;
    if (!tokens) return BMMC_OK;
    if ((!rows && n_rows) || !slot || !out) return BMMC_ERR_INVALID_ARG;
    const int ws = weights ? dtype_bytes(weight_type) : 4;
    if (misaligned(rows, es) || misaligned(out, es) || misaligned(slot, 4) || misaligned(weights, ws))
        return BMMC_ERR_MISALIGNED;
    const Rows to{out, tokens, out_stride * es, hidden * es};
    if (may_overlap({rows, n_rows, row_stride * es, hidden * es}, to) ||
        may_overlap({slot, 1, 0, tokens * choices * 4}, to) || may_overlap({weights, 1, 0, tokens * choices * ws}, to))
        return BMMC_ERR_ALIAS;
    if ((s = all_reachable(device, {rows, slot, weights, out})) != BMMC_OK) return s;
    const Way way = way_of(hidden, es, {(uint64_t)(uintptr_t)rows, (uint64_t)(uintptr_t)out, (uint64_t)(row_stride * es),
                                   (uint64_t)(out_stride * es), (uint64_t)(hidden * es)});
    const int words = way.words;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const chk::Spans spans = spans_of({{rows, n_rows, row_stride * es, hidden * es}, {slot, 1, 0, tokens * choices * 4},
                                       {weights, 1, 0, tokens * choices * ws}}, {to});
    (void)spans;
    by_type(type, way, [&](auto e, auto width, auto across) {
        using T = decltype(e);
        constexpr int W = decltype(width)::value;
        constexpr bool A = decltype(across)::value;
        const Cover c = cover(tokens, words, 128);
        const int64_t bytes = choices * hidden * es;  // of a token's rows
        if (choices <= kStagedChoices && tokens * words > kFewWords &&
            (way.bytes == 16 ? choices <= 2 && bytes >= 8192 : bytes >= 4096 && (A || choices <= 4))) {
            const Parts p = parts_of<T>(hidden, (choices <= 2 ? kStagedWords : 800) / choices);
            s = launch(combine_staged_kernel<T>, dim3((unsigned)tokens, p.count), dim3(p.threads),
                       (size_t)choices * (p.words + 1) * 16, st, nullptr, static_cast<const char*>(rows), row_stride * es,
                       n_rows, slot, weights, int(weight_type == BMMC_F32), choices, (int)hidden, p.words,
                       magic_of(p.words + 1), static_cast<char*>(out), out_stride * es BMMC_SPANS_ARG(spans));
            return;
        }
        auto kernel = combine_kernel<T, W, 2, A>;
        if constexpr (!A)
            if (choices > 2) kernel = choices <= 4 ? combine_kernel<T, W, 4, A> : combine_kernel<T, W, 8, A>;
        s = launch(kernel, c.grid, c.block, 0, st, nullptr, static_cast<const char*>(rows), row_stride * es, n_rows, slot,
                   weights, int(weight_type == BMMC_F32), tokens, choices, (int)hidden, static_cast<char*>(out),
                   out_stride * es BMMC_SPANS_ARG(spans));
    });
    return s;
}

bmmc_status expert_combine_backward(const void* grad, int64_t grad_stride, const void* rows, int64_t row_stride,
                                    int64_t n_rows, const int32_t* slot, const void* weights, int weight_type,
                                    int64_t tokens, int choices, int64_t hidden, int type, void* grad_rows,
                                    int64_t grad_row_stride, void* grad_weights, void* stream) {
    int es = 0;
    const bool device = device_pointers(type);
    bmmc_status s = check_moves(tokens, choices, hidden, n_rows, type, &es);
    if (s != BMMC_OK) return s;
    if (weight_type != BMMC_F32 && weight_type != type) return BMMC_ERR_UNSUPPORTED_ELEM;
    if (bad_stride(grad_stride, tokens) || bad_stride(row_stride, n_rows) ||
        bad_output_stride(grad_row_stride, hidden, n_rows))
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
    if ((s = all_reachable(device, {grad, rows, slot, weights, grad_rows, grad_weights})) != BMMC_OK) return s;
    const Way way = way_of(hidden, es, {(uint64_t)(uintptr_t)grad, (uint64_t)(uintptr_t)rows, (uint64_t)(uintptr_t)grad_rows,
                                   (uint64_t)(grad_stride * es), (uint64_t)(row_stride * es),
                                   (uint64_t)(grad_row_stride * es), (uint64_t)(hidden * es)});
    const int words = way.words;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const int most = choices <= 2 || !way.bytes ? 128 : 256;
    int x = 4;
    while (x < words && x < most) x <<= 1;
    const dim3 block(x, 256 / x);
    const unsigned blocks = (unsigned)((tokens + block.y - 1) / block.y);
    const chk::Spans spans = spans_of({in[0], in[1], in[2], in[3]}, {gr, gw});
    (void)spans;
    by_type(type, way, [&](auto e, auto width, auto across) {
        using T = decltype(e);
        constexpr int W = decltype(width)::value;
        constexpr bool A = decltype(across)::value;
        if (A && choices <= kStagedChoices && tokens * words > kFewWords && hidden * es >= 1024) {
            const Parts p = parts_of<T>(hidden, kStagedWords / (choices + 1));
            s = launch(combine_backward_staged_kernel<T>, dim3((unsigned)tokens), dim3(p.threads),
                       (size_t)(choices + 1) * (p.words + 3) * 16, st, nullptr, static_cast<const char*>(grad),
                       grad_stride * es, static_cast<const char*>(rows), row_stride * es, n_rows, slot, weights,
                       int(weight_type == BMMC_F32), choices, (int)hidden, p.words, magic_of(p.words + 3),
                       static_cast<char*>(grad_rows), grad_row_stride * es, grad_weights BMMC_SPANS_ARG(spans));
            return;
        }
        auto kernel = combine_backward_kernel<T, W, 2, A>;
        if constexpr (!A)
            if (choices > 2) kernel = combine_backward_kernel<T, W, 4, A>;
        s = launch(kernel, dim3(blocks), block, 0, st, nullptr, static_cast<const char*>(grad), grad_stride * es,
                   static_cast<const char*>(rows), row_stride * es, n_rows, slot, weights, int(weight_type == BMMC_F32),
                   tokens, choices, (int)hidden, static_cast<char*>(grad_rows), grad_row_stride * es,
                   grad_weights BMMC_SPANS_ARG(spans));
    });
    return s;
}

}  // extern "C"

namespace bmmc {
cudaError_t bounds_record_experts(unsigned long long out[chk::kRecordWords], bool clear) {
    return chk::read_record(out, clear);
}
}  // namespace bmmc
