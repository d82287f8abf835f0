// Host-side checks shared by the entry points that move tokens by maps held
// on the device (experts.cu, rotary.cu, paged_cache8.cu, embedding.cu,
// balance.cu).  Each includes bounds.cuh before this header.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cstdint>
#include <initializer_list>
#include <type_traits>

#include "../../include/bmmc.h"
#include "launch.hpp"

namespace bmmc {

constexpr int64_t kMaxStride = (int64_t)1 << 40;  // elements
constexpr int64_t kMaxTokens = ((int64_t)1 << 31) - 1;

// SMs of a GB300.  Rules that ask whether a call fills the machine count in
// them; on another number of SMs they choose another form, with the same
// results.
constexpr int kSms = 152;

// Whether a stride is out of range, or `n` steps of it lead further than any
// memory (so that byte offsets stay far below 2^63).
inline bool bad_stride(int64_t stride, int64_t n) {
    return stride < 0 || stride > kMaxStride || (n > 1 && stride > ((int64_t)1 << 50) / (n - 1));
}

// Bytes of one element; 0 for an unknown type.
inline int dtype_bytes(int type) {
    switch (type) {
        case BMMC_F32: return 4;
        case BMMC_F16: case BMMC_BF16: return 2;
    }
    return 0;
}

// An array of `rows` rows, `stride` bytes apart, `span` bytes each.
struct Rows {
    const void* base;
    int64_t rows, stride, span;
    uintptr_t lo() const { return (uintptr_t)base; }
    uintptr_t hi() const { return rows < 1 ? lo() : lo() + (uintptr_t)((rows - 1) * stride + span); }
};

// The ranges a checked build's launch may read and write (others drop them).
inline chk::Spans spans_of(std::initializer_list<Rows> rd, std::initializer_list<Rows> wr) {
    chk::Spans s{};
    if constexpr (chk::kEnabled) {
        for (const Rows& r : rd)
            if (r.base && r.rows > 0) s.rd[s.n_rd++] = chk::Span{r.lo(), r.hi()};
        for (const Rows& r : wr)
            if (r.base && r.rows > 0) s.wr[s.n_wr++] = chk::Span{r.lo(), r.hi()};
    }
    return s;
}

// Whether two arrays may share bytes.  Rows with one common stride that do
// not run into each other are told apart (slices of one fused projection);
// any other two whose address ranges meet count as overlapping.
inline bool may_overlap(const Rows& a, const Rows& b) {
    if (!a.base || !b.base || a.rows < 1 || b.rows < 1) return false;
    if (a.hi() <= b.lo() || b.hi() <= a.lo()) return false;
    if (a.stride != b.stride || a.stride <= 0) return true;
    const int64_t s = a.stride;
    int64_t d = (int64_t)(b.lo() - a.lo()) % s;
    if (d < 0) d += s;
    return !(d >= a.span && d + b.span <= s);
}

// Whether two arrays of the same sizes and strides, b `distance` behind a, share
// no address though their ranges meet.  The elements of each have addresses of
// their own, so its dimensions nest.  From the slowest one inwards: rows that
// lie in each other's gaps do not meet; where both rows of one number lie
// within the stride, only those can meet, and their insides decide.  In bytes;
// runs are the innermost, dense dimension.
template <int N>
bool lie_between(int64_t run_a, int64_t run_b, const int64_t (&sizes)[N], const int64_t (&strides)[N], int64_t distance) {
    int order[N];
    for (int i = 0; i < N; ++i) order[i] = i;
    std::sort(order, order + N, [&](int x, int y) { return strides[x] > strides[y]; });
    for (int k = 0; k < N; ++k) {
        const int64_t s = strides[k], d = s ? (distance % s + s) % s : 0;
        if (sizes[k] < 2) continue;
        __int128 rest = 0;
        for (int j = 0; j < N; ++j)
            if (sizes[j] > 1 && strides[j] % s) rest += (__int128)(sizes[j] - 1) * strides[j];
        if (d >= run_a + rest && d + run_b + rest <= s) return true;
    }
    for (int k = 0; k < N; ++k) {
        const int64_t s = strides[order[k]];
        if (sizes[order[k]] < 2) continue;
        __int128 rest = 0;
        for (int j = k + 1; j < N; ++j)
            if (sizes[order[j]] > 1) rest += (__int128)(sizes[order[j]] - 1) * strides[order[j]];
        if (run_a + rest > s || run_b + rest > s) return false;  // (no nest: only where runs have gaps, see below)
        const int64_t d = (distance % s + s) % s;  // from a row of a to the row of b that starts behind it
        if (d >= run_a + rest) {
            if (d + run_b + rest <= s) return true;
            distance = d - s;
        } else {
            if (d + run_b + rest > s) return false;
            distance = d;
        }
    }
    return distance >= run_a || distance + run_b <= 0;
}

// The same for two arrays of the same sizes whose strides may differ: a dimension
// with two strides is taken as a part of the runs, gaps and all.
template <int N>
bool lie_between(int64_t run_a, int64_t run_b, const int64_t (&sizes)[N], const int64_t (&a)[N], const int64_t (&b)[N],
                 int64_t distance) {
    int64_t nest[N];
    for (int i = 0; i < N; ++i) {
        nest[i] = a[i] == b[i] ? sizes[i] : 1;
        if (nest[i] == sizes[i]) continue;
        run_a += (sizes[i] - 1) * a[i];
        run_b += (sizes[i] - 1) * b[i];
    }
    return lie_between(run_a, run_b, nest, a, distance);
}

// Whether the elements of an array with these sizes and strides (elements;
// the innermost dimension has unit stride) have addresses of their own.
template <int N>
bool one_to_one(int64_t inner, const int64_t (&sizes)[N], const int64_t (&strides)[N]) {
    int order[N];
    for (int i = 0; i < N; ++i) order[i] = i;
    std::sort(order, order + N, [&](int x, int y) { return strides[x] < strides[y]; });
    __int128 span = inner;  // addresses the faster dimensions reach over
    for (int k = 0; k < N; ++k) {
        const int i = order[k];
        if (sizes[i] < 2) continue;
        if (strides[i] < span) return false;
        span += (__int128)(sizes[i] - 1) * strides[i];
    }
    return true;
}

// The widest word (16, 8, 4 or 2 bytes, at least one element) that divides
// every address, stride and length given in bytes.
inline int word_bytes(int elem, std::initializer_list<uint64_t> all) {
    uint64_t m = 16;
    for (uint64_t v : all) m |= v;
    const int w = (int)(m & (~m + 1));  // lowest set bit: at most 16
    return w < elem ? elem : w;
}

// Takes the flag off a call's type (or width of ids).
inline bool device_pointers(int& type) {
    const bool device = type >= 0 && (type & BMMC_DEVICE_POINTERS);
    if (device) type &= ~BMMC_DEVICE_POINTERS;
    return device;
}

inline bmmc_status all_reachable(bool device, std::initializer_list<const void*> ps) {
    if (device) return BMMC_OK;
    for (const void* p : ps)
        if (p) {
            const bmmc_status s = pointer_reachable(p);
            if (s != BMMC_OK) return s;
        }
    return BMMC_OK;
}

// Launch a kernel with some attributes.
template <class... P, class... A>
bmmc_status launch_with(void (*kernel)(P...), dim3 grid, dim3 block, size_t smem, cudaStream_t st,
                        cudaLaunchAttribute* attributes, unsigned count, const A&... args) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cfg.attrs = attributes;
    cfg.numAttrs = count;
    if (cudaLaunchKernelEx(&cfg, kernel, P(args)...) == cudaSuccess) return BMMC_OK;
    cudaGetLastError();
    return BMMC_ERR_CUDA;
}

// The same with one attribute or none.
template <class... P, class... A>
bmmc_status launch(void (*kernel)(P...), dim3 grid, dim3 block, size_t smem, cudaStream_t st,
                   cudaLaunchAttribute* attribute, const A&... args) {
    return launch_with(kernel, grid, block, smem, st, attribute, attribute ? 1 : 0, args...);
}

// Lets a kernel have `smem` bytes of dynamic shared memory, kMostSmem at most;
// each device is told once.
constexpr size_t kMostSmem = 200 * 1024;

template <auto Kernel>
bmmc_status allow_smem(size_t smem) {
    static std::atomic<uint64_t> allowed{0};  // devices that were told, bit by bit (others are told every time)
    if (smem <= 40 * 1024) return BMMC_OK;    // (48 KB with the static arrays are always allowed)
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess && dev < 64 && (allowed.load(std::memory_order_relaxed) >> dev & 1)) return BMMC_OK;
    if (e == cudaSuccess) e = cudaFuncSetAttribute(Kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kMostSmem);
    if (e != cudaSuccess) {
        cudaGetLastError();
        return BMMC_ERR_CUDA;
    }
    if (dev < 64) allowed.fetch_or((uint64_t)1 << dev, std::memory_order_relaxed);
    return BMMC_OK;
}

// How the words of the tokens' rows are dealt out: blocks of x * y threads
// take y tokens and x words of each; gridDim.y parts make up a row.
struct Cover {
    dim3 grid, block;
};

constexpr int kMostParts = 65535;

// Up to this many words (one for every thread of the machine) the blocks are
// smaller, so that more of the machine takes part.
constexpr int64_t kFewWords = kSms * 2048;

inline Cover cover(int64_t tokens, int words, int most) {
    // a grid has 65535 parts at most: rows of 2^24 elements are up to 2^23 words
    while ((words + most - 1) / most > kMostParts) most <<= 1;
    const int parts = (words + most - 1) / most, need = (words + parts - 1) / parts;
    int x = 4;
    while (x < 32 && x < need) x <<= 1;
    if (x < need) x = (need + 31) / 32 * 32;
    const int y = x >= most ? 1 : most / x;
    Cover c;
    c.block = dim3(x, y);
    c.grid = dim3((unsigned)((tokens + y - 1) / y), (unsigned)((words + x - 1) / x));
    return c;
}

// How rows of `hidden` elements are walked: in words of 16 or 8 bytes where
// all addresses, strides and lengths (or'ed into `bits`, in bytes) are
// multiples of them, else across the words' bounds.
struct Way {
    int bytes;   // 16, 8 or 0: across
    int words;   // of a row; across: at most
};

inline Way way_of(int64_t hidden, int es, std::initializer_list<uint64_t> bits) {
    const int wb = word_bytes(es, bits);
    if (wb >= 8) return {wb, (int)(hidden * es / wb)};
    const int W = 16 / es;
    return {0, (int)((hidden + 2 * (W - 1)) / W)};
}

// Calls f(T{}, elements per word, across).
template <class T, class F>
void by_way(const Way& way, F&& f) {
    constexpr int es = sizeof(T);
    if (way.bytes == 16) f(T{}, std::integral_constant<int, 16 / es>{}, std::false_type{});
    else if (way.bytes == 8) f(T{}, std::integral_constant<int, 8 / es>{}, std::false_type{});
    else f(T{}, std::integral_constant<int, 16 / es>{}, std::true_type{});
}

template <class F>
void by_type(int type, const Way& way, F&& f) {
    switch (type) {
        case BMMC_F32: by_way<float>(way, f); break;
        case BMMC_F16: by_way<__half>(way, f); break;
        default: by_way<__nv_bfloat16>(way, f); break;
    }
}

// Rows that are written lie apart.
inline bool bad_output_stride(int64_t stride, int64_t hidden, int64_t rows) {
    return bad_stride(stride, rows) || (rows > 1 && stride < hidden);
}

inline bool misaligned(const void* p, size_t bytes) { return (uintptr_t)p & (bytes - 1); }

}  // namespace bmmc
