// Host-side checks shared by the entry points that move tokens by maps held
// on the device (experts.cu, rotary.cu).  Each includes bounds.cuh before this
// header.
#pragma once

#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>
#include <initializer_list>

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

// Launch a kernel, with one attribute or none.
template <class... P, class... A>
bmmc_status launch(void (*kernel)(P...), dim3 grid, dim3 block, size_t smem, cudaStream_t st,
                   cudaLaunchAttribute* attribute, const A&... args) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cfg.attrs = attribute;
    cfg.numAttrs = attribute ? 1 : 0;
    if (cudaLaunchKernelEx(&cfg, kernel, P(args)...) == cudaSuccess) return BMMC_OK;
    cudaGetLastError();
    return BMMC_ERR_CUDA;
}

}  // namespace bmmc
