// A router's balance loss with the number of choices of each expert, and its
// gradient: expert_balance and expert_balance_backward (declared in
// include/bmmc.h).
//
// With p[t] the softmax of token t's logits, c[e] the routed choices of expert
// e, C their sum, n the tokens that have one and f[e] = c[e] / C:
//   loss = E * sum over e of f[e] * (sum over those tokens of p[t][e]) / n,
//   d loss / d logit[t][e] = E / n * p[t][e] * (f[e] - sum over j of f[j] * p[t][j]),
// as the counts do not depend on the logits.
#include <cuda_runtime.h>

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
constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kMaxBlocks = 2 * kSms;

template <class T>
__device__ __forceinline__ float logit(const T* row, int e) {
    return BMMC_RD_OK(row + e, sizeof(T)) ? to_f32(row[e]) : 0.0f;
}

// Whether a token's choices hold one that is routed, and (in hist) how many
// each expert has of them; by a warp.
template <class Id, bool COUNT>
__device__ __forceinline__ bool routed(const Id* ids, int choices, int experts, int lane, Slots<int> hist) {
    bool any = false;
    for (int k = lane; k < choices; k += 32) {
        const Id id = BMMC_RD_OK(ids + k, sizeof(Id)) ? ids[k] : (Id)-1;
        const bool there = id >= 0 && id < (Id)experts;
        if (COUNT && there) hist.add((int)id, 1);
        any |= there;
    }
    return __any_sync(~0u, any);
}

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
    for (int d = 16; d; d >>= 1) v = fmaxf(v, __shfl_xor_sync(~0u, v, d));
    return v;
}
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int d = 16; d; d >>= 1) v += __shfl_xor_sync(~0u, v, d);
    return v;
}

// What a row's softmax subtracts and divides by, by a warp.  A row whose
// logits are all -inf has shares of zero: nothing is subtracted from it, its
// sum is zero and *over is zero.
template <class T>
__device__ __forceinline__ float softmax_of(const T* row, int experts, int lane, float* over) {
    float m = -INFINITY, sum = 0.0f;
    for (int e = lane; e < experts; e += 32) m = fmaxf(m, logit(row, e));
    m = warp_max(m);
    if (m == -INFINITY) m = 0.0f;
    for (int e = lane; e < experts; e += 32) sum += expf(logit(row, e) - m);
    sum = warp_sum(sum);
    *over = sum == 0.0f ? 0.0f : 1.0f / sum;
    return m;
}

// Each block's sums of p[t][e] over its tokens, and its counts.
template <class T, class Id>
__global__ void __launch_bounds__(kThreads) balance_part_kernel(const char* __restrict__ logits, int64_t stride,
                                                                const Id* __restrict__ ids, int64_t tokens, int choices,
                                                                int experts, float* __restrict__ sums,
                                                                int* __restrict__ counts BMMC_SPANS_PARAM) {
    extern __shared__ int s_mem[];
    BMMC_SPANS_ENTER(s_mem, chk_dynamic_bytes());
    const Slots<int> mem(s_mem, (kWarps + 1) * experts + 1), hist = mem.part(0, experts + 1);
    const Slots<float> all(reinterpret_cast<float*>(s_mem + experts + 1), kWarps * experts);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const Slots<float> mine = all.part(warp * experts, experts);
    for (int e = threadIdx.x; e <= experts; e += kThreads) hist.set(e, 0);
    for (int e = lane; e < experts; e += 32) mine.set(e, 0.0f);
    __syncthreads();
    for (int64_t t = (int64_t)blockIdx.x * kWarps + warp; t < tokens; t += (int64_t)gridDim.x * kWarps) {
        if (!routed<Id, true>(ids + t * choices, choices, experts, lane, hist)) continue;
        if (lane == 0) hist.add(experts, 1);
        const T* const row = reinterpret_cast<const T*>(logits + t * stride);
        float over;
        const float m = softmax_of(row, experts, lane, &over);
        for (int e = lane; e < experts; e += 32) mine.set(e, mine.get(e) + expf(logit(row, e) - m) * over);
    }
    __syncthreads();
    for (int e = threadIdx.x; e <= experts; e += kThreads) {
        float sum = 0.0f;
        if (e < experts)
            for (int w = 0; w < kWarps; ++w) sum += all.get(w * experts + e);
        const int64_t at = (int64_t)blockIdx.x * (experts + 1) + e;
        if (BMMC_WR_OK(sums + at, 4)) sums[at] = sum;
        if (BMMC_WR_OK(counts + at, 4)) counts[at] = hist.get(e);
    }
}

// The blocks' sums and counts joined, in their order.
__global__ void __launch_bounds__(1024) balance_join_kernel(const float* __restrict__ sums, const int* __restrict__ counts,
                                                            int blocks, int experts, float* __restrict__ loss,
                                                            int* __restrict__ out_counts BMMC_SPANS_PARAM) {
    __shared__ double s_dot[32];
    __shared__ long long s_all[32];
    __shared__ int s_tokens[1];
    BMMC_SPANS_ENTER(s_dot, sizeof(s_dot), s_all, sizeof(s_all), s_tokens, sizeof(s_tokens));
    const Slots<double> dots(s_dot, 32);
    const Slots<long long> alls(s_all, 32);
    const Slots<int> there(s_tokens, 1);
    double dot = 0.0;
    long long all = 0;
    for (int e = threadIdx.x; e <= experts; e += 1024) {
        double sum = 0.0;
        int count = 0;
#pragma unroll 8
        for (int b = 0; b < blocks; ++b) {
            const int64_t at = (int64_t)b * (experts + 1) + e;
            sum += BMMC_RD_OK(sums + at, 4) ? sums[at] : 0.0f;
            count += BMMC_RD_OK(counts + at, 4) ? counts[at] : 0;
        }
        if (BMMC_WR_OK(out_counts + e, 4)) out_counts[e] = count;
        if (e == experts) there.set(0, count);
        else if (count) dot += sum * count, all += count;  // (an expert without choices has no part, whatever its sum)
    }
    for (int d = 16; d; d >>= 1) {
        dot += __shfl_xor_sync(~0u, dot, d);
        all += __shfl_xor_sync(~0u, all, d);
    }
    if ((threadIdx.x & 31) == 0) dots.set(threadIdx.x >> 5, dot), alls.set(threadIdx.x >> 5, all);
    __syncthreads();
    if (threadIdx.x) return;
    dot = 0.0, all = 0;
    for (int w = 0; w < 32; ++w) dot += dots.get(w), all += alls.get(w);
    const int n = there.get(0);
    if (BMMC_WR_OK(loss, 4)) *loss = n ? (float)(dot * experts / ((double)all * n)) : 0.0f;
}

template <class T, class Id>
__global__ void __launch_bounds__(kThreads) balance_backward_kernel(
    const float* __restrict__ grad, const char* __restrict__ logits, int64_t stride, const Id* __restrict__ ids,
    int64_t tokens, int choices, int experts, const int* __restrict__ counts, char* __restrict__ out, int64_t out_stride
        BMMC_SPANS_PARAM) {
    extern __shared__ int s_mem[];
    __shared__ int s_all[kWarps];
    BMMC_SPANS_ENTER(s_mem, chk_dynamic_bytes(), s_all, sizeof(s_all));
    const Slots<float> share(reinterpret_cast<float*>(s_mem), experts);
    const Slots<int> alls(s_all, kWarps);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int all = 0;
    for (int e = threadIdx.x; e < experts; e += kThreads) all += BMMC_RD_OK(counts + e, 4) ? counts[e] : 0;
    for (int d = 16; d; d >>= 1) all += __shfl_xor_sync(~0u, all, d);
    if (lane == 0) alls.set(warp, all);
    __syncthreads();
    all = 0;
    for (int w = 0; w < kWarps; ++w) all += alls.get(w);
    const int n = BMMC_RD_OK(counts + experts, 4) ? counts[experts] : 0;
    for (int e = threadIdx.x; e < experts; e += kThreads)
        share.set(e, all ? (BMMC_RD_OK(counts + e, 4) ? (float)counts[e] : 0.0f) / (float)all : 0.0f);
    const float factor = n ? (BMMC_RD_OK(grad, 4) ? *grad : 0.0f) * ((float)experts / (float)n) : 0.0f;
    __syncthreads();
    for (int64_t t = (int64_t)blockIdx.x * kWarps + warp; t < tokens; t += (int64_t)gridDim.x * kWarps) {
        T* const to = reinterpret_cast<T*>(out + t * out_stride);
        const T* const row = reinterpret_cast<const T*>(logits + t * stride);
        if (!routed<Id, false>(ids + t * choices, choices, experts, lane, Slots<int>(s_mem, 0))) {
            for (int e = lane; e < experts; e += 32)
                if (BMMC_WR_OK(to + e, sizeof(T))) to[e] = from_f32<T>(0.0f);
            continue;
        }
        float over, dot = 0.0f;
        const float m = softmax_of(row, experts, lane, &over);
        for (int e = lane; e < experts; e += 32) dot += expf(logit(row, e) - m) * over * share.get(e);
        dot = warp_sum(dot);
        for (int e = lane; e < experts; e += 32)
            if (BMMC_WR_OK(to + e, sizeof(T)))
                to[e] = from_f32<T>(factor * (expf(logit(row, e) - m) * over) * (share.get(e) - dot));
    }
}

int blocks_of(int64_t tokens) {
    const int64_t b = (tokens + kWarps - 1) / kWarps;
    return (int)(b < kMaxBlocks ? (b < 1 ? 1 : b) : kMaxBlocks);
}

bmmc_status check_router(int64_t tokens, int choices, int experts, int id_bytes) {
    if (id_bytes != 4 && id_bytes != 8) return BMMC_ERR_UNSUPPORTED_ELEM;
    if (tokens < 0 || choices < 1 || choices > EXPERT_MAX_CHOICES || tokens > kMaxTokens / choices || experts < 1 ||
        experts > kMaxExperts)
        return BMMC_ERR_INVALID_ARG;
    return BMMC_OK;
}

template <class F>
bmmc_status by_types(int type, int id_bytes, F&& f) {
    const auto ids = [&](auto t) { return id_bytes == 4 ? f(t, int32_t{}) : f(t, int64_t{}); };
    if (type == BMMC_F32) return ids(float{});
    return type == BMMC_F16 ? ids(__half{}) : ids(__nv_bfloat16{});
}

template <class K>
bool allow(K kernel, size_t smem) {
    if (smem <= 48 * 1024 || cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) == cudaSuccess)
        return true;
    cudaGetLastError();
    return false;
}

}  // namespace

extern "C" {

bmmc_status expert_balance_workspace(int64_t tokens, int choices, int experts, size_t* bytes) {
    if (!bytes) return BMMC_ERR_INVALID_ARG;
    *bytes = 0;
    const bmmc_status s = check_router(tokens, choices, experts, 4);
    if (s == BMMC_OK) *bytes = (size_t)blocks_of(tokens) * (experts + 1) * 8;
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
    if (!workspace || workspace_bytes < need) return BMMC_ERR_NO_SCRATCH;
    if (misaligned(logits, es) || misaligned(ids, id_bytes) || misaligned(loss, 4) || misaligned(counts, 4) ||
        misaligned(workspace, 16))
        return BMMC_ERR_MISALIGNED;
    const Rows in[2] = {{logits, tokens, stride * es, experts * (int64_t)es}, {ids, 1, 0, tokens * choices * id_bytes}};
    const Rows out[3] = {{loss, 1, 0, 4}, {counts, 1, 0, (experts + 1) * 4ll}, {workspace, 1, 0, (int64_t)need}};
    for (int i = 0; i < 3; ++i) {
        if (may_overlap(in[0], out[i]) || may_overlap(in[1], out[i])) return BMMC_ERR_ALIAS;
        for (int j = 0; j < i; ++j)
            if (may_overlap(out[i], out[j])) return BMMC_ERR_ALIAS;
    }
    if ((s = all_reachable(device, {logits, ids, loss, counts, workspace})) != BMMC_OK) return s;
    const chk::Spans spans = spans_of({in[0], in[1], out[2]}, {out[0], out[1], out[2]});
    (void)spans;
    const int blocks = blocks_of(tokens);
    float* const sums = static_cast<float*>(workspace);
    int* const parts = static_cast<int*>(workspace) + (size_t)blocks * (experts + 1);
    const size_t smem = ((kWarps + 1) * (size_t)experts + 1) * 4;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    s = by_types(type, id_bytes, [&](auto t, auto id) {
        using T = decltype(t);
        using Id = decltype(id);
        const auto kernel = balance_part_kernel<T, Id>;
        if (!allow(kernel, smem)) return BMMC_ERR_CUDA;
        return launch(kernel, dim3(blocks), dim3(kThreads), smem, st, nullptr, static_cast<const char*>(logits), stride * es,
                      static_cast<const Id*>(ids), tokens, choices, experts, sums, parts BMMC_SPANS_ARG(spans));
    });
    if (s != BMMC_OK) return s;
    return launch(balance_join_kernel, dim3(1), dim3(1024), 0, st, nullptr, (const float*)sums, (const int*)parts, blocks,
                  experts, loss, counts BMMC_SPANS_ARG(spans));
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
    return by_types(type, id_bytes, [&](auto t, auto id) {
        using T = decltype(t);
        using Id = decltype(id);
        return launch(balance_backward_kernel<T, Id>, dim3(blocks_of(tokens)), dim3(kThreads), (size_t)experts * 4,
                      static_cast<cudaStream_t>(stream), nullptr, grad, static_cast<const char*>(logits), stride * es,
                      static_cast<const Id*>(ids), tokens, choices, experts, (const int*)counts,
                      static_cast<char*>(grad_logits), grad_stride * es BMMC_SPANS_ARG(spans));
    });
}

}  // extern "C"

namespace bmmc {
cudaError_t bounds_record_balance(unsigned long long out[chk::kRecordWords], bool clear) {
    return chk::read_record(out, clear);
}
}  // namespace bmmc
