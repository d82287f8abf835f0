// Keys and values in a paged cache of 8 bits, written with a scale for each
// head of each entry, and a cache's entries read back in the order of the
// sequences: paged_append_quantised and paged_read (declared in
// include/bmmc.h).
//
// A head y of D elements has the scale s = max |y| / M, M the largest value of
// the 8-bit type, and the values round(y / s).
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>
#include <type_traits>

#include "../../include/bmmc.h"
#define BMMC_CHK_FILE 10  // site tag of this file in bounds-checked builds
#include "bounds.cuh"
#include "paged_places.cuh"
#include "token_moves.hpp"
#include "token_words.cuh"

using namespace bmmc;

namespace {

constexpr int kThreads = 128, kWarps = kThreads / 32;

// The 8-bit types: the factor 1 / M of a scale, two values side by side, and
// what a value stands for.  What is encoded is at most M * (1 + 2^-22) in
// magnitude (the three roundings of y * (1 / (max * (1 / M))) are 2^-24 each),
// which rounds to M; or NaN, which becomes NaN, or 0 as a whole number.
struct E4m3 {
    using Code = unsigned char;
    static constexpr float kOver = 1.0f / 448.0f;
    static __device__ __forceinline__ unsigned encode(float a, float b) {
        return __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
    }
    // the values of the codes in the low half of c
    static __device__ __forceinline__ float2 decode(unsigned c) {
        return __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)c, __NV_E4M3)));
    }
};
struct I8 {
    using Code = signed char;
    static constexpr float kOver = 1.0f / 127.0f;
    static __device__ __forceinline__ unsigned encode(float a, float b) {
        return __byte_perm(__float2int_rn(a), __float2int_rn(b), 0x5540) & 0xffffu;
    }
    // (c + 128 in the last bits of 2^23, less 2^23 + 128: the conversion of a
    // byte has a quarter of the rate)
    static __device__ __forceinline__ float2 decode(unsigned c) {
        c ^= 0x8080u;
        return make_float2(__uint_as_float(__byte_perm(c, 0x4b000000u, 0x7440)) - 8388736.0f,
                           __uint_as_float(__byte_perm(c, 0x4b000000u, 0x7441)) - 8388736.0f);
    }
};

constexpr float kLeastScale = 0x1p-126f;  // so that 1 / scale is finite, and zeros have one

// The scale of a head whose largest |y| is `most`.  A head that holds an
// infinity or a NaN has the scale NaN.
template <class Q>
__device__ __forceinline__ float scale_of(float most) {
    return most < INFINITY ? fmaxf(__fmul_rn(most, Q::kOver), kLeastScale) : __uint_as_float(0x7fffffffu);
}

// The larger of a and |b|, NaN where one of them is.
__device__ __forceinline__ float larger(float a, float b) {
    float y;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(fabsf(b)));
    return y;
}

// Where the scales of a cache lie; strides in bytes.
struct Scales {
    char* data;
    int64_t page, slot, head;
    __device__ __forceinline__ float* at(int p, int s, int h) const {
        return reinterpret_cast<float*>(data + p * page + s * slot + h * head);
    }
};

// ---- append --------------------------------------------------------------------

struct QuantisedParams {
    MoveParams moves;
    Scales scales[2];
    int dims[3];
    int stage;  // floats of a warp's staged heads
};

constexpr int kMostThreads = 256;
constexpr int kHeadsAtOnce = 2;  // heads whose words a thread has in flight

// W values times `over` as W codes, written as one word.
template <class Q, int W>
__device__ __forceinline__ void put_codes(char* to, const float (&y)[W], float over) {
    if (!BMMC_WR_OK(to, W)) return;
    const auto two = [&](int i) { return Q::encode(__fmul_rn(y[i], over), W > 1 ? __fmul_rn(y[W > 1 ? i + 1 : 0], over) : 0.0f); };
    if constexpr (W == 1) {
        *reinterpret_cast<unsigned char*>(to) = (unsigned char)two(0);
    } else if constexpr (W == 2) {
        *reinterpret_cast<unsigned short*>(to) = (unsigned short)two(0);
    } else {
        unsigned c[W / 4];
#pragma unroll
        for (int i = 0; i < W; i += 4) c[i / 4] = two(i) | two(i + 2) << 16;
        if constexpr (W == 8) *reinterpret_cast<uint2*>(to) = make_uint2(c[0], c[1]);
        else *reinterpret_cast<unsigned*>(to) = c[0];
    }
}

// A word's elements (and, TWO, those half a head on) turned.
template <int W, bool TWO, int N>
__device__ __forceinline__ void turn_words(float (&x)[W], float (&y)[W], const float2 (&r)[N]) {
    if constexpr (TWO) {
#pragma unroll
        for (int i = 0; i < W; ++i) {
            const float v = x[i];
            x[i] = turned_first(v, y[i], r[i]);
            y[i] = turned_second(v, y[i], r[i]);
        }
    } else {
#pragma unroll
        for (int i = 0; i < W; i += 2) {
            const float v = x[i];
            x[i] = turned_first(v, x[i + 1], r[i / 2]);
            x[i + 1] = turned_second(v, x[i + 1], r[i / 2]);
        }
    }
}

// A thread's words of one kind of heads of its token: keys (Q 0, turned), values
// (1) and queries (2, turned, not quantised).  The kind is known when this is
// compiled, so that what describes it lies at fixed places: with one loop over
// the kinds it was fetched again for every head, and the append of 16001 tokens
// took 88 us.
template <class T, class Q, bool ADJACENT, int PART>
__device__ __forceinline__ void append_part(const QuantisedParams& qp, int64_t t, bool there, int in, Slots<float2> turn,
                                            int64_t to, int page, int slot) {
    constexpr int W = 16 / sizeof(T);
    constexpr bool kTurned = PART != 1, kPlaced = PART != 2;
    constexpr bool kTwo = kTurned && !ADJACENT;  // an item that is turned has two words
    constexpr int kTurns = kTwo ? W : W / 2;
    const MoveParams& p = qp.moves;
    const Heads& h = p.part[PART];
    const int down = (in * h.magic) >> 16, step = (1 << p.group_log2) / h.across, j0 = in - down * h.across;
    there = there && down < step;
    const char* const src = h.src + t * h.src_token + down * h.src_head;
    char* const dst = h.dst + to + down * h.dst_head;
    const int64_t src_step = step * h.src_head, dst_step = step * h.dst_head;
    const int half = p.pairs * (int)sizeof(T);
    const auto load = [&](Pack<T, W>& y, bool want, const char* from) {
        if (want && BMMC_RD_OK(from, 16)) y.load(from);
        else y.word = uint4{};
    };
    // (a cache's heads have a thread for each word: one j)
    for (int j = j0; j == j0 || j < h.items; j += h.across) {
        const bool mine = there && j < h.items, turned = kTurned && mine && j < h.turning, two = kTwo && turned;
        const int at = (kTwo && j >= h.turning ? j + h.turning : j) * W;
        float2 r[kTurns];
        if (turned)
#pragma unroll
            for (int i = 0; i < kTurns; ++i) r[i] = turn.get(j * kTurns + i);
        const char* from = src + at * (int)sizeof(T);
        char* row = dst + at * (kPlaced ? 1 : (int)sizeof(T));
        // `first`: of the heads that the lanes of a warp take at once; the same for all of them
        for (int first = 0; first < h.heads; first += kHeadsAtOnce * step) {
            Pack<T, W> a[kHeadsAtOnce], b[kHeadsAtOnce];
#pragma unroll
            for (int u = 0; u < kHeadsAtOnce; ++u) {
                const bool put = mine && first + u * step + down < h.heads;
                load(a[u], put, from);
                if (kTwo) load(b[u], put && two, from + half);
                from += src_step;
            }
#pragma unroll
            for (int u = 0; u < kHeadsAtOnce; ++u) {
                if (u && first + u * step >= h.heads) break;  // no lane has one
                const bool put = mine && first + u * step + down < h.heads;
                float x[W], y[W];
#pragma unroll
                for (int i = 0; i < W; ++i) x[i] = a[u].get(i), y[i] = kTwo ? b[u].get(i) : 0.0f;
                if (turned) turn_words<W, kTwo>(x, y, r);
                if constexpr (!kPlaced) {
                    a[u].set(x);
                    if (put && BMMC_WR_OK(row, 16)) a[u].store(row);
                    if (two) {
                        b[u].set(y);
                        if (put && BMMC_WR_OK(row + half, 16)) b[u].store(row + half);
                    }
                } else {
                    float most = 0.0f;  // (lanes without a word have zeros)
#pragma unroll
                    for (int i = 0; i < W; ++i) most = larger(most, x[i]);
                    if (two)
#pragma unroll
                        for (int i = 0; i < W; ++i) most = larger(most, y[i]);
                    for (int d = h.across >> 1; d; d >>= 1) most = larger(most, __shfl_xor_sync(~0u, most, d));
                    const float scale = scale_of<Q>(most), over = __frcp_rn(scale);
                    if (put) {
                        put_codes<Q, W>(row, x, over);
                        if (two) put_codes<Q, W>(row + p.pairs, y, over);
                        if (j == 0) {
                            float* const s = qp.scales[PART == 1].at(page, slot, first + u * step + down);
                            if (BMMC_WR_OK(s, 4)) *s = scale;
                        }
                    }
                }
                row += dst_step;
            }
        }
    }
}

// Heads made of words of 16 bytes: a block takes some tokens, a group of
// threads each, and a thread its word (two, where a pair's elements lie half a
// head apart) of one head after another, two at a time, its cosines and sines
// in registers.  The threads of a head are neighbouring lanes, a power of two of
// them, which find its largest element by exchange.  A head stays in registers from
// load to store; under the 64 of a thread the variants of 16-bit heads with pairs half
// a head apart keep some of the rest aside (bf16: 76 bytes written, 124 read a thread;
// f16: 52 and 84; 80 registers, which hold all, were slower, see below).
//
// 16001 tokens of 32 + 8 + 8 heads of 128 bf16 into e4m3 pages 68 us for 53 us of
// bytes (the same heads into pages of their own type 63 for 58): 53 million warp
// instructions, two thirds of the issue slots, of them three quarters the turns,
// products and conversions themselves; and the start of a block.  One head at a time
// instead of two 78 us, twice the threads a token 102, half of them 74; 80 registers
// a thread 69.  Staged by element in shared memory it took 208.  256 single tokens
// 4.2 us.  Keys and values alone into whole numbers, unturned, 40 us for 14.6 of bytes:
// 64 % of the issue slots, 115 instructions of a warp a head (it has two at a time), the
// block's start included, and 42 % of the warps there.
template <class T, class Q, bool ADJACENT>
__global__ void __launch_bounds__(kMostThreads, 4) append_words_kernel(const __grid_constant__ QuantisedParams qp BMMC_SPANS_PARAM) {
    extern __shared__ float2 s_turn[];  // [tokens of the block][pairs] cos, sin
    __shared__ int64_t s_place[2][kMaxTokensPerBlock];
    __shared__ float s_position[kMaxTokensPerBlock];
    __shared__ int s_slot[2][kMaxTokensPerBlock];
    BMMC_SPANS_ENTER(s_turn, chk::dyn_smem_bytes(), s_place, sizeof(s_place), s_position, sizeof(s_position), s_slot,
                     sizeof(s_slot));
    const MoveParams& p = qp.moves;
    const int tid = threadIdx.x, per_block = blockDim.x >> p.group_log2;
    const Slots<float2> turns(s_turn, per_block * p.pairs);
    const Slots<int64_t> places(&s_place[0][0], 2 * kMaxTokensPerBlock);
    const Slots<float> place_numbers(s_position, kMaxTokensPerBlock);
    const Slots<int> slots(&s_slot[0][0], 2 * kMaxTokensPerBlock);
    const int64_t t0 = (int64_t)blockIdx.x * per_block;
    const int nt = (int)min((int64_t)per_block, p.tokens - t0);
    // a block of a small call takes one part only
    const int first_part = gridDim.y > 1 ? blockIdx.y : 0, last_part = gridDim.y > 1 ? first_part + 1 : p.parts;
    begin_block(p, t0, nt, first_part, last_part, turns, places, place_numbers, slots);
    const int k = tid >> p.group_log2, in = tid & ((1 << p.group_log2) - 1);
    const bool there = k < nt;
    const int64_t t = there ? t0 + k : t0;
    const Slots<float2> turn = turns.part(there ? k * p.pairs : 0, p.pairs);
    if (first_part <= 1) {
        const int page = there ? slots.get(k) : -1, slot = there ? slots.get(kMaxTokensPerBlock + k) : 0;
        const int64_t key_at = places.get(there ? k : 0), value_at = places.get(kMaxTokensPerBlock + (there ? k : 0));
        if (first_part == 0) append_part<T, Q, ADJACENT, 0>(qp, t, there && page >= 0, in, turn, key_at, page, slot);
        if (last_part > 1) append_part<T, Q, ADJACENT, 1>(qp, t, there && page >= 0, in, turn, value_at, page, slot);
    }
    if (last_part > 2) append_part<T, Q, ADJACENT, 2>(qp, t, there, in, turn, t * p.part[2].dst_token, 0, 0);
}

// Threads of a token and of a head, as for heads that are only moved: in a
// small call as many as a part has words, so that all its loads are in flight at
// once, and the parts go to blocks of their own; in one that fills the machine a
// quarter, so that cosines and sines serve several heads.
template <class T, class Q>
bmmc_status launch_append_words(QuantisedParams& qp, const chk::Spans& spans, cudaStream_t st) {
    (void)spans;
    constexpr int W = 16 / sizeof(T);
    MoveParams& p = qp.moves;
    int64_t most = std::max(1, p.pairs / kAhead);
    int least = 2;
    for (int q = 0; q < p.parts; ++q) {
        Heads& h = p.part[q];
        const int pairs = h.turned ? p.pairs : 0;
        h.turning = p.adjacent ? 2 * pairs / W : pairs / W;
        h.items = h.turning + (qp.dims[q] - 2 * pairs) / W;
        most = std::max(most, (int64_t)h.heads * h.items);
        if (h.place)
            while ((1 << least) < h.items) ++least;
    }
    int full = 2;
    while (full < 8 && (1 << full) < most) ++full;
    const bool small = (p.tokens << full) <= kSms * 1024;
    int group = std::max(least, small ? std::min(full, 7) : most > 1024 ? full : std::max(2, full - 2));
    int threads = small ? std::max(64, 1 << group) : std::max(kThreads, 1 << group);
    while ((threads >> group) > kMaxTokensPerBlock) ++group;
    while ((threads >> group) > 1 && (threads >> group) * p.pairs * sizeof(float2) > 32 * 1024) ++group;
    p.group_log2 = group;
    for (int q = 0; q < p.parts; ++q) {
        Heads& h = p.part[q];
        h.across = 1;
        if (h.place)
            while (h.across < h.items) h.across <<= 1;
        else
            h.across = std::min(h.items, 1 << group);
        h.magic = (65536 + h.across - 1) / h.across;
        const bool dense = p.device && (h.heads < 2 || h.src_head == (int64_t)qp.dims[q] * (int)sizeof(T));
        h.ahead = dense ? std::min((unsigned)(h.heads * qp.dims[q] * sizeof(T)), 65536u) : 0u;
    }
    const int per_block = threads >> group;
    const bool split = p.tokens / per_block * p.parts * threads <= kSms * 1024;
    const dim3 grid((unsigned)((p.tokens + per_block - 1) / per_block), split ? p.parts : 1);
    const auto kernel = p.adjacent ? append_words_kernel<T, Q, true> : append_words_kernel<T, Q, false>;
    return launch(kernel, grid, dim3(threads), (size_t)per_block * p.pairs * sizeof(float2), st, nullptr, qp BMMC_SPANS_ARG(spans));
}

// W floats of shared memory as words of up to 16 bytes, which warps move without
// meeting in a bank.
template <int W>
struct FloatWord;
template <> struct FloatWord<8> { using type = float4; };
template <> struct FloatWord<4> { using type = float4; };
template <> struct FloatWord<2> { using type = float2; };
template <> struct FloatWord<1> { using type = float; };

constexpr int kRowFloats = 1024;  // of a warp's heads in shared memory, or one head
constexpr int kRowBatch = 32;     // most heads of a warp at a time

// Any heads, in words of W elements: a warp brings some heads into shared memory
// in 32 bits, turns their pairs there by element, finds their scales, and writes
// them in words of W codes.  16001 tokens as above with 37 pairs 134 us (an element
// a lane 235): bound by its instructions, the walk of each pair and the exchange
// for each head's scale.  Heads of 66, in words of two elements, 162 us.
template <class T, class Q, int W>
__global__ void __launch_bounds__(kThreads) append_rows_kernel(const __grid_constant__ QuantisedParams qp BMMC_SPANS_PARAM) {
    extern __shared__ float4 s_stage[];  // a warp's heads each, then [tokens of the block][pairs] cos, sin
    __shared__ int64_t s_place[2][kMaxTokensPerBlock];
    __shared__ float s_position[kMaxTokensPerBlock];
    __shared__ int s_slot[2][kMaxTokensPerBlock];
    __shared__ struct {
        const char* src[kRowBatch];
        char* dst[kRowBatch];      // NULL: not written
        float* scale[kRowBatch];   // where it goes
        float over[kRowBatch];
        int turns[kRowBatch];      // where its token's turns start
    } s_rows[kWarps];
    BMMC_SPANS_ENTER(s_stage, chk::dyn_smem_bytes(), s_place, sizeof(s_place), s_position, sizeof(s_position), s_slot,
                     sizeof(s_slot), s_rows, sizeof(s_rows));
    using F = typename FloatWord<W>::type;
    constexpr int kF = W * 4 / (int)sizeof(F);  // words of floats
    using Word = Pack<T, W>;
    const MoveParams& p = qp.moves;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, per_block = blockDim.x >> p.group_log2;
    const Slots<float4> all(s_stage, kWarps * qp.stage / 4 + (per_block * p.pairs + 1) / 2);
    const Slots<float2> turns(reinterpret_cast<float2*>(s_stage + kWarps * qp.stage / 4), per_block * p.pairs);
    const Slots<float> stage(reinterpret_cast<float*>(s_stage) + warp * qp.stage, qp.stage);
    const Slots<F> staged(reinterpret_cast<F*>(s_stage + warp * qp.stage / 4), qp.stage * 4 / (int)sizeof(F));
    const Slots<int64_t> places(&s_place[0][0], 2 * kMaxTokensPerBlock);
    const Slots<float> place_numbers(s_position, kMaxTokensPerBlock);
    const Slots<int> slots(&s_slot[0][0], 2 * kMaxTokensPerBlock);
    auto& mine = s_rows[warp];
    const Slots<const char*> src(mine.src, kRowBatch);
    const Slots<char*> dst(mine.dst, kRowBatch);
    const Slots<float*> scales(mine.scale, kRowBatch);
    const Slots<float> over(mine.over, kRowBatch);
    const Slots<int> turns_of(mine.turns, kRowBatch);
    const int64_t t0 = (int64_t)blockIdx.x * per_block;
    const int nt = (int)min((int64_t)per_block, p.tokens - t0);
    const int first_part = gridDim.y > 1 ? blockIdx.y : 0, last_part = gridDim.y > 1 ? first_part + 1 : p.parts;
    begin_block(p, t0, nt, first_part, last_part, turns, places, place_numbers, slots);
    for (int q = first_part; q < last_part; ++q) {
        const Heads& h = p.part[q];
        const int dim = qp.dims[q];
        for (int r0 = warp * h.batch; r0 < nt * h.heads; r0 += kWarps * h.batch) {
            const int rows = min(h.batch, nt * h.heads - r0);
            if (lane < rows) {
                const int k = (r0 + lane) / h.heads, head = r0 + lane - k * h.heads;
                const int64_t to = h.place ? places.get((h.place - 1) * kMaxTokensPerBlock + k) : (t0 + k) * h.dst_token;
                src.set(lane, h.src + (t0 + k) * h.src_token + head * h.src_head);
                dst.set(lane, to < 0 ? nullptr : h.dst + to + head * h.dst_head);
                turns_of.set(lane, k * p.pairs);
                if (h.place && to >= 0)
                    scales.set(lane, qp.scales[h.place - 1].at(slots.get(k), slots.get(kMaxTokensPerBlock + k), head));
            }
            __syncwarp();
#pragma unroll 4
            for (int x = lane; x < rows * h.words; x += 32) {
                const int row = h.words == 1 ? x : (int)__umulhi(x, h.words_magic);
                const char* const from = src.get(row) + (x - row * h.words) * (int)sizeof(Word);
                Word y;
                if (BMMC_RD_OK(from, sizeof(Word))) y.load(from);
#pragma unroll
                for (int i = 0; i < kF; ++i) {
                    F f;
                    float* const v = reinterpret_cast<float*>(&f);
#pragma unroll
                    for (int j = 0; j < W / kF; ++j) v[j] = y.get(i * (W / kF) + j);
                    staged.set(x * kF + i, f);
                }
            }
            __syncwarp();
            if (h.turned && p.pairs) {
#pragma unroll 2
                for (int x = lane; x < rows * p.pairs; x += 32) {
                    const int row = quotient(x, p.pairs, p.pairs_magic), i = x - row * p.pairs;
                    const int a = row * dim + (p.adjacent ? 2 * i : i), b = a + (p.adjacent ? 1 : p.pairs);
                    const float2 r = turns.get(turns_of.get(row) + i);
                    const float u = stage.get(a), v = stage.get(b);
                    stage.set(a, turned_first(u, v, r));
                    stage.set(b, turned_second(u, v, r));
                }
                __syncwarp();
            }
            if (h.place) {
#pragma unroll 2
                for (int row = 0; row < rows; ++row) {
                    float most = 0.0f;
                    for (int e = lane; e < dim; e += 32) most = larger(most, stage.get(row * dim + e));
                    for (int d = 16; d; d >>= 1) most = larger(most, __shfl_xor_sync(~0u, most, d));
                    if (lane == 0) {
                        const float scale = scale_of<Q>(most);
                        over.set(row, __frcp_rn(scale));
                        float* const to = scales.get(row);
                        if (dst.get(row) && BMMC_WR_OK(to, 4)) *to = scale;
                    }
                }
                __syncwarp();
            }
#pragma unroll 2
            for (int x = lane; x < rows * h.words; x += 32) {
                const int row = h.words == 1 ? x : (int)__umulhi(x, h.words_magic);
                char* const row_to = dst.get(row);
                if (!row_to) continue;
                float v[W];
#pragma unroll
                for (int i = 0; i < kF; ++i) {
                    const F f = staged.get(x * kF + i);
#pragma unroll
                    for (int j = 0; j < W / kF; ++j) v[i * (W / kF) + j] = reinterpret_cast<const float*>(&f)[j];
                }
                if (h.place) {
                    put_codes<Q, W>(row_to + (x - row * h.words) * W, v, over.get(row));
                } else {
                    Word y;
                    y.set(v);
                    char* const to = row_to + (x - row * h.words) * (int)sizeof(Word);
                    if (BMMC_WR_OK(to, sizeof(Word))) y.store(to);
                }
            }
            __syncwarp();
        }
    }
}

template <class T, class Q, int W>
bmmc_status launch_append_rows(QuantisedParams& qp, const chk::Spans& spans, cudaStream_t st) {
    (void)spans;
    MoveParams& p = qp.moves;
    int per_block = p.tokens >= kSms * 32 ? 4 : 1;
    while (per_block > 1 && per_block * p.pairs * sizeof(float2) > 32 * 1024) per_block >>= 1;
    p.group_log2 = 0;  // threads of a token: the kernel takes as many tokens as there is room for turns
    while ((kThreads >> p.group_log2) > per_block) ++p.group_log2;
    qp.stage = kRowFloats;
    for (int q = 0; q < p.parts; ++q) qp.stage = std::max(qp.stage, (qp.dims[q] + 3) & ~3);
    for (int q = 0; q < p.parts; ++q) {
        Heads& h = p.part[q];
        h.words = qp.dims[q] / W;
        h.words_magic = (unsigned)((((uint64_t)1 << 32) + h.words - 1) / h.words);
        // no more heads a warp than its share
        h.batch = std::max(1, std::min({qp.stage / qp.dims[q], kRowBatch, (per_block * h.heads + kWarps - 1) / kWarps}));
        const bool dense = p.device && W * sizeof(T) == 16 && (h.heads < 2 || h.src_head == (int64_t)qp.dims[q] * (int)sizeof(T));
        h.ahead = dense ? std::min((unsigned)(h.heads * qp.dims[q] * sizeof(T)), 65536u) : 0u;
    }
    const size_t smem = (size_t)kWarps * qp.stage * 4 + (size_t)per_block * p.pairs * sizeof(float2);
    constexpr auto kernel = append_rows_kernel<T, Q, W>;
    const bmmc_status allowed = allow_smem<kernel>(smem);
    if (allowed != BMMC_OK) return allowed;
    const bool split = p.tokens * p.parts <= kSms * 8;
    return launch(kernel, dim3((unsigned)((p.tokens + per_block - 1) / per_block), split ? p.parts : 1), dim3(kThreads), smem, st,
                  nullptr, qp BMMC_SPANS_ARG(spans));
}

// Words of as many elements as bits (of the heads, es bytes each) and cache_bits
// (of the caches) are multiples of.
template <class T, class Q>
bmmc_status launch_append(QuantisedParams& qp, uint64_t bits, uint64_t cache_bits, const chk::Spans& spans, cudaStream_t st) {
    constexpr int es = sizeof(T);
    int W = word_bytes(es, {bits}) / es;
    while (W > 1 && (cache_bits & (uint64_t)(W - 1))) W >>= 1;
    if constexpr (es == 2)
        if (W == 8) return launch_append_rows<T, Q, 8>(qp, spans, st);
    if (W == 4) return launch_append_rows<T, Q, 4>(qp, spans, st);
    return W == 2 ? launch_append_rows<T, Q, 2>(qp, spans, st) : launch_append_rows<T, Q, 1>(qp, spans, st);
}

// ---- read ----------------------------------------------------------------------

constexpr int kReadThreads = 256;
constexpr int kReadRows = 64;  // rows of a block, at most
constexpr int kReadEach = 8;   // rows of a thread, at most
constexpr int kReadAhead = 4;  // rows whose words a thread has in flight

struct ReadParams {
    MoveParams moves;  // part[0], part[1]: from the caches to the rows; lengths: each sequence's first entry
    Scales scales[2];
    int dims[2];
    int rows;           // of a block
    int words[2];       // of a head
    uint64_t magic[2];  // wide_magic_of(words)
};

// W elements of the result from what the cache holds: themselves, or W codes
// and their scale.
template <class T, class Q, int W>
struct Held {
    using Word = typename WordOf<W * (int)sizeof(T)>::type;
    Word word;
    __device__ __forceinline__ void load(const char* p) { word = *reinterpret_cast<const Word*>(p); }
    __device__ __forceinline__ Pack<T, W> value(float) const {
        Pack<T, W> y;
        y.word = word;
        return y;
    }
    static constexpr int kBytes = W * (int)sizeof(T);
};
template <class T, class Q, int W>
struct Coded {
    static constexpr int kBytes = W;
    unsigned c[W > 4 ? 2 : 1];
    __device__ __forceinline__ void load(const char* p) {
        if constexpr (W == 8) {
            const uint2 v = *reinterpret_cast<const uint2*>(p);
            c[0] = v.x, c[1] = v.y;
        } else if constexpr (W == 4) {
            c[0] = *reinterpret_cast<const unsigned*>(p);
        } else if constexpr (W == 2) {
            c[0] = *reinterpret_cast<const unsigned short*>(p);
        } else {
            c[0] = *reinterpret_cast<const unsigned char*>(p);
        }
    }
    __device__ __forceinline__ Pack<T, W> value(float scale) const {
        float v[W];
        if constexpr (W == 1) {
            v[0] = __fmul_rn(Q::decode(c[0]).x, scale);
        } else {
#pragma unroll
            for (int i = 0; i < W; i += 2) {
                const float2 y = Q::decode(c[i / 4] >> (i % 4 * 8) & 0xffffu);
                v[i] = __fmul_rn(y.x, scale), v[i + 1] = __fmul_rn(y.y, scale);
            }
        }
        Pack<T, W> y;
        y.set(v);
        return y;
    }
};

// A block takes some rows: its warps find their places, then a thread takes the
// same word of each (SIDE: of some; the others go to threads beside it), several
// rows at a time.  Pure movement: 65536 entries of 8 heads of 128, keys and values,
// from e4m3 to bf16 68.2 us for 60.0 us of bytes, from whole numbers 71.6, bf16 as they
// are 82.8 for 79.1; an element a lane took 173.  Eight rows a thread, four in flight:
// the places' chain (starts, table) is waited for once a block.  One head an entry 24 us
// (7.5): the chain.
template <class T, class Q, int W, bool SIDE>
__global__ void __launch_bounds__(kReadThreads) read_words_kernel(const __grid_constant__ ReadParams rp BMMC_SPANS_PARAM) {
    __shared__ int64_t s_place[2][kReadRows];
    __shared__ int s_page[kReadRows], s_slot[kReadRows];
    BMMC_SPANS_ENTER(s_place, sizeof(s_place), s_page, sizeof(s_page), s_slot, sizeof(s_slot));
    constexpr bool kCoded = !std::is_void_v<Q>;
    using Word = std::conditional_t<kCoded, Coded<T, Q, W>, Held<T, Q, W>>;
    const Slots<int64_t> places(&s_place[0][0], 2 * kReadRows);
    const Slots<int> pages(s_page, kReadRows), slots(s_slot, kReadRows);
    const MoveParams& p = rp.moves;
    const int tid = threadIdx.y * blockDim.x + threadIdx.x, lane = tid & 31, warps = (int)(blockDim.x * blockDim.y) >> 5;
    const int64_t t0 = (int64_t)blockIdx.x * rp.rows;
    const int n = (int)min((int64_t)rp.rows, p.tokens - t0);
    for (int i = tid >> 5; i < n; i += warps) {
        const Place place = place_of(p, t0 + i, find_sequence_warp(p.starts, p.sequences, t0 + i, lane));
        if (lane == 0) {
            places.set(i, place.byte[0]), places.set(kReadRows + i, place.byte[1]);
            pages.set(i, place.page), slots.set(i, place.slot);
        }
    }
    __syncthreads();
    const auto part = [&](auto which) {
        constexpr int q = decltype(which)::value;
        const Heads& h = p.part[q];
        for (int j = threadIdx.x; j < h.heads * rp.words[q]; j += blockDim.x) {
            const int head = wide_quotient(j, rp.magic[q]), at = (j - head * rp.words[q]) * W;
            const char* const src = h.src + head * h.src_head + at * (Word::kBytes / W);
            const int first = SIDE ? threadIdx.y : 0, step = SIDE ? blockDim.y : 1;
            char* to = h.dst + (t0 + first) * h.dst_token + head * h.dst_head + at * (int)sizeof(T);
            for (int r = first; r < n; r += kReadAhead * step) {
                Word word[kReadAhead];
                float scale[kReadAhead];
                bool there[kReadAhead];
#pragma unroll
                for (int u = 0; u < kReadAhead; ++u) {
                    const int i = r + u * step, page = i < n ? pages.get(i) : -1;
                    there[u] = page >= 0;
                    const char* const from = src + (there[u] ? places.get(q * kReadRows + i) : 0);
                    there[u] = there[u] && BMMC_RD_OK(from, Word::kBytes);
                    if (there[u]) word[u].load(from);
                    scale[u] = 0.0f;
                    if (kCoded && there[u]) {
                        const float* const s = rp.scales[q].at(page, slots.get(i), head);
                        if (BMMC_RD_OK(s, 4)) scale[u] = *s;
                    }
                }
#pragma unroll
                for (int u = 0; u < kReadAhead; ++u) {
                    if (r + u * step >= n) break;
                    Pack<T, W> y;
                    if (there[u]) y = word[u].value(scale[u]);
                    else y.word = typename Pack<T, W>::Word{};
                    if (BMMC_WR_OK(to, sizeof(y))) y.store(to);
                    to += step * h.dst_token;
                }
            }
        }
    };
    part(std::integral_constant<int, 0>{});
    part(std::integral_constant<int, 1>{});
}

template <class T, class Q, int W>
bmmc_status launch_read_words(ReadParams& rp, const chk::Spans& spans, cudaStream_t st) {
    (void)spans;
    const int64_t tokens = rp.moves.tokens;
    int most = 1;
    for (int q = 0; q < 2; ++q) {
        rp.words[q] = rp.dims[q] / W;
        rp.magic[q] = wide_magic_of(rp.words[q]);
        most = std::max(most, rp.moves.part[q].heads * rp.words[q]);
    }
    // threads of a row, and rows side by side; several rows a thread where the
    // blocks still fill the machine
    int x = 8, each = 1;
    while (x < kReadThreads && x < most) x <<= 1;
    const int y = std::max(1, 64 / x);
    while (each < kReadEach && tokens * x >= kSms * 2048 * each * 2) each <<= 1;
    rp.rows = y * each;
    return launch(y > 1 ? read_words_kernel<T, Q, W, true> : read_words_kernel<T, Q, W, false>, dim3((unsigned)((tokens + rp.rows - 1) / rp.rows)), dim3(x, y), 0, st, nullptr,
                  rp BMMC_SPANS_ARG(spans));
}

// Elements of a word: as many as out_bits (16 bytes at most) and cache_bits
// (cs bytes an element) are multiples of.
template <class T, class Q>
bmmc_status launch_read(ReadParams& rp, uint64_t out_bits, uint64_t cache_bits, const chk::Spans& spans, cudaStream_t st) {
    constexpr int es = sizeof(T), cs = std::is_void_v<Q> ? es : 1;
    int W = word_bytes(es, {out_bits}) / es;
    while (W > 1 && (cache_bits & (uint64_t)(W * cs - 1))) W >>= 1;
    if constexpr (es == 2)
        if (W == 8) return launch_read_words<T, Q, 8>(rp, spans, st);
    if (W == 4) return launch_read_words<T, Q, 4>(rp, spans, st);
    if (W == 2) return launch_read_words<T, Q, 2>(rp, spans, st);
    return launch_read_words<T, Q, 1>(rp, spans, st);
}

// ---- host ----------------------------------------------------------------------

// Checks the scales of a cache of these pages, [pages][page_size][heads] floats.
bmmc_status read_scales(const paged_cache_t& s, int64_t pages, int64_t page_size, int64_t heads, Scales& to, Rows& rows) {
    const bmmc_status status = check_cache(s, pages, page_size, heads, 1, 4);
    if (status != BMMC_OK) return status;
    to = Scales{static_cast<char*>(s.data), s.page_stride * 4, s.slot_stride * 4, s.head_stride * 4};
    rows = cache_rows(s, pages, page_size, heads, 1, 4);
    return BMMC_OK;
}

// Whether two arrays [pages][page_size][heads] of runs of run_* bytes, with strides
// in elements of *_bytes, lie between each other: by page, entry or head.
bool lies_between(const paged_cache_t& a, int64_t run_a, int a_bytes, const paged_cache_t& b, int64_t run_b, int b_bytes,
                  int64_t pages, int64_t page_size, int64_t heads) {
    const int64_t sizes[3] = {pages, page_size, heads};
    const int64_t strides_a[3] = {a.page_stride * a_bytes, a.slot_stride * a_bytes, a.head_stride * a_bytes};
    const int64_t strides_b[3] = {b.page_stride * b_bytes, b.slot_stride * b_bytes, b.head_stride * b_bytes};
    return lie_between(run_a, run_b, sizes, strides_a, strides_b, (int64_t)((uintptr_t)b.data - (uintptr_t)a.data));
}

// Whether two results lie between each other, by token or by head.
bool heads_between(const token_heads_t& k, const token_heads_t& v, int64_t tokens, int es) {
    if ((tokens > 1 && k.token_stride != v.token_stride) || (k.heads > 1 && k.head_stride != v.head_stride)) return false;
    const int64_t sizes[2] = {tokens, k.heads}, strides[2] = {k.token_stride * es, k.head_stride * es};
    return lie_between(k.dim * es, v.dim * es, sizes, strides, (int64_t)((uintptr_t)v.data - (uintptr_t)k.data));
}

template <class F>
bmmc_status by_cache_type(int type, int64_t cache_type, F&& f) {
    const auto cache = [&](auto t) { return cache_type == BMMC_I8 ? f(t, I8{}) : f(t, E4m3{}); };
    if (type == BMMC_F32) return cache(float{});
    return type == BMMC_F16 ? cache(__half{}) : cache(__nv_bfloat16{});
}

}  // namespace

extern "C" {

bmmc_status paged_append_quantised(const paged_append_quantised_args_t* args, void* stream) {
    if (!args) return BMMC_ERR_INVALID_ARG;
    const paged_append_args_t& a = args->append;
    if (a.tokens < 0 || a.tokens > kMaxTokens) return BMMC_ERR_INVALID_ARG;
    int type = a.type < 0 || a.type > 0xfff ? -1 : (int)a.type;
    const bool device = device_pointers(type);
    const int es = dtype_bytes(type);
    if (!es || (args->cache_type != BMMC_E4M3 && args->cache_type != BMMC_I8)) return BMMC_ERR_UNSUPPORTED_ELEM;
    if (!a.tokens) return BMMC_OK;
    AppendCall c;
    bmmc_status s = read_append(a, es, 1, device, c);
    if (s != BMMC_OK) return s;
    QuantisedParams qp{};
    Rows scales[2];
    const paged_cache_t* from[2] = {&args->k_scales, &args->v_scales};
    for (int i = 0; i < 2; ++i)
        if ((s = read_scales(*from[i], a.pages, a.page_size, a.k.heads, qp.scales[i], scales[i])) != BMMC_OK) return s;
    for (const Rows& r : scales) {
        for (const Rows& m : c.maps)
            if (may_overlap(r, m)) return BMMC_ERR_ALIAS;
        if (may_overlap(r, c.k) || may_overlap(r, c.v) || may_overlap(r, c.q) || may_overlap(r, c.written[2]) ||
            meets_turns(r, a.turns, a.tokens))
            return BMMC_ERR_ALIAS;
    }
    // scales may lie between the caches' values (behind each head's, or behind an entry's) and between each other
    const paged_cache_t* values[2] = {&a.k_cache, &a.v_cache};
    for (int i = 0; i < 2; ++i)
        for (int j = 0; j < 2; ++j)
            if (may_overlap(scales[i], c.written[j]) &&
                !lies_between(*from[i], 4, 4, *values[j], c.dims[j], 1, a.pages, a.page_size, a.k.heads))
                return BMMC_ERR_ALIAS;
    if (may_overlap(scales[0], scales[1]) && !lies_between(*from[0], 4, 4, *from[1], 4, 4, a.pages, a.page_size, a.k.heads))
        return BMMC_ERR_ALIAS;
    if ((s = append_reachable(a, device)) != BMMC_OK) return s;
    if ((s = all_reachable(device, {args->k_scales.data, args->v_scales.data})) != BMMC_OK) return s;
    qp.moves = c.moves;
    qp.moves.adjacent = a.turns.flags & ROTARY_ADJACENT;
    for (int i = 0; i < 3; ++i) qp.dims[i] = c.dims[i];
    const chk::Spans spans = spans_of({c.k, c.v, c.q, turn_rows(a.turns, a.tokens, 0), turn_rows(a.turns, a.tokens, 1),
                                       turn_rows(a.turns, a.tokens, 2), c.maps[0], c.maps[1], c.maps[2]},
                                      {c.written[0], c.written[1], c.written[2], scales[0], scales[1]});
    // heads of words: their lengths, addresses and pairs in words of 16 bytes, their values in what those become
    const int W = 16 / es;
    bool words = word_bytes(es, {c.in_bits, c.q_bits, pair_bits(a.turns, es)}) == 16 &&
                 !(c.cache_bits & (uint64_t)(W - 1));
    for (int i = 0; i < 2; ++i) {
        const int64_t two = i == 0 && !qp.moves.adjacent ? a.turns.pairs : 0;  // elements in an item's second word
        words = words && (c.dims[i] - two) / W <= 32;
    }
    return by_cache_type(type, args->cache_type, [&](auto t, auto q) {
        if (words) return launch_append_words<decltype(t), decltype(q)>(qp, spans, static_cast<cudaStream_t>(stream));
        return launch_append<decltype(t), decltype(q)>(qp, c.in_bits | c.q_bits, c.cache_bits | c.dims[0] | c.dims[1], spans,
                                                       static_cast<cudaStream_t>(stream));
    });
}

bmmc_status paged_read(const paged_read_args_t* a, void* stream) {
    if (!a || a->tokens < 0 || a->tokens > kMaxTokens) return BMMC_ERR_INVALID_ARG;
    int type = a->type < 0 || a->type > 0xfff ? -1 : (int)a->type;
    const bool device = device_pointers(type);
    const int es = dtype_bytes(type);
    if (!es) return BMMC_ERR_UNSUPPORTED_ELEM;
    const bool quantised = a->cache_type == BMMC_E4M3 || a->cache_type == BMMC_I8;
    if (!quantised && a->cache_type != type) return BMMC_ERR_UNSUPPORTED_ELEM;
    const int cs = quantised ? 1 : es;
    if (!a->tokens) return BMMC_OK;
    if (a->sequences < 0 || a->sequences > kMaxTokens || !a->starts || (a->sequences && a->table_columns && !a->table) ||
        a->table_columns < 0 || a->table_columns > kMaxTokens || bad_stride(a->table_stride, a->sequences) || a->pages < 0 ||
        a->pages > kMaxTokens || a->page_size < 1 || a->page_size > kMaxTokens || a->k.heads != a->v.heads)
        return BMMC_ERR_INVALID_ARG;
    if ((uintptr_t)a->starts % 4 || (uintptr_t)a->firsts % 4 || (uintptr_t)a->table % 4) return BMMC_ERR_MISALIGNED;
    const token_heads_t* to[2] = {&a->k, &a->v};
    const paged_cache_t *cache[2] = {&a->k_cache, &a->v_cache}, *scale[2] = {&a->k_scales, &a->v_scales};
    ReadParams rp{};
    MoveParams& p = rp.moves;
    Rows in[7] = {}, out[2];
    uint64_t cache_bits = 0, out_bits = 0;
    bmmc_status s;
    for (int i = 0; i < 2; ++i) {
        if ((s = check_heads(*to[i], a->tokens, es)) != BMMC_OK) return s;
        if (!writable(*to[i], a->tokens)) return BMMC_ERR_INVALID_ARG;
        // (a cache that is only read may hold an entry's elements at one address)
        const paged_cache_t& m = *cache[i];
        if ((!m.data && a->pages) || bad_stride(m.page_stride, a->pages) || bad_stride(m.slot_stride, a->page_size) ||
            bad_stride(m.head_stride, to[i]->heads))
            return BMMC_ERR_INVALID_ARG;
        if ((uintptr_t)m.data % cs) return BMMC_ERR_MISALIGNED;
        out[i] = rows_of(*to[i], a->tokens, es);
        in[i] = cache_rows(m, a->pages, a->page_size, to[i]->heads, to[i]->dim, cs);
        if (quantised) {
            const paged_cache_t& x = *scale[i];
            if ((!x.data && a->pages) || bad_stride(x.page_stride, a->pages) || bad_stride(x.slot_stride, a->page_size) ||
                bad_stride(x.head_stride, to[i]->heads))
                return BMMC_ERR_INVALID_ARG;
            if ((uintptr_t)x.data % 4) return BMMC_ERR_MISALIGNED;
            rp.scales[i] = Scales{static_cast<char*>(x.data), x.page_stride * 4, x.slot_stride * 4, x.head_stride * 4};
            in[2 + i] = cache_rows(x, a->pages, a->page_size, to[i]->heads, 1, 4);
        } else if (scale[i]->data) {
            return BMMC_ERR_INVALID_ARG;
        }
        Heads& h = p.part[i];
        h.src = static_cast<const char*>(m.data);
        h.src_head = m.head_stride * cs;
        h.dst = static_cast<char*>(to[i]->data);
        h.dst_token = to[i]->token_stride * es;
        h.dst_head = to[i]->head_stride * es;
        h.heads = (int)to[i]->heads;
        p.page_stride[i] = m.page_stride * cs;
        p.slot_stride[i] = m.slot_stride * cs;
        rp.dims[i] = (int)to[i]->dim;
        cache_bits |= (uint64_t)(uintptr_t)m.data | (uint64_t)p.page_stride[i] | (uint64_t)p.slot_stride[i] | (uint64_t)h.src_head;
        out_bits |= address_bits(*to[i], es);
    }
    in[4] = Rows{a->starts, 1, 0, (a->sequences + 1) * 4};
    in[5] = Rows{a->firsts, 1, 0, a->sequences * 4};
    in[6] = Rows{a->table, a->sequences, a->table_stride * 4, a->table_columns * 4};
    for (const Rows& r : in)
        if (may_overlap(r, out[0]) || may_overlap(r, out[1])) return BMMC_ERR_ALIAS;
    if (may_overlap(out[0], out[1]) && !heads_between(a->k, a->v, a->tokens, es)) return BMMC_ERR_ALIAS;
    if ((s = all_reachable(device, {a->k.data, a->v.data, a->k_cache.data, a->v_cache.data, a->k_scales.data, a->v_scales.data,
                                    a->starts, a->firsts, a->table})) != BMMC_OK)
        return s;
    p.parts = 2;
    p.device = device;
    p.tokens = a->tokens;
    p.starts = a->starts;
    p.lengths = a->firsts;
    p.table = a->table;
    p.sequences = a->sequences;
    p.table_stride = a->table_stride;
    p.table_columns = a->table_columns;
    p.pages = a->pages;
    p.page_size = (int)a->page_size;
    const chk::Spans spans = spans_of({in[0], in[1], in[2], in[3], in[4], in[5], in[6]}, {out[0], out[1]});
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (quantised)
        return by_cache_type(type, a->cache_type, [&](auto t, auto q) {
            return launch_read<decltype(t), decltype(q)>(rp, out_bits, cache_bits, spans, st);
        });
    // (values of the result's own type are only moved)
    return es == 4 ? launch_read<float, void>(rp, out_bits, cache_bits, spans, st)
                   : launch_read<__half, void>(rp, out_bits, cache_bits, spans, st);
}

}  // extern "C"

namespace bmmc {
cudaError_t bounds_record_paged_cache8(unsigned long long out[chk::kRecordWords], bool clear) {
    return chk::read_record(out, clear);
}
}  // namespace bmmc
