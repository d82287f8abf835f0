// Vectors of tensor elements as the token-moving kernels load and store them.
// Each source includes bounds.cuh, with its own BMMC_CHK_FILE tag, before this
// header.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

namespace bmmc {

// x / d for x, d < 2^16, with magic_of(d) = 2^32 / d rounded up.
inline unsigned magic_of(int d) { return d > 1 ? (unsigned)((((uint64_t)1 << 32) + d - 1) / d) : 0; }
__device__ __forceinline__ int quotient(int x, int d, unsigned magic) { return d == 1 ? x : (int)__umulhi(x, magic); }

// A shared array, or a part of one, whose elements are reached by number.  In
// bounds-checked builds each number is tested against the length, and each
// address against the arrays that the kernel registered; otherwise it is a
// pointer.
template <class T>
struct Slots {
    T* p;
#ifdef BMMC_BOUNDS_CHECK
    int n;
    __device__ __forceinline__ Slots(T* p_, int n_) : p(p_), n(n_) {}
    __device__ __forceinline__ bool ok(int i, int line = __builtin_LINE()) const {
        return chk::slot_ok(p, i, 1, n, sizeof(T), BMMC_CHK_FILE * 100000 + line);
    }
    // (a part that does not lie in the array has no elements)
    __device__ __forceinline__ Slots part(int first, int count, int line = __builtin_LINE()) const {
        return Slots(p + first, chk::slot_ok(p, first, count, n, sizeof(T), BMMC_CHK_FILE * 100000 + line) ? count : 0);
    }
    __device__ __forceinline__ T get(int i, int line = __builtin_LINE()) const { return ok(i, line) ? p[i] : T{}; }
    __device__ __forceinline__ void set(int i, T v, int line = __builtin_LINE()) const {
        if (ok(i, line)) p[i] = v;
    }
    __device__ __forceinline__ void add(int i, T v, int line = __builtin_LINE()) const {
        if (ok(i, line)) atomicAdd(p + i, v);
    }
#else
    __device__ __forceinline__ Slots(T* p_, int) : p(p_) {}
    __device__ __forceinline__ bool ok(int) const { return true; }
    __device__ __forceinline__ Slots part(int first, int) const { return Slots(p + first, 0); }
    __device__ __forceinline__ T get(int i) const { return p[i]; }
    __device__ __forceinline__ void set(int i, T v) const { p[i] = v; }
    __device__ __forceinline__ void add(int i, T v) const { atomicAdd(p + i, v); }
#endif
};

template <int BYTES> struct WordOf;
template <> struct WordOf<16> { using type = uint4; };
template <> struct WordOf<8> { using type = uint2; };
template <> struct WordOf<4> { using type = uint32_t; };
template <> struct WordOf<2> { using type = uint16_t; };

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
// Round to nearest even, once per output.
template <class T> __device__ __forceinline__ T from_f32(float v);
template <> __device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <> __device__ __forceinline__ __half from_f32<__half>(float v) { return __float2half_rn(v); }
template <> __device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }
// Two at once: the 16-bit types have one instruction for a pair.
__device__ __forceinline__ void pair_from_f32(float* o, float a, float b) { o[0] = a; o[1] = b; }
__device__ __forceinline__ void pair_from_f32(__half* o, float a, float b) {
    *reinterpret_cast<__half2*>(o) = __floats2half2_rn(a, b);
}
__device__ __forceinline__ void pair_from_f32(__nv_bfloat16* o, float a, float b) {
    *reinterpret_cast<__nv_bfloat162*>(o) = __floats2bfloat162_rn(a, b);
}

// A word read if `want`, else zero: without a branch, so that the loads of a
// batch are all on their way before the first of them is waited for.
__device__ __forceinline__ void load_if(bool want, uint4& v, const void* p) {
    asm("{\n .reg .pred q;\n setp.ne.u32 q, %4, 0;\n mov.u32 %0, 0;\n mov.u32 %1, 0;\n mov.u32 %2, 0;\n mov.u32 %3, 0;\n"
        " @q ld.global.nc.v4.u32 {%0, %1, %2, %3}, [%5];\n}"
        : "=&r"(v.x), "=&r"(v.y), "=&r"(v.z), "=&r"(v.w)
        : "r"((int)want), "l"(p));
}
__device__ __forceinline__ void load_if(bool want, uint2& v, const void* p) {
    asm("{\n .reg .pred q;\n setp.ne.u32 q, %2, 0;\n mov.u32 %0, 0;\n mov.u32 %1, 0;\n"
        " @q ld.global.nc.v2.u32 {%0, %1}, [%3];\n}"
        : "=&r"(v.x), "=&r"(v.y)
        : "r"((int)want), "l"(p));
}

// 16 bytes cut out of two neighbouring words, `shift` bytes behind the
// first one's start; a warp's shifts are mostly the same.
__device__ __forceinline__ uint4 cut(const uint4& a, const uint4& b, unsigned shift) {
    const unsigned bits = (shift & 3) * 8;
    uint32_t w0 = a.x, w1 = a.y, w2 = a.z, w3 = a.w, w4 = b.x;
    switch (shift >> 2) {
        case 1: w0 = a.y, w1 = a.z, w2 = a.w, w3 = b.x, w4 = b.y; break;
        case 2: w0 = a.z, w1 = a.w, w2 = b.x, w3 = b.y, w4 = b.z; break;
        case 3: w0 = a.w, w1 = b.x, w2 = b.y, w3 = b.z, w4 = b.w; break;
        default: break;
    }
    return make_uint4(__funnelshift_r(w0, w1, bits), __funnelshift_r(w1, w2, bits), __funnelshift_r(w2, w3, bits),
                      __funnelshift_r(w3, w4, bits));
}

// W elements of type T, moved as one word.
template <class T, int W>
struct Pack {
    using Word = typename WordOf<W * sizeof(T)>::type;
    union {
        Word word;
        T e[W];
    };
    __device__ Pack() {}
    __device__ __forceinline__ void load(const void* p) { word = *reinterpret_cast<const Word*>(p); }
    __device__ __forceinline__ void store(void* p) const { *reinterpret_cast<Word*>(p) = word; }
    __device__ __forceinline__ float get(int i) const { return to_f32(e[i]); }
    __device__ __forceinline__ void set(const float (&v)[W]) {
        if constexpr (W == 1) {
            e[0] = from_f32<T>(v[0]);
        } else {
#pragma unroll
            for (int i = 0; i < W; i += 2) pair_from_f32(e + i, v[i], v[i + 1]);
        }
    }
};

// How a row of `length` elements at any element-aligned address is walked in
// packs.  Aligned rows (ACROSS false): pack w is elements w * W and up.  Rows
// whose address or length is no multiple of the word (ACROSS true, packs of
// 16 bytes): the packs are the aligned words of the row that is written, the
// first and the last of them partly outside, and rows that are read are cut
// to fit out of the two aligned words around each pack.  Only words that hold
// bytes of the row are read: the bytes next to it that come along lie in the
// row's own 16-byte granules.
template <class T, int W, bool ACROSS>
struct Walk {
    static_assert(!ACROSS || W * sizeof(T) == 16, "packs of 16 bytes");
    int length, lead = 0;  // lead: elements between the first word's start and the row's
    __device__ __forceinline__ Walk(int n, const void* written) : length(n) {
        if (ACROSS) lead = ((unsigned)reinterpret_cast<uintptr_t>(written) & 15u) / sizeof(T);
    }
    __device__ __forceinline__ int at(int w) const { return w * W - lead; }  // first element of pack w
    __device__ __forceinline__ bool in(int w) const { return at(w) < length; }
    __device__ __forceinline__ int packs() const { return (length + lead + W - 1) / W; }

    // A pack on its way: fetch starts the loads (of nothing where !want), get
    // takes the pack.
    struct Fetch {
        typename Pack<T, W>::Word a, b;
        unsigned shift;
    };
    __device__ __forceinline__ void fetch(Fetch& f, bool want, const char* row, int w) const {
        const char* p = row + (int64_t)at(w) * sizeof(T);
        if constexpr (ACROSS) {
            const char* const end = row + (int64_t)length * sizeof(T);
            f.shift = (unsigned)reinterpret_cast<uintptr_t>(p) & 15u;
            p -= f.shift;
            load_if(want && p + 16 > row && BMMC_RD_WORD_OK(p, 16), f.a, p);
            load_if(want && f.shift && p + 16 < end && BMMC_RD_WORD_OK(p + 16, 16), f.b, p + 16);
        } else {
            load_if(want && BMMC_RD_OK(p, sizeof(f.a)), f.a, p);
        }
    }
    __device__ __forceinline__ Pack<T, W> get(const Fetch& f) const {
        Pack<T, W> y;
        if constexpr (ACROSS) y.word = cut(f.a, f.b, f.shift);
        else y.word = f.a;
        return y;
    }
    __device__ __forceinline__ void store(const Pack<T, W>& y, char* row, int w) const {
        const int a = at(w);
        if (!ACROSS || (a >= 0 && a + W <= length)) {
            if (BMMC_WR_OK(row + (int64_t)a * sizeof(T), sizeof(y))) y.store(row + (int64_t)a * sizeof(T));
        } else {
#pragma unroll
            for (int i = 0; i < W; ++i)
                if (a + i >= 0 && a + i < length && BMMC_WR_OK(reinterpret_cast<T*>(row) + a + i, sizeof(T))) reinterpret_cast<T*>(row)[a + i] = y.e[i];
        }
    }
    // zero in the elements of pack w that lie outside the row
    __device__ __forceinline__ void trim(Pack<T, W>& y, int w) const {
        if constexpr (ACROSS) {
            const int a = at(w);
            if (a >= 0 && a + W <= length) return;
#pragma unroll
            for (int i = 0; i < W; ++i)
                if (a + i < 0 || a + i >= length) y.e[i] = from_f32<T>(0.0f);
        }
    }
};

}  // namespace bmmc
