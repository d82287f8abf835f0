// Vectors of tensor elements as the token-moving kernels load and store them.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

namespace bmmc {

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

}  // namespace bmmc
