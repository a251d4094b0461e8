// Elements of the three types that the step's kernels take, and vectors of
// them as 16-byte accesses.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cstdint>
#include <type_traits>

#include "../../include/csgmv.h"

namespace csgmv {

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }
template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }
template <>
__device__ __forceinline__ __half from_f32<__half>(float v) { return __float2half_rn(v); }

// V elements as they lie in memory: one access of V * sizeof(T) bytes where
// that is at most 16, else several of 16.
template <typename T, int V>
struct alignas(V * sizeof(T) > 16 ? 16 : V * sizeof(T)) Vec {
    T e[V];
};
template <typename T, int V>
__device__ __forceinline__ Vec<T, V> ld_vec(const T *p) {
    constexpr int B = V * (int)sizeof(T);
    Vec<T, V> v;
    if constexpr (B % 16 == 0) {
#pragma unroll
        for (int i = 0; i < B / 16; ++i) reinterpret_cast<uint4 *>(&v)[i] = reinterpret_cast<const uint4 *>(p)[i];
    } else if constexpr (B == 8) {
        *reinterpret_cast<uint2 *>(&v) = *reinterpret_cast<const uint2 *>(p);
    } else if constexpr (B == 4) {
        *reinterpret_cast<uint32_t *>(&v) = *reinterpret_cast<const uint32_t *>(p);
    } else {
        static_assert(V == 1, "vectors of 4, 8 or 16 bytes times n");
        v.e[0] = p[0];
    }
    return v;
}
template <typename T, int V>
__device__ __forceinline__ void st_vec(T *p, const Vec<T, V> &v) {
    constexpr int B = V * (int)sizeof(T);
    if constexpr (B % 16 == 0) {
#pragma unroll
        for (int i = 0; i < B / 16; ++i) reinterpret_cast<uint4 *>(p)[i] = reinterpret_cast<const uint4 *>(&v)[i];
    } else if constexpr (B == 8) {
        *reinterpret_cast<uint2 *>(p) = *reinterpret_cast<const uint2 *>(&v);
    } else if constexpr (B == 4) {
        *reinterpret_cast<uint32_t *>(p) = *reinterpret_cast<const uint32_t *>(&v);
    } else {
        p[0] = v.e[0];
    }
}

// All of a vector from and to f32, by words where that takes fewer instructions (two
// centred norms with gates: 5.2 TB/s, by single elements 4.0).
template <typename T, int V>
__device__ __forceinline__ void widen(const Vec<T, V> &x, float (&v)[V]) {
    if constexpr (std::is_same_v<T, __nv_bfloat16> && V > 1) {  // (upper halves of f32: a shift and a mask)
#pragma unroll
        for (int i = 0; i < V; i += 2) {
            const uint32_t w = reinterpret_cast<const uint32_t *>(x.e)[i / 2];
            v[i] = __uint_as_float(w << 16), v[i + 1] = __uint_as_float(w & 0xffff0000u);
        }
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] = to_f32(x.e[i]);
    }
}
template <typename T, int V>
__device__ __forceinline__ Vec<T, V> narrow(const float (&v)[V]) {
    Vec<T, V> x;
    if constexpr (std::is_same_v<T, __nv_bfloat16> && V > 1) {
#pragma unroll
        for (int i = 0; i < V; i += 2) *reinterpret_cast<__nv_bfloat162 *>(&x.e[i]) = __floats2bfloat162_rn(v[i], v[i + 1]);
    } else if constexpr (std::is_same_v<T, __half> && V > 1) {
#pragma unroll
        for (int i = 0; i < V; i += 2) *reinterpret_cast<__half2 *>(&x.e[i]) = __floats2half2_rn(v[i], v[i + 1]);
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) x.e[i] = from_f32<T>(v[i]);
    }
    return x;
}

inline int dtype_bytes(int dtype) { return dtype == CSGMV_DTYPE_F32 ? 4 : 2; }

}  // namespace csgmv
