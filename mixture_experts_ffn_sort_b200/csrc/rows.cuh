// rows.cuh -- loads, stores and conversions of row elements in the three row
// types (bf16, f16, f32), for the kernels that move and reduce rows.
#pragma once

#include <string.h>

#include "device_common.cuh"

namespace moe {

// V bytes as one load or store.
template <int V>
struct RawVec;
template <>
struct RawVec<16> {
    using type = uint4;
};
template <>
struct RawVec<8> {
    using type = uint2;
};
template <>
struct RawVec<4> {
    using type = uint32_t;
};
template <>
struct RawVec<2> {
    using type = uint16_t;
};
template <int V>
using raw_t = typename RawVec<V>::type;

__device__ __forceinline__ float elem_to_float(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float elem_to_float(__half v) { return __half2float(v); }
__device__ __forceinline__ float elem_to_float(float v) { return v; }

// V bytes of elements -> fp32 values, and back with one rounding each.
template <class E, int V>
__device__ __forceinline__ void unpack(const raw_t<V>& raw, float (&f)[V / sizeof(E)]) {
    constexpr int N = V / sizeof(E);
    E e[N];
    memcpy(e, &raw, V);
#pragma unroll
    for (int i = 0; i < N; ++i) f[i] = elem_to_float(e[i]);
}

__device__ __forceinline__ void pair_to(__nv_bfloat162* o, float a, float b) { *o = __floats2bfloat162_rn(a, b); }
__device__ __forceinline__ void pair_to(__half2* o, float a, float b) { *o = __floats2half2_rn(a, b); }

template <class E>
struct PairOf;
template <>
struct PairOf<__nv_bfloat16> {
    using type = __nv_bfloat162;
    static __device__ __forceinline__ __nv_bfloat16 one(float v) { return __float2bfloat16_rn(v); }
};
template <>
struct PairOf<__half> {
    using type = __half2;
    static __device__ __forceinline__ __half one(float v) { return __float2half_rn(v); }
};

template <class E, int V>
__device__ __forceinline__ raw_t<V> pack(const float (&f)[V / sizeof(E)]) {
    constexpr int N = V / sizeof(E);
    raw_t<V> raw;
    if constexpr (sizeof(E) == 4) {
        memcpy(&raw, f, V);
    } else if constexpr (N == 1) {
        const E e = PairOf<E>::one(f[0]);
        memcpy(&raw, &e, V);
    } else {
        typename PairOf<E>::type e[N / 2];
#pragma unroll
        for (int i = 0; i < N / 2; ++i) pair_to(&e[i], f[2 * i], f[2 * i + 1]);
        memcpy(&raw, e, V);
    }
    return raw;
}

template <int V>
__device__ __forceinline__ raw_t<V> zero_raw() {
    raw_t<V> z;
    memset(&z, 0, V);
    return z;
}

}  // namespace moe
