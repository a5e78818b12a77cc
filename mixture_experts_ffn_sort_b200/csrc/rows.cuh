// rows.cuh -- loads, stores and conversions of row elements in the three row
// types (bf16, f16, f32), for the kernels that move and reduce rows.
#pragma once

#include <string.h>

#include "device_common.cuh"

namespace moe {

__device__ __forceinline__ float elem_to_float(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float elem_to_float(__half v) { return __half2float(v); }
__device__ __forceinline__ float elem_to_float(float v) { return v; }

template <class E>
__device__ __forceinline__ E elem_from_float(float v);
template <>
__device__ __forceinline__ __nv_bfloat16 elem_from_float(float v) { return __float2bfloat16_rn(v); }
template <>
__device__ __forceinline__ __half elem_from_float(float v) { return __float2half_rn(v); }
template <>
__device__ __forceinline__ float elem_from_float(float v) { return v; }

// 16 bytes of elements -> fp32 values, and back with one rounding each.
template <class E>
constexpr int kVec = 16 / static_cast<int>(sizeof(E));

template <class E>
__device__ __forceinline__ void unpack(const uint4& raw, float (&f)[kVec<E>]) {
    E e[kVec<E>];
    memcpy(e, &raw, 16);
#pragma unroll
    for (int i = 0; i < kVec<E>; ++i) f[i] = elem_to_float(e[i]);
}

__device__ __forceinline__ uint4 pack_as(const float (&f)[8], __nv_bfloat16) {
    return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                      pack_bf16x2(f[6], f[7]));
}
__device__ __forceinline__ uint4 pack_as(const float (&f)[8], __half) {
    __half2 h[4];
    uint4 raw;
#pragma unroll
    for (int i = 0; i < 4; ++i) h[i] = __floats2half2_rn(f[2 * i], f[2 * i + 1]);
    memcpy(&raw, h, 16);
    return raw;
}
__device__ __forceinline__ uint4 pack_as(const float (&f)[4], float) {
    return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
}
template <class E>
__device__ __forceinline__ uint4 pack(const float (&f)[kVec<E>]) {
    return pack_as(f, E{});
}

// acc += w * elements, the fp32 additions two at a time.
template <class E>
__device__ __forceinline__ void add_weighted(float (&acc)[kVec<E>], const uint4& raw, float w) {
    float f[kVec<E>];
    unpack<E>(raw, f);
#pragma unroll
    for (int i = 0; i < kVec<E>; i += 2)
        asm("{\n\t.reg .b64 a, b, c;\n\t"
            "mov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %4};\n\tmov.b64 c, {%0, %1};\n\t"
            "fma.rn.f32x2 c, a, b, c;\n\tmov.b64 {%0, %1}, c;\n\t}"
            : "+f"(acc[i]), "+f"(acc[i + 1])
            : "f"(f[i]), "f"(f[i + 1]), "f"(w));
}

// i / d for i * d < 2^63, d < 2^31: the high half of a product with
// M = ceil(2^64 / d).  M d - 2^64 = e < d, so i M / 2^64 exceeds i / d by
// i e / (d 2^64) < 1 / d, too little to reach the next whole number.
struct FastDiv {
    unsigned long long magic;  // 0: d == 1
    unsigned d;
    __host__ explicit FastDiv(unsigned v) : magic(v == 1 ? 0 : ~0ull / v + 1), d(v) {}
    __device__ __forceinline__ long div(long i) const {
        return magic ? static_cast<long>(__umul64hi(static_cast<unsigned long long>(i), magic)) : i;
    }
};

// ---------------------------------------------------------------- rows that do not start on 16 bytes
//
// When a row's bytes are no multiple of 16, rows start at any multiple of their
// element.  16 bytes from any place are two aligned blocks and a shift, the
// second of them an L1 hit of the neighbouring thread's first; only a block that
// reaches out of the whole tensor (its last one) is read element by element.
// 4-byte words need a shift by half a word at most.

__device__ __forceinline__ uint4 load_block(const char* base, long a, long total) {
    if (a >= 0 && a + 16 <= total) return __ldg(reinterpret_cast<const uint4*>(base + a));
    uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const long b = a + 2 * i;
        if (b >= 0 && b + 2 <= total)
            w[i >> 1] |= static_cast<uint32_t>(__ldg(reinterpret_cast<const uint16_t*>(base + b))) << (16 * (i & 1));
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// Bytes [sh, sh + 16) of two 16-byte blocks, 0 < sh < 16.
__device__ __forceinline__ uint4 shift_blocks(const uint4& lo, const uint4& hi, int sh) {
    uint32_t w0 = lo.x, w1 = lo.y, w2 = lo.z, w3 = lo.w, w4 = hi.x, w5 = hi.y;
    if (sh & 8) {
        w0 = lo.z; w1 = lo.w; w2 = hi.x; w3 = hi.y; w4 = hi.z; w5 = hi.w;
    }
    if (sh & 4) {
        w0 = w1; w1 = w2; w2 = w3; w3 = w4; w4 = w5;
    }
    const int bits = (sh & 3) * 8;
    return make_uint4(__funnelshift_r(w0, w1, bits), __funnelshift_r(w1, w2, bits), __funnelshift_r(w2, w3, bits),
                      __funnelshift_r(w3, w4, bits));
}

// Bytes [at, at + 16) of a tensor of `total` bytes at the 16-byte aligned
// `base` (zeros outside of it).
__device__ __forceinline__ uint4 load_window(const char* base, long at, long total) {
    const long a = at & ~15L;
    const int sh = static_cast<int>(at & 15);
    const uint4 lo = load_block(base, a, total);
    if (sh == 0) return lo;
    return shift_blocks(lo, load_block(base, a + 16, total), sh);
}

// One row as the 4-byte words of memory that it touches: word k holds its
// bytes [4 k - lead, 4 k - lead + 4), where lead is 2 for a row that starts
// within a word (HALF: rows of an odd number of 2-byte elements) and 0 otherwise.
template <bool HALF>
struct RowWords {
    const char* base;  // word 0
    int row_bytes, lead;
    long left;  // bytes of the tensor from word 0 on
    __device__ __forceinline__ RowWords(const char* tensor, long row, long bytes, long total)
        : row_bytes(static_cast<int>(bytes)) {
        const long at = row * bytes;
        lead = HALF ? static_cast<int>(at & 2) : 0;
        base = tensor + (at - lead);
        left = total - (at - lead);
    }
    __device__ __forceinline__ int count() const { return (row_bytes + lead + 3) >> 2; }
    // Word k (outside of 0 .. count(): the nearest); its halves that belong to
    // other rows are those rows'.
    __device__ __forceinline__ uint32_t word(int k) const {
        k = min(max(k, 0), count() - 1);
        // The tensor's last word may be half a word.
        return !HALF || 4L * k + 4 <= left ? __ldg(reinterpret_cast<const uint32_t*>(base) + k)
                                           : __ldg(reinterpret_cast<const uint16_t*>(base) + 2 * k);
    }
    // Word k of a row of the other start, out of word k and beside(k).
    __device__ __forceinline__ uint32_t beside(int k) const { return word(lead ? k + 1 : k - 1); }
    __device__ __forceinline__ uint32_t shifted(uint32_t same, uint32_t next) const {
        return lead ? __funnelshift_r(same, next, 16) : __funnelshift_r(next, same, 16);
    }
};

// Word k of the row at byte `at` of a tensor (counted as in RowWords), without the halves outside the row.
template <bool HALF>
__device__ __forceinline__ void store_word(char* tensor, long at, long row_bytes, int k, uint32_t v) {
    const int lead = HALF ? static_cast<int>(at & 2) : 0;
    const int from = 4 * k - lead, bytes = static_cast<int>(row_bytes);
    char* o = tensor + at + from;
    if (from >= 0 && from + 4 <= bytes) {
        *reinterpret_cast<uint32_t*>(o) = v;
    } else if (HALF) {
        if (from >= 0 && from + 2 <= bytes) *reinterpret_cast<uint16_t*>(o) = static_cast<uint16_t>(v);
        if (from == -2) *reinterpret_cast<uint16_t*>(o + 2) = static_cast<uint16_t>(v >> 16);
    }
}

// The words at + 128 k (k = 0..3) of shared memory at any 2-byte place `at` of
// `base` (16-byte aligned, 4 bytes of room after the last word).
__device__ __forceinline__ uint4 load_shared_words(const char* base, int at) {
    const uint32_t* p = reinterpret_cast<const uint32_t*>(base + (at & ~3));
    uint4 v = make_uint4(p[0], p[32], p[64], p[96]);
    if (at & 2) {
        v.x = __funnelshift_r(v.x, p[1], 16);
        v.y = __funnelshift_r(v.y, p[33], 16);
        v.z = __funnelshift_r(v.z, p[65], 16);
        v.w = __funnelshift_r(v.w, p[97], 16);
    }
    return v;
}

// Those words to p + 128 k (4-byte aligned), where p is byte `rel` of a row of `row_bytes`.
template <class E>
__device__ __forceinline__ void store_words(char* p, const uint4& v, long rel, long row_bytes) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const long r = rel + 128 * k;
        char* o = p + 128 * k;
        if (r >= 0 && r + 4 <= row_bytes) {
            *reinterpret_cast<uint32_t*>(o) = w[k];
        } else if (sizeof(E) == 2) {  // half a word at the row's first or last byte
            if (r >= 0 && r + 2 <= row_bytes) *reinterpret_cast<uint16_t*>(o) = static_cast<uint16_t>(w[k]);
            if (r + 2 >= 0 && r + 4 <= row_bytes) *reinterpret_cast<uint16_t*>(o + 2) = static_cast<uint16_t>(w[k] >> 16);
        }
    }
}

// Elements [from, to) of a vector to `p`, where element 0 belongs (aligned to
// its element): one store when that is the whole vector and p is aligned.
template <class E>
__device__ __forceinline__ void store_part(char* p, const uint4& v, int from, int to) {
    if (from <= 0 && to >= kVec<E> && (reinterpret_cast<uintptr_t>(p) & 15) == 0) {
        *reinterpret_cast<uint4*>(p) = v;
    } else {
        E e[kVec<E>];
        memcpy(e, &v, 16);
#pragma unroll
        for (int i = 0; i < kVec<E>; ++i)
            if (i >= from && i < to) reinterpret_cast<E*>(p)[i] = e[i];
    }
}

}  // namespace moe
