// grad_clip.cu -- the global 2-norm of many gradient tensors and clipping by
// it (moe_grad_sumsq, moe_grad_clip).
//
// The tensors' addresses travel in the kernel's parameters (no copy of a table
// to the device, so the calls can be captured in a graph), a launch taking up
// to GradTable::kMax of them.  Every tensor is cut into chunks of 16 KB on
// 16-byte boundaries of its own memory; a grid of a few blocks per SM walks
// all chunks of the launch.  Values are squared and added in fp32 over one
// 16-byte vector, then in fp64 per thread, per block (a partial sum in the
// workspace) and over the partials, always in the same order.
#include "launch.h"
#include "rows.cuh"

namespace moe {

namespace {

constexpr int kThreads = 256;
constexpr int kUnroll = 4;
constexpr long kChunk = static_cast<long>(kThreads) * 16 * kUnroll;  // bytes of a tensor per step of a block
constexpr int kMaxBlocks = 148 * 8;

template <int CAP>
struct GradTable {
    const void* src[CAP];
    void* dst[CAP];
    long numel_type[CAP];  // numel * 4 + dtype
    int first[CAP + 1];    // first chunk of each tensor; first[n] = chunks in all
    int n;
};

// The tensor holding chunk c: the last one whose first chunk is <= c.
template <int CAP>
__device__ __forceinline__ int tensor_of(const GradTable<CAP>& tab, int c) {
    int lo = 0, hi = tab.n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (tab.first[mid] <= c) lo = mid;
        else hi = mid;
    }
    return lo;
}

__device__ __forceinline__ double block_sum(double v, double* sh) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
    const int warp = threadIdx.x >> 5;
    __syncthreads();
    if ((threadIdx.x & 31) == 0) sh[warp] = v;
    __syncthreads();
    double s = 0.;
#pragma unroll
    for (int i = 0; i < kThreads / 32; ++i) s += sh[i];
    return s;
}

// The squares of one 16-byte vector: in fp32, and in fp64 where fp32 would
// overflow or lose them.
template <class E>
__device__ __forceinline__ double vec_sumsq(const uint4& raw) {
    constexpr int N = 16 / sizeof(E);
    float f[N];
    unpack<E, 16>(raw, f);
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < N; ++i) s = fmaf(f[i], f[i], s);
    if (s > 1e-20f && s < 1e30f) return s;
    double d = 0.;
#pragma unroll
    for (int i = 0; i < N; ++i) d = fma(static_cast<double>(f[i]), static_cast<double>(f[i]), d);
    return d;
}

// Elements [begin, end) of a tensor that chunk k covers, as byte offsets from
// the tensor's 16-byte boundary `base` (the element range starts at `skip`).
template <class E>
__device__ __forceinline__ double chunk_sumsq(const void* src, long numel, long k) {
    const uintptr_t a = reinterpret_cast<uintptr_t>(src);
    const char* base = reinterpret_cast<const char*>(a & ~uintptr_t(15));
    const long skip = static_cast<long>(a & 15), end = skip + numel * static_cast<long>(sizeof(E));
    const long lo = k * kChunk;
    double acc = 0.;
    uint4 v[kUnroll];
    bool whole[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
        const long o = lo + (static_cast<long>(u) * kThreads + threadIdx.x) * 16;
        whole[u] = o >= skip && o + 16 <= end;
        if (whole[u]) v[u] = __ldg(reinterpret_cast<const uint4*>(base + o));
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
        if (whole[u]) {
            acc += vec_sumsq<E>(v[u]);
        } else {  // the first or last vector of the tensor, or beyond it
            const long o = lo + (static_cast<long>(u) * kThreads + threadIdx.x) * 16;
            for (long b = o; b < o + 16; b += sizeof(E))
                if (b >= skip && b < end) {
                    const double f = elem_to_float(*reinterpret_cast<const E*>(base + b));
                    acc = fma(f, f, acc);
                }
        }
    }
    return acc;
}

template <int CAP>
__global__ void __launch_bounds__(kThreads) sumsq_kernel(const __grid_constant__ GradTable<CAP> tab,
                                                         double* __restrict__ partial) {
    __shared__ double sh[kThreads / 32];
    double acc = 0.;
    const int chunks = tab.first[tab.n];
    for (int c = blockIdx.x; c < chunks; c += gridDim.x) {
        const int i = tensor_of(tab, c);
        const long k = c - tab.first[i], n = tab.numel_type[i] >> 2;
        switch (tab.numel_type[i] & 3) {
            case MOE_DTYPE_BF16: acc += chunk_sumsq<__nv_bfloat16>(tab.src[i], n, k); break;
            case MOE_DTYPE_F16: acc += chunk_sumsq<__half>(tab.src[i], n, k); break;
            default: acc += chunk_sumsq<float>(tab.src[i], n, k); break;
        }
    }
    acc = block_sum(acc, sh);
    if (threadIdx.x == 0) partial[blockIdx.x] = acc;
}

__device__ __forceinline__ double sum_partials(const double* __restrict__ partial, int n, double* sh) {
    double acc = 0.;
    for (int i = threadIdx.x; i < n; i += kThreads) acc += partial[i];
    return block_sum(acc, sh);
}

__global__ void __launch_bounds__(kThreads) finish_kernel(const double* __restrict__ partial, int n,
                                                          double* __restrict__ sumsq, float* __restrict__ norm) {
    __shared__ double sh[kThreads / 32];
    const double s = sum_partials(partial, n, sh);
    if (threadIdx.x == 0) {
        if (sumsq) *sumsq = s;
        if (norm) *norm = static_cast<float>(sqrt(s));
    }
}

template <class E>
__device__ __forceinline__ void chunk_scale(const void* src, void* dst, long numel, long k, float f) {
    const uintptr_t a = reinterpret_cast<uintptr_t>(src), d = reinterpret_cast<uintptr_t>(dst);
    const long skip = static_cast<long>(a & 15), end = skip + numel * static_cast<long>(sizeof(E));
    const char* base = reinterpret_cast<const char*>(a - skip);
    char* to = reinterpret_cast<char*>(d - skip);  // 16-byte aligned when src and dst share their offset
    const bool together = ((a ^ d) & 15) == 0;
    const long lo = k * kChunk;
    uint4 v[kUnroll];
    bool whole[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
        const long o = lo + (static_cast<long>(u) * kThreads + threadIdx.x) * 16;
        whole[u] = together && o >= skip && o + 16 <= end;
        if (whole[u]) v[u] = *reinterpret_cast<const uint4*>(base + o);
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
        const long o = lo + (static_cast<long>(u) * kThreads + threadIdx.x) * 16;
        if (whole[u]) {
            float g[16 / sizeof(E)];
            unpack<E, 16>(v[u], g);
#pragma unroll
            for (int i = 0; i < static_cast<int>(16 / sizeof(E)); ++i) g[i] *= f;
            *reinterpret_cast<uint4*>(to + o) = pack<E, 16>(g);
        } else {
            for (long b = o; b < o + 16; b += sizeof(E))
                if (b >= skip && b < end) {
                    const float g[1] = {elem_to_float(*reinterpret_cast<const E*>(base + b)) * f};
                    *reinterpret_cast<raw_t<sizeof(E)>*>(to + b) = pack<E, sizeof(E)>(g);
                }
        }
    }
}

template <int CAP>
__global__ void __launch_bounds__(kThreads) scale_kernel(const __grid_constant__ GradTable<CAP> tab,
                                                         const double* __restrict__ partial, int n_partial,
                                                         const double* __restrict__ sumsq, float max_norm, float eps,
                                                         float* __restrict__ norm_out) {
    __shared__ double sh[kThreads / 32];
    const double s = sumsq ? *sumsq : sum_partials(partial, n_partial, sh);
    const double norm = sqrt(s);
    if (norm_out && blockIdx.x == 0 && threadIdx.x == 0) *norm_out = static_cast<float>(norm);
    const double ratio = static_cast<double>(max_norm) / (norm + static_cast<double>(eps));
    const float f = ratio >= 1. || norm == 0. ? 1.f : static_cast<float>(ratio);  // NaN stays NaN
    const int chunks = tab.first[tab.n];
    for (int c = blockIdx.x; c < chunks; c += gridDim.x) {
        const int i = tensor_of(tab, c);
        const long k = c - tab.first[i], n = tab.numel_type[i] >> 2;
        if (f == 1.f && tab.src[i] == tab.dst[i]) continue;  // in place, nothing to clip
        switch (tab.numel_type[i] & 3) {
            case MOE_DTYPE_BF16: chunk_scale<__nv_bfloat16>(tab.src[i], tab.dst[i], n, k, f); break;
            case MOE_DTYPE_F16: chunk_scale<__half>(tab.src[i], tab.dst[i], n, k, f); break;
            default: chunk_scale<float>(tab.src[i], tab.dst[i], n, k, f); break;
        }
    }
}

constexpr int kCap = 1000;

long chunks_of(const moe_tensor_ref& r) {
    if (r.numel == 0) return 0;
    const long skip = static_cast<long>(reinterpret_cast<uintptr_t>(r.data) & 15);
    return (skip + r.numel * dtype_bytes(r.dtype) + kChunk - 1) / kChunk;
}

// Fills the table with refs[*at ..): up to CAP non-empty tensors (their chunks
// fit an int: grad_chunks_fit).  False when none is left.
template <int CAP>
bool fill(GradTable<CAP>* tab, const moe_tensor_ref* refs, int n, int* at) {
    tab->n = 0;
    long chunks = 0;
    for (; *at < n && tab->n < CAP; ++*at) {
        const moe_tensor_ref& r = refs[*at];
        const long c = chunks_of(r);
        if (c == 0) continue;
        const int i = tab->n++;
        tab->src[i] = r.data;
        tab->dst[i] = r.out;
        tab->numel_type[i] = r.numel * 4 + r.dtype;
        tab->first[i] = static_cast<int>(chunks);
        chunks += c;
    }
    tab->first[tab->n] = static_cast<int>(chunks);
    return tab->n > 0;
}

int grid_of(int chunks) { return chunks < kMaxBlocks ? chunks : kMaxBlocks; }

}  // namespace

// One set of partial sums for every launch of up to kCap tensors.
size_t grad_workspace_bytes(int n) {
    return (static_cast<size_t>(n) + kCap - 1) / kCap * kMaxBlocks * sizeof(double);
}

bool grad_chunks_fit(const moe_tensor_ref* refs, int n) {
    long chunks = 0;
    for (int i = 0; i < n; ++i)
        if ((chunks += chunks_of(refs[i])) > 0x7fffffffL) return false;
    return true;
}

static cudaError_t launch_partials(const moe_tensor_ref* refs, int n, double* partial, int* n_partial,
                                   cudaStream_t stream) {
    GradTable<kCap> tab;
    *n_partial = 0;
    for (int at = 0; fill(&tab, refs, n, &at);) {
        const int grid = grid_of(tab.first[tab.n]);
        sumsq_kernel<kCap><<<grid, kThreads, 0, stream>>>(tab, partial + *n_partial);
        *n_partial += grid;
        cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

cudaError_t launch_grad_sumsq(const moe_tensor_ref* refs, int n, double* sumsq, float* norm, void* ws,
                              cudaStream_t stream) {
    int np = 0;
    cudaError_t e = launch_partials(refs, n, static_cast<double*>(ws), &np, stream);
    if (e != cudaSuccess) return e;
    finish_kernel<<<1, kThreads, 0, stream>>>(static_cast<double*>(ws), np, sumsq, norm);
    return cudaGetLastError();
}

cudaError_t launch_grad_clip(const moe_tensor_ref* refs, int n, const double* sumsq, float max_norm, float eps,
                             float* norm, void* ws, cudaStream_t stream) {
    int np = 0;
    if (!sumsq) {
        cudaError_t e = launch_partials(refs, n, static_cast<double*>(ws), &np, stream);
        if (e != cudaSuccess) return e;
    }
    GradTable<kCap> tab;
    bool any = false;
    for (int at = 0; fill(&tab, refs, n, &at); any = true) {
        scale_kernel<kCap><<<grid_of(tab.first[tab.n]), kThreads, 0, stream>>>(
            tab, static_cast<const double*>(ws), np, sumsq, max_norm, eps, any ? nullptr : norm);
        cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess) return e;
    }
    if (!any && norm) {  // no values: the norm alone
        tab.n = 0;
        tab.first[0] = 0;
        scale_kernel<kCap><<<1, kThreads, 0, stream>>>(tab, static_cast<const double*>(ws), np, sumsq, max_norm, eps, norm);
        return cudaGetLastError();
    }
    return cudaSuccess;
}

}  // namespace moe
