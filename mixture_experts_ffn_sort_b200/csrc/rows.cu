// rows.cu -- rows sorted by expert and back (moe_permute, moe_unpermute) and
// the gradients (moe_unpermute_bwd), for bf16, f16 and f32 rows.
//
// Everything here is indexed by token: inv_route gives the sorted position of
// each of a token's K routes, so a token's row is read once for its K copies
// (permute), its K sorted rows are summed in slot order by one thread per
// column vector (unpermute, a fixed order), and no two tokens write the same
// row.  A position outside [0, T*K) is skipped: -1 silently, anything else
// with MOE_STATUS_BAD_MAP.  All of it is bound by memory: a few operations for
// every element read or written.
#include "launch.h"
#include "rows.cuh"

namespace moe {

namespace {

constexpr int kThreads = 256;

// The sorted position of a route, or -1; flags corrupt entries.
__device__ __forceinline__ int32_t position(const int32_t* __restrict__ inv, long r, long R, bool* bad) {
    const int32_t p = __ldg(inv + r);
    if (p >= 0 && p < R) return p;
    if (p != -1) *bad = true;
    return -1;
}

// Zeros in the sorted rows [*n_rows, R) (grid-stride over the whole grid).
template <int V>
__device__ __forceinline__ void zero_tail(const int32_t* __restrict__ n_rows, long R, long vecs, void* rows) {
    if (!n_rows) return;
    long n = __ldg(n_rows);
    n = n < 0 ? 0 : n;
    raw_t<V>* o = static_cast<raw_t<V>*>(rows);
    for (long i = n * vecs + static_cast<long>(blockIdx.x) * blockDim.x + threadIdx.x; i < R * vecs;
         i += static_cast<long>(gridDim.x) * blockDim.x)
        o[i] = zero_raw<V>();
}

template <int V>
__global__ void __launch_bounds__(kThreads) permute_kernel(const void* __restrict__ x,
                                                           const int32_t* __restrict__ inv,
                                                           const int32_t* __restrict__ n_rows, int T, int K,
                                                           long vecs, void* __restrict__ x_sorted,
                                                           int32_t* __restrict__ status) {
    const long R = static_cast<long>(T) * K, total = static_cast<long>(T) * vecs;
    const raw_t<V>* in = static_cast<const raw_t<V>*>(x);
    raw_t<V>* out = static_cast<raw_t<V>*>(x_sorted);
    bool bad = false;
    for (long i = static_cast<long>(blockIdx.x) * blockDim.x + threadIdx.x; i < total;
         i += static_cast<long>(gridDim.x) * blockDim.x) {
        const long t = i / vecs, c = i - t * vecs;
        const raw_t<V> v = __ldg(in + i);
        for (int j = 0; j < K; ++j) {
            const int32_t p = position(inv, t * K + j, R, &bad);
            if (p >= 0) out[p * vecs + c] = v;
        }
    }
    zero_tail<V>(n_rows, R, vecs, x_sorted);
    if (bad) report_status(status, MOE_STATUS_BAD_MAP);
}

template <class E, int V>
__global__ void __launch_bounds__(kThreads) unpermute_kernel(const void* __restrict__ y_sorted,
                                                             const int32_t* __restrict__ inv,
                                                             const float* __restrict__ w,
                                                             const void* __restrict__ y_shared, int T, int K,
                                                             long vecs, void* __restrict__ out,
                                                             int32_t* __restrict__ status) {
    constexpr int N = V / sizeof(E);
    const long R = static_cast<long>(T) * K, total = static_cast<long>(T) * vecs;
    const raw_t<V>* in = static_cast<const raw_t<V>*>(y_sorted);
    bool bad = false;
    for (long i = static_cast<long>(blockIdx.x) * blockDim.x + threadIdx.x; i < total;
         i += static_cast<long>(gridDim.x) * blockDim.x) {
        const long t = i / vecs, c = i - t * vecs;
        float acc[N];
#pragma unroll
        for (int n = 0; n < N; ++n) acc[n] = 0.f;
        for (int j = 0; j < K; ++j) {
            const int32_t p = position(inv, t * K + j, R, &bad);
            const float wj = w ? __ldg(w + t * K + j) : 1.f;
            if (p < 0 || wj == 0.f) continue;
            float f[N];
            unpack<E, V>(__ldg(in + p * vecs + c), f);
#pragma unroll
            for (int n = 0; n < N; ++n) acc[n] = fmaf(wj, f[n], acc[n]);
        }
        if (y_shared) {
            float f[N];
            unpack<E, V>(__ldg(static_cast<const raw_t<V>*>(y_shared) + i), f);
#pragma unroll
            for (int n = 0; n < N; ++n) acc[n] += f[n];
        }
        static_cast<raw_t<V>*>(out)[i] = pack<E, V>(acc);
    }
    if (bad) report_status(status, MOE_STATUS_BAD_MAP);
}

// One warp per route: dy = w * dout, dw = <dout, y> over the row.
template <class E, int V>
__global__ void __launch_bounds__(kThreads) unpermute_bwd_kernel(
    const void* __restrict__ dout, const void* __restrict__ y_sorted, const int32_t* __restrict__ inv,
    const float* __restrict__ w, const int32_t* __restrict__ n_rows, int T, int K, long vecs,
    void* __restrict__ dy_sorted, float* __restrict__ dw, int32_t* __restrict__ status) {
    constexpr int N = V / sizeof(E);
    const long R = static_cast<long>(T) * K;
    const int lane = threadIdx.x & 31;
    bool bad = false;
    for (long r = (static_cast<long>(blockIdx.x) * blockDim.x + threadIdx.x) >> 5; r < R;
         r += (static_cast<long>(gridDim.x) * blockDim.x) >> 5) {
        const int32_t p = position(inv, r, R, &bad);
        const float wr = w ? __ldg(w + r) : 1.f;
        float dot = 0.f;
        if (p >= 0) {
            const raw_t<V>* d = static_cast<const raw_t<V>*>(dout) + (r / K) * vecs;
            for (long c = lane; c < vecs; c += 32) {
                float fd[N];
                unpack<E, V>(__ldg(d + c), fd);
                if (dw) {
                    float fy[N];
                    unpack<E, V>(__ldg(static_cast<const raw_t<V>*>(y_sorted) + p * vecs + c), fy);
#pragma unroll
                    for (int n = 0; n < N; ++n) dot = fmaf(fd[n], fy[n], dot);
                }
                if (dy_sorted) {
#pragma unroll
                    for (int n = 0; n < N; ++n) fd[n] = wr == 0.f ? 0.f : wr * fd[n];
                    static_cast<raw_t<V>*>(dy_sorted)[p * vecs + c] = pack<E, V>(fd);
                }
            }
        }
        if (dw) {
#pragma unroll
            for (int off = 16; off > 0; off >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, off);
            if (lane == 0) dw[r] = dot;
        }
    }
    if (dy_sorted) zero_tail<V>(n_rows, R, vecs, dy_sorted);
    if (bad) report_status(status, MOE_STATUS_BAD_MAP);
}

// Bytes per load: the largest power of two up to 16 that divides a row (rows
// start 16-byte aligned, so every row is then aligned to it).
int vec_bytes(long row_bytes) {
    for (int v = 16; v > 2; v >>= 1)
        if (row_bytes % v == 0) return v;
    return 2;
}

int grid_for(long threads) {
    const long blocks = (threads + kThreads - 1) / kThreads;
    return static_cast<int>(blocks < 1 ? 1 : blocks > 148L * 64 ? 148L * 64 : blocks);
}

}  // namespace

cudaError_t launch_permute(const RowsArgs& a, const void* x, void* x_sorted, cudaStream_t stream) {
    const long row = static_cast<long>(a.H) * dtype_bytes(a.dtype);
    const int v = vec_bytes(row);
    const long vecs = row / v;
    const int grid = grid_for(a.T * vecs);
    switch (v) {
        case 16: permute_kernel<16><<<grid, kThreads, 0, stream>>>(x, a.inv, a.n_rows, a.T, a.K, vecs, x_sorted, a.status); break;
        case 8: permute_kernel<8><<<grid, kThreads, 0, stream>>>(x, a.inv, a.n_rows, a.T, a.K, vecs, x_sorted, a.status); break;
        case 4: permute_kernel<4><<<grid, kThreads, 0, stream>>>(x, a.inv, a.n_rows, a.T, a.K, vecs, x_sorted, a.status); break;
        default: permute_kernel<2><<<grid, kThreads, 0, stream>>>(x, a.inv, a.n_rows, a.T, a.K, vecs, x_sorted, a.status); break;
    }
    return cudaGetLastError();
}

#define MOE_ROWS_DISPATCH(LAUNCH)                        \
    switch (a.dtype * 100 + v) {                         \
        case MOE_DTYPE_BF16 * 100 + 16: LAUNCH(__nv_bfloat16, 16) break; \
        case MOE_DTYPE_BF16 * 100 + 8: LAUNCH(__nv_bfloat16, 8) break;   \
        case MOE_DTYPE_BF16 * 100 + 4: LAUNCH(__nv_bfloat16, 4) break;   \
        case MOE_DTYPE_BF16 * 100 + 2: LAUNCH(__nv_bfloat16, 2) break;   \
        case MOE_DTYPE_F16 * 100 + 16: LAUNCH(__half, 16) break;         \
        case MOE_DTYPE_F16 * 100 + 8: LAUNCH(__half, 8) break;           \
        case MOE_DTYPE_F16 * 100 + 4: LAUNCH(__half, 4) break;           \
        case MOE_DTYPE_F16 * 100 + 2: LAUNCH(__half, 2) break;           \
        case MOE_DTYPE_F32 * 100 + 16: LAUNCH(float, 16) break;          \
        case MOE_DTYPE_F32 * 100 + 8: LAUNCH(float, 8) break;            \
        default: LAUNCH(float, 4) break;                                 \
    }

cudaError_t launch_unpermute(const RowsArgs& a, const void* y_sorted, const float* w, const void* y_shared, void* out,
                             cudaStream_t stream) {
    const long row = static_cast<long>(a.H) * dtype_bytes(a.dtype);
    const int v = vec_bytes(row);
    const long vecs = row / v;
    const int grid = grid_for(a.T * vecs);
#define MOE_LAUNCH(E, V)                                                                                        \
    unpermute_kernel<E, V><<<grid, kThreads, 0, stream>>>(y_sorted, a.inv, w, y_shared, a.T, a.K, vecs, out, a.status);
    MOE_ROWS_DISPATCH(MOE_LAUNCH)
#undef MOE_LAUNCH
    return cudaGetLastError();
}

cudaError_t launch_unpermute_bwd(const RowsArgs& a, const void* dout, const void* y_sorted, const float* w,
                                 void* dy_sorted, float* dw, cudaStream_t stream) {
    const long row = static_cast<long>(a.H) * dtype_bytes(a.dtype);
    const int v = vec_bytes(row);
    const long vecs = row / v;
    const int grid = grid_for(static_cast<long>(a.T) * a.K * 32);
#define MOE_LAUNCH(E, V)                                                                                          \
    unpermute_bwd_kernel<E, V><<<grid, kThreads, 0, stream>>>(dout, y_sorted, a.inv, w, a.n_rows, a.T, a.K, vecs, \
                                                              dy_sorted, dw, a.status);
    MOE_ROWS_DISPATCH(MOE_LAUNCH)
#undef MOE_LAUNCH
    return cudaGetLastError();
}

}  // namespace moe
