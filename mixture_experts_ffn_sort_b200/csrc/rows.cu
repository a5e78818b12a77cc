// rows.cu -- rows sorted by expert and back (moe_permute, moe_unpermute) and
// the gradients (moe_unpermute_bwd), for bf16, f16 and f32 rows.
//
// Everything here is indexed by token: inv_route gives the sorted position of
// each of a token's K routes, so a token's row is read once for its K copies
// (permute), its K sorted rows are summed in slot order by one thread per
// 16-byte column (unpermute, a fixed order), and no two tokens write the same
// row.  A position outside [0, T*K) is skipped: -1 silently, anything else
// with MOE_STATUS_BAD_MAP.  All of it is bound by memory: a few operations for
// every element read or written.
//
// Each kernel has two forms: rows whose bytes are a multiple of 16 are moved
// by aligned 16-byte vectors; other rows (SHIFT) by the shifted windows of
// rows.cuh, on the alignment of the tensor that is K times the larger one.
#include <type_traits>

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
__device__ __forceinline__ void zero_tail(const int32_t* __restrict__ n_rows, long R, long row_bytes, void* rows) {
    if (!n_rows) return;
    long n = __ldg(n_rows);
    if (n >= R) return;
    n = n < 0 ? 0 : n;
    char* o = static_cast<char*>(rows);
    const long begin = n * row_bytes, end = R * row_bytes;  // multiples of 2
    for (long b = (begin & ~15L) + (static_cast<long>(blockIdx.x) * blockDim.x + threadIdx.x) * 16; b < end;
         b += static_cast<long>(gridDim.x) * blockDim.x * 16) {
        if (b >= begin && b + 16 <= end) {
            *reinterpret_cast<uint4*>(o + b) = make_uint4(0, 0, 0, 0);
        } else {
            for (long i = b; i < b + 16; i += 2)
                if (i >= begin && i < end) *reinterpret_cast<uint16_t*>(o + i) = 0;
        }
    }
}

// x_sorted[inv[t, j]] = x[t].  One thread per 16-byte column of a token: one
// load, K stores.  SHIFT: one thread per 16-byte block of the sorted rows.
template <class E, bool SHIFT>
__global__ void __launch_bounds__(kThreads) permute_kernel(const char* __restrict__ x,
                                                           const int32_t* __restrict__ inv,
                                                           const int32_t* __restrict__ n_rows, int T, int K,
                                                           long row_bytes, const FastDiv vecs,
                                                           char* __restrict__ x_sorted, int32_t* __restrict__ status) {
    const long R = static_cast<long>(T) * K, total = static_cast<long>(T) * vecs.d;
    bool bad = false;
    for (long i = static_cast<long>(blockIdx.x) * blockDim.x + threadIdx.x; i < total;
         i += static_cast<long>(gridDim.x) * blockDim.x) {
        const long t = vecs.div(i), c = i - t * vecs.d;
        uint4 v;
        if (!SHIFT) v = __ldg(reinterpret_cast<const uint4*>(x) + i);
#pragma unroll 4
        for (int j = 0; j < K; ++j) {
            const int32_t p = position(inv, t * K + j, R, &bad);
            if (p < 0) continue;
            const long row = p * row_bytes;
            if (!SHIFT) {
                reinterpret_cast<uint4*>(x_sorted + row)[c] = v;
            } else {
                const long rel = 16 * c - (row & 15);  // the block's first byte within the row
                if (rel >= row_bytes) continue;
                v = load_window(x, t * row_bytes + rel, T * row_bytes);
                constexpr long S = sizeof(E);
                const int to = static_cast<int>((row_bytes - rel) / S < 16 ? (row_bytes - rel) / S : 16);
                store_part<E>(x_sorted + row + rel, v, static_cast<int>(-rel / S), to);
            }
        }
    }
    zero_tail(n_rows, R, row_bytes, x_sorted);
    if (bad) report_status(status, MOE_STATUS_BAD_MAP);
}

// Slots of a batch at most.
constexpr int kBatch = 4;

// out[t] = sum_j w[t, j] y[inv[t, j]] (+ y_shared[t]).  One thread per 16-byte
// column of a token; slots in batches: all positions, then all rows, then the
// sums in slot order, so that the loads of a batch are in flight together.
template <class E, bool SHIFT>
__global__ void __launch_bounds__(kThreads) unpermute_kernel(const char* __restrict__ y_sorted,
                                                             const int32_t* __restrict__ inv,
                                                             const float* __restrict__ w,
                                                             const char* __restrict__ y_shared, int T, int K,
                                                             int batch, long row_bytes, const FastDiv vecs,
                                                             char* __restrict__ out, int32_t* __restrict__ status) {
    constexpr int N = kVec<E>;
    constexpr int B = kBatch;
    const long R = static_cast<long>(T) * K, total = static_cast<long>(T) * vecs.d;
    bool bad = false;
    for (long i = static_cast<long>(blockIdx.x) * blockDim.x + threadIdx.x; i < total;
         i += static_cast<long>(gridDim.x) * blockDim.x) {
        const long t = vecs.div(i), c = i - t * vecs.d;
        float acc[N];
#pragma unroll
        for (int n = 0; n < N; ++n) acc[n] = 0.f;
        for (int j0 = 0; j0 < K; j0 += batch) {
            const int n_here = K - j0 < batch ? K - j0 : batch;
            int32_t p[B];
            float wj[B];
#pragma unroll
            for (int b = 0; b < B; ++b) {
                p[b] = -1;
                wj[b] = 1.f;
                if (b < n_here) {
                    p[b] = position(inv, t * K + j0 + b, R, &bad);
                    if (w) wj[b] = __ldg(w + t * K + j0 + b);
                    if (wj[b] == 0.f) p[b] = -1;
                }
            }
            uint4 v[B];
#pragma unroll
            for (int b = 0; b < B; ++b) {
                if (p[b] < 0) continue;
                const long row = p[b] * row_bytes;
                if (SHIFT) v[b] = load_window(y_sorted, row + 16 * c, R * row_bytes);
                else v[b] = __ldg(reinterpret_cast<const uint4*>(y_sorted + row) + c);
            }
#pragma unroll
            for (int b = 0; b < B; ++b) {
                if (p[b] < 0) continue;
                float f[N];
                unpack<E>(v[b], f);
#pragma unroll
                for (int n = 0; n < N; ++n) acc[n] = fmaf(wj[b], f[n], acc[n]);
            }
        }
        const long at = t * row_bytes + 16 * c;
        if (y_shared) {
            float f[N];
            unpack<E>(SHIFT ? load_window(y_shared, at, T * row_bytes)
                            : __ldg(reinterpret_cast<const uint4*>(y_shared + at)), f);
#pragma unroll
            for (int n = 0; n < N; ++n) acc[n] += f[n];
        }
        if (SHIFT) store_part<E>(out + at, pack<E>(acc), 0, static_cast<int>((row_bytes - 16 * c) / sizeof(E)));
        else *reinterpret_cast<uint4*>(out + at) = pack<E>(acc);
    }
    if (bad) report_status(status, MOE_STATUS_BAD_MAP);
}

// dy[p] = w dout[t], dw = <dout[t], y[p]> for p = inv[t, j].  G threads per
// route, each with every G-th 16-byte vector, U of them at a time; the dot
// product is summed over the lanes by a butterfly and, for G > 32, over the
// warps in order.  SHIFT: vectors on the alignment of the sorted rows.
template <class E, bool SHIFT, int G>
__global__ void __launch_bounds__(kThreads) unpermute_bwd_kernel(
    const char* __restrict__ dout, const char* __restrict__ y_sorted, const int32_t* __restrict__ inv,
    const float* __restrict__ w, const int32_t* __restrict__ n_rows, int T, const FastDiv K, long row_bytes,
    char* __restrict__ dy_sorted, float* __restrict__ dw, int32_t* __restrict__ status) {
    constexpr int N = kVec<E>;
    constexpr int U = SHIFT ? 2 : 4;
    constexpr int PER = kThreads / G;  // routes of a block at a time
    constexpr long S = sizeof(E);
    __shared__ float sh[kThreads / 32];
    const long R = static_cast<long>(T) * K.d;
    const int lane = threadIdx.x % G;
    bool bad = false;
    for (long r0 = static_cast<long>(blockIdx.x) * PER; r0 < R; r0 += static_cast<long>(gridDim.x) * PER) {
        const long r = r0 + threadIdx.x / G;
        const int32_t p = r < R ? position(inv, r, R, &bad) : -1;
        float dot = 0.f;
        if (p >= 0) {
            const float wr = w ? __ldg(w + r) : 1.f;
            const long t = K.div(r), row = p * row_bytes;
            const long lead = SHIFT ? row & 15 : 0;  // bytes of the first block before the row
            const long blocks = (lead + row_bytes + 15) >> 4;
            const char* d = dout + t * row_bytes;
            for (long c0 = lane; c0 < blocks; c0 += G * U) {
                uint4 vd[U], vy[U];
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const long c = c0 + u * G;
                    if (c >= blocks) continue;
                    const long rel = 16 * c - lead;
                    vd[u] = SHIFT ? load_window(dout, t * row_bytes + rel, T * row_bytes)
                                  : __ldg(reinterpret_cast<const uint4*>(d) + c);
                    if (dw)
                        vy[u] = SHIFT ? load_block(y_sorted, row + rel, R * row_bytes)
                                      : __ldg(reinterpret_cast<const uint4*>(y_sorted + row) + c);
                }
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const long c = c0 + u * G;
                    if (c >= blocks) continue;
                    const long rel = 16 * c - lead;
                    float fd[N];
                    unpack<E>(vd[u], fd);
                    // Elements of this vector that belong to the row.
                    const int from = SHIFT ? static_cast<int>(-rel / S) : 0;
                    const int to = SHIFT && row_bytes - rel < 16 ? static_cast<int>((row_bytes - rel) / S) : N;
                    if (dw) {
                        float fy[N];
                        unpack<E>(vy[u], fy);
#pragma unroll
                        for (int n = 0; n < N; ++n)
                            if (!SHIFT || (n >= from && n < to)) dot = fmaf(fd[n], fy[n], dot);
                    }
                    if (dy_sorted) {
#pragma unroll
                        for (int n = 0; n < N; ++n) fd[n] = wr == 0.f ? 0.f : wr * fd[n];
                        if (SHIFT) store_part<E>(dy_sorted + row + rel, pack<E>(fd), from, to);
                        else reinterpret_cast<uint4*>(dy_sorted + row)[c] = pack<E>(fd);
                    }
                }
            }
        }
        if (dw) {
#pragma unroll
            for (int off = (G < 32 ? G : 32) / 2; off > 0; off >>= 1)
                dot += __shfl_xor_sync(0xffffffffu, dot, off);
            if (G > 32) {
                __syncthreads();
                if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = dot;
                __syncthreads();
                dot = 0.f;
                const int first = threadIdx.x / G * (G / 32);
#pragma unroll
                for (int i = 0; i < G / 32; ++i) dot += sh[first + i];
            }
            if (lane == 0 && r < R) dw[r] = dot;
        }
    }
    if (dy_sorted) zero_tail(n_rows, R, row_bytes, dy_sorted);
    if (bad) report_status(status, MOE_STATUS_BAD_MAP);
}

int grid_for(long threads) {
    const long blocks = (threads + kThreads - 1) / kThreads;
    return static_cast<int>(blocks < 1 ? 1 : blocks > 148L * 64 ? 148L * 64 : blocks);
}

long row_bytes_of(const RowsArgs& a) { return static_cast<long>(a.H) * dtype_bytes(a.dtype); }

// Calls f(E, SHIFT) for the row type and alignment.
template <class F>
void dispatch(const RowsArgs& a, F f) {
    const bool shift = row_bytes_of(a) % 16 != 0;
    switch (a.dtype) {
        case MOE_DTYPE_BF16: shift ? f(__nv_bfloat16{}, std::true_type{}) : f(__nv_bfloat16{}, std::false_type{}); break;
        case MOE_DTYPE_F16: shift ? f(__half{}, std::true_type{}) : f(__half{}, std::false_type{}); break;
        default: shift ? f(float{}, std::true_type{}) : f(float{}, std::false_type{}); break;
    }
}

}  // namespace

cudaError_t launch_permute(const RowsArgs& a, const void* x, void* x_sorted, cudaStream_t stream) {
    const long row = row_bytes_of(a);
    // Shifted rows may touch one 16-byte block more than they have.
    const FastDiv vecs(static_cast<unsigned>(row % 16 ? row / 16 + 2 : row / 16));
    const int grid = grid_for(static_cast<long>(a.T) * vecs.d);
    dispatch(a, [&](auto e, auto shift) {
        permute_kernel<decltype(e), decltype(shift)::value><<<grid, kThreads, 0, stream>>>(
            static_cast<const char*>(x), a.inv, a.n_rows, a.T, a.K, row, vecs, static_cast<char*>(x_sorted), a.status);
    });
    return cudaGetLastError();
}

cudaError_t launch_unpermute(const RowsArgs& a, const void* y_sorted, const float* w, const void* y_shared, void* out,
                             cudaStream_t stream) {
    const long row = row_bytes_of(a);
    const FastDiv vecs(static_cast<unsigned>((row + 15) / 16));
    const int grid = grid_for(static_cast<long>(a.T) * vecs.d);
    dispatch(a, [&](auto e, auto shift) {
        constexpr int B = kBatch;
        const int batches = (a.K + B - 1) / B, batch = (a.K + batches - 1) / batches;
        unpermute_kernel<decltype(e), decltype(shift)::value><<<grid, kThreads, 0, stream>>>(
            static_cast<const char*>(y_sorted), a.inv, w, static_cast<const char*>(y_shared), a.T, a.K, batch, row,
            vecs, static_cast<char*>(out), a.status);
    });
    return cudaGetLastError();
}

cudaError_t launch_unpermute_bwd(const RowsArgs& a, const void* dout, const void* y_sorted, const float* w,
                                 void* dy_sorted, float* dw, cudaStream_t stream) {
    const long row = row_bytes_of(a), R = static_cast<long>(a.T) * a.K, vecs = (row + 15) / 16;
    const FastDiv K(static_cast<unsigned>(a.K));
    // Threads per route: a warp when every lane then has work, fewer for short
    // rows, a whole block while the routes are too few to fill the GPU with warps.
    const int g = vecs <= 8 ? 8 : vecs <= 64 || R >= 148 * 16 ? 32 : 256;
    dispatch(a, [&](auto e, auto shift) {
        auto launch = [&](auto G) {
            constexpr int kG = decltype(G)::value;
            unpermute_bwd_kernel<decltype(e), decltype(shift)::value, kG><<<grid_for(R * kG), kThreads, 0, stream>>>(
                static_cast<const char*>(dout), static_cast<const char*>(y_sorted), a.inv, w, a.n_rows, a.T, K, row,
                static_cast<char*>(dy_sorted), dw, a.status);
        };
        if (g == 8) launch(std::integral_constant<int, 8>{});
        else if (g == 32) launch(std::integral_constant<int, 32>{});
        else launch(std::integral_constant<int, 256>{});
    });
    return cudaGetLastError();
}

}  // namespace moe
