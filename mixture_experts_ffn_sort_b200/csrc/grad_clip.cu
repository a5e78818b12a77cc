// grad_clip.cu -- the global 2-norm of many gradient tensors and clipping by
// it (moe_grad_sumsq, moe_grad_clip).
//
// The tensors' addresses travel in the kernel's parameters (no copy of a table
// to the device, so the calls can be captured in a graph), a launch taking up
// to kCap of them.  Every tensor is cut into chunks on 16-byte boundaries of its
// own memory.  A grid of a few blocks per SM sums the chunks of a launch; a grid
// of the same size or, for large lists, a block for every chunk scales them; a
// list of a few chunks is clipped by one cluster of blocks.
// Values are squared and added in fp32 over one 16-byte vector, then in fp64 per
// thread, per block (a partial sum in the workspace) and over the partials,
// always in the same order.
//
// Bound by memory: 769 bf16 tensors of 2 MB are summed in 245 us, 6.6 TB/s, and
// scaled into other memory in 495 us, 6.5 TB/s.  The norm has to be known before
// anything is scaled, so what does not fit L2 is read twice.
#include <type_traits>

#include "launch_after.cuh"
#include "router_common.cuh"
#include "rows.cuh"
#include "train.h"

namespace moe {

namespace {

constexpr int kThreads = 256;  // that share a chunk (of a block, or of one of the groups of a larger one)
__device__ __forceinline__ int chunk_thread() { return threadIdx.x % kThreads; }
// A chunk is U vectors of 16 bytes a thread, all in flight together.
template <int U>
constexpr long kChunk = static_cast<long>(kThreads) * 16 * U;
constexpr int kScaleU = 4;
constexpr int kPerSm = 4;
constexpr int kMaxBlocks = 148 * kPerSm;

template <int CAP>
struct GradTable {
    const void* src[CAP];
    void* dst[CAP];
    long numel_type[CAP];  // numel * 4 + dtype
    int first[CAP + 1];    // first chunk of each tensor; first[n] = chunks in all
    // Where to look for a chunk's tensor: hint[h] holds chunk h << shift, the
    // last one the last chunk.
    static constexpr int kHints = CAP < 1000 ? 2 * CAP : 1024;
    uint16_t hint[kHints + 1];
    int shift, n;
};

// The tensor holding chunk c: the last one whose first chunk is <= c, between
// two hints.  (A search through all of 1000 tensors waits for ten parameters
// one after the other: 10.0 us against 9.0 us for 800 tensors of 8 KB.)
template <int CAP>
__device__ __forceinline__ int tensor_of(const GradTable<CAP>& tab, int c) {
    int lo = tab.hint[c >> tab.shift], hi = tab.hint[(c >> tab.shift) + 1] + 1;
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
// overflow or lose them.  (From 1e-36 on, eight squares that are rounded to
// multiples of 2^-149 are off by less than 2^-26 of their sum.)
template <class E>
__device__ __forceinline__ double vec_sumsq(const uint4& raw) {
    constexpr int N = 16 / sizeof(E);
    float f[N];
    unpack<E>(raw, f);
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < N; ++i) s = fmaf(f[i], f[i], s);
    if ((s > 1e-36f && s < 1e30f) || !(raw.x | raw.y | raw.z | raw.w)) return s;
    double d = 0.;
#pragma unroll
    for (int i = 0; i < N; ++i) d = fma(static_cast<double>(f[i]), static_cast<double>(f[i]), d);
    return d;
}

// The bytes of a tensor that one step of a block covers: chunk k, as offsets
// from the tensor's 16-byte boundary (its elements are [skip, end) of them).
template <int U>
struct Span {
    long lo, skip, end;
    template <class E>
    static __device__ __forceinline__ Span of(const void* src, long numel, long k) {
        const long skip = static_cast<long>(reinterpret_cast<uintptr_t>(src) & 15);
        return {k * kChunk<U>, skip, skip + numel * static_cast<long>(sizeof(E))};
    }
    __device__ __forceinline__ bool inside() const { return lo >= skip && lo + kChunk<U> <= end; }
    __device__ __forceinline__ long at(int u) const {
        return lo + (static_cast<long>(u) * kThreads + chunk_thread()) * 16;
    }
};

// Calls f(byte offset) for this thread's element of the vectors that only in
// part belong to the tensor: its first (before the first 16-byte boundary, or
// all of a tensor within 16 bytes) and its last.  Lanes 0..7 take the elements
// of the first, 32..39 those of the last.
template <class E, int U, class F>
__device__ __forceinline__ void part_elements(const Span<U>& s, F f) {
    const int i = threadIdx.x & 31;
    if (i >= kVec<E> || chunk_thread() >= 64) return;
    const bool first = chunk_thread() < 32;
    const long last = s.end & ~15L;  // start of the last vector, if it is not whole
    const long o = first ? 0 : last;
    if (o < s.lo || o >= s.lo + kChunk<U>) return;
    if (first ? s.skip == 0 && s.end >= 16 : last == s.end || last == 0) return;
    const long b = o + i * static_cast<long>(sizeof(E));
    if (b >= s.skip && b < s.end) f(b);
}

template <class E, int U>
__device__ __forceinline__ double chunk_sumsq(const void* src, long numel, long k) {
    const Span<U> s = Span<U>::template of<E>(src, numel, k);
    const char* base = static_cast<const char*>(src) - s.skip;
    double acc = 0.;
    uint4 v[U];
    if (s.inside()) {
#pragma unroll
        for (int u = 0; u < U; ++u) v[u] = __ldg(reinterpret_cast<const uint4*>(base + s.at(u)));
    } else {  // the tensor's first or last chunk
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const long o = s.at(u);
            v[u] = make_uint4(0, 0, 0, 0);
            if (o >= s.skip && o + 16 <= s.end) v[u] = __ldg(reinterpret_cast<const uint4*>(base + o));
        }
        part_elements<E, U>(s, [&](long b) {
            const double f = elem_to_float(*reinterpret_cast<const E*>(base + b));
            acc = f * f;
        });
    }
#pragma unroll
    for (int u = 0; u < U; ++u) acc += vec_sumsq<E>(v[u]);
    return acc;
}

// The squares of the table's chunk c (this thread's share).
template <int CAP, int U>
__device__ __forceinline__ double table_sumsq(const GradTable<CAP>& tab, int c) {
    const int i = tensor_of(tab, c);
    const long k = c - tab.first[i], n = tab.numel_type[i] >> 2;
    switch (tab.numel_type[i] & 3) {
        case MOE_DTYPE_BF16: return chunk_sumsq<__nv_bfloat16, U>(tab.src[i], n, k);
        case MOE_DTYPE_F16: return chunk_sumsq<__half, U>(tab.src[i], n, k);
        default: return chunk_sumsq<float, U>(tab.src[i], n, k);
    }
}

template <int CAP, int U>
__global__ void __launch_bounds__(kThreads, kPerSm) sumsq_kernel(const __grid_constant__ GradTable<CAP> tab,
                                                         double* __restrict__ partial) {
    __shared__ double sh[kThreads / 32];
    grid_dependency_wait();
    double acc = 0.;
    const int chunks = tab.first[tab.n];
    for (int c = blockIdx.x; c < chunks; c += gridDim.x) acc += table_sumsq<CAP, U>(tab, c);
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
    grid_dependency_wait();  // the partial sums
    const double s = sum_partials(partial, n, sh);
    if (threadIdx.x == 0) {
        if (sumsq) *sumsq = s;
        if (norm) *norm = static_cast<float>(sqrt(s));
    }
}

// The factor for a sum of squares.
__device__ __forceinline__ double clip_factor(double sumsq, float max_norm, float eps, double* norm) {
    *norm = sqrt(sumsq);
    const double over = *norm + static_cast<double>(eps), ratio = static_cast<double>(max_norm) / over;
    return ratio >= 1. || over == 0. ? 1. : ratio;  // 0 / 0 clips nothing, NaN stays NaN
}

// Whether the factor, rounded to fp32 as f, is too small for one of its normal numbers.
__device__ __forceinline__ bool subnormal(float f, double ratio) { return f < 0x1p-126f && ratio > 0.; }

template <class E>
__device__ __forceinline__ uint4 scaled(const uint4& v, float f) {
    float g[kVec<E>];
    unpack<E>(v, g);
#pragma unroll
    for (int i = 0; i < kVec<E>; ++i) g[i] *= f;
    return pack<E>(g);
}

template <class E, int U>
__device__ __forceinline__ void chunk_scale(const void* src, void* dst, long numel, long k, float f) {
    const Span<U> s = Span<U>::template of<E>(src, numel, k);
    const char* base = static_cast<const char*>(src) - s.skip;
    char* to = static_cast<char*>(dst) - s.skip;
    const bool together = (reinterpret_cast<uintptr_t>(to) & 15) == 0;  // src and dst share their offset
    if (together) {
        uint4 v[U];
        const bool inside = s.inside();
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (inside || (s.at(u) >= s.skip && s.at(u) + 16 <= s.end))
                v[u] = *reinterpret_cast<const uint4*>(base + s.at(u));
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (inside || (s.at(u) >= s.skip && s.at(u) + 16 <= s.end))
                *reinterpret_cast<uint4*>(to + s.at(u)) = scaled<E>(v[u], f);
        if (!inside)
            part_elements<E, U>(s, [&](long b) {
                *reinterpret_cast<E*>(to + b) =
                    elem_from_float<E>(elem_to_float(*reinterpret_cast<const E*>(base + b)) * f);
            });
        return;
    }
    // Another offset: element by element, neighbouring threads on neighbouring elements.
    const long first = s.lo > s.skip ? s.lo : s.skip, past = s.lo + kChunk<U> < s.end ? s.lo + kChunk<U> : s.end;
#pragma unroll 8
    for (long b = first + chunk_thread() * static_cast<long>(sizeof(E)); b < past; b += kThreads * sizeof(E))
        *reinterpret_cast<E*>(to + b) =
            elem_from_float<E>(elem_to_float(*reinterpret_cast<const E*>(base + b)) * f);
}

template <int CAP>
__device__ __forceinline__ void table_scale(const GradTable<CAP>& tab, int c, float f) {
    const int i = tensor_of(tab, c);
    const long k = c - tab.first[i], n = tab.numel_type[i] >> 2;
    if (f == 1.f && tab.src[i] == tab.dst[i]) return;  // in place, nothing to clip
    switch (tab.numel_type[i] & 3) {
        case MOE_DTYPE_BF16: chunk_scale<__nv_bfloat16, kScaleU>(tab.src[i], tab.dst[i], n, k, f); break;
        case MOE_DTYPE_F16: chunk_scale<__half, kScaleU>(tab.src[i], tab.dst[i], n, k, f); break;
        default: chunk_scale<float, kScaleU>(tab.src[i], tab.dst[i], n, k, f); break;
    }
}

template <class E>
__device__ __forceinline__ void chunk_scale_small(const void* src, void* dst, long numel, long k, float a, float b) {
    const Span<kScaleU> s = Span<kScaleU>::template of<E>(src, numel, k);
    const long per = kChunk<kScaleU> / static_cast<long>(sizeof(E)), lead = s.skip / static_cast<long>(sizeof(E));
    const long first = k * per > lead ? k * per - lead : 0;
    const long past = (k + 1) * per - lead < numel ? (k + 1) * per - lead : numel;
    for (long i = first + chunk_thread(); i < past; i += kThreads)
        static_cast<E*>(dst)[i] = elem_from_float<E>(elem_to_float(static_cast<const E*>(src)[i]) * a * b);
}

// Chunks c, c - step, ... of the table (this thread's share) by a factor below
// fp32's normal numbers: a, which has all of its bits, then b, a power of two.
// Not inlined, and element by element, because it is hardly ever taken: as a
// second factor for every vector it took 769 bf16 tensors of 2 MB from 719 to 728
// us, inlined beside the other loop to 722 us.
template <int CAP>
__device__ __noinline__ void table_scale_small(const GradTable<CAP>& tab, int c, int step, double ratio) {
    const int e = max(ilogb(ratio) + 1, -149);
    const float a = static_cast<float>(ldexp(ratio, -e)), b = ldexpf(1.f, e);
    for (; c >= 0; c -= step) {
        const int i = tensor_of(tab, c);
        const long k = c - tab.first[i], n = tab.numel_type[i] >> 2;
        switch (tab.numel_type[i] & 3) {
            case MOE_DTYPE_BF16: chunk_scale_small<__nv_bfloat16>(tab.src[i], tab.dst[i], n, k, a, b); break;
            case MOE_DTYPE_F16: chunk_scale_small<__half>(tab.src[i], tab.dst[i], n, k, a, b); break;
            default: chunk_scale_small<float>(tab.src[i], tab.dst[i], n, k, a, b); break;
        }
    }
}

template <int CAP>
__global__ void __launch_bounds__(kThreads, kPerSm) scale_kernel(const __grid_constant__ GradTable<CAP> tab,
                                                         const double* __restrict__ partial, int n_partial,
                                                         const double* __restrict__ sumsq, float max_norm, float eps,
                                                         float* __restrict__ norm_out) {
    __shared__ double sh[kThreads / 32];
    grid_dependency_wait();  // the partial sums
    const double s = sumsq ? *sumsq : sum_partials(partial, n_partial, sh);
    double norm;
    const double ratio = clip_factor(s, max_norm, eps, &norm);
    const float f = static_cast<float>(ratio);
    if (norm_out && blockIdx.x == 0 && threadIdx.x == 0) *norm_out = static_cast<float>(norm);
    const int chunks = tab.first[tab.n];
    // The last ones first: they may still be in L2 from the sum.
    if (subnormal(f, ratio)) return table_scale_small(tab, chunks - 1 - static_cast<int>(blockIdx.x), gridDim.x, ratio);
    for (int b = blockIdx.x; b < chunks; b += gridDim.x) table_scale(tab, chunks - 1 - b, f);
}

// Both steps for a small list, in one launch that reads it once: a cluster of
// blocks, each of four groups of threads that take a chunk and keep it in
// registers, exchanges the blocks' sums through distributed shared memory, adds
// them in the same order everywhere, and scales.
constexpr int kClusterBlocks = 8;
constexpr int kClusterThreads = 4 * kThreads;

template <class E>
__device__ __forceinline__ double kept_sumsq(const Span<kScaleU>& s, const char* base, const uint4 (&v)[kScaleU]) {
    double acc = 0.;
    part_elements<E, kScaleU>(s, [&](long b) {
        const double f = elem_to_float(*reinterpret_cast<const E*>(base + b));
        acc = f * f;
    });
#pragma unroll
    for (int u = 0; u < kScaleU; ++u) acc += vec_sumsq<E>(v[u]);
    return acc;
}

template <class E>
__device__ __forceinline__ void kept_scale(const Span<kScaleU>& s, const char* base, char* to,
                                           const uint4 (&v)[kScaleU], float f) {
#pragma unroll
    for (int u = 0; u < kScaleU; ++u)
        if (s.at(u) >= s.skip && s.at(u) + 16 <= s.end) *reinterpret_cast<uint4*>(to + s.at(u)) = scaled<E>(v[u], f);
    part_elements<E, kScaleU>(s, [&](long b) {
        *reinterpret_cast<E*>(to + b) = elem_from_float<E>(elem_to_float(*reinterpret_cast<const E*>(base + b)) * f);
    });
}

template <int CAP>
__global__ void __cluster_dims__(kClusterBlocks, 1, 1) __launch_bounds__(kClusterThreads, 1)
    clip_cluster_kernel(const __grid_constant__ GradTable<CAP> tab, float max_norm, float eps,
                        float* __restrict__ norm_out) {
    __shared__ double warps[kClusterThreads / 32];
    __shared__ double blocks[kClusterBlocks];
    cluster_arrive();  // waited for before the first store into another block
    const uint32_t rank = cluster_ctarank();
    const int c = static_cast<int>(rank) * (kClusterThreads / kThreads) + threadIdx.x / kThreads;
    const bool have = c < tab.first[tab.n];
    const int i = have ? tensor_of(tab, c) : 0;
    const int type = static_cast<int>(tab.numel_type[i] & 3);
    const char* src = static_cast<const char*>(tab.src[i]);
    const Span<kScaleU> s = type == MOE_DTYPE_F32
                                ? Span<kScaleU>::template of<float>(src, tab.numel_type[i] >> 2, c - tab.first[i])
                                : Span<kScaleU>::template of<__half>(src, tab.numel_type[i] >> 2, c - tab.first[i]);
    const char* base = src - s.skip;
    grid_dependency_wait();
    uint4 v[kScaleU];
#pragma unroll
    for (int u = 0; u < kScaleU; ++u) {
        v[u] = make_uint4(0, 0, 0, 0);
        if (have && s.at(u) >= s.skip && s.at(u) + 16 <= s.end) v[u] = *reinterpret_cast<const uint4*>(base + s.at(u));
    }
    double acc = 0.;
    if (have)
        acc = type == MOE_DTYPE_BF16  ? kept_sumsq<__nv_bfloat16>(s, base, v)
              : type == MOE_DTYPE_F16 ? kept_sumsq<__half>(s, base, v)
                                      : kept_sumsq<float>(s, base, v);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, off);
    if ((threadIdx.x & 31) == 0) warps[threadIdx.x >> 5] = acc;
    __syncthreads();
    cluster_wait();
    if (threadIdx.x < kClusterBlocks) {  // this block's sum, to every block of the cluster
        double sum = 0.;
        for (int w = 0; w < kClusterThreads / 32; ++w) sum += warps[w];
        asm volatile("st.shared::cluster.f64 [%0], %1;" ::"r"(cluster_map_shared(smem_u32(&blocks[rank]), threadIdx.x)),
                     "d"(sum)
                     : "memory");
    }
    cluster_sync_all();
    double sum = 0.;
#pragma unroll
    for (int w = 0; w < kClusterBlocks; ++w) sum += blocks[w];
    double norm;
    const double ratio = clip_factor(sum, max_norm, eps, &norm);
    const float f = static_cast<float>(ratio);
    if (norm_out && rank == 0 && threadIdx.x == 0) *norm_out = static_cast<float>(norm);
    char* dst = static_cast<char*>(tab.dst[i]);
    if (!have || (f == 1.f && src == dst)) return;
    if (subnormal(f, ratio)) {
        table_scale_small(tab, c, c + 1, ratio);
    } else if (((reinterpret_cast<uintptr_t>(src) ^ reinterpret_cast<uintptr_t>(dst)) & 15) == 0) {
        char* to = dst - s.skip;
        if (type == MOE_DTYPE_BF16) kept_scale<__nv_bfloat16>(s, base, to, v, f);
        else if (type == MOE_DTYPE_F16) kept_scale<__half>(s, base, to, v, f);
        else kept_scale<float>(s, base, to, v, f);
    } else {
        table_scale(tab, c, f);
    }
}

// Tensors of a launch: the table is 28 bytes for each, and 2 KB of hints, and a
// kernel's parameters hold 32,764.  Every launch copies the whole table, about
// 3 us on the host for the largest, so there are smaller ones.
constexpr int kCap = 1000;

template <int V>
using Int = std::integral_constant<int, V>;

// Calls f with the size of table that n tensors take.
template <class F>
cudaError_t with_table(int n, F f) {
    return n <= 32 ? f(Int<32>{}) : n <= 128 ? f(Int<128>{}) : n <= 256 ? f(Int<256>{}) : n <= 512 ? f(Int<512>{})
                                                                                             : f(Int<kCap>{});
}

long chunks_of(const moe_tensor_ref& r, long chunk) {
    if (r.numel == 0) return 0;
    const long skip = static_cast<long>(reinterpret_cast<uintptr_t>(r.data) & 15);
    return (skip + r.numel * dtype_bytes(r.dtype) + chunk - 1) / chunk;
}

// Fills the table with refs[*at ..): up to CAP non-empty tensors in chunks of
// so many bytes (which fit an int: grad_chunks_fit).  False when none is left.
template <int CAP>
bool fill(GradTable<CAP>* tab, const moe_tensor_ref* refs, int n, int* at, long chunk) {
    tab->n = 0;
    long chunks = 0;
    for (; *at < n && tab->n < CAP; ++*at) {
        const moe_tensor_ref& r = refs[*at];
        const long c = chunks_of(r, chunk);
        if (c == 0) continue;
        const int i = tab->n++;
        tab->src[i] = r.data;
        tab->dst[i] = r.out;
        tab->numel_type[i] = r.numel * 4 + r.dtype;
        tab->first[i] = static_cast<int>(chunks);
        chunks += c;
    }
    tab->first[tab->n] = static_cast<int>(chunks);
    tab->shift = 0;
    while ((chunks - 1) >> tab->shift >= GradTable<CAP>::kHints) ++tab->shift;
    int i = 0, h = 0;
    for (; static_cast<long>(h) << tab->shift < chunks; ++h) {
        while (tab->first[i + 1] <= h << tab->shift) ++i;
        tab->hint[h] = static_cast<uint16_t>(i);
    }
    tab->hint[h] = static_cast<uint16_t>(tab->n ? tab->n - 1 : 0);
    return tab->n > 0;
}

int grid_of(int chunks) { return chunks < kMaxBlocks ? chunks : kMaxBlocks; }

// Lists of at least kLarge bytes keep every block busy with 8 vectors a thread.
// Measured for 769 tensors of 2 MB: their sum 248 us against 320 us with 4, and
// the scaling with a block a chunk 510 us against 565 us with a grid that stays
// (before the hints of GradTable, which took it to 495 us).  Below it, more and smaller chunks spread better and one launch less
// counts for more (9 tensors, 6 MB: both in 5.6 us against 7.7 us).
constexpr long kLarge = 64L << 20;

// Lists of as many chunks (16 KB or less) as a cluster has groups of threads are
// clipped by one launch: 9 fp32 tensors of 8 KB take 3.9 us a call in a loop of
// calls, which the host bounds, against 5.8 us with two launches, and 3.5 us
// against 4.1 us of the GPU's time in a graph.
constexpr int kClusterChunks = kClusterBlocks * kClusterThreads / kThreads;

bool is_large(const moe_tensor_ref* refs, int n) {
    long bytes = 0;
    for (int i = 0; i < n; ++i) bytes += refs[i].numel * dtype_bytes(refs[i].dtype);
    return bytes >= kLarge;
}

template <int CAP, int U>
cudaError_t launch_partial(const GradTable<CAP>& tab, double* partial, int* n_partial, cudaStream_t stream) {
    const int grid = grid_of(tab.first[tab.n]);
    double* to = partial + *n_partial;
    *n_partial += grid;
    return launch_after(sumsq_kernel<CAP, U>, grid, kThreads, 0, stream, tab, to);
}

template <int CAP>
cudaError_t launch_partials(const moe_tensor_ref* refs, int n, bool large, double* partial, int* n_partial,
                            cudaStream_t stream) {
    GradTable<CAP> tab;
    *n_partial = 0;
    cudaError_t e = cudaSuccess;
    for (int at = 0; e == cudaSuccess && fill(&tab, refs, n, &at, large ? kChunk<8> : kChunk<kScaleU>);)
        e = large ? launch_partial<CAP, 8>(tab, partial, n_partial, stream)
                  : launch_partial<CAP, kScaleU>(tab, partial, n_partial, stream);
    return e;
}

template <int CAP>
cudaError_t launch_scale(const GradTable<CAP>& tab, bool large, const double* partial, int n_partial,
                         const double* sumsq, float max_norm, float eps, float* norm, cudaStream_t stream) {
    const int chunks = tab.first[tab.n];
    return launch_after(scale_kernel<CAP>, chunks == 0 ? 1 : large ? chunks : grid_of(chunks), kThreads, 0, stream, tab,
                        partial, n_partial, sumsq, max_norm, eps, norm);
}

template <int CAP>
cudaError_t launch_clip(const moe_tensor_ref* refs, int n, const double* sumsq, float max_norm, float eps, float* norm,
                        double* partial, cudaStream_t stream) {
    const bool large = is_large(refs, n);
    GradTable<CAP> tab;
    int np = 0, at = 0;
    cudaError_t e = cudaSuccess;
    if (!sumsq && !large && n <= CAP) {  // one table for both launches
        const bool any = fill(&tab, refs, n, &at, kChunk<kScaleU>);
        if constexpr (CAP == 32) {  // more tensors are more chunks
            if (any && tab.first[tab.n] <= kClusterChunks)
                return launch_after(clip_cluster_kernel<CAP>, kClusterBlocks, kClusterThreads, 0, stream, tab, max_norm,
                                    eps, norm);
        }
        if (any) e = launch_partial<CAP, kScaleU>(tab, partial, &np, stream);
        return e != cudaSuccess ? e : launch_scale(tab, false, partial, np, sumsq, max_norm, eps, norm, stream);
    }
    if (!sumsq) {
        e = launch_partials<CAP>(refs, n, large, partial, &np, stream);
        if (e == cudaSuccess && large) {  // one block adds the partial sums for all
            double* total = partial + np;
            e = launch_after(finish_kernel, 1, kThreads, 0, stream, partial, np, total, norm);
            sumsq = total;
            norm = nullptr;
        }
        if (e != cudaSuccess) return e;
    }
    bool any = false;
    for (; e == cudaSuccess && fill(&tab, refs, n, &at, kChunk<kScaleU>); any = true)
        e = launch_scale(tab, large, partial, np, sumsq, max_norm, eps, any ? nullptr : norm, stream);
    if (e == cudaSuccess && !any && norm)  // no values: the norm alone (the table is empty)
        e = launch_scale(tab, large, partial, np, sumsq, max_norm, eps, norm, stream);
    return e;
}

}  // namespace

// One set of partial sums for every launch of up to kCap tensors, and their total.
size_t grad_workspace_bytes(int n) {
    if (n == 0) return 0;
    return ((static_cast<size_t>(n) + kCap - 1) / kCap * kMaxBlocks + 2) * sizeof(double);
}

bool grad_chunks_fit(const moe_tensor_ref* refs, int n) {
    long chunks = 0;
    for (int i = 0; i < n; ++i)
        if ((chunks += chunks_of(refs[i], kChunk<kScaleU>)) > 0x7fffffffL) return false;
    return true;
}

cudaError_t launch_grad_sumsq(const moe_tensor_ref* refs, int n, double* sumsq, float* norm, void* ws,
                              cudaStream_t stream) {
    int np = 0;
    double* partial = static_cast<double*>(ws);
    const bool large = is_large(refs, n);
    const cudaError_t e =
        with_table(n, [&](auto cap) { return launch_partials<decltype(cap)::value>(refs, n, large, partial, &np, stream); });
    return e != cudaSuccess ? e : launch_after(finish_kernel, 1, kThreads, 0, stream, partial, np, sumsq, norm);
}

cudaError_t launch_grad_clip(const moe_tensor_ref* refs, int n, const double* sumsq, float max_norm, float eps,
                             float* norm, void* ws, cudaStream_t stream) {
    return with_table(n, [&](auto cap) {
        return launch_clip<decltype(cap)::value>(refs, n, sumsq, max_norm, eps, norm, static_cast<double*>(ws), stream);
    });
}

}  // namespace moe
