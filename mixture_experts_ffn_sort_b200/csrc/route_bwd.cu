// route_bwd.cu -- the gradient of the routing (moe_route_bwd): from the K
// route weights of a token to its E logits, the choice held fixed.
//
// G lanes per token (8, 16 or 32, at least K), lane j holding choice j, so that
// a warp has the loads of several tokens in flight.  The K scores are
// recomputed from the K chosen logits (softmax relative to the largest of them,
// which cancels), then dl_j = scaling * q_j * (G_j - sum_i G_i q_i), times
// (1 - s_j) for sigmoid scores.  The rows of a warp's tokens are written as
// zeros and the K chosen gradients are stored over them, after the loads: zeros
// that go first delay them (21.5 us against 19.1 us with a warp a token).  The
// full softmax needs the whole row and has a kernel of its own.
//
// 32768 tokens of 512 experts, top-10, sigmoid: 16.4 us, 6.2 TB/s of 67 MB
// written and 35 MB read, since each of the ten scattered logits of a row
// brings its whole piece of DRAM.
#include "launch_after.cuh"
#include "route_device.cuh"
#include "train.h"

namespace moe {

namespace {

constexpr uint32_t kFull = 0xffffffffu;

template <int G>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
    for (int off = G / 2; off > 0; off >>= 1) v += __shfl_xor_sync(kFull, v, off);
    return v;
}
template <int G>
__device__ __forceinline__ float group_max(float v) {
#pragma unroll
    for (int off = G / 2; off > 0; off >>= 1) v = fmaxf(v, __shfl_xor_sync(kFull, v, off));
    return v;
}

// Zeros in p[0 .. n) by one warp, p aligned to floats.
__device__ __forceinline__ void warp_zero(float* p, long n, int lane) {
    const long head = static_cast<long>((0 - (reinterpret_cast<uintptr_t>(p) >> 2)) & 3);
    if (lane < head && lane < n) p[lane] = 0.f;
    const long quads = n > head ? (n - head) >> 2 : 0;
    for (long i = lane; i < quads; i += 32) reinterpret_cast<float4*>(p + head)[i] = make_float4(0.f, 0.f, 0.f, 0.f);
    const long rest = head + 4 * quads + lane;
    if (rest < n) p[rest] = 0.f;
}

// Choices of the same expert: the lowest lane of a token collects them.  (Each
// carries `term`, the token's part of the row; it counts once.)  Returns
// whether this lane has something to store.
__device__ __forceinline__ bool collect(int token, int id, bool here, int lane, float term, float* d) {
    const uint32_t same = __match_any_sync(kFull, here ? token * MOE_MAX_E + id : -1 - lane);
    const bool first = here && (same & ((1u << lane) - 1u)) == 0;
    if (__any_sync(kFull, here && !first)) {
        float sum = *d;
        for (int i = 0; i < 32; ++i) {
            const float di = __shfl_sync(kFull, *d, i);
            if (first && i != lane && ((same >> i) & 1u)) sum += di - term;
        }
        *d = sum;
    }
    return first;
}

template <bool SOFTMAX, bool RENORM, int G>
__global__ void __launch_bounds__(256) route_bwd_kernel(const float* __restrict__ logits,
                                                        const int32_t* __restrict__ ids,
                                                        const float* __restrict__ dw, int T, int E, int K,
                                                        float scaling, const uint8_t* __restrict__ zero_mask,
                                                        float* __restrict__ dlogits, int32_t* __restrict__ status) {
    static_assert(!SOFTMAX || RENORM, "the full softmax has a kernel of its own");
    constexpr int TPW = 32 / G;  // tokens of a warp
    const int t0 = ((blockIdx.x * blockDim.x + threadIdx.x) >> 5) * TPW;
    grid_dependency_wait();
    if (t0 >= T) return;
    const int lane = threadIdx.x & 31, j = lane % G;
    const int t = t0 + lane / G;
    const bool on = j < K && t < T;
    const size_t o = static_cast<size_t>(t) * K + j;

    const int id = on ? __ldg(ids + o) : -1;
    const bool here = id >= 0 && id < E;
    if (on && !here) report_status(status, MOE_STATUS_BAD_ID);
    const float g = here && !(zero_mask && zero_mask[o]) ? __ldg(dw + o) : 0.f;
    const float l = here ? __ldg(logits + static_cast<size_t>(t) * E + id) : -INFINITY;

    float s;
    if (SOFTMAX) {
        float lmax = group_max<G>(l);
        if (lmax == -INFINITY) lmax = 0.f;  // no score above 0
        s = here ? expf(l - lmax) : 0.f;
    } else {
        s = here ? sigmoid(l) : 0.f;
    }
    float q = s, mean = 0.f;
    if (RENORM) {
        const float z = group_sum<G>(s);
        q = z == 0.f ? 0.f : s / z;  // every score below fp32's range: no gradient
        mean = group_sum<G>(g * q);
    }
    float d = scaling * q * (g - mean);
    if (!SOFTMAX) d *= here ? sigmoid(-l) : 0.f;  // 1 - s without the cancellation
    warp_zero(dlogits + static_cast<size_t>(t0) * E, static_cast<long>(min(TPW, T - t0)) * E, lane);
    const bool first = collect(lane / G, id, here, lane, 0.f, &d);
    __syncwarp();  // the rows' zeros before the chosen logits
    if (first) dlogits[static_cast<size_t>(t) * E + id] = d;
}

// The softmax over all experts, not renormalised: every logit has a gradient.
// One warp per token, which reads the row once and keeps its scores, EPL a
// lane.  32768 tokens of 512 experts, top-10: 31.0 us, 4.3 TB/s of 134 MB (33.8
// us with the row read for the maximum, the sum and the result); the exponentials
// and the chain of four sums over the warp hold it back.
template <int EPL>
__global__ void __launch_bounds__(256) route_bwd_full_kernel(const float* __restrict__ logits,
                                                             const int32_t* __restrict__ ids,
                                                             const float* __restrict__ dw, int T, int E, int K,
                                                             float scaling, const uint8_t* __restrict__ zero_mask,
                                                             float* __restrict__ dlogits,
                                                             int32_t* __restrict__ status) {
    const int t = (blockIdx.x * blockDim.x + threadIdx.x) >> 5, lane = threadIdx.x & 31;
    grid_dependency_wait();
    if (t >= T) return;
    const float* lg = logits + static_cast<size_t>(t) * E;
    float* out = dlogits + static_cast<size_t>(t) * E;
    const size_t o = static_cast<size_t>(t) * K + lane;

    const int id = lane < K ? __ldg(ids + o) : -1;
    float p[EPL], lmax = -INFINITY;
#pragma unroll
    for (int i = 0; i < EPL; ++i) p[i] = lane + 32 * i < E ? __ldg(lg + lane + 32 * i) : -INFINITY;
    const bool here = id >= 0 && id < E;
    if (lane < K && !here) report_status(status, MOE_STATUS_BAD_ID);
    const float g = here && !(zero_mask && zero_mask[o]) ? __ldg(dw + o) : 0.f;
    const float l = here ? __ldg(lg + id) : -INFINITY;  // in L1 from the row
#pragma unroll
    for (int i = 0; i < EPL; ++i) lmax = fmaxf(lmax, p[i]);
    lmax = group_max<32>(lmax);
    if (lmax == -INFINITY) lmax = 0.f;  // no score above 0: no gradient (z = 0)
    float z = 0.f;
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
        p[i] = expf(p[i] - lmax);
        z += p[i];
    }
    z = group_sum<32>(z);
    const float rz = z == 0.f ? 0.f : 1.f / z;
    const float q = here ? expf(l - lmax) * rz : 0.f;
    const float mean = group_sum<32>(g * q), row = -scaling * mean;
    float d = scaling * q * (g - mean);
    const bool first = collect(0, id, here, lane, row * q, &d);
#pragma unroll
    for (int i = 0; i < EPL; ++i)
        if (lane + 32 * i < E) out[lane + 32 * i] = row * (p[i] * rz);
    __syncwarp();  // the row before the chosen logits
    if (first) out[id] = d;
}

}  // namespace

cudaError_t launch_route_bwd(const float* logits, const int32_t* ids, const float* dw, int T, int E, int K,
                             const RouteCfg& cfg, const uint8_t* zero_mask, float* dlogits, int32_t* status,
                             cudaStream_t stream) {
    auto launch = [&](auto kernel, int G) {
        const int tokens = 8 * (32 / G);  // of a block
        return launch_after(kernel, (T + tokens - 1) / tokens, 256, 0, stream, logits, ids, dw, T, E, K, cfg.scaling,
                            zero_mask, dlogits, status);
    };
    if (cfg.score == MOE_SCORE_SOFTMAX) {
        if (!cfg.renormalize)
            return E <= 64    ? launch(route_bwd_full_kernel<2>, 32)
                   : E <= 128 ? launch(route_bwd_full_kernel<4>, 32)
                   : E <= 256 ? launch(route_bwd_full_kernel<8>, 32)
                   : E <= 512 ? launch(route_bwd_full_kernel<16>, 32)
                              : launch(route_bwd_full_kernel<32>, 32);
        return K <= 8 ? launch(route_bwd_kernel<true, true, 8>, 8)
                      : K <= 16 ? launch(route_bwd_kernel<true, true, 16>, 16)
                                : launch(route_bwd_kernel<true, true, 32>, 32);
    }
    if (cfg.renormalize)
        return K <= 8 ? launch(route_bwd_kernel<false, true, 8>, 8)
                      : K <= 16 ? launch(route_bwd_kernel<false, true, 16>, 16)
                                : launch(route_bwd_kernel<false, true, 32>, 32);
    return K <= 8 ? launch(route_bwd_kernel<false, false, 8>, 8)
                  : K <= 16 ? launch(route_bwd_kernel<false, false, 16>, 16)
                            : launch(route_bwd_kernel<false, false, 32>, 32);
}

}  // namespace moe
