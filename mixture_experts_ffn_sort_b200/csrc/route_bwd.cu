// route_bwd.cu -- the gradient of the routing (moe_route_bwd): from the K
// route weights of a token to its E logits, the choice held fixed.
//
// G lanes per token (8, 16 or 32, at least K), lane j holding choice j, so that
// a warp has the loads of several tokens in flight.  The K
// scores are recomputed from the K chosen logits (softmax relative to the
// largest of them, which cancels; the full normaliser, when the weights are
// not renormalised, needs the whole row), then dl_j = scaling * q_j *
// (G_j - sum_i G_i q_i), times (1 - s_j) for sigmoid scores.  The rows of a
// warp's tokens are written as zeros (or as the unchosen experts' softmax
// term) and the K chosen gradients are stored over them, after the loads: zeros
// that go first delay them (21.5 us against 19.1 us with a warp a token).
//
// 32768 tokens of 512 experts, top-10, sigmoid: 16.4 us, 6.2 TB/s of 67 MB
// written and 35 MB read, since each of the ten scattered logits of a row
// brings its whole piece of DRAM.
#include "launch.h"
#include "launch_after.cuh"
#include "route_device.cuh"

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

template <bool SOFTMAX, bool RENORM, int G>
__global__ void __launch_bounds__(256) route_bwd_kernel(const float* __restrict__ logits,
                                                        const int32_t* __restrict__ ids,
                                                        const float* __restrict__ dw, int T, int E, int K,
                                                        float scaling, const uint8_t* __restrict__ zero_mask,
                                                        float* __restrict__ dlogits, int32_t* __restrict__ status) {
    constexpr int TPW = 32 / G;  // tokens of a warp
    const int t0 = ((blockIdx.x * blockDim.x + threadIdx.x) >> 5) * TPW;
    grid_dependency_wait();
    if (t0 >= T) return;
    const int lane = threadIdx.x & 31, j = lane % G;
    const int t = t0 + lane / G;
    const bool on = j < K && t < T;
    const float* lg = logits + static_cast<size_t>(t) * E;
    float* out = dlogits + static_cast<size_t>(t) * E;
    const size_t o = static_cast<size_t>(t) * K + j;

    const int id = on ? __ldg(ids + o) : -1;
    const bool here = id >= 0 && id < E;
    if (on && !here) report_status(status, MOE_STATUS_BAD_ID);
    const float g = on && !(zero_mask && zero_mask[o]) ? __ldg(dw + o) : 0.f;
    const float gj = here ? g : 0.f;
    const float l = here ? __ldg(lg + id) : -INFINITY;

    float s = 0.f, q = 0.f, lmax = 0.f, rz = 0.f;
    if (SOFTMAX) {
        lmax = l;
        if (!RENORM && t < T)
            for (int e = j; e < E; e += G) lmax = fmaxf(lmax, __ldg(lg + e));
        lmax = group_max<G>(lmax);
        if (lmax == -INFINITY) lmax = 0.f;  // no score above 0: no gradient (z = 0)
        s = here ? expf(l - lmax) : 0.f;
        float z = RENORM ? s : 0.f;
        if (!RENORM && t < T)
            for (int e = j; e < E; e += G) z += expf(__ldg(lg + e) - lmax);
        z = group_sum<G>(z);
        rz = z == 0.f ? 0.f : 1.f / z;
        q = here ? s * rz : 0.f;
    } else {
        s = here ? sigmoid(l) : 0.f;
        q = s;
        if (RENORM) {
            const float sum = group_sum<G>(s);
            q = sum == 0.f ? 0.f : s / sum;  // every score below fp32's range: no gradient
        }
    }
    const float mean = SOFTMAX || RENORM ? group_sum<G>(gj * q) : 0.f;
    float d = scaling * q * (gj - mean);
    if (!SOFTMAX) d *= here ? sigmoid(-l) : 0.f;  // 1 - s without the cancellation
    if (SOFTMAX && !RENORM) {
        if (t < T)
            for (int e = j; e < E; e += G) out[e] = -scaling * (expf(__ldg(lg + e) - lmax) * rz) * mean;
    } else {
        warp_zero(dlogits + static_cast<size_t>(t0) * E, static_cast<long>(min(TPW, T - t0)) * E, lane);
    }
    // Choices of the same expert: the lowest lane collects them.
    const uint32_t same = __match_any_sync(kFull, here ? (lane / G) * MOE_MAX_E + id : -1 - lane);
    const bool first = here && (same & ((1u << lane) - 1u)) == 0;
    if (__any_sync(kFull, here && !first)) {
        // (Each choice of a full softmax carries the row's term; it counts once.)
        const float term = SOFTMAX && !RENORM ? -scaling * q * mean : 0.f;
        float sum = d;
        for (int i = 0; i < 32; ++i) {
            const float di = __shfl_sync(kFull, d, i);
            if (first && i != lane && ((same >> i) & 1u)) sum += di - term;
        }
        d = sum;
    }
    __syncwarp();  // the rows' zeros before the chosen logits
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
        // The full softmax reads and writes whole rows: a warp for each.
        if (!cfg.renormalize) return launch(route_bwd_kernel<true, false, 32>, 32);
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
