// route_bwd.cu -- the gradient of the routing (moe_route_bwd): from the K
// route weights of a token to its E logits, the choice held fixed.
//
// One warp per token, lane j holding choice j.  The K scores are recomputed
// from the K chosen logits (softmax relative to the largest of them, which
// cancels; the full normaliser, when the weights are not renormalised, needs
// the whole row), then dl_j = scaling * q_j * (G_j - sum_i G_i q_i), times
// (1 - s_j) for sigmoid scores.  The row is written as zeros (or as the
// unchosen experts' softmax term) and the K chosen logits are stored over it.
#include "launch.h"
#include "route_device.cuh"

namespace moe {

namespace {

constexpr uint32_t kFull = 0xffffffffu;

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(kFull, v, off);
    return v;
}
__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) v = fmaxf(v, __shfl_xor_sync(kFull, v, off));
    return v;
}

template <bool SOFTMAX, bool RENORM>
__global__ void __launch_bounds__(256) route_bwd_kernel(const float* __restrict__ logits,
                                                        const int32_t* __restrict__ ids,
                                                        const float* __restrict__ dw, int T, int E, int K,
                                                        float scaling, const uint8_t* __restrict__ zero_mask,
                                                        float* __restrict__ dlogits, int32_t* __restrict__ status) {
    const int t = (blockIdx.x * blockDim.x + threadIdx.x) >> 5;
    if (t >= T) return;
    const int lane = threadIdx.x & 31;
    const float* lg = logits + static_cast<size_t>(t) * E;
    float* out = dlogits + static_cast<size_t>(t) * E;
    const size_t o = static_cast<size_t>(t) * K + lane;

    const int id = lane < K ? __ldg(ids + o) : -1;
    const bool here = id >= 0 && id < E;
    if (lane < K && !here) report_status(status, MOE_STATUS_BAD_ID);
    const float G = here && !(zero_mask && zero_mask[o]) ? __ldg(dw + o) : 0.f;
    const float l = here ? __ldg(lg + id) : -INFINITY;

    float s = 0.f, q = 0.f, lmax = 0.f, rz = 0.f;
    if (SOFTMAX) {
        lmax = l;
        if (!RENORM)
            for (int e = lane; e < E; e += 32) lmax = fmaxf(lmax, __ldg(lg + e));
        lmax = warp_max(lmax);
        s = here ? expf(l - lmax) : 0.f;
        float z = RENORM ? s : 0.f;
        if (!RENORM)
            for (int e = lane; e < E; e += 32) z += expf(__ldg(lg + e) - lmax);
        z = warp_sum(z);
        rz = 1.f / z;
        q = here ? s * rz : 0.f;
    } else {
        s = here ? sigmoid(l) : 0.f;
        q = s;
        if (RENORM) {
            const float sum = warp_sum(s);
            q = sum > 0.f ? s / sum : 0.f;  // every score below fp32's range: no gradient
        }
    }
    const bool centred = SOFTMAX || RENORM;
    const float mean = centred ? warp_sum(G * q) : 0.f;
    float d = scaling * q * (G - mean);
    if (!SOFTMAX) d *= here ? sigmoid(-l) : 0.f;  // 1 - s without the cancellation
    if (SOFTMAX && !RENORM) {
        for (int e = lane; e < E; e += 32) out[e] = -scaling * (expf(__ldg(lg + e) - lmax) * rz) * mean;
    } else {
        for (int e = lane; e < E; e += 32) out[e] = 0.f;
    }
    // Choices of the same expert: the lowest lane collects them.
    const uint32_t same = __match_any_sync(kFull, here ? id : -1 - lane);
    const bool first = here && (same & ((1u << lane) - 1u)) == 0;
    if (__any_sync(kFull, here && !first)) {
        // (Each choice of a full softmax carries the row's term; it counts once.)
        const float term = SOFTMAX && !RENORM ? -scaling * q * mean : 0.f;
        float sum = d;
        for (int j = 0; j < K; ++j) {
            const float dj = __shfl_sync(kFull, d, j);
            if (first && j != lane && ((same >> j) & 1u)) sum += dj - term;
        }
        d = sum;
    }
    __syncwarp();  // the row's zeros before the chosen logits
    if (first) out[id] = d;
}

}  // namespace

cudaError_t launch_route_bwd(const float* logits, const int32_t* ids, const float* dw, int T, int E, int K,
                             const RouteCfg& cfg, const uint8_t* zero_mask, float* dlogits, int32_t* status,
                             cudaStream_t stream) {
    const int blocks = (T + 7) / 8;
#define MOE_LAUNCH(S, N) \
    route_bwd_kernel<S, N><<<blocks, 256, 0, stream>>>(logits, ids, dw, T, E, K, cfg.scaling, zero_mask, dlogits, status)
    if (cfg.score == MOE_SCORE_SOFTMAX) {
        if (cfg.renormalize) MOE_LAUNCH(true, true);
        else MOE_LAUNCH(true, false);
    } else {
        if (cfg.renormalize) MOE_LAUNCH(false, true);
        else MOE_LAUNCH(false, false);
    }
#undef MOE_LAUNCH
    return cudaGetLastError();
}

}  // namespace moe
