// train.h -- internal host-side launchers of the training calls' kernels (C++
// only; the public boundary is include/moe_ffn.h).
#pragma once

#include "../../include/moe_ffn.h"
#include "launch.h"

namespace moe {

// ---------------------------------------------------------------- rows and their gradients (training)
inline int dtype_bytes(int dtype) { return dtype == MOE_DTYPE_F32 ? 4 : 2; }
struct RowsArgs {
    const int32_t* inv;     // [T, K] sorted positions
    const int32_t* n_rows;  // sorted rows in use (device), or NULL
    int T, K, H;
    int dtype;  // MOE_DTYPE_*
    int32_t* status;
};
cudaError_t launch_permute(const RowsArgs& a, const void* x, void* x_sorted, cudaStream_t stream);
cudaError_t launch_unpermute(const RowsArgs& a, const void* y_sorted, const float* w, const void* y_shared, void* out,
                             cudaStream_t stream);
cudaError_t launch_unpermute_bwd(const RowsArgs& a, const void* dout, const void* y_sorted, const float* w,
                                 void* dy_sorted, float* dw, cudaStream_t stream);
cudaError_t launch_route_bwd(const float* logits, const int32_t* ids, const float* dw, int T, int E, int K,
                             const RouteCfg& cfg, const uint8_t* zero_mask, float* dlogits, int32_t* status,
                             cudaStream_t stream);

// ---------------------------------------------------------------- gradient norm and clipping
size_t grad_workspace_bytes(int n);
// Whether the chunks that the kernels cut the tensors into can be counted in an int (about 35 TB).
bool grad_chunks_fit(const moe_tensor_ref* refs, int n);
cudaError_t launch_grad_sumsq(const moe_tensor_ref* refs, int n, double* sumsq, float* norm, void* ws,
                              cudaStream_t stream);
cudaError_t launch_grad_clip(const moe_tensor_ref* refs, int n, const double* sumsq, float max_norm, float eps,
                             float* norm, void* ws, cudaStream_t stream);

}  // namespace moe
