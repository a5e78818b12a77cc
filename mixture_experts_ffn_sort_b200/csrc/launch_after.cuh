// launch_after.cuh -- launches of the training kernels.
//
// They are programmatic dependents of whatever runs before them in the stream:
// their blocks take their places while that kernel's last ones finish, and
// start by waiting for all of it (grid_dependency_wait), before any memory is read or
// written.  A kernel launched this way has to begin with that wait.
#pragma once

#include <cuda_runtime.h>

namespace moe {

template <class... P, class... A>
cudaError_t launch_after(void (*kernel)(P...), int grid, int threads, size_t smem, cudaStream_t stream,
                         const A&... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(grid));
    cfg.blockDim = dim3(static_cast<unsigned>(threads));
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr = {};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

}  // namespace moe
