// launch_after.cuh -- launches of the training kernels.
//
// They are programmatic dependents of whatever runs before them in the stream:
// their blocks take their places while that kernel's last ones finish, and
// start by waiting for all of it (grid_dependency_wait), before any memory is read or
// written.  A kernel launched this way has to begin with that wait: nothing but
// its parameters and its own shared memory comes before it, and no block leaves
// without it (the next kernel waits for this one alone).
//
// That is also what makes read-only loads (__ldg, const __restrict__) right
// here.  They promise memory that does not change while the kernel runs, and a
// dependent is running while its predecessor still writes.  Every one of them
// stands behind the wait and within a condition on the thread's index: an
// ordinary load may not move across the wait's memory clobber, one of memory
// taken for constant may, but not out of its condition.  A new kernel has to keep
// it so.
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
