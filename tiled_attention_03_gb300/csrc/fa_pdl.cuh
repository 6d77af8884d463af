// fa_pdl.cuh -- programmatic dependent launch (internal): a kernel launched with
// launch_after() may be set up while the kernel before it in the stream still runs. It
// calls after_previous() before it touches memory, which waits until that kernel has
// finished and its stores are visible; let_next_start() is the other side, and orders
// nothing. Between two kernels of a few microseconds this hides the launch, about 1 us.
#pragma once

#include <cuda_runtime.h>

namespace fa {

__device__ __forceinline__ void after_previous() {
    asm volatile("griddepcontrol.wait;" ::: "memory");
}
__device__ __forceinline__ void let_next_start() {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

template <typename... Want, typename... Have>
cudaError_t launch_after(void (*kernel)(Want...), dim3 grid, unsigned threads, size_t smem,
                         cudaStream_t stream, const Have &...args) {
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

}  // namespace fa
