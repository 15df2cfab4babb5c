// pdl.cuh -- programmatic dependent launch: between the decode passes, and of kernels that
// start while the stream's last one ends.
#pragma once

#include <cuda_runtime.h>

namespace diffattn {

// The next kernel on the stream, if launched with programmatic stream
// serialisation, may start its blocks once every CTA of this grid has
// executed this (or exited).
__device__ __forceinline__ void pdl_launch_dependents() {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// Wait until the grids this one depends on have completed and their memory
// writes are visible (returns at once without such a dependency).
__device__ __forceinline__ void pdl_wait() {
    asm volatile("griddepcontrol.wait;" ::: "memory");
}

// Launch a kernel that may start before the stream's last one is over, if that one lets
// it; it executes pdl_wait before it touches anything but its own shared memory.
template <typename... P, typename... A>
int pdl_launch(void (*kernel)(P...), dim3 grid, unsigned threads, size_t smem, cudaStream_t stream, const A&... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...) == cudaSuccess ? 0 : -1;
}

}  // namespace diffattn
