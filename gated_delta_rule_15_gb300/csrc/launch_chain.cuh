// launch_chain.cuh -- launches whose blocks may start while the kernel before them in the stream ends.
#pragma once

#include <cuda_runtime.h>

#include "common.cuh"

namespace dr {

// In the kernel before: its successor's blocks may take SMs that have no work left.
__device__ __forceinline__ void let_next_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
// In the successor, by every block, in front of the first access to what the kernel before writes and of the first write of
// its own: waits until that kernel has ended.
__device__ __forceinline__ void wait_for_last() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

template <class... P, class... A>
int launch_after(void (*kernel)(P...), unsigned blocks, unsigned threads, size_t smem, cudaStream_t stream, const A &...args) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(blocks);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...) == cudaSuccess ? kOk : kErrCuda;
}

}  // namespace dr
