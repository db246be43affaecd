// Launching the post-training kernels: each may start before the work ahead of it in the stream
// has ended (programmatic dependent launch) and waits for it on the device before it touches
// memory, so that chains of short kernels hide one another's start.
#pragma once

#include <cuda_runtime.h>

namespace vl {

template <typename K, typename... Args>
cudaError_t launch_pdl(K kernel, long long grid, dim3 threads, size_t smem, cudaStream_t st, Args... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid, 1, 1);
    cfg.blockDim = threads;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

}  // namespace vl
