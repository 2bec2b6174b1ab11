// Launch that may overlap the end of the kernel before it on the stream
// (programmatic dependent launch): the kernel's set-up runs early, and
// dependency_wait() comes before its first access to memory that others write
// or read. Reads behind it are plain loads: a read-only load (__ldg, or a const
// __restrict__ parameter) is taken to give the same value anywhere in the
// kernel, so that the compiler may move it ahead of the wait.
#pragma once

#include <cuda_runtime.h>

#include <utility>

namespace mdcn {

template <typename... Params, typename... Args>
cudaError_t launch_dependent(void (*kernel)(Params...), dim3 grid, int threads, int smem, cudaStream_t st, Args&&... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(static_cast<unsigned>(threads));
    cfg.dynamicSmemBytes = static_cast<size_t>(smem);
    cfg.stream = st;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, std::forward<Args>(args)...);
    return e == cudaSuccess ? cudaGetLastError() : e;
}

#ifdef __CUDACC__
__device__ __forceinline__ void dependency_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
#endif

}  // namespace mdcn
