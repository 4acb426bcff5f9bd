// pdl.h -- programmatic dependent launch: a kernel may be set up while the one before it on its stream
// ends.  Every thread of every CTA of a kernel that is launched so calls wait_for_previous() before its first access
// to memory that an earlier kernel may touch; the wait ends when the kernels before have completed and their
// writes are visible.  (A kernel that returned without waiting could complete before its predecessor, and let
// its successor run too early.)  Only the products call dependents_may_launch(), at their end; elsewhere the end
// of the kernel is the trigger.  Earlier triggers gave the next kernel's CTAs room beside the running ones and
// were slower (2048 tokens routed 6.5 us against 5.0, the expert half for one token 70 against 59).
#pragma once

#include <cuda_runtime.h>

namespace coli {

__device__ __forceinline__ void dependents_may_launch() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void wait_for_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// kernel<<<grid, block, smem, st>>>(args...), in clusters of `cluster` CTAs.
template <typename... Params, typename... Args>
cudaError_t launch_early(void (*kernel)(Params...), dim3 grid, int block, size_t smem, cudaStream_t st, int cluster, Args &&...args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(block);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = cluster;
    at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, Params(args)...);
}

}  // namespace coli
