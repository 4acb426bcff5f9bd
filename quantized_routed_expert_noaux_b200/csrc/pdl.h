// pdl.h -- programmatic dependent launch: a kernel may be set up while the one before it on its stream
// ends.  Every thread of every CTA of a kernel that is launched so calls wait_for_previous() before its first access
// to memory that an earlier kernel may touch; the wait ends when the kernels before have completed and their
// writes are visible.  (A kernel that returned without waiting could complete before its predecessor, and let
// its successor run too early.)  The products call dependents_may_launch() at their end.  The 8-bit quantiser calls
// it first (the product behind it is set up meanwhile), and so does the sort of many slots (the copies behind it
// load their rows meanwhile): after wait_for_previous(), so that what is read before the successor's own wait
// is complete.  Elsewhere the end of the kernel is the trigger; earlier ones gave the next kernel's CTAs room
// beside the running ones and were slower (2048 tokens routed 6.5 us against 5.0, the fp4 expert half for one
// token 70 against 59).
#pragma once

#include <atomic>
#include <cuda_runtime.h>
#include <stdint.h>

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

// The kernel's shared-memory attribute lasts as long as the context: set once per device (twice is
// harmless).
template <typename K>
cudaError_t allow_smem(K *kernel, size_t bytes, std::atomic<uint64_t> &ready) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess || (dev < 64 && (ready.load(std::memory_order_relaxed) >> dev & 1))) return e;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(bytes));
    if (e == cudaSuccess && dev < 64) ready.fetch_or(1ull << dev, std::memory_order_relaxed);
    return e;
}

}  // namespace coli
