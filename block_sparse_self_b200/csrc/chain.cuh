// chain.cuh -- launches that overlap the end of the kernel before them.
//
// The training calls launch several short kernels after one another; for small
// inputs their launches, set-up and tails are most of the time.  A chained
// launch (programmatic stream serialization) starts once every CTA of the
// kernel before it has called grid_release() or ended, not once it has
// completed.  What makes that sound, for every kernel of a chain:
//  - the first kernel of a chain is launched normally: what the caller wrote
//    before the call is complete, and any kernel of the chain may read it at once;
//  - every thread calls grid_wait(), which returns when the kernel before has
//    completed and its writes are visible: before the first use of anything that
//    the chain itself wrote, and before any write; a kernel that needs nothing of
//    the chain and writes only buffers of its own calls it before it ends.
//    So a kernel completes after all kernels before it, and completion of the
//    last is completion of all, which the caller's next (normal) launch waits for.
//  - a kernel that allocates tensor memory releases the next one only after that:
//    a CTA of the next kernel must not take it and then wait for this one.  That holds
//    for the last kernel too: what follows it is the caller's, perhaps a chained launch
//    of another library that allocates tensor memory.
//  - what the chain itself wrote is read with chain_load(), never by __ldg() or through
//    const __restrict__: while a kernel waits, the kernel before may still be writing it,
//    so it is not read-only for the kernel's lifetime, and a load that may assume so is
//    not held behind grid_wait().  __ldg() is for the caller's inputs.
// Without a chained launch before it grid_wait() returns at once.
// 7 blocks of 128, D = 64, 3 heads: a backward pass every 27.0 us against 41.0 with normal
// launches; as a graph 24.7 against 31.2.
#pragma once

#include <cuda_runtime.h>

namespace vsa {

__device__ __forceinline__ void grid_release() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void grid_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// An ordinary load: it stays behind grid_wait(), which clobbers memory.
template <typename T>
__device__ __forceinline__ T chain_load(const T *p) { return *p; }

template <typename... P, typename... A>
inline cudaError_t launch_kernel(bool chained, void (*kern)(P...), dim3 grid, dim3 block, size_t smem, cudaStream_t st,
                                 const A &...args) {
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cfg.attrs = &at;
    cfg.numAttrs = chained ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kern, args...);
}

}  // namespace vsa
