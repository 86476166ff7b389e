// overlap.cuh -- launches whose start overlaps the end of the kernel before them
// on the stream (programmatic dependent launch), for the operators around the
// layer: a decoder step is a chain of short kernels, and the gap between two of
// them is as long as the shortest.
//
// Rules that make it safe, whatever ran before on the stream:
//  - a kernel launched this way calls overlap_wait() before it reads anything
//    that an earlier kernel may have written and before it writes anything at all
//    (it may prefetch what never changes: weights in the library's own copy), and
//    reads it with ordinary or L2 loads, not through the read-only path.  The
//    wait ends when the kernel before has finished and its writes are visible;
//  - a kernel that is followed by such a launch may call overlap_trigger() as early
//    as it likes: that only lets the next kernel's blocks start, and their wait is
//    for its end.  As every kernel waits in turn, the end of one means the end of
//    all before it.
#pragma once

#include <cuda_runtime.h>

namespace moe {

__device__ __forceinline__ void overlap_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void overlap_trigger() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// Launches kern with clusters of `cluster` CTAs (1: none), overlapping the kernel before it.
template <typename... Params, typename... Args>
cudaError_t launch_overlapped(void (*kern)(Params...), dim3 grid, dim3 block, int smem, int cluster, cudaStream_t st,
                              Args &&...args)
{
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = (size_t)smem;
    cfg.stream = st;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = (unsigned)cluster;
    at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kern, static_cast<Params>(args)...);
}

}  // namespace moe
