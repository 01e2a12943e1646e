// Launches that begin while the one before them on the stream still runs.
#pragma once

#include "moe_internal.cuh"

namespace ep {

namespace {

// device: what the launch before this one wrote is there (an ordinary launch goes on at once)
__device__ __forceinline__ void wait_for_launch_before() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
// device: this CTA has begun; the launch behind may
__device__ __forceinline__ void let_next_launch_begin() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// Launches `kernel` in clusters of `cluster` CTAs (0: as the kernel says).
template <typename... P, typename... A>
cudaError_t launch_in_order(int order, void (*kernel)(P...), dim3 grid, int threads, size_t smem, int cluster,
                            cudaStream_t st, const A &...args) {
    cudaLaunchConfig_t c{};
    c.gridDim = grid;
    c.blockDim = dim3((unsigned)threads);
    c.dynamicSmemBytes = smem;
    c.stream = st;
    cudaLaunchAttribute attr[2]{};
    int n = 0;
    if (order != kFirst) {
        attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[n++].val.programmaticStreamSerializationAllowed = 1;
    }
    if (cluster) {
        attr[n].id = cudaLaunchAttributeClusterDimension;
        attr[n].val.clusterDim.x = (unsigned)cluster;
        attr[n].val.clusterDim.y = attr[n].val.clusterDim.z = 1;
        ++n;
    }
    c.attrs = attr;
    c.numAttrs = (unsigned)n;
    return cudaLaunchKernelEx(&c, kernel, args...);
}

}  // namespace

}  // namespace ep
