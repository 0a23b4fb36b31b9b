// launch.cuh -- kernels of one call chained by programmatic dependent launch.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "internal.h"

namespace ss {

// Kernels are launched while the one before them on the stream still runs (its
// last CTAs, where it does not say otherwise): each lets its own successor launch,
// sets itself up, and waits for the one before to be done before it reads or
// writes anything.  A kernel that waited is done only after all before it, so the
// next one's wait covers them too.  Without such a predecessor the wait returns at
// once.
__device__ __forceinline__ void launch_after() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void wait_before() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// Launch of `grid` CTAs in clusters of `cluster` (0: as the kernel says), after
// the kernel before it on the stream or (chained) overlapping its end.
template <class... P, class... A>
int launch(void (*kernel)(P...), int64_t grid, int threads, int smem, int cluster, bool chained, cudaStream_t st,
           A&&... args) {
    if (grid > INT32_MAX) return SS_EOVERFLOW;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = (size_t)smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2] = {};
    unsigned n = 0;
    if (chained) {
        attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[n++].val.programmaticStreamSerializationAllowed = 1;
    }
    if (cluster > 0) {
        attr[n].id = cudaLaunchAttributeClusterDimension;
        attr[n].val.clusterDim.x = (unsigned)cluster;
        attr[n].val.clusterDim.y = attr[n].val.clusterDim.z = 1;
        ++n;
    }
    cfg.attrs = attr;
    cfg.numAttrs = n;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...);
    return e == cudaSuccess ? check_launch() : cuda_fail(e);
}

// Launch of `grid` CTAs that may wait for one another: all resident at once, or
// kNotResident and nothing launched (where the stream has a part of the SMs only).
constexpr int kNotResident = 1;

template <class... P, class... A>
int launch_cooperative(void (*kernel)(P...), int64_t grid, int threads, cudaStream_t st, A&&... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3((unsigned)threads);
    cfg.stream = st;
    cudaLaunchAttribute attr[1] = {};
    attr[0].id = cudaLaunchAttributeCooperative;
    attr[0].val.cooperative = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...);
    if (e == cudaErrorCooperativeLaunchTooLarge) {
        cudaGetLastError();
        return kNotResident;
    }
    return e == cudaSuccess ? check_launch() : cuda_fail(e);
}

}  // namespace ss
