// Programmatic dependent launches: a kernel is put on its SMs while the one
// before it on the stream still runs, and waits there for that one's results.
// A decode step is a chain of kernels of a few microseconds, and a launch
// after another's end costs between one and two of them.
#pragma once

#include "pa_device.cuh"

namespace pa {

// First in a kernel launched by launch_dependent, before any global access, in
// every thread: waits until the kernel before it on the stream is done and its
// writes are visible (as that kernel's own wait does for the one before it).
// Plain loads are ordered behind it.  Read-only ones (__ldg, ld.global.nc) are
// not for memory that a kernel before may write: they hold for memory that nobody
// writes while this kernel is there, and it is there early.
__device__ __forceinline__ void dependent_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// Once every CTA of the grid has come by here, or has ended, the kernel after
// this one may be put on the SMs.
__device__ __forceinline__ void dependent_release() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// whether np bytes from p on and nq bytes from q on have any in common
inline bool overlaps(const void *p, size_t np, const void *q, size_t nq) {
    const uintptr_t a = reinterpret_cast<uintptr_t>(p), b = reinterpret_cast<uintptr_t>(q);
    return a < b + nq && b < a + np;
}

// `cluster` CTAs along x to a thread-block cluster (0: none).
template <class... Params, class... Actual>
inline cudaError_t launch_dependent(void (*kernel)(Params...), dim3 grid, int threads, size_t smem, int cluster,
                                    cudaStream_t stream, Actual &&...args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cluster;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, static_cast<Params>(args)...);
}

}  // namespace pa
