// launch.cuh -- launches with attributes, and the shared-memory allowance of a kernel.
#pragma once
#include <atomic>
#include <cuda_runtime.h>

namespace fa {

// A launch, or (behind) one as the programmatic dependent of the launch before it on the stream; `cluster` neighbouring
// CTAs along x form a cluster.
template <class... Params, class... Args>
cudaError_t launch_behind(void (*kern)(Params...), dim3 grid, int threads, size_t smem, bool behind, int cluster,
                          cudaStream_t s, Args... args) {
    cudaLaunchAttribute attrs[2];
    int n = 0;
    if (behind) {
        attrs[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attrs[n++].val.programmaticStreamSerializationAllowed = 1;
    }
    if (cluster > 1) {
        attrs[n].id = cudaLaunchAttributeClusterDimension;
        attrs[n].val.clusterDim.x = cluster;
        attrs[n].val.clusterDim.y = attrs[n].val.clusterDim.z = 1;
        ++n;
    }
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cfg.attrs = attrs;
    cfg.numAttrs = n;
    return cudaLaunchKernelEx(&cfg, kern, Params(args)...);
}

// Lets `kern` use `bytes` of dynamic shared memory, once per device and kernel (`done`: that kernel's devices so far;
// the call costs a launch's host time over again).
inline cudaError_t allow_smem(const void *kern, int bytes, std::atomic<unsigned long long> &done) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const unsigned long long bit = 1ull << (dev & 63);
    if (dev < 64 && (done.load(std::memory_order_relaxed) & bit)) return cudaSuccess;
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess && dev < 64) done.fetch_or(bit, std::memory_order_relaxed);
    return e;
}

}  // namespace fa
