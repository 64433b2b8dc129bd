// launch.h -- kernel launches that allocate nothing and throw nothing, as they run
// below C entry points.
#pragma once

#include <cuda_runtime.h>

#include "subset.h"

namespace pa {

// The largest shared-memory carveout, asked for once per (device, kernel): consecutive kernels of the library never make
// the SMs reconfigure between them.
inline void carveout_noted(const void *kernel) noexcept {
    static DoneOnce once;
    int dev = 0;
    bool done;
    if (cudaGetDevice(&dev) != cudaSuccess) return;
    std::atomic<const void *> *slot = once.find(dev, kernel, done);
    if (done) return;
    cudaFuncSetAttribute(kernel, cudaFuncAttributePreferredSharedMemoryCarveout, 100);
    DoneOnce::note(slot, kernel);
}

// A launch with programmatic stream serialization allowed, in clusters of `cluster` CTAs.
template <typename... KArgs, typename... Args>
inline cudaError_t launch_soon(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem, cudaStream_t stream, unsigned cluster,
                               Args... args) noexcept {
    carveout_noted(reinterpret_cast<const void *>(kernel));
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, static_cast<KArgs>(args)...);
}

}  // namespace pa
