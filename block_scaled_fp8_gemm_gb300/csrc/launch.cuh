// launch.cuh -- kernel launches with a cluster, or overlapping the kernel before them.
#pragma once

#include <cuda_runtime.h>

namespace gemmar {

// Launch with a cluster of `splits` along y; with `early` the kernel may start while the
// one before it in the stream still runs (it calls grid_wait before it reads that one's
// results, and every CTA does before it ends).
template <typename... Params, typename... Args>
cudaError_t launch(void (*kernel)(Params...), dim3 grid, int threads, size_t smem, int splits, bool early,
                   cudaStream_t st, Args... args)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attrs[2];
    cfg.attrs = attrs;
    if (splits > 1) {
        attrs[cfg.numAttrs].id = cudaLaunchAttributeClusterDimension;
        attrs[cfg.numAttrs].val.clusterDim.x = 1;
        attrs[cfg.numAttrs].val.clusterDim.y = (unsigned)splits;
        attrs[cfg.numAttrs++].val.clusterDim.z = 1;
    }
    if (early) {
        attrs[cfg.numAttrs].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attrs[cfg.numAttrs++].val.programmaticStreamSerializationAllowed = 1;
    }
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

}  // namespace gemmar
