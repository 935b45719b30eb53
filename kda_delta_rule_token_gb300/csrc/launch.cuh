// A launch whose CTAs may come while the kernel before it in the stream still ends
// (programmatic dependent launch).  Every kernel that is launched so waits for the one before
// (ptx::griddep_wait) before it reads or writes memory that others use.  The wait is each kernel's own: what
// the kernel before it has waited for reaches it by that kernel's end alone, so that all
// of a call's kernels, and the next call's first one, see what came before them.  The first kernels
// of the calls for several continuations are launched so too: calls in a row, between other work, took
// 2 to 3 us less each when that came in (64 sequences reordered 18.4 -> 15.8 us, 14.6 now; 64 samples'
// attention 46.6 -> 44.1, 42.6 now).
#pragma once

#include <cuda_runtime.h>

#include <utility>

#include "kda_internal.cuh"

namespace kda {

// `cluster`: CTAs of a cluster along the grid's x.
template <class... Params, class... Args>
cudaError_t launch_clusters_behind(void (*kernel)(Params...), dim3 grid, int cluster, int threads, size_t smem, cudaStream_t stream, Args&&... args) {
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)cluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, std::forward<Args>(args)...);
    count_launches(1);
    if (e != cudaSuccess) cudaGetLastError();   // returned, not left for others to find
    return e;
}

template <class... Params, class... Args>
cudaError_t launch_behind(void (*kernel)(Params...), dim3 grid, int threads, size_t smem, cudaStream_t stream, Args&&... args) {
    return launch_clusters_behind(kernel, grid, 1, threads, smem, stream, std::forward<Args>(args)...);
}

}  // namespace kda
