// ds_host.h -- error reporting and launches shared by the library's host code.
#pragma once

#include <cuda_runtime.h>

namespace ds {

// Message of the calling thread's most recent failure (ds_last_error_detail).
extern thread_local char g_detail[512];

// Records a message and returns `status`.
int fail(int status, const char *fmt, ...) __attribute__((format(printf, 2, 3)));
int fail_cuda(cudaError_t e, const char *what);

// Launches with programmatic dependent launch: the grid may be scheduled while
// the previous kernel on the stream drains.  The kernel calls
// dependent_grid_wait() before it touches memory, reads that with plain loads
// (neither __ldg nor const __restrict__), and calls allow_dependent_grid().
// CTAs come in clusters of `cluster`.
template <typename... Params, typename... Args>
cudaError_t launch_clusters(void (*kernel)(Params...), unsigned cluster, unsigned grid, unsigned threads,
                            size_t smem, cudaStream_t stream, Args &&...args)
{
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cluster;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, static_cast<Params>(args)...);
}

template <typename... Params, typename... Args>
cudaError_t launch_overlapped(void (*kernel)(Params...), unsigned grid, unsigned threads, size_t smem,
                              cudaStream_t stream, Args &&...args)
{
    return launch_clusters(kernel, 1, grid, threads, smem, stream, static_cast<Args &&>(args)...);
}

// The current device's ordinal and its SM count, asked of CUDA once a device.
int current_device(int *dev, int *sms);

}  // namespace ds
