// Host-side helpers shared by the translation units of the C ABI.
#pragma once

#include <cstdint>

#include <cuda.h>
#include <cuda_runtime.h>

#include "../../include/tsenor.h"

namespace tsenor {

// Records the message tsenor_last_error returns; the status is TSENOR_ERR_CUDA.
tsenor_status cuda_fail(cudaError_t e, const char* what);

inline bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// encode(), a call of the driver's tensor map encoder: it wants a context, which a host thread has only once it has called the
// runtime, so that the first call of a thread may have to make it and try again.  (By setting the device that is set: it
// allocates nothing and waits for nothing, which would end a capture that another thread has under way.)
template <typename F>
cudaError_t with_context(F encode) {
    CUresult r = encode();
    int device;
    if (r != CUDA_SUCCESS && cudaGetDevice(&device) == cudaSuccess && cudaSetDevice(device) == cudaSuccess) r = encode();
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

// Launches a kernel whose threads call prior_done() (pdl.h) before they touch global memory: it may start,
// and set itself up, while the kernel before it on the stream still runs.  cluster: CTAs
// of a cluster, 1 for none.
template <typename... P, typename... A>
cudaError_t launch_early(void (*kernel)(P...), int64_t grid, int block, size_t smem, int cluster, cudaStream_t st, A... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned(grid));
    cfg.blockDim = dim3(unsigned(block));
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = unsigned(cluster);
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, P(args)...);
}

// Lets launches of a kernel on the current device ask for up to `most` bytes of dynamic shared memory.  The limit belongs to
// the kernel, which all host threads share: `most` is a constant of the kernel, never what one launch needs.
template <typename... P>
cudaError_t allow_shared(void (*kernel)(P...), unsigned most) {
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, int(most));
}

// How many clusters of a kernel the current device runs at once.
template <typename... P>
cudaError_t clusters_that_fit(int* count, void (*kernel)(P...), int block, size_t smem, int cluster) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned(cluster));
    cfg.blockDim = dim3(unsigned(block));
    cfg.dynamicSmemBytes = smem;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = unsigned(cluster);
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaOccupancyMaxActiveClusters(count, kernel, &cfg);
}

// Counters on the current device that tsenor_error_count adds up and resets: rows that failed in the distillation kernels,
// and warps of tsenor_matmul's kernels whose limited wait ran out.
cudaError_t row_failures(unsigned long long** counter);
cudaError_t stalls(unsigned long long** counter);

}  // namespace tsenor
