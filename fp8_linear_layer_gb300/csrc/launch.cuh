// launch.cuh -- kernels whose launch overlaps the end of the kernel before them
// on the stream (programmatic dependent launch).
//
// Every kernel launched this way calls await_dependency() before its first
// access to global memory: it returns when the kernel before has completed and its
// writes are visible, so the order of the stream holds.  What that kernel may have
// written is not read through the non-coherent path (__ldg), whose data must not
// change while the reading kernel runs.  One that then calls
// release_dependents() lets the next kernel's blocks take the places of blocks
// that finish, with their set-up done by the time the last one does: a product of
// one token behind another takes 6.5 us instead of 7.5 at 7168 x 2048, 12.9
// instead of 14.7 at 4096 x 14336.  (Released before the wait, blocks of the next
// kernel gather on the SMs that finish first: slower than without.)
#pragma once
#include <cuda_runtime.h>

#include "per_device.h"

namespace fp8ll {

// lets the kernel have `bytes` of dynamic shared memory on the current device, on
// first use (`allowed`: the kernel's own); 0 or a negative error
template <typename Kernel>
int allow_shared_memory(PerDevice& allowed, Kernel* kern, size_t bytes) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return -3;
    return allowed.get(dev, [kern, bytes] {
        return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(bytes)) ==
                       cudaSuccess
                   ? 0
                   : -3;
    });
}

__device__ __forceinline__ void release_dependents() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void await_dependency() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

template <typename... Params, typename... Args>
cudaError_t launch_dependent_clusters(void (*kern)(Params...), dim3 grid, unsigned cluster, unsigned block, size_t smem,
                                      cudaStream_t stream, Args&&... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(block);
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
    cfg.numAttrs = cluster > 0 ? 2 : 1;
    const cudaError_t rc = cudaLaunchKernelEx(&cfg, kern, static_cast<Params>(args)...);
    if (rc != cudaSuccess) cudaGetLastError();  // the caller reports it: not left for the next check of other code
    return rc;
}

template <typename... Params, typename... Args>
cudaError_t launch_dependent(void (*kern)(Params...), unsigned grid, unsigned block, size_t smem, cudaStream_t stream,
                             Args&&... args) {
    return launch_dependent_clusters(kern, dim3(grid), 0, block, smem, stream, static_cast<Args&&>(args)...);
}

}  // namespace fp8ll
