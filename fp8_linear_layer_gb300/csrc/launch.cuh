// launch.cuh -- a kernel whose launch overlaps the end of the kernel before it on
// the stream (programmatic dependent launch).
//
// The first kernel calls release_dependents() as it starts: the second one's
// blocks may then take the places of blocks that finish, with their set-up done
// by the time the last one does.  The second kernel calls await_dependency()
// before its first access to memory: it returns when the first kernel has
// completed and its writes are visible, so the pair behaves as two launches in
// stream order.
#pragma once
#include <cuda_runtime.h>

namespace fp8ll {

__device__ __forceinline__ void release_dependents() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void await_dependency() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

template <typename... Params, typename... Args>
cudaError_t launch_dependent(void (*kern)(Params...), unsigned grid, unsigned block, size_t smem, cudaStream_t stream,
                             Args&&... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(block);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, static_cast<Params>(args)...);
}

}  // namespace fp8ll
