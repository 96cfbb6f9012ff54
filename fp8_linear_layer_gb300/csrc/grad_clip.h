// grad_clip.h -- host interface of the gradient norm and clipping kernels.
#pragma once
#include <cstdint>
#include <cuda_runtime.h>

#include "fp8ll.h"

namespace fp8ll {

constexpr int kClipTensorsPerLaunch = 1000;  // 32 bytes each: the kernel parameters hold 32,764
constexpr int kClipMaxBlocks = 2048;         // partial sums of one launch
constexpr int kClipChunk = 8192;             // elements a CTA takes at a time
constexpr int kClipMaxTensors = 1 << 17;     // tensors of one call
// What pass 1 leaves in L2 (129 MB, two halves) for pass 2.  Measured on 470 MB
// of fp32: 224 us with 32 MB, 219 with 64, 219 with 96 (and 411 of the 470 MB
// come from DRAM again).
constexpr int64_t kClipKeepBytes = 64ll << 20;

// norm of all tensors; with `scale` also the scaled tensors
int launch_grad_norm(int64_t count, const fp8ll_grad_t* grads, int scale, float max_norm, float* norm,
                     float* partials, cudaStream_t stream, int num_sms);

}  // namespace fp8ll
