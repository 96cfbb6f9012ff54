// rmsnorm.cu -- root-mean-square norm with the residual's addition and an fp8
// output, and its backward pass.
//
//   h = bf16(x + r)                     (the residual stream; h = x without r)
//   rstd = 1 / sqrt(mean_c h^2 + eps)   (0 where that root is 0)
//   y = fl32(fl32(h rstd) gamma)        -> fp8 codes and scales, and / or bf16
//
// The norm is taken of the rounded h, which is what the stream carries on and
// what the backward pass reads.  y is cast from fp32: the cast sees the value
// before any bf16 rounding, so an element is rounded once.
//
// Bound by HBM: 8192 x 4096 with residual, 1x128: 38 us, 0.91 of the measured copy
// rate (48.9 without the loads ahead and with every lane's own divisions); the
// columns kernel 20 us more at that size.
#include "norm_kernels.cuh"

namespace fp8ll {

int launch_rmsnorm(const NormParams& p, int recipe, int fmt, cudaStream_t stream, int num_sms) {
    switch (recipe * 2 + fmt) {
        case 0: return launch_norm<false, 0, kRecipeBlock>(p, stream, num_sms);
        case 1: return launch_norm<false, 1, kRecipeBlock>(p, stream, num_sms);
        case 2: return launch_norm<false, 0, kRecipeMx>(p, stream, num_sms);
        case 3: return launch_norm<false, 1, kRecipeMx>(p, stream, num_sms);
        case 4: return launch_norm<false, 0, kRecipeTensor>(p, stream, num_sms);
        case 5: return launch_norm<false, 1, kRecipeTensor>(p, stream, num_sms);
        default: return -3;
    }
}

int launch_rmsnorm_grad(const NormGradParams& p, cudaStream_t stream, int num_sms) {
    const int64_t nv = p.cols / 8;
    auto threads = [nv](int V) { return static_cast<int>(((nv + V - 1) / V + 31) / 32 * 32); };
    // up to 1024 columns a row needs no more than a warp: 25.8 us at 32768 x 512
    // against 35.8 with 64 threads per row and a barrier
    if (nv <= 16) return launch_grad<false, 1, 256, false, true, 16>(p, 256, num_sms, 4, stream);
    if (nv <= 32) return launch_grad<false, 1, 256, false, true, 32>(p, 256, num_sms, 4, stream);
    if (nv <= 64) return launch_grad<false, 2, 256, false, true, 32>(p, 256, num_sms, 2, stream);
    if (nv <= 128) return launch_grad<false, 4, 256, false, true, 32>(p, 256, num_sms, 1, stream);
    // two vectors a thread while the CTA stays within 512 threads, else dgamma
    // moves to shared memory: 102.6 us at 4096 x 14336 against 132.9 with spilled
    // registers
    int T = threads(2);
    if (T <= 512) return launch_grad<false, 2, 512, false, true, 0>(p, T, num_sms, 512 / T, stream);
    T = threads(4);
    if (T <= 512) return launch_grad<false, 4, 512, true, true, 0>(p, T, num_sms, 1, stream);
    return launch_grad<false, 8, 512, true, false, 0>(p, threads(8), num_sms, 1, stream);
}

}  // namespace fp8ll
