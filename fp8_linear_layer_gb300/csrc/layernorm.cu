// layernorm.cu -- layer norm with the residual's addition and an fp8 output, and
// its backward pass.
//
//   h = bf16(x + r)                               (the residual stream; h = x without r)
//   mean = sum_c h / C,  rstd = 1 / sqrt(sum_c (h - mean)^2 / C + eps)   (0 where that root is 0)
//   y = fma(fl(fl(h - mean) rstd), gamma, beta)   -> fp8 codes and scales, and / or bf16
//
// The deviations are summed in a second pass over the row, which stays in
// registers, so that a mean far from zero costs no digits.
//
// Bound by HBM where there are rows enough: 8192 x 4096 with residual on 1x128 40.6
// us, 0.87 of the measured copy rate; the columns kernel 20 us more at that size
// (half of h from L2, and a pass over a tile for the maxima in front of the cast's).
// The backward pass 16384 x 7168 with the residual's gradient 169 us, 0.83: one row
// at a time per SM there, 1260 cycles of instructions in the 2950 that it takes.  (Two
// rows at a time, the next four copied to shared memory ahead by cp.async: 166.)
#include "norm_kernels.cuh"

namespace fp8ll {
int launch_layernorm(const NormParams& p, int recipe, int fmt, cudaStream_t stream, int num_sms) {
    switch (recipe * 2 + fmt) {
        case 0: return launch_norm<true, 0, kRecipeBlock>(p, stream, num_sms);
        case 1: return launch_norm<true, 1, kRecipeBlock>(p, stream, num_sms);
        case 2: return launch_norm<true, 0, kRecipeMx>(p, stream, num_sms);
        case 3: return launch_norm<true, 1, kRecipeMx>(p, stream, num_sms);
        case 4: return launch_norm<true, 0, kRecipeTensor>(p, stream, num_sms);
        case 5: return launch_norm<true, 1, kRecipeTensor>(p, stream, num_sms);
        default: return -3;
    }
}

int launch_layernorm_grad(const NormGradParams& p, cudaStream_t stream, int num_sms) {
    const int64_t nv = p.cols / 8;
    auto threads = [nv](int V) { return static_cast<int>(((nv + V - 1) / V + 31) / 32 * 32); };
    if (nv <= 16) return launch_grad<true, 1, 256, false, true, 16, 3>(p, 256, num_sms, 3, stream);
    if (nv <= 32) return launch_grad<true, 1, 256, false, true, 32, 3>(p, 256, num_sms, 3, stream);
    if (nv <= 64) return launch_grad<true, 2, 256, false, true, 32, 2>(p, 256, num_sms, 2, stream);
    if (nv <= 128) return launch_grad<true, 4, 256, false, true, 32>(p, 256, num_sms, 1, stream);
    int T = threads(2);
    if (T <= 512) return launch_grad<true, 2, 512, false, true, 0>(p, T, num_sms, 512 / T, stream);
    T = threads(4);
    if (T <= 512) return launch_grad<true, 4, 512, true, true, 0>(p, T, num_sms, 1, stream);
    return launch_grad<true, 8, 512, true, false, 0>(p, threads(8), num_sms, 1, stream);
}

}  // namespace fp8ll
