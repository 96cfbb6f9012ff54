// layernorm.cu -- layer norm with the residual's addition and an fp8 output, and
// its backward pass.
//
//   h = bf16(x + r)                               (the residual stream; h = x without r)
//   mean = sum_c h / C,  rstd = 1 / sqrt(sum_c (h - mean)^2 / C + eps)   (0 where that root is 0)
//   y = fma(fl(fl(h - mean) rstd), gamma, beta)   -> fp8 codes and scales, and / or bf16
//
// The deviations are summed in a second pass over the row, which stays in
// registers, so that a mean far from zero costs no digits.
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
    if (nv <= 16) return launch_grad<true, 1, 256, false, true, 16>(p, 256, num_sms, 4, stream);
    if (nv <= 32) return launch_grad<true, 1, 256, false, true, 32>(p, 256, num_sms, 4, stream);
    if (nv <= 64) return launch_grad<true, 2, 256, false, true, 32>(p, 256, num_sms, 2, stream);
    if (nv <= 128) return launch_grad<true, 4, 256, false, true, 32>(p, 256, num_sms, 1, stream);
    int T = threads(2);
    if (T <= 512) return launch_grad<true, 2, 512, false, true, 0>(p, T, num_sms, 512 / T, stream);
    T = threads(4);
    if (T <= 512) return launch_grad<true, 4, 512, true, true, 0>(p, T, num_sms, 1, stream);
    return launch_grad<true, 8, 512, true, false, 0>(p, threads(8), num_sms, 1, stream);
}

}  // namespace fp8ll
