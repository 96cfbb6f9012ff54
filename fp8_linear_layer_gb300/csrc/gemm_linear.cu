// gemm_linear.cu -- instantiations of the 1x128 GEMM with the bias, activation
// and residual epilogue.
#include "gemm_kernel.cuh"

namespace fp8ll {

int launch_gemm_linear(const TensorMaps& maps, const GemmParams& p, int epi, cudaStream_t stream, int grid) {
    switch (epi) {
        case kEpiLinear: return launch_gemm_impl<kEpiLinear>(maps, p, stream, grid);
        case kEpiLinearGelu: return launch_gemm_impl<kEpiLinearGelu>(maps, p, stream, grid);
        case kEpiLinearAny: return launch_gemm_impl<kEpiLinearAny>(maps, p, stream, grid);
        case kEpiLinearGeluAny: return launch_gemm_impl<kEpiLinearGeluAny>(maps, p, stream, grid);
        default: return -1;
    }
}

}  // namespace fp8ll
