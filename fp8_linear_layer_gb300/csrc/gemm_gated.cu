// gemm_gated.cu -- instantiations of the 1x128 GEMM with the gated epilogue (both
// projections of a tile, the activation and their product) and its data gradient,
// whole and with the K blocks of each tile split.
#include "gemm_kernel.cuh"

namespace fp8ll {

// one tile per cluster of SPLIT CTAs
template <int EPI, int SPLIT>
static int launch_split(const TensorMaps& maps, const GemmParams& p, cudaStream_t stream) {
    int dev = 0;
    if (configure_gemm<EPI, SPLIT>(&dev) != 0) return -3;
    return launch_dependent_clusters(gemm_fp8_kernel<EPI, SPLIT>, dim3(SPLIT * p.total_tiles), SPLIT, kThreads,
                                     smem_bytes<EPI, SPLIT>(), stream, maps, p) == cudaSuccess
               ? 0
               : -3;
}

template <int EPI>
static int launch(const TensorMaps& maps, const GemmParams& p, int parts, cudaStream_t stream, int grid) {
    switch (parts) {
        case 4: return launch_split<EPI, 4>(maps, p, stream);
        case 2: return launch_split<EPI, 2>(maps, p, stream);
        default: return launch_gemm_impl<EPI>(maps, p, stream, grid);
    }
}

// The gradient's rows are dear: in parts from fewer K blocks on than the linear GEMM.
// us in one, two and four parts:
//   300 x 1024 over 1024   13.0   11.8   11.3
//   1000 x 2048 over 1024  13.4   12.5
//                     512  11.0   11.1
int gemm_gated_grad_parts(const GemmParams& p) { return gemm_parts(p, kGatesSplitBlocks, kGatesSplitBlocks); }

int launch_gemm_gated(const TensorMaps& maps, const GemmParams& p, int epi, int parts, cudaStream_t stream, int grid) {
    switch (epi) {
        case kEpiGatedSilu: return launch<kEpiGatedSilu>(maps, p, parts, stream, grid);
        case kEpiGatedGelu: return launch<kEpiGatedGelu>(maps, p, parts, stream, grid);
        case kEpiGatedSiluGrad: return launch<kEpiGatedSiluGrad>(maps, p, parts, stream, grid);
        case kEpiGatedGeluGrad: return launch<kEpiGatedGeluGrad>(maps, p, parts, stream, grid);
        default: return -1;
    }
}

}  // namespace fp8ll
