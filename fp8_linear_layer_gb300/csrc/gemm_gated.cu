// gemm_gated.cu -- instantiations of the 1x128 GEMM with the gated epilogue (both
// projections of a tile, the activation and their product) and its data gradient,
// whole and with the K blocks of each tile split.
//
//   Z = A B^T + bias,  Y = act(Z_gate) Z_up        B: the gate's rows, then the up projection's
//   C = A B^T,  dZ = (C Z_up act'(Z_gate), C act(Z_gate))
//
// Forward: a tile's 256 rows of B are 128 of each projection, loaded as two boxes, so
// the K loop, its MMAs and its promotion are the linear GEMM's, and the two sums of an
// output lie in one thread's registers: Z goes to memory only where the backward pass
// wants it.  The CTA pairs of the other recipes load one projection each.  Bound by
// the promotion of K blocks (1x128) and by the tensor core: 8192 x 14336 over 4096,
// 1013 us (1899 TFLOP/s), with Z 1071; MXFP8 597 and 624, per tensor 556 and 640.
// Gradient: four bytes read and four written per output of the product, which an
// epilogue of two warps per scheduler handles a step at a time (7.5 us a tile, of 26):
// 8192 x 14336 over 4096, 628 us (1532 TFLOP/s), MXFP8 387.  With B's rows ordered it
// needs no shuffles: per tensor 347 (with them 376).
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

// The ordered epilogue takes 5 us a tile instead of 7.5, but the K loop in front of it
// comes out with 296 instructions a warp and block instead of 280: 0.66 us for 0.58.
// us, ordered / not (8192 x 14336 over 128: 156 / 214):
//   K blocks         8            16            20            24            28            32
//   8192 x 14336  256 / 293     382 / 403     446 / 459     508 / 513     573 / 570     637 / 627
//   8192 x 4096   80.7 / 88.0  117.4 / 120.7 136.4 / 137.1 155.2 / 153.1 174.5 / 169.7 193.2 / 186.1
//   2048 x 5632   36.5 / 40.6   52.0 / 54.5   59.7 / 61.3   67.8 / 68.3   75.9 / 75.2   83.6 / 82.3
// They cross between 20 and 28 blocks; at 24 the one taken is at most 1.4% behind.
// (Epilogues of other shapes moved these by a few per cent and not the crossing point.)
bool gemm_gated_grad_ordered(const GemmParams& p) { return p.groups[0].nkb <= 24; }

int launch_gemm_gated(const TensorMaps& maps, const GemmParams& p, int epi, int parts, cudaStream_t stream, int grid) {
    switch (epi) {
        case kEpiGatedSilu: return launch<kEpiGatedSilu>(maps, p, parts, stream, grid);
        case kEpiGatedGelu: return launch<kEpiGatedGelu>(maps, p, parts, stream, grid);
        case kEpiGatedSiluGrad: return launch<kEpiGatedSiluGrad>(maps, p, parts, stream, grid);
        case kEpiGatedGeluGrad: return launch<kEpiGatedGeluGrad>(maps, p, parts, stream, grid);
        case kEpiGatedSiluGradOrdered: return launch_gemm_impl<kEpiGatedSiluGradOrdered>(maps, p, stream, grid);
        case kEpiGatedGeluGradOrdered: return launch_gemm_impl<kEpiGatedGeluGradOrdered>(maps, p, stream, grid);
        default: return -1;
    }
}

}  // namespace fp8ll
