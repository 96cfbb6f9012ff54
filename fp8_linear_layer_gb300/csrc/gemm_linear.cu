// gemm_linear.cu -- instantiations of the 1x128 GEMM with the bias, activation
// and residual epilogue, whole and with the K blocks of each tile split.
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

// As many as run at once in clusters, where the K loop that they save is longer than
// the exchange of the sums (about 4 us; part of it is won back because a part's
// threads store fewer rows).  With a residual / with GELU, residual and Z, us in
// one, two and four parts:
//   1000 x 2112 over 7168   38.6 / 41.1   25.7 / 27.8
//                    1536   12.4 / 15.4   12.6 / 14.4
//                    1024   10.1 / 13.0   11.4 / 13.1
//   600 x 1024 over 2048    14.6 / 17.2   13.0 / 14.7   12.9 / 14.0
//                   1536    12.2 / 14.9   11.8 / 13.5   12.5 / 13.3
// and where rows are not 16-byte aligned, which makes every row that is stored dearer:
//   600 x 1023 over 1536    16.4 / 22.9   12.7 / 16.3   12.1 / 14.1
//                   1024    14.0 / 20.5   11.5 / 15.3   11.5 / 13.5
int gemm_linear_parts(const GemmParams& p) {
    const int nkb = p.groups[0].nkb;
    const bool odd_rows = p.N % 8 != 0;
    if (nkb >= (odd_rows ? 8 : 16) && p.total_tiles <= gemm_split_slots<4>()) return 4;
    if (nkb >= (odd_rows ? 8 : 12) && p.total_tiles <= gemm_split_slots<2>()) return 2;
    return 1;
}

template <int SPLIT>
static int launch_split(const TensorMaps& maps, const GemmParams& p, int epi, cudaStream_t stream) {
    switch (epi) {
        case kEpiLinear: return launch_gemm_split<kEpiLinear, SPLIT>(maps, p, stream);
        case kEpiLinearGelu: return launch_gemm_split<kEpiLinearGelu, SPLIT>(maps, p, stream);
        case kEpiLinearAny: return launch_gemm_split<kEpiLinearAny, SPLIT>(maps, p, stream);
        case kEpiLinearGeluAny: return launch_gemm_split<kEpiLinearGeluAny, SPLIT>(maps, p, stream);
        default: return -1;
    }
}

int launch_gemm_linear_parts(const TensorMaps& maps, const GemmParams& p, int epi, int parts, cudaStream_t stream) {
    return parts == 4 ? launch_split<4>(maps, p, epi, stream) : launch_split<2>(maps, p, epi, stream);
}

}  // namespace fp8ll
