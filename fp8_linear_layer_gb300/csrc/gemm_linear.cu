// gemm_linear.cu -- instantiations of the 1x128 GEMM with the bias, activation
// and residual epilogue, whole and with the K blocks of each tile split.
#include <atomic>

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

// clusters of SPLIT CTAs that run at once on the current device (GPCs' sizes
// leave SMs over), asked once; 0 where that is not known
template <int SPLIT>
static int split_slots() {
    static std::atomic<int> known[64];
    int dev = 0;
    if (configure_gemm<kEpiLinearAny, SPLIT>(&dev) != 0) return 0;
    int n = known[dev].load(std::memory_order_relaxed);
    if (n == 0) {
        cudaLaunchAttribute attr;
        attr.id = cudaLaunchAttributeClusterDimension;
        attr.val.clusterDim.x = SPLIT;
        attr.val.clusterDim.y = 1;
        attr.val.clusterDim.z = 1;
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(SPLIT, 1, 1);
        cfg.blockDim = dim3(kThreads, 1, 1);
        cfg.dynamicSmemBytes = smem_bytes<kEpiLinearAny, SPLIT>();
        cfg.attrs = &attr;
        cfg.numAttrs = 1;
        if (cudaOccupancyMaxActiveClusters(&n, gemm_fp8_kernel<kEpiLinearAny, SPLIT>, &cfg) != cudaSuccess) {
            cudaGetLastError();
            return 0;
        }
        known[dev].store(n, std::memory_order_relaxed);
    }
    return n;
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
//   1000 x 2111 over 768    14.3 / 19.5   13.4 / 15.4
//   1000 x 2110 over 768    11.8 / 15.5   12.2 / 14.0
int gemm_linear_parts(const GemmParams& p) {
    const int nkb = p.groups[0].nkb;
    const bool odd_rows = p.N % 8 != 0;
    if (nkb >= (odd_rows ? 6 : 16) && p.total_tiles <= split_slots<4>()) return 4;
    if (nkb >= (odd_rows ? 6 : 12) && p.total_tiles <= split_slots<2>()) return 2;
    return 1;
}

// one tile per cluster of SPLIT CTAs
template <int EPI, int SPLIT>
static int launch_split_impl(const TensorMaps& maps, const GemmParams& p, cudaStream_t stream) {
    int dev = 0;
    if (configure_gemm<EPI, SPLIT>(&dev) != 0) return -3;
    return launch_dependent_clusters(gemm_fp8_kernel<EPI, SPLIT>, dim3(SPLIT * p.total_tiles), SPLIT, kThreads,
                                     smem_bytes<EPI, SPLIT>(), stream, maps, p) == cudaSuccess
               ? 0
               : -3;
}

template <int SPLIT>
static int launch_split(const TensorMaps& maps, const GemmParams& p, int epi, cudaStream_t stream) {
    switch (epi) {
        case kEpiLinear: return launch_split_impl<kEpiLinear, SPLIT>(maps, p, stream);
        case kEpiLinearGelu: return launch_split_impl<kEpiLinearGelu, SPLIT>(maps, p, stream);
        case kEpiLinearAny: return launch_split_impl<kEpiLinearAny, SPLIT>(maps, p, stream);
        case kEpiLinearGeluAny: return launch_split_impl<kEpiLinearGeluAny, SPLIT>(maps, p, stream);
        default: return -1;
    }
}

int launch_gemm_linear_parts(const TensorMaps& maps, const GemmParams& p, int epi, int parts, cudaStream_t stream) {
    return parts == 4 ? launch_split<4>(maps, p, epi, stream) : launch_split<2>(maps, p, epi, stream);
}

}  // namespace fp8ll
