// gemm_rows.h -- host interface of the linear GEMM for few rows of A.
#pragma once
#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

#include "rmsnorm.h"

namespace fp8ll {

constexpr int kRowsFeatures = 128;  // rows of B per output tile: the MMA's M

// tokens (rows of A) per output tile: the MMA's N
inline int rows_tokens(int64_t M) { return M <= 16 ? 16 : M <= 32 ? 32 : M <= 64 ? 64 : 128; }

// CTAs that share the K blocks of an output tile, at most 8
int rows_cluster(int64_t M, int64_t N, int64_t nkb);

// Whether this kernel is taken.  Up to 64 tokens always (1x128 / MXFP8 at 64
// tokens: 16.3 / 14.9 us against the tile kernels' 18.9 / 18.0 at 14336 features
// over 4096, 16.0 / 15.1 against 26.4 / 27.1 at 4096 over 14336).  Beyond that
// where K is split four or eight ways: 256 x 2112 over 7168 takes 14.2 us on 1x128
// operands, 18.6 in the tile kernel's four parts; 512 x 1024 over 4096 takes 9.0 us
// on MXFP8 operands, 13.8 in the pair kernel's two.  A split in two is left to the
// tile kernels where they split K themselves (1x128, 256 x 4096 over 14336: 39.1 us,
// 29.6 in four parts) or K is short (256 x 4096 over 1024: 11.4 / 10.2 against 9.4 /
// 8.5).  It is taken for MXFP8 and per-tensor operands from K = 4096 (128 x 8192 over
// 4096: 14.2 against 15.1; within 5% either way elsewhere), and for rows that are
// not 16-byte aligned, which cost this kernel's epilogue less (256 x 2001 over 512
// with GELU, residual and Z: 13.8 / 12.9 against 19.4 / 23.8).
inline bool rows_kernel_taken(int64_t M, int64_t N, int64_t K, int recipe) {
    if (M <= 64) return true;
    const int c = rows_cluster(M, N, K / 128);
    if (c != 2) return c >= 4;
    return recipe == kRecipeBlock ? N % 8 != 0 && K < 768 : N % 8 != 0 || K >= 4096;
}

struct RowsMaps {
    CUtensorMap w, x;    // codes: boxes of 128 rows of B, of rows_tokens(M) rows of A, 128 bytes each
    CUtensorMap sw, sx;  // 1x128: their scales, one K block; MXFP8: one 512-byte scale atom
};

struct RowsParams {
    int32_t M, N, nkb;
    int32_t cluster;        // CTAs that share the K blocks of an output tile (set by the launcher)
    uint32_t idesc;         // tcgen05 instruction descriptor without the MMA's N
    int32_t gelu;
    int32_t debug_starve;   // test hook: the producer issues no loads
    uint64_t budget_ns;     // wall-clock budget of each pipeline wait
    int* status;
    int64_t groups_w, groups_x;  // MXFP8: 128-row groups per K block of the scale arrays
    const float* tsw;       // per tensor: the scales
    const float* tsx;
    const uint16_t* bias;   // bf16 [N] or null
    const uint16_t* res;    // bf16 [M][ldr] or null
    int64_t ldr;
    uint16_t* out;          // bf16 [M][N]
    uint16_t* aux;          // bf16 [M][N] or null
};

int launch_gemm_rows(const RowsMaps& maps, RowsParams p, int recipe, cudaStream_t stream);

}  // namespace fp8ll
