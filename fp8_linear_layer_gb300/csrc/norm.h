// norm.h -- what the norm kernels receive: the root-mean-square norm's, and the
// layer norm's, which is the same of the centred row, plus beta.
#pragma once
#include <cstdint>
#include <cuda_runtime.h>

namespace fp8ll {

constexpr int kRecipeBlock = 0;   // one fp32 scale per 128 elements
constexpr int kRecipeMx = 1;      // one UE8M0 scale per 32 elements
constexpr int kRecipeTensor = 2;  // one fp32 scale per tensor
constexpr int64_t kNormMaxCols = 32768;
// the backward pass keeps two fp32 sums per column in shared memory
constexpr int64_t kLayerNormMaxCols = 28672;

struct NormParams {
    const uint16_t* x;         // bf16 [rows][ldx]
    const uint16_t* residual;  // bf16 [rows][ldr] or null
    const uint16_t* gamma;     // bf16 [cols]
    const uint16_t* beta;      // layer norm: bf16 [cols] or null
    int64_t rows, cols, ldx, ldr;
    int64_t ahead;  // a CTA asks for the row so many behind its own in L2 (0: for none)
    float eps;
    uint16_t* h;    // bf16 [rows][cols] or null: x + residual
    float* mean;    // layer norm: [rows]
    float* rstd;    // [rows]
    uint16_t* y;    // bf16 [rows][cols] or null
    uint8_t* qr;    // row codes [rows][cols] or null
    uint8_t* qc;    // column codes [cols][rows] or null
    float* sr;      // 1x128: scales of the row codes [cols/128][sldr]
    float* sc;      // 1x128: scales of the column codes [rows/128][sldc]
    int64_t sldr, sldc;
    uint8_t* sfr;   // MXFP8: scale bytes of the row and of the column codes
    uint8_t* sfc;
    const float* amax_in;  // per-tensor: the amax to cast with, the scale made of it, max|y|
    float* scale;
    float* amax_out;
};

struct NormGradParams {
    const uint16_t* dy;    // bf16 [rows][lddy]
    const uint16_t* h;     // bf16 [rows][ldh]
    const uint16_t* gamma;
    const float* mean;     // layer norm
    const float* rstd;
    const uint16_t* dres;  // bf16 [rows][ldres] or null
    int64_t rows, cols, lddy, ldh, ldres;
    uint16_t* dx;          // bf16 [rows][cols]
    float* dgamma;         // [cols]
    float* dbeta;          // layer norm: [cols] or null
    int accumulate;
    float* partials;       // [bands][cols], layer norm [bands][2][cols]
};

int launch_rmsnorm(const NormParams& p, int recipe, int fmt, cudaStream_t stream, int num_sms);
int launch_layernorm(const NormParams& p, int recipe, int fmt, cudaStream_t stream, int num_sms);
// most bands of partial dgamma sums that the gradients' launches write, on any device
constexpr int kGradMaxBands = 1024;
inline int64_t norm_grad_max_bands(int64_t rows) { return rows < kGradMaxBands ? rows : kGradMaxBands; }
int launch_rmsnorm_grad(const NormGradParams& p, cudaStream_t stream, int num_sms);
int launch_layernorm_grad(const NormGradParams& p, cudaStream_t stream, int num_sms);

}  // namespace fp8ll
