// api_block.cu -- C ABI of the norms, their backward passes, dropout and gradient
// clipping: host-side validation and launches.  No allocation, no synchronization.
#include <cmath>
#include <cstdint>
#include <initializer_list>

#include "dropout.h"
#include "fp8ll.h"
#include "grad_clip.h"
#include "internal.h"
#include "norm.h"

using namespace fp8ll;

namespace {

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

struct Range {
    const void* p;
    int64_t bytes;
};

// true when two ranges share a byte (a null or empty range shares none)
bool share(const Range& a, const Range& b) {
    if (!a.p || !b.p || a.bytes <= 0 || b.bytes <= 0) return false;
    const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
    return x < y + static_cast<uintptr_t>(b.bytes) && y < x + static_cast<uintptr_t>(a.bytes);
}

// rows of ld elements whose extent, in bytes of up to 4 an element, stays within 64 bits
bool spans(int64_t rows, int64_t ld) { return ld < (1LL << 36) && (rows < 2 || ld <= (1LL << 60) / rows); }

// center: the layer norm's, with mean and beta
bool valid_norm(const NormParams& p, bool center, int fmt) {
    if (fmt != FP8LL_E4M3 && fmt != FP8LL_E5M2) return false;
    if (p.cols % 128 != 0 || p.cols > (center ? kLayerNormMaxCols : kNormMaxCols) || p.rows > (1LL << 31) - 1)
        return false;
    if (center && (!p.mean || !aligned(p.mean, 4) || !aligned(p.beta, 16))) return false;
    if (!(p.eps >= 0.0f) || std::isinf(p.eps)) return false;
    if (!p.x || !aligned(p.x, 16) || p.ldx < p.cols || p.ldx % 8 != 0 || !spans(p.rows, p.ldx)) return false;
    if (p.residual && (!aligned(p.residual, 16) || p.ldr < p.cols || p.ldr % 8 != 0 || !spans(p.rows, p.ldr)))
        return false;
    if (p.residual && !p.h) return false;
    if (!p.gamma || !aligned(p.gamma, 16) || !p.rstd || !aligned(p.rstd, 4)) return false;
    if (!aligned(p.h, 16) || !aligned(p.y, 16) || !aligned(p.qr, 16) || !aligned(p.qc, 16)) return false;
    if (!p.y && !p.qr && !p.qc) return false;
    if (p.qc && p.rows % 128 != 0) return false;
    return true;
}

// every output apart from every other and from the inputs; h may take the
// place of x or of the residual, element by element
bool apart(const NormParams& p, const Range* scales, int num_scales) {
    const int64_t n = p.rows * p.cols;
    const Range x{p.x, ((p.rows - 1) * p.ldx + p.cols) * 2}, g{p.gamma, p.cols * 2}, b{p.beta, p.cols * 2};
    const Range r{p.residual, ((p.rows - 1) * p.ldr + p.cols) * 2};
    Range out[12] = {{p.h, 2 * n}, {p.rstd, 4 * p.rows}, {p.y, 2 * n}, {p.qr, n}, {p.qc, n}, {p.mean, 4 * p.rows}};
    int count = 6;
    for (int i = 0; i < num_scales; ++i) out[count++] = scales[i];
    for (int i = 0; i < count; ++i) {
        const bool h_on_x = i == 0 && p.h == p.x && p.ldx == p.cols;
        const bool h_on_r = i == 0 && p.h == p.residual && p.ldr == p.cols;
        if ((share(out[i], x) && !h_on_x) || (share(out[i], r) && !h_on_r) || share(out[i], g) || share(out[i], b))
            return false;
        for (int j = 0; j < i; ++j)
            if (share(out[i], out[j])) return false;
    }
    return true;
}

int launch(const NormParams& p, bool center, int recipe, int fmt, fp8ll_stream_t stream) {
    int sms = 0;
    const int rc = current_device_sms(&sms);
    if (rc != FP8LL_OK) return rc;
    const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    return (center ? launch_layernorm(p, recipe, fmt, s, sms) : launch_rmsnorm(p, recipe, fmt, s, sms)) == 0
               ? FP8LL_OK
               : FP8LL_ERR_LAUNCH;
}

NormParams norm_params(const void* x, const void* residual, const void* gamma, int64_t rows, int64_t cols,
                          int64_t ldx, int64_t ldr, float eps, void* h, float* rstd, void* y, uint8_t* q_rows,
                          uint8_t* q_cols) {
    NormParams p = {};
    p.x = static_cast<const uint16_t*>(x);
    p.residual = static_cast<const uint16_t*>(residual);
    p.gamma = static_cast<const uint16_t*>(gamma);
    p.rows = rows;
    p.cols = cols;
    p.ldx = ldx;
    p.ldr = residual ? ldr : 0;
    p.eps = eps;
    p.h = static_cast<uint16_t*>(h);
    p.rstd = rstd;
    p.y = static_cast<uint16_t*>(y);
    p.qr = q_rows;
    p.qc = q_cols;
    return p;
}

// The three recipes' calls, of either norm, from parameters without the scales.
int block_norm(NormParams p, bool center, int fmt, float* scale_rows, int64_t scale_ld_rows, float* scale_cols,
               int64_t scale_ld_cols, fp8ll_stream_t stream) {
    if (p.rows < 0 || p.cols < 0 || (fmt != FP8LL_E4M3 && fmt != FP8LL_E5M2)) return FP8LL_ERR_INVALID_ARG;
    if (p.rows == 0 || p.cols == 0) return FP8LL_OK;
    if (!valid_norm(p, center, fmt)) return FP8LL_ERR_INVALID_ARG;
    Range scales[2] = {{nullptr, 0}, {nullptr, 0}};
    if (p.qr) {
        if (!scale_rows || !aligned(scale_rows, 16) || scale_ld_rows < p.rows || scale_ld_rows % 4 != 0 ||
            scale_ld_rows >= (1LL << 36))
            return FP8LL_ERR_INVALID_ARG;
        p.sr = scale_rows;
        p.sldr = scale_ld_rows;
        scales[0] = Range{scale_rows, ((p.cols / 128 - 1) * scale_ld_rows + p.rows) * 4};
    }
    if (p.qc) {
        if (!scale_cols || !aligned(scale_cols, 16) || scale_ld_cols < p.cols || scale_ld_cols % 4 != 0 ||
            scale_ld_cols >= (1LL << 36))
            return FP8LL_ERR_INVALID_ARG;
        p.sc = scale_cols;
        p.sldc = scale_ld_cols;
        scales[1] = Range{scale_cols, ((p.rows / 128 - 1) * scale_ld_cols + p.cols) * 4};
    }
    if (!apart(p, scales, 2)) return FP8LL_ERR_INVALID_ARG;
    return launch(p, center, kRecipeBlock, fmt, stream);
}

int mx_norm(NormParams p, bool center, int fmt, uint8_t* sf_rows, uint8_t* sf_cols, fp8ll_stream_t stream) {
    if (p.rows < 0 || p.cols < 0 || (fmt != FP8LL_E4M3 && fmt != FP8LL_E5M2)) return FP8LL_ERR_INVALID_ARG;
    if (p.rows == 0 || p.cols == 0) return FP8LL_OK;
    if (!valid_norm(p, center, fmt)) return FP8LL_ERR_INVALID_ARG;
    if ((p.qr && (!sf_rows || !aligned(sf_rows, 16))) || (p.qc && (!sf_cols || !aligned(sf_cols, 16))))
        return FP8LL_ERR_INVALID_ARG;
    p.sfr = p.qr ? sf_rows : nullptr;
    p.sfc = p.qc ? sf_cols : nullptr;
    const Range scales[2] = {{p.sfr, static_cast<int64_t>(fp8_mx_sf_bytes(p.rows, p.cols))},
                             {p.sfc, p.qc ? static_cast<int64_t>(fp8_mx_sf_bytes(p.cols, p.rows)) : 0}};
    if (!apart(p, scales, 2)) return FP8LL_ERR_INVALID_ARG;
    return launch(p, center, kRecipeMx, fmt, stream);
}

int tensor_norm(NormParams p, bool center, int fmt, const float* amax_in, float* scale, float* amax_out,
                fp8ll_stream_t stream) {
    if (p.rows < 0 || p.cols < 0 || (fmt != FP8LL_E4M3 && fmt != FP8LL_E5M2)) return FP8LL_ERR_INVALID_ARG;
    if (p.rows == 0 || p.cols == 0) return FP8LL_OK;
    if (!valid_norm(p, center, fmt)) return FP8LL_ERR_INVALID_ARG;
    if (!amax_in || !aligned(amax_in, 4) || !scale || !aligned(scale, 4) || !aligned(amax_out, 4))
        return FP8LL_ERR_INVALID_ARG;
    // the kernels read *amax_in while they write the scale and the new amax
    if (scale == amax_in || amax_out == amax_in) return FP8LL_ERR_INVALID_ARG;
    p.amax_in = amax_in;
    p.scale = scale;
    p.amax_out = amax_out;
    const Range scales[2] = {{scale, 4}, {amax_out, 4}}, in{amax_in, 4};
    if (!apart(p, scales, 2)) return FP8LL_ERR_INVALID_ARG;
    const int64_t n = p.rows * p.cols;
    for (const Range& out :
         {Range{p.h, 2 * n}, {p.rstd, 4 * p.rows}, {p.y, 2 * n}, {p.qr, n}, {p.qc, n}, {p.mean, 4 * p.rows}})
        if (share(out, in)) return FP8LL_ERR_INVALID_ARG;
    return launch(p, center, kRecipeTensor, fmt, stream);
}

NormParams layernorm_params(const void* x, const void* residual, const void* gamma, const void* beta, int64_t rows,
                            int64_t cols, int64_t ldx, int64_t ldr, float eps, void* h, float* mean, float* rstd,
                            void* y, uint8_t* q_rows, uint8_t* q_cols) {
    NormParams p = norm_params(x, residual, gamma, rows, cols, ldx, ldr, eps, h, rstd, y, q_rows, q_cols);
    p.beta = static_cast<const uint16_t*>(beta);
    p.mean = mean;
    return p;
}

// The backward pass of either norm.
int norm_backward(NormGradParams p, bool center, void* workspace, size_t workspace_bytes, int64_t need,
                  fp8ll_stream_t stream) {
    const int64_t rows = p.rows, cols = p.cols;
    if (rows < 0 || cols < 0 || (p.accumulate != 0 && p.accumulate != 1)) return FP8LL_ERR_INVALID_ARG;
    if (cols == 0) return FP8LL_OK;
    if (cols % 8 != 0 || cols > (center ? kLayerNormMaxCols : kNormMaxCols) || !p.dgamma || !aligned(p.dgamma, 16) ||
        !aligned(p.dbeta, 16))
        return FP8LL_ERR_INVALID_ARG;
    const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    int sms = 0;
    if (rows == 0) {  // a sum over no rows
        if (share(Range{p.dgamma, cols * 4}, Range{p.dbeta, cols * 4})) return FP8LL_ERR_INVALID_ARG;
        const int rc = current_device_sms(&sms);
        if (rc != FP8LL_OK || p.accumulate) return rc;
        const size_t bytes = static_cast<size_t>(cols) * 4;
        if (cudaMemsetAsync(p.dgamma, 0, bytes, s) != cudaSuccess) return FP8LL_ERR_LAUNCH;
        return !p.dbeta || cudaMemsetAsync(p.dbeta, 0, bytes, s) == cudaSuccess ? FP8LL_OK : FP8LL_ERR_LAUNCH;
    }
    if (rows > (1LL << 31) - 1) return FP8LL_ERR_INVALID_ARG;
    if (!p.dy || !p.h || !p.gamma || !p.rstd || !p.dx || (center && !p.mean)) return FP8LL_ERR_INVALID_ARG;
    if (!aligned(p.dy, 16) || !aligned(p.h, 16) || !aligned(p.gamma, 16) || !aligned(p.rstd, 4) ||
        !aligned(p.mean, 4) || !aligned(p.dres, 16) || !aligned(p.dx, 16))
        return FP8LL_ERR_INVALID_ARG;
    if (p.lddy < cols || p.lddy % 8 != 0 || !spans(rows, p.lddy) || p.ldh < cols || p.ldh % 8 != 0 ||
        !spans(rows, p.ldh))
        return FP8LL_ERR_INVALID_ARG;
    if (p.dres && (p.ldres < cols || p.ldres % 8 != 0 || !spans(rows, p.ldres))) return FP8LL_ERR_INVALID_ARG;
    if (!workspace || !aligned(workspace, 16) || static_cast<int64_t>(workspace_bytes) < need)
        return FP8LL_ERR_WORKSPACE;
    const Range in[6] = {{p.dy, ((rows - 1) * p.lddy + cols) * 2},
                         {p.dres, p.dres ? ((rows - 1) * p.ldres + cols) * 2 : 0},
                         {p.h, ((rows - 1) * p.ldh + cols) * 2},
                         {p.gamma, cols * 2},
                         {p.rstd, rows * 4},
                         {p.mean, rows * 4}};
    const Range out[4] = {{p.dx, rows * cols * 2}, {p.dgamma, cols * 4}, {workspace, need}, {p.dbeta, cols * 4}};
    for (int i = 0; i < 4; ++i) {
        for (int j = 0; j < 6; ++j) {
            // dx may take the place of dy or of the residual's gradient, element by element
            const bool in_place =
                i == 0 && ((j == 0 && p.dx == p.dy && p.lddy == cols) || (j == 1 && p.dx == p.dres && p.ldres == cols));
            if (share(out[i], in[j]) && !in_place) return FP8LL_ERR_INVALID_ARG;
        }
        for (int j = 0; j < i; ++j)
            if (share(out[i], out[j])) return FP8LL_ERR_INVALID_ARG;
    }
    const int rc = current_device_sms(&sms);
    if (rc != FP8LL_OK) return rc;
    p.partials = static_cast<float*>(workspace);
    return (center ? launch_layernorm_grad(p, s, sms) : launch_rmsnorm_grad(p, s, sms)) == 0 ? FP8LL_OK
                                                                                              : FP8LL_ERR_LAUNCH;
}

NormGradParams grad_params(const void* dy, const void* h, const void* gamma, const float* rstd, const void* dres,
                           int64_t rows, int64_t cols, int64_t lddy, int64_t ldh, int64_t ldres, void* dx,
                           float* dgamma, int accumulate) {
    NormGradParams p = {};
    p.dy = static_cast<const uint16_t*>(dy);
    p.h = static_cast<const uint16_t*>(h);
    p.gamma = static_cast<const uint16_t*>(gamma);
    p.rstd = rstd;
    p.dres = static_cast<const uint16_t*>(dres);
    p.rows = rows;
    p.cols = cols;
    p.lddy = lddy;
    p.ldh = ldh;
    p.ldres = ldres;
    p.dx = static_cast<uint16_t*>(dx);
    p.dgamma = dgamma;
    p.accumulate = accumulate;
    return p;
}

}  // namespace

extern "C" {

int fp8_rmsnorm_quantize(const void* x_bf16, const void* residual_bf16, const void* gamma_bf16, int64_t rows,
                         int64_t cols, int64_t ldx, int64_t ldr, float eps, int fmt, void* h_bf16, float* rstd,
                         void* y_bf16, uint8_t* q_rows, float* scale_rows, int64_t scale_ld_rows, uint8_t* q_cols,
                         float* scale_cols, int64_t scale_ld_cols, fp8ll_stream_t stream) {
    return block_norm(norm_params(x_bf16, residual_bf16, gamma_bf16, rows, cols, ldx, ldr, eps, h_bf16, rstd, y_bf16,
                                  q_rows, q_cols),
                      false, fmt, scale_rows, scale_ld_rows, scale_cols, scale_ld_cols, stream);
}

int fp8_mx_rmsnorm_quantize(const void* x_bf16, const void* residual_bf16, const void* gamma_bf16, int64_t rows,
                            int64_t cols, int64_t ldx, int64_t ldr, float eps, int fmt, void* h_bf16, float* rstd,
                            void* y_bf16, uint8_t* q_rows, uint8_t* sf_rows, uint8_t* q_cols, uint8_t* sf_cols,
                            fp8ll_stream_t stream) {
    return mx_norm(norm_params(x_bf16, residual_bf16, gamma_bf16, rows, cols, ldx, ldr, eps, h_bf16, rstd, y_bf16,
                               q_rows, q_cols),
                   false, fmt, sf_rows, sf_cols, stream);
}

int fp8_tensor_rmsnorm_quantize(const void* x_bf16, const void* residual_bf16, const void* gamma_bf16, int64_t rows,
                                int64_t cols, int64_t ldx, int64_t ldr, float eps, int fmt, const float* amax_in,
                                void* h_bf16, float* rstd, void* y_bf16, uint8_t* q_rows, uint8_t* q_cols,
                                float* scale, float* amax_out, fp8ll_stream_t stream) {
    return tensor_norm(norm_params(x_bf16, residual_bf16, gamma_bf16, rows, cols, ldx, ldr, eps, h_bf16, rstd, y_bf16,
                                   q_rows, q_cols),
                       false, fmt, amax_in, scale, amax_out, stream);
}

int fp8_layernorm_quantize(const void* x_bf16, const void* residual_bf16, const void* gamma_bf16, const void* beta_bf16,
                           int64_t rows, int64_t cols, int64_t ldx, int64_t ldr, float eps, int fmt, void* h_bf16,
                           float* mean, float* rstd, void* y_bf16, uint8_t* q_rows, float* scale_rows,
                           int64_t scale_ld_rows, uint8_t* q_cols, float* scale_cols, int64_t scale_ld_cols,
                           fp8ll_stream_t stream) {
    return block_norm(layernorm_params(x_bf16, residual_bf16, gamma_bf16, beta_bf16, rows, cols, ldx, ldr, eps, h_bf16,
                                       mean, rstd, y_bf16, q_rows, q_cols),
                      true, fmt, scale_rows, scale_ld_rows, scale_cols, scale_ld_cols, stream);
}

int fp8_mx_layernorm_quantize(const void* x_bf16, const void* residual_bf16, const void* gamma_bf16,
                              const void* beta_bf16, int64_t rows, int64_t cols, int64_t ldx, int64_t ldr, float eps,
                              int fmt, void* h_bf16, float* mean, float* rstd, void* y_bf16, uint8_t* q_rows,
                              uint8_t* sf_rows, uint8_t* q_cols, uint8_t* sf_cols, fp8ll_stream_t stream) {
    return mx_norm(layernorm_params(x_bf16, residual_bf16, gamma_bf16, beta_bf16, rows, cols, ldx, ldr, eps, h_bf16,
                                    mean, rstd, y_bf16, q_rows, q_cols),
                   true, fmt, sf_rows, sf_cols, stream);
}

int fp8_tensor_layernorm_quantize(const void* x_bf16, const void* residual_bf16, const void* gamma_bf16,
                                  const void* beta_bf16, int64_t rows, int64_t cols, int64_t ldx, int64_t ldr,
                                  float eps, int fmt, const float* amax_in, void* h_bf16, float* mean, float* rstd,
                                  void* y_bf16, uint8_t* q_rows, uint8_t* q_cols, float* scale, float* amax_out,
                                  fp8ll_stream_t stream) {
    return tensor_norm(layernorm_params(x_bf16, residual_bf16, gamma_bf16, beta_bf16, rows, cols, ldx, ldr, eps, h_bf16,
                                        mean, rstd, y_bf16, q_rows, q_cols),
                       true, fmt, amax_in, scale, amax_out, stream);
}

size_t fp8_rmsnorm_workspace_size(int64_t rows, int64_t cols) {
    if (rows < 1 || cols < 1 || cols > kNormMaxCols) return 0;
    return static_cast<size_t>(norm_grad_max_bands(rows)) * static_cast<size_t>(cols) * sizeof(float);
}

int fp8_rmsnorm_backward(const void* dy_bf16, const void* h_bf16, const void* gamma_bf16, const float* rstd,
                         const void* residual_grad_bf16, int64_t rows, int64_t cols, int64_t lddy, int64_t ldh,
                         int64_t ldres, void* dx_bf16, float* dgamma, int accumulate, void* workspace,
                         size_t workspace_bytes, fp8ll_stream_t stream) {
    return norm_backward(grad_params(dy_bf16, h_bf16, gamma_bf16, rstd, residual_grad_bf16, rows, cols, lddy, ldh,
                                     ldres, dx_bf16, dgamma, accumulate),
                         false, workspace, workspace_bytes,
                         static_cast<int64_t>(fp8_rmsnorm_workspace_size(rows, cols)), stream);
}

size_t fp8_layernorm_workspace_size(int64_t rows, int64_t cols) {
    if (rows < 1 || cols < 1 || cols > kLayerNormMaxCols) return 0;
    return static_cast<size_t>(norm_grad_max_bands(rows)) * 2 * static_cast<size_t>(cols) * sizeof(float);
}

int fp8_layernorm_backward(const void* dy_bf16, const void* h_bf16, const void* gamma_bf16, const float* mean,
                           const float* rstd, const void* residual_grad_bf16, int64_t rows, int64_t cols, int64_t lddy,
                           int64_t ldh, int64_t ldres, void* dx_bf16, float* dgamma, float* dbeta, int accumulate,
                           void* workspace, size_t workspace_bytes, fp8ll_stream_t stream) {
    NormGradParams p = grad_params(dy_bf16, h_bf16, gamma_bf16, rstd, residual_grad_bf16, rows, cols, lddy, ldh, ldres,
                                   dx_bf16, dgamma, accumulate);
    p.mean = mean;
    p.dbeta = dbeta;
    return norm_backward(p, true, workspace, workspace_bytes,
                         static_cast<int64_t>(fp8_layernorm_workspace_size(rows, cols)), stream);
}

int fp8_dropout(const void* x_bf16, const void* residual_bf16, int64_t rows, int64_t cols, int64_t ldx, int64_t ldr,
                double p, uint64_t seed, uint32_t site, int64_t step, const int64_t* step_dev, void* out_bf16,
                fp8ll_stream_t stream) {
    if (rows < 0 || cols < 0 || !(p >= 0.0 && p < 1.0)) return FP8LL_ERR_INVALID_ARG;
    if (rows == 0 || cols == 0) return FP8LL_OK;
    if (rows >= kDropoutMaxElements || cols >= kDropoutMaxElements / rows + 1 || rows * cols >= kDropoutMaxElements)
        return FP8LL_ERR_INVALID_ARG;
    if (!x_bf16 || !aligned(x_bf16, 2) || ldx < cols || !spans(rows, ldx) || !out_bf16 || !aligned(out_bf16, 2))
        return FP8LL_ERR_INVALID_ARG;
    if (residual_bf16 && (!aligned(residual_bf16, 2) || ldr < cols || !spans(rows, ldr))) return FP8LL_ERR_INVALID_ARG;
    if (!aligned(step_dev, 8)) return FP8LL_ERR_INVALID_ARG;
    const Range out{out_bf16, rows * cols * 2}, x{x_bf16, ((rows - 1) * ldx + cols) * 2};
    const Range res{residual_bf16, residual_bf16 ? ((rows - 1) * ldr + cols) * 2 : 0}, counter{step_dev, 8};
    // the output may take the place of x or of the residual, element by element
    if (share(out, x) && !(out_bf16 == x_bf16 && (ldx == cols || rows == 1))) return FP8LL_ERR_INVALID_ARG;
    if (share(out, res) && !(out_bf16 == residual_bf16 && (ldr == cols || rows == 1))) return FP8LL_ERR_INVALID_ARG;
    if (share(out, counter)) return FP8LL_ERR_INVALID_ARG;
    int sms = 0;
    const int rc = current_device_sms(&sms);
    if (rc != FP8LL_OK) return rc;
    DropoutParams d = {};
    d.x = static_cast<const uint16_t*>(x_bf16);
    d.res = static_cast<const uint16_t*>(residual_bf16);
    d.out = static_cast<uint16_t*>(out_bf16);
    d.rows = rows;
    d.cols = cols;
    d.ldx = ldx;
    d.ldr = residual_bf16 ? ldr : 0;
    d.threshold = static_cast<uint32_t>(p * 4294967296.0);
    d.scale = static_cast<float>(1.0 / (1.0 - p));
    d.key0 = static_cast<uint32_t>(seed);
    d.key1 = static_cast<uint32_t>(seed >> 32);
    d.site = site;
    d.step = static_cast<uint64_t>(step);
    d.step_dev = step_dev;
    return launch_dropout(d, reinterpret_cast<cudaStream_t>(stream), sms) == 0 ? FP8LL_OK : FP8LL_ERR_LAUNCH;
}

size_t fp8_grad_norm_workspace_size(int64_t count) {
    if (count < 0) return 0;
    const int64_t launches = count == 0 ? 1 : (count + kClipTensorsPerLaunch - 1) / kClipTensorsPerLaunch;
    return static_cast<size_t>(launches) * kClipMaxBlocks * sizeof(float);
}

static int grad_call(int64_t count, const fp8ll_grad_t* grads, int scale, float max_norm, float* norm,
                     void* workspace, size_t workspace_bytes, fp8ll_stream_t stream) {
    if (count < 0 || count > kClipMaxTensors || (count > 0 && !grads) || !norm || !aligned(norm, 4))
        return FP8LL_ERR_INVALID_ARG;
    if (scale && !(max_norm >= 0.0f)) return FP8LL_ERR_INVALID_ARG;
    const int64_t need = static_cast<int64_t>(fp8_grad_norm_workspace_size(count));
    const Range nr{norm, 4}, ws{workspace, need};
    int64_t total = 0;
    for (int64_t i = 0; i < count; ++i) {
        const fp8ll_grad_t& g = grads[i];
        if (g.n < 0 || g.n >= (1LL << 40) || (g.dtype != FP8LL_F32 && g.dtype != FP8LL_BF16))
            return FP8LL_ERR_INVALID_ARG;
        total += g.n;
        if (total >= (1LL << 43)) return FP8LL_ERR_INVALID_ARG;  // chunk numbers are 32 bits
        if (g.n == 0) continue;
        const int size = g.dtype == FP8LL_F32 ? 4 : 2;
        if (!g.grad || !aligned(g.grad, size)) return FP8LL_ERR_INVALID_ARG;
        const Range in{g.grad, g.n * size};
        if (share(in, nr) || share(in, ws)) return FP8LL_ERR_INVALID_ARG;
        if (!scale) continue;
        if (!g.out || !aligned(g.out, size)) return FP8LL_ERR_INVALID_ARG;
        const Range out{g.out, g.n * size};
        if ((g.out != g.grad && share(in, out)) || share(out, nr) || share(out, ws)) return FP8LL_ERR_INVALID_ARG;
    }
    if (!workspace || !aligned(workspace, 16) || static_cast<int64_t>(workspace_bytes) < need)
        return FP8LL_ERR_WORKSPACE;
    if (share(nr, ws)) return FP8LL_ERR_INVALID_ARG;
    int sms = 0;
    const int rc = current_device_sms(&sms);
    if (rc != FP8LL_OK) return rc;
    return launch_grad_norm(count, grads, scale, max_norm, norm, static_cast<float*>(workspace),
                            reinterpret_cast<cudaStream_t>(stream), sms) == 0
               ? FP8LL_OK
               : FP8LL_ERR_LAUNCH;
}

int fp8_grad_norm(int64_t count, const fp8ll_grad_t* grads, float* norm, void* workspace, size_t workspace_bytes,
                  fp8ll_stream_t stream) {
    return grad_call(count, grads, 0, 0.0f, norm, workspace, workspace_bytes, stream);
}

int fp8_clip_grads(int64_t count, const fp8ll_grad_t* grads, float max_norm, float* norm, void* workspace,
                   size_t workspace_bytes, fp8ll_stream_t stream) {
    return grad_call(count, grads, 1, max_norm, norm, workspace, workspace_bytes, stream);
}

}  // extern "C"
