// api_block.cu -- C ABI of the norm, its backward pass and gradient clipping:
// host-side validation and launches.  No allocation, no synchronization.
#include <cmath>
#include <cstdint>
#include <initializer_list>

#include "fp8ll.h"
#include "grad_clip.h"
#include "internal.h"
#include "rmsnorm.h"

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

bool valid_norm(const RmsNormParams& p, int fmt) {
    if (fmt != FP8LL_E4M3 && fmt != FP8LL_E5M2) return false;
    if (p.cols % 128 != 0 || p.cols > kNormMaxCols || p.rows > (1LL << 31) - 1) return false;
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
bool apart(const RmsNormParams& p, const Range* scales, int num_scales) {
    const int64_t n = p.rows * p.cols;
    const Range x{p.x, ((p.rows - 1) * p.ldx + p.cols) * 2}, g{p.gamma, p.cols * 2};
    const Range r{p.residual, ((p.rows - 1) * p.ldr + p.cols) * 2};
    Range out[12] = {{p.h, 2 * n}, {p.rstd, 4 * p.rows}, {p.y, 2 * n}, {p.qr, n}, {p.qc, n}};
    int count = 5;
    for (int i = 0; i < num_scales; ++i) out[count++] = scales[i];
    for (int i = 0; i < count; ++i) {
        const bool h_on_x = i == 0 && p.h == p.x && p.ldx == p.cols;
        const bool h_on_r = i == 0 && p.h == p.residual && p.ldr == p.cols;
        if ((share(out[i], x) && !h_on_x) || (share(out[i], r) && !h_on_r) || share(out[i], g)) return false;
        for (int j = 0; j < i; ++j)
            if (share(out[i], out[j])) return false;
    }
    return true;
}

int launch(const RmsNormParams& p, int recipe, int fmt, fp8ll_stream_t stream) {
    int sms = 0;
    const int rc = current_device_sms(&sms);
    if (rc != FP8LL_OK) return rc;
    return launch_rmsnorm(p, recipe, fmt, reinterpret_cast<cudaStream_t>(stream), sms) == 0 ? FP8LL_OK
                                                                                           : FP8LL_ERR_LAUNCH;
}

RmsNormParams norm_params(const void* x, const void* residual, const void* gamma, int64_t rows, int64_t cols,
                          int64_t ldx, int64_t ldr, float eps, void* h, float* rstd, void* y, uint8_t* q_rows,
                          uint8_t* q_cols) {
    RmsNormParams p = {};
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

}  // namespace

extern "C" {

int fp8_rmsnorm_quantize(const void* x_bf16, const void* residual_bf16, const void* gamma_bf16, int64_t rows,
                         int64_t cols, int64_t ldx, int64_t ldr, float eps, int fmt, void* h_bf16, float* rstd,
                         void* y_bf16, uint8_t* q_rows, float* scale_rows, int64_t scale_ld_rows, uint8_t* q_cols,
                         float* scale_cols, int64_t scale_ld_cols, fp8ll_stream_t stream) {
    if (rows < 0 || cols < 0 || (fmt != FP8LL_E4M3 && fmt != FP8LL_E5M2)) return FP8LL_ERR_INVALID_ARG;
    if (rows == 0 || cols == 0) return FP8LL_OK;
    RmsNormParams p = norm_params(x_bf16, residual_bf16, gamma_bf16, rows, cols, ldx, ldr, eps, h_bf16, rstd, y_bf16,
                                  q_rows, q_cols);
    if (!valid_norm(p, fmt)) return FP8LL_ERR_INVALID_ARG;
    Range scales[2] = {{nullptr, 0}, {nullptr, 0}};
    if (q_rows) {
        if (!scale_rows || !aligned(scale_rows, 16) || scale_ld_rows < rows || scale_ld_rows % 4 != 0 ||
            scale_ld_rows >= (1LL << 36))
            return FP8LL_ERR_INVALID_ARG;
        p.sr = scale_rows;
        p.sldr = scale_ld_rows;
        scales[0] = Range{scale_rows, ((cols / 128 - 1) * scale_ld_rows + rows) * 4};
    }
    if (q_cols) {
        if (!scale_cols || !aligned(scale_cols, 16) || scale_ld_cols < cols || scale_ld_cols % 4 != 0 ||
            scale_ld_cols >= (1LL << 36))
            return FP8LL_ERR_INVALID_ARG;
        p.sc = scale_cols;
        p.sldc = scale_ld_cols;
        scales[1] = Range{scale_cols, ((rows / 128 - 1) * scale_ld_cols + cols) * 4};
    }
    if (!apart(p, scales, 2)) return FP8LL_ERR_INVALID_ARG;
    return launch(p, kRecipeBlock, fmt, stream);
}

int fp8_mx_rmsnorm_quantize(const void* x_bf16, const void* residual_bf16, const void* gamma_bf16, int64_t rows,
                            int64_t cols, int64_t ldx, int64_t ldr, float eps, int fmt, void* h_bf16, float* rstd,
                            void* y_bf16, uint8_t* q_rows, uint8_t* sf_rows, uint8_t* q_cols, uint8_t* sf_cols,
                            fp8ll_stream_t stream) {
    if (rows < 0 || cols < 0 || (fmt != FP8LL_E4M3 && fmt != FP8LL_E5M2)) return FP8LL_ERR_INVALID_ARG;
    if (rows == 0 || cols == 0) return FP8LL_OK;
    RmsNormParams p = norm_params(x_bf16, residual_bf16, gamma_bf16, rows, cols, ldx, ldr, eps, h_bf16, rstd, y_bf16,
                                  q_rows, q_cols);
    if (!valid_norm(p, fmt)) return FP8LL_ERR_INVALID_ARG;
    if ((q_rows && (!sf_rows || !aligned(sf_rows, 16))) || (q_cols && (!sf_cols || !aligned(sf_cols, 16))))
        return FP8LL_ERR_INVALID_ARG;
    p.sfr = q_rows ? sf_rows : nullptr;
    p.sfc = q_cols ? sf_cols : nullptr;
    const Range scales[2] = {{p.sfr, static_cast<int64_t>(fp8_mx_sf_bytes(rows, cols))},
                             {p.sfc, q_cols ? static_cast<int64_t>(fp8_mx_sf_bytes(cols, rows)) : 0}};
    if (!apart(p, scales, 2)) return FP8LL_ERR_INVALID_ARG;
    return launch(p, kRecipeMx, fmt, stream);
}

int fp8_tensor_rmsnorm_quantize(const void* x_bf16, const void* residual_bf16, const void* gamma_bf16, int64_t rows,
                                int64_t cols, int64_t ldx, int64_t ldr, float eps, int fmt, const float* amax_in,
                                void* h_bf16, float* rstd, void* y_bf16, uint8_t* q_rows, uint8_t* q_cols,
                                float* scale, float* amax_out, fp8ll_stream_t stream) {
    if (rows < 0 || cols < 0 || (fmt != FP8LL_E4M3 && fmt != FP8LL_E5M2)) return FP8LL_ERR_INVALID_ARG;
    if (rows == 0 || cols == 0) return FP8LL_OK;
    RmsNormParams p = norm_params(x_bf16, residual_bf16, gamma_bf16, rows, cols, ldx, ldr, eps, h_bf16, rstd, y_bf16,
                                  q_rows, q_cols);
    if (!valid_norm(p, fmt)) return FP8LL_ERR_INVALID_ARG;
    if (!amax_in || !aligned(amax_in, 4) || !scale || !aligned(scale, 4) || !aligned(amax_out, 4))
        return FP8LL_ERR_INVALID_ARG;
    // the kernels read *amax_in while they write the scale and the new amax
    if (scale == amax_in || amax_out == amax_in) return FP8LL_ERR_INVALID_ARG;
    p.amax_in = amax_in;
    p.scale = scale;
    p.amax_out = amax_out;
    const Range scales[2] = {{scale, 4}, {amax_out, 4}}, in{amax_in, 4};
    if (!apart(p, scales, 2)) return FP8LL_ERR_INVALID_ARG;
    const int64_t n = rows * cols;
    for (const Range& out : {Range{h_bf16, 2 * n}, {rstd, 4 * rows}, {y_bf16, 2 * n}, {q_rows, n}, {q_cols, n}})
        if (share(out, in)) return FP8LL_ERR_INVALID_ARG;
    return launch(p, kRecipeTensor, fmt, stream);
}

size_t fp8_rmsnorm_workspace_size(int64_t rows, int64_t cols) {
    if (rows < 1 || cols < 1 || cols > kNormMaxCols) return 0;
    return static_cast<size_t>(rmsnorm_grad_max_bands(rows)) * static_cast<size_t>(cols) * sizeof(float);
}

int fp8_rmsnorm_backward(const void* dy_bf16, const void* h_bf16, const void* gamma_bf16, const float* rstd,
                         const void* residual_grad_bf16, int64_t rows, int64_t cols, int64_t lddy, int64_t ldh,
                         int64_t ldres, void* dx_bf16, float* dgamma, int accumulate, void* workspace,
                         size_t workspace_bytes, fp8ll_stream_t stream) {
    if (rows < 0 || cols < 0 || (accumulate != 0 && accumulate != 1)) return FP8LL_ERR_INVALID_ARG;
    if (cols == 0) return FP8LL_OK;
    if (cols % 8 != 0 || cols > kNormMaxCols || !dgamma || !aligned(dgamma, 16)) return FP8LL_ERR_INVALID_ARG;
    int sms = 0;
    if (rows == 0) {  // a sum over no rows
        const int rc = current_device_sms(&sms);
        if (rc != FP8LL_OK || accumulate) return rc;
        return cudaMemsetAsync(dgamma, 0, static_cast<size_t>(cols) * 4, reinterpret_cast<cudaStream_t>(stream)) ==
                       cudaSuccess
                   ? FP8LL_OK
                   : FP8LL_ERR_LAUNCH;
    }
    if (rows > (1LL << 31) - 1) return FP8LL_ERR_INVALID_ARG;
    if (!dy_bf16 || !h_bf16 || !gamma_bf16 || !rstd || !dx_bf16) return FP8LL_ERR_INVALID_ARG;
    if (!aligned(dy_bf16, 16) || !aligned(h_bf16, 16) || !aligned(gamma_bf16, 16) || !aligned(rstd, 4) ||
        !aligned(residual_grad_bf16, 16) || !aligned(dx_bf16, 16))
        return FP8LL_ERR_INVALID_ARG;
    if (lddy < cols || lddy % 8 != 0 || !spans(rows, lddy) || ldh < cols || ldh % 8 != 0 || !spans(rows, ldh))
        return FP8LL_ERR_INVALID_ARG;
    if (residual_grad_bf16 && (ldres < cols || ldres % 8 != 0 || !spans(rows, ldres))) return FP8LL_ERR_INVALID_ARG;
    const int64_t need = static_cast<int64_t>(fp8_rmsnorm_workspace_size(rows, cols));
    if (!workspace || !aligned(workspace, 16) || static_cast<int64_t>(workspace_bytes) < need)
        return FP8LL_ERR_WORKSPACE;
    const Range in[5] = {{dy_bf16, ((rows - 1) * lddy + cols) * 2},
                         {residual_grad_bf16, residual_grad_bf16 ? ((rows - 1) * ldres + cols) * 2 : 0},
                         {h_bf16, ((rows - 1) * ldh + cols) * 2},
                         {gamma_bf16, cols * 2},
                         {rstd, rows * 4}};
    const Range out[3] = {{dx_bf16, rows * cols * 2}, {dgamma, cols * 4}, {workspace, need}};
    for (int i = 0; i < 3; ++i) {
        for (int j = 0; j < 5; ++j) {
            // dx may take the place of dy or of the residual's gradient, element by element
            const bool in_place = i == 0 && ((j == 0 && dx_bf16 == dy_bf16 && lddy == cols) ||
                                             (j == 1 && dx_bf16 == residual_grad_bf16 && ldres == cols));
            if (share(out[i], in[j]) && !in_place) return FP8LL_ERR_INVALID_ARG;
        }
        for (int j = 0; j < i; ++j)
            if (share(out[i], out[j])) return FP8LL_ERR_INVALID_ARG;
    }
    const int rc = current_device_sms(&sms);
    if (rc != FP8LL_OK) return rc;
    RmsNormGradParams p = {};
    p.dy = static_cast<const uint16_t*>(dy_bf16);
    p.h = static_cast<const uint16_t*>(h_bf16);
    p.gamma = static_cast<const uint16_t*>(gamma_bf16);
    p.rstd = rstd;
    p.dres = static_cast<const uint16_t*>(residual_grad_bf16);
    p.rows = rows;
    p.cols = cols;
    p.lddy = lddy;
    p.ldh = ldh;
    p.ldres = ldres;
    p.dx = static_cast<uint16_t*>(dx_bf16);
    p.dgamma = dgamma;
    p.accumulate = accumulate;
    p.partials = static_cast<float*>(workspace);
    return launch_rmsnorm_grad(p, reinterpret_cast<cudaStream_t>(stream), sms) == 0 ? FP8LL_OK : FP8LL_ERR_LAUNCH;
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
