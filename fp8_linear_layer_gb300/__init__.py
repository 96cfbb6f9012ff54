"""GB300 (sm_103a) block-scaled FP8 GEMMs for a training linear layer.

Y = X W^T + b: the forward GEMM with bias / tanh-GELU epilogues, the data-
gradient GEMM with the GELU-derivative and bias-gradient epilogue, and the
accumulating fp32 weight-gradient GEMM plus its k-grouped MoE variant (and the
same GEMMs on MXFP8 operands, scaled by the tensor core), all in
hand-written CUDA behind the C ABI of include/fp8ll.h.  Around the layer, the
operators of a pre-norm residual block: RMS and layer norm with the residual's
addition and an fp8 output, their backward passes, dropout whose mask is never
stored, the GEMM with bias, activation and residual and the gated GEMM (also for a
few tokens), the gated one's data gradient, and gradient clipping.  This package is the Python
binding (ctypes) over that library (``binding``, ``block``), the training step
of one layer (``linear``) and a feed-forward block (``feedforward``) built from
those calls.
"""
from .binding import (ACC_FAST, ACC_FULL, ACT_GELU, ACT_NONE, ACT_SILU, E4M3, E5M2, EPI_BIAS, EPI_BIAS_GELU, EPI_DGELU,
                      EPI_DGELU_BGRAD, EPI_NONE, EXPORTS, Fp8Error, Fp8Tensor, cast_f32, debug_starve_next_gemm, device_status,
                      empty_fp8, gemm_dgrad, gemm_dgrad_quant, gemm_fprop, gemm_wgrad, grouped_wgrad, lib, quantize, quantize_dual,
                      scale_ld, status_string, workspace_size, Fp8MxTensor, empty_mx, mx_gemm_dgrad, mx_gemm_fprop,
                      mx_gemm_wgrad, mx_quantize, mx_sf_bytes, Fp8TensorScaled, amax_history_update,
                      empty_tensor_scaled, tensor_amax, tensor_gemm_dgrad, tensor_gemm_fprop, tensor_gemm_wgrad,
                      tensor_quantize, bgrad_from_operand, quantize_dbias, mx_quantize_dbias)
from .block import (GradList, LayerNorm, RmsNorm, clip_grads, dropout, empty_layernorm, empty_mx_layernorm,
                    empty_mx_rmsnorm, empty_rmsnorm, empty_tensor_layernorm, empty_tensor_rmsnorm, gemm_gated,
                    gemm_gated_dgrad, gemm_linear, grad_norm, layernorm_backward, layernorm_quantize,
                    layernorm_workspace, mx_gemm_gated, mx_gemm_gated_dgrad, mx_gemm_linear,
                    mx_layernorm_quantize, mx_rmsnorm_quantize, rmsnorm_backward, rmsnorm_quantize,
                    rmsnorm_workspace, tensor_gemm_gated, tensor_gemm_gated_dgrad, tensor_gemm_linear,
                    tensor_layernorm_quantize, tensor_rmsnorm_quantize)

__all__ = ["ACC_FAST", "ACC_FULL", "ACT_GELU", "ACT_NONE", "E4M3", "E5M2", "EPI_BIAS", "EPI_BIAS_GELU", "EPI_DGELU", "EPI_DGELU_BGRAD",
           "EPI_NONE", "EXPORTS", "Fp8Error", "Fp8Tensor", "cast_f32", "debug_starve_next_gemm", "device_status",
           "empty_fp8", "gemm_dgrad", "gemm_dgrad_quant", "gemm_fprop", "gemm_wgrad", "grouped_wgrad", "lib", "quantize", "quantize_dual", "scale_ld",
           "status_string", "workspace_size", "Fp8MxTensor", "empty_mx", "mx_gemm_dgrad", "mx_gemm_fprop",
           "mx_gemm_wgrad", "mx_quantize", "mx_sf_bytes", "Fp8TensorScaled", "amax_history_update",
           "empty_tensor_scaled", "tensor_amax", "tensor_gemm_dgrad", "tensor_gemm_fprop", "tensor_gemm_wgrad",
           "tensor_quantize", "bgrad_from_operand", "quantize_dbias", "mx_quantize_dbias", "GradList", "RmsNorm",
           "clip_grads", "empty_mx_rmsnorm", "empty_rmsnorm", "empty_tensor_rmsnorm", "gemm_linear", "grad_norm",
           "mx_gemm_linear", "mx_rmsnorm_quantize", "rmsnorm_backward", "rmsnorm_quantize", "rmsnorm_workspace",
           "tensor_gemm_linear", "tensor_rmsnorm_quantize", "LayerNorm", "dropout", "empty_layernorm",
           "empty_mx_layernorm", "empty_tensor_layernorm", "layernorm_backward", "layernorm_quantize",
           "layernorm_workspace", "mx_layernorm_quantize", "tensor_layernorm_quantize", "ACT_SILU", "gemm_gated",
           "gemm_gated_dgrad", "mx_gemm_gated", "mx_gemm_gated_dgrad", "tensor_gemm_gated", "tensor_gemm_gated_dgrad"]
