"""The operators of a pre-norm residual block around the FP8 linear layer:
RMS norm with the residual's addition and an fp8 output, its backward pass, the
matrix product with bias, activation and residual, and gradient clipping.

Argument marshalling only, as in ``binding``: every computation happens in the
CUDA library, on torch's current stream.
"""
import ctypes
from dataclasses import dataclass
from typing import Optional, Sequence

import torch

from . import binding as B
from .binding import (ACC_FULL, ACT_GELU, ACT_NONE, Fp8MxTensor, Fp8Tensor, Fp8TensorScaled, _check, _ptr, _stream,
                      empty_fp8, empty_mx, lib)


# -------------------------------------------------------------------- norm ----

@dataclass
class RmsNorm:
    """What a norm leaves: the residual stream h (with a residual; otherwise the
    stream is x, and h may be left out), rstd [rows], and the requested forms of its output: ``rows`` and
    ``cols`` (fp8 operands, ``cols`` the transposed one), ``y`` (bf16).
    ``amax`` [1]: max|y| (per-tensor scaling)."""
    h: Optional[torch.Tensor]
    rstd: torch.Tensor
    rows: Optional[object] = None
    cols: Optional[object] = None
    y: Optional[torch.Tensor] = None
    amax: Optional[torch.Tensor] = None


def _empty_norm(make, rows, cols, fmt, rows_too, cols_too, residual, y, device):
    stream = torch.empty((rows, cols), dtype=torch.bfloat16, device=device) if residual else None
    return RmsNorm(stream, torch.empty((rows,), dtype=torch.float32, device=device),
                   make(rows, cols, fmt, device) if rows_too else None,
                   make(cols, rows, fmt, device) if cols_too else None,
                   torch.empty((rows, cols), dtype=torch.bfloat16, device=device) if y else None)


def empty_rmsnorm(rows: int, cols: int, fmt: int, rows_too: bool = True, cols_too: bool = False,
                  residual: bool = False, y: bool = False, device="cuda") -> RmsNorm:
    """Outputs of ``rmsnorm_quantize``, to be used call after call."""
    return _empty_norm(empty_fp8, rows, cols, fmt, rows_too, cols_too, residual, y, device)


def empty_mx_rmsnorm(rows: int, cols: int, fmt: int, rows_too: bool = True, cols_too: bool = False,
                     residual: bool = False, y: bool = False, device="cuda") -> RmsNorm:
    """Outputs of ``mx_rmsnorm_quantize``."""
    return _empty_norm(empty_mx, rows, cols, fmt, rows_too, cols_too, residual, y, device)


def empty_tensor_rmsnorm(rows: int, cols: int, fmt: int, rows_too: bool = True, cols_too: bool = False,
                         residual: bool = False, y: bool = False, device="cuda") -> RmsNorm:
    """Outputs of ``tensor_rmsnorm_quantize``: both orientations share one scale."""
    scale = torch.empty((1,), dtype=torch.float32, device=device)

    def make(r, k, f, dev):
        return Fp8TensorScaled(torch.empty((r, k), dtype=torch.uint8, device=dev), scale, f)

    out = _empty_norm(make, rows, cols, fmt, rows_too, cols_too, residual, y, device)
    out.amax = torch.empty((1,), dtype=torch.float32, device=device)
    return out


def _norm_args(x, gamma, eps, fmt, residual, out):
    assert x.dtype == torch.bfloat16 and x.dim() == 2 and x.stride(1) == 1
    rows, cols = x.shape
    assert gamma.dtype == torch.bfloat16 and gamma.is_contiguous() and gamma.numel() == cols
    if residual is not None:
        assert residual.dtype == torch.bfloat16 and residual.shape == x.shape and residual.stride(1) == 1
        assert out.h is not None, "the sum x + residual needs its place (h)"
    for t in (out.h, out.y):
        assert t is None or (t.dtype == torch.bfloat16 and t.shape == x.shape and t.is_contiguous())
    assert out.rstd.dtype == torch.float32 and out.rstd.is_contiguous() and out.rstd.numel() == rows
    for t, shape in ((out.rows, (rows, cols)), (out.cols, (cols, rows))):
        assert t is None or (t.fmt == fmt and tuple(t.q.shape) == shape and t.q.is_contiguous())
    return (_ptr(x), _ptr(residual), _ptr(gamma), rows, cols, x.stride(0) if rows > 1 else cols,
            (residual.stride(0) if rows > 1 else cols) if residual is not None else 0, float(eps), int(fmt))


def _operand_ptrs(t, scale):
    return (None, None) if t is None else (_ptr(t.q), _ptr(getattr(t, scale)))


def rmsnorm_quantize(x: torch.Tensor, gamma: torch.Tensor, eps: float, fmt: int,
                     residual: Optional[torch.Tensor] = None, out: Optional[RmsNorm] = None, rows: bool = True,
                     cols: bool = False, y: bool = False) -> RmsNorm:
    """h = x + residual (bf16), then its RMS norm y = h rstd gamma cast from
    fp32 with one scale per 128 elements: row codes for the forward product
    (``rows``), transposed codes for the weight gradient (``cols``), bf16
    (``y``).  With ``out`` its buffers are used, and say which forms are made."""
    if out is None:
        out = empty_rmsnorm(x.shape[0], x.shape[1], fmt, rows, cols, residual is not None, y, x.device)
    args = _norm_args(x, gamma, eps, fmt, residual, out)
    qr, sr = _operand_ptrs(out.rows, "scale")
    qc, sc = _operand_ptrs(out.cols, "scale")
    _check(lib().fp8_rmsnorm_quantize(*args, _ptr(out.h), _ptr(out.rstd), _ptr(out.y), qr, sr,
                                      out.rows.scale.stride(0) if qr else 0, qc, sc,
                                      out.cols.scale.stride(0) if qc else 0, _stream()), "fp8_rmsnorm_quantize")
    return out


def mx_rmsnorm_quantize(x: torch.Tensor, gamma: torch.Tensor, eps: float, fmt: int,
                        residual: Optional[torch.Tensor] = None, out: Optional[RmsNorm] = None, rows: bool = True,
                        cols: bool = False, y: bool = False) -> RmsNorm:
    """``rmsnorm_quantize`` with MXFP8 operands (one power-of-two scale per 32 elements)."""
    if out is None:
        out = empty_mx_rmsnorm(x.shape[0], x.shape[1], fmt, rows, cols, residual is not None, y, x.device)
    args = _norm_args(x, gamma, eps, fmt, residual, out)
    _check(lib().fp8_mx_rmsnorm_quantize(*args, _ptr(out.h), _ptr(out.rstd), _ptr(out.y),
                                         *_operand_ptrs(out.rows, "sf"), *_operand_ptrs(out.cols, "sf"), _stream()),
           "fp8_mx_rmsnorm_quantize")
    return out


def tensor_rmsnorm_quantize(x: torch.Tensor, gamma: torch.Tensor, eps: float, fmt: int, amax_in: torch.Tensor,
                            residual: Optional[torch.Tensor] = None, out: Optional[RmsNorm] = None,
                            rows: bool = True, cols: bool = False, y: bool = False) -> RmsNorm:
    """``rmsnorm_quantize`` with one scale for the tensor, made of ``amax_in``
    (a 1-element device tensor: the largest amax of earlier steps); ``amax``
    of the result receives this call's max|y|."""
    if out is None:
        out = empty_tensor_rmsnorm(x.shape[0], x.shape[1], fmt, rows, cols, residual is not None, y, x.device)
    args = _norm_args(x, gamma, eps, fmt, residual, out)
    assert amax_in.dtype == torch.float32 and amax_in.numel() == 1
    made = [t for t in (out.rows, out.cols) if t is not None]
    assert len(made) < 2 or made[0].scale.data_ptr() == made[1].scale.data_ptr(), "both orientations share one scale"
    scale = made[0].scale if made else torch.empty((1,), dtype=torch.float32, device=x.device)
    _check(lib().fp8_tensor_rmsnorm_quantize(*args, _ptr(amax_in), _ptr(out.h), _ptr(out.rstd), _ptr(out.y),
                                             _ptr(out.rows.q) if out.rows is not None else None,
                                             _ptr(out.cols.q) if out.cols is not None else None, _ptr(scale),
                                             _ptr(out.amax), _stream()), "fp8_tensor_rmsnorm_quantize")
    return out


def rmsnorm_workspace(rows: int, cols: int, device="cuda") -> torch.Tensor:
    """Workspace of ``rmsnorm_backward``."""
    return torch.empty((int(lib().fp8_rmsnorm_workspace_size(int(rows), int(cols))) // 4,), dtype=torch.float32,
                       device=device)


def rmsnorm_backward(dy: torch.Tensor, h: torch.Tensor, gamma: torch.Tensor, rstd: torch.Tensor,
                     residual_grad: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                     dgamma: Optional[torch.Tensor] = None, accumulate: bool = False,
                     workspace: Optional[torch.Tensor] = None):
    """(dx, dgamma) of y = h rstd gamma: dx (bf16) is the gradient of h, with the
    gradient that reaches h around the norm (``residual_grad``) added; dgamma
    (fp32) is written, or added to with ``accumulate``."""
    assert h.dim() == 2 and dy.shape == h.shape and dy.dtype == h.dtype == torch.bfloat16
    assert dy.stride(1) == 1 and h.stride(1) == 1
    rows, cols = h.shape
    assert gamma.dtype == torch.bfloat16 and gamma.is_contiguous() and gamma.numel() == cols
    assert rstd.dtype == torch.float32 and rstd.is_contiguous() and rstd.numel() == rows
    r = residual_grad
    assert r is None or (r.dtype == torch.bfloat16 and r.shape == h.shape and r.stride(1) == 1)
    if out is None:
        out = torch.empty((rows, cols), dtype=torch.bfloat16, device=h.device)
    if dgamma is None:
        assert not accumulate, "accumulate needs dgamma"
        dgamma = torch.empty((cols,), dtype=torch.float32, device=h.device)
    if workspace is None:
        workspace = rmsnorm_workspace(rows, cols, h.device)
    assert out.dtype == torch.bfloat16 and out.shape == h.shape and out.is_contiguous()
    assert dgamma.dtype == torch.float32 and dgamma.is_contiguous() and dgamma.numel() == cols

    def ld(t):
        return t.stride(0) if rows > 1 else cols

    _check(lib().fp8_rmsnorm_backward(_ptr(dy), _ptr(h), _ptr(gamma), _ptr(rstd), _ptr(r), rows, cols, ld(dy), ld(h),
                                      ld(r) if r is not None else 0, _ptr(out), _ptr(dgamma), int(bool(accumulate)),
                                      _ptr(workspace), workspace.numel() * workspace.element_size(), _stream()),
           "fp8_rmsnorm_backward")
    return out, dgamma


# ----------------------------------------------------------------- product ----

def _linear_args(M, N, bias, act, residual, out, aux, want_aux, device):
    if out is None:
        out = torch.empty((M, N), dtype=torch.bfloat16, device=device)
    if aux is None and want_aux:
        assert act == ACT_GELU, "only an activation has a pre-activation to keep"
        aux = torch.empty((M, N), dtype=torch.bfloat16, device=device)
    for t in (out, aux):
        assert t is None or (t.dtype == torch.bfloat16 and tuple(t.shape) == (M, N) and t.is_contiguous())
    assert bias is None or (bias.dtype == torch.bfloat16 and bias.is_contiguous() and bias.numel() == N)
    ldr = 0
    if residual is not None:
        assert residual.dtype == torch.bfloat16 and tuple(residual.shape) == (M, N)
        assert N == 1 or residual.stride(1) == 1
        ldr = residual.stride(0) if M > 1 else N
    return out, aux, (_ptr(bias), int(act), _ptr(residual), ldr)


def gemm_linear(A: Fp8Tensor, W: Fp8Tensor, bias: Optional[torch.Tensor] = None, act: int = ACT_NONE,
                residual: Optional[torch.Tensor] = None, acc: int = ACC_FULL, out: Optional[torch.Tensor] = None,
                aux: Optional[torch.Tensor] = None, want_aux: bool = False):
    """Y (bf16 [M][N]) = act(A W^T + bias) + residual, rounded once; returns (Y,
    Z-or-None), Z = A W^T + bias with ``want_aux`` or ``aux`` (GELU only).
    ``out`` may be the residual itself.  Few rows run a kernel of their own."""
    M, N = A.rows, W.rows
    out, aux, args = _linear_args(M, N, bias, act, residual, out, aux, want_aux, A.q.device)
    assert A.k == W.k
    oa, ob = A.operand(), W.operand()
    _check(lib().fp8_gemm_linear(M, N, A.k, ctypes.byref(oa), ctypes.byref(ob), *args, int(acc), _ptr(out),
                                 _ptr(aux), _stream()), "fp8_gemm_linear")
    return out, aux


def mx_gemm_linear(A: Fp8MxTensor, W: Fp8MxTensor, bias: Optional[torch.Tensor] = None, act: int = ACT_NONE,
                   residual: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                   aux: Optional[torch.Tensor] = None, want_aux: bool = False):
    """``gemm_linear`` on MXFP8 operands."""
    M, N = A.rows, W.rows
    out, aux, args = _linear_args(M, N, bias, act, residual, out, aux, want_aux, A.q.device)
    assert A.k == W.k
    oa, ob = A.operand(), W.operand()
    _check(lib().fp8_mx_gemm_linear(M, N, A.k, ctypes.byref(oa), ctypes.byref(ob), *args, _ptr(out), _ptr(aux),
                                    _stream()), "fp8_mx_gemm_linear")
    return out, aux


def tensor_gemm_linear(A: Fp8TensorScaled, W: Fp8TensorScaled, bias: Optional[torch.Tensor] = None,
                       act: int = ACT_NONE, residual: Optional[torch.Tensor] = None,
                       out: Optional[torch.Tensor] = None, aux: Optional[torch.Tensor] = None,
                       want_aux: bool = False):
    """``gemm_linear`` on per-tensor scaled operands."""
    M, N = A.rows, W.rows
    out, aux, args = _linear_args(M, N, bias, act, residual, out, aux, want_aux, A.q.device)
    assert A.k == W.k
    oa, ob = A.operand(), W.operand()
    _check(lib().fp8_tensor_gemm_linear(M, N, A.k, ctypes.byref(oa), ctypes.byref(ob), *args, _ptr(out), _ptr(aux),
                                        _stream()), "fp8_tensor_gemm_linear")
    return out, aux


# ---------------------------------------------------------------- clipping ----

class GradList:
    """The gradient tensors of a model (fp32 or bf16, contiguous), with where
    their clipped values go (``out``: the tensors themselves by default), the
    norm's place on the device and the workspace: built once, used every step.
    It holds the tensors; what they contain is read at each call."""

    def __init__(self, grads: Sequence[torch.Tensor], out: Optional[Sequence[torch.Tensor]] = None):
        self.grads = list(grads)
        self.out = self.grads if out is None else list(out)
        assert len(self.out) == len(self.grads)
        for g, o in zip(self.grads, self.out):
            assert g.dtype in (torch.float32, torch.bfloat16) and g.is_contiguous()
            assert o.dtype == g.dtype and o.shape == g.shape and o.is_contiguous() and o.device == g.device
            assert g.device == self.grads[0].device
        device = self.grads[0].device if self.grads else torch.device("cuda")
        self.table = (B.GradStruct * len(self.grads))(*[
            B.GradStruct(g.data_ptr(), o.data_ptr(), g.numel(), B.F32 if g.dtype == torch.float32 else B.BF16, 0)
            for g, o in zip(self.grads, self.out)])
        self.norm = torch.empty((1,), dtype=torch.float32, device=device)
        self.workspace = torch.empty((int(lib().fp8_grad_norm_workspace_size(len(self.grads))) // 4,),
                                     dtype=torch.float32, device=device)

    def _tail(self):
        return _ptr(self.norm), _ptr(self.workspace), self.workspace.numel() * 4, _stream()


def grad_norm(grads) -> torch.Tensor:
    """The L2 norm over all elements of all tensors (a ``GradList`` or a
    sequence of tensors), as a 1-element fp32 device tensor."""
    g = grads if isinstance(grads, GradList) else GradList(grads)
    _check(lib().fp8_grad_norm(len(g.grads), g.table, *g._tail()), "fp8_grad_norm")
    return g.norm


def clip_grads(grads, max_norm: float) -> torch.Tensor:
    """Scales every tensor by min(1, max_norm / (norm + 1e-6)), norm the L2 norm
    over all of them, and returns the norm (device, 1 element)."""
    g = grads if isinstance(grads, GradList) else GradList(grads)
    _check(lib().fp8_clip_grads(len(g.grads), g.table, float(max_norm), *g._tail()), "fp8_clip_grads")
    return g.norm
