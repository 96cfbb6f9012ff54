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
from .binding import (ACC_FULL, ACT_GELU, ACT_NONE, Fp8MxTensor, Fp8Tensor, Fp8TensorScaled, _check, empty_fp8,
                      empty_mx, lib)

_bf16, _f32, _u8 = torch.bfloat16, torch.float32, torch.uint8
_C = torch._C


def _stream() -> int:
    """torch's current stream as the address that the library takes (the same
    stream as ``torch.cuda.current_stream()``, without building its object: a
    call of few tokens is bound by what the host does)."""
    return _C._cuda_getCurrentRawStream(_C._cuda_getDevice())


def _ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    """Address of a tensor on the GPU (or none): the kernels take no host memory."""
    if t is None:
        return None
    assert t.is_cuda
    return t.data_ptr()


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


def _rows(t, shape):
    """Leading dimension of a bf16 matrix of this shape with packed rows, on the GPU."""
    ld, one = t.stride()
    assert t.dtype is _bf16 and t.shape == shape and (one == 1 or shape[1] == 1) and t.is_cuda
    return ld if shape[0] > 1 else shape[1]


def _packed(t, dtype, shape):
    """Address of a contiguous tensor of this type and shape, on the GPU (or none)."""
    if t is None:
        return None
    assert t.dtype is dtype and t.shape == shape and t.is_contiguous() and t.is_cuda
    return t.data_ptr()


def _norm_args(x, shape, gamma, eps, fmt, residual, out):
    rows, cols = shape
    ldx, ldr = _rows(x, shape), 0
    if residual is not None:
        ldr = _rows(residual, shape)
        assert out.h is not None, "the sum x + residual needs its place (h)"
    return (x.data_ptr(), None if residual is None else residual.data_ptr(), _packed(gamma, _bf16, (cols,)), rows, cols,
            ldx, ldr, eps, fmt)


def _norm_outs(shape, out):
    return _packed(out.h, _bf16, shape), _packed(out.rstd, _f32, (shape[0],)), _packed(out.y, _bf16, shape)


def _codes(t, fmt, rows, cols):
    assert t.fmt == fmt
    return _packed(t.q, _u8, (rows, cols))


def rmsnorm_quantize(x: torch.Tensor, gamma: torch.Tensor, eps: float, fmt: int,
                     residual: Optional[torch.Tensor] = None, out: Optional[RmsNorm] = None, rows: bool = True,
                     cols: bool = False, y: bool = False) -> RmsNorm:
    """h = x + residual (bf16), then its RMS norm y = h rstd gamma cast from
    fp32 with one scale per 128 elements: row codes for the forward product
    (``rows``), transposed codes for the weight gradient (``cols``), bf16
    (``y``).  With ``out`` its buffers are used, and say which forms are made."""
    shape = x.shape
    m, k = shape
    if out is None:
        out = empty_rmsnorm(m, k, fmt, rows, cols, residual is not None, y, x.device)
    args = _norm_args(x, shape, gamma, eps, fmt, residual, out)
    qr = sr = qc = sc = None
    ldr = ldc = 0
    if out.rows is not None:
        qr, sr, ldr = _codes(out.rows, fmt, m, k), _ptr(out.rows.scale), out.rows.scale.stride()[0]
    if out.cols is not None:
        qc, sc, ldc = _codes(out.cols, fmt, k, m), _ptr(out.cols.scale), out.cols.scale.stride()[0]
    _check(lib().fp8_rmsnorm_quantize(*args, *_norm_outs(shape, out), qr, sr, ldr, qc, sc, ldc, _stream()),
           "fp8_rmsnorm_quantize")
    return out


def mx_rmsnorm_quantize(x: torch.Tensor, gamma: torch.Tensor, eps: float, fmt: int,
                        residual: Optional[torch.Tensor] = None, out: Optional[RmsNorm] = None, rows: bool = True,
                        cols: bool = False, y: bool = False) -> RmsNorm:
    """``rmsnorm_quantize`` with MXFP8 operands (one power-of-two scale per 32 elements)."""
    shape = x.shape
    m, k = shape
    if out is None:
        out = empty_mx_rmsnorm(m, k, fmt, rows, cols, residual is not None, y, x.device)
    args = _norm_args(x, shape, gamma, eps, fmt, residual, out)
    qr = sr = qc = sc = None
    if out.rows is not None:
        qr, sr = _codes(out.rows, fmt, m, k), _ptr(out.rows.sf)
    if out.cols is not None:
        qc, sc = _codes(out.cols, fmt, k, m), _ptr(out.cols.sf)
    _check(lib().fp8_mx_rmsnorm_quantize(*args, *_norm_outs(shape, out), qr, sr, qc, sc, _stream()),
           "fp8_mx_rmsnorm_quantize")
    return out


def tensor_rmsnorm_quantize(x: torch.Tensor, gamma: torch.Tensor, eps: float, fmt: int, amax_in: torch.Tensor,
                            residual: Optional[torch.Tensor] = None, out: Optional[RmsNorm] = None,
                            rows: bool = True, cols: bool = False, y: bool = False) -> RmsNorm:
    """``rmsnorm_quantize`` with one scale for the tensor, made of ``amax_in``
    (a 1-element device tensor: the largest amax of earlier steps); ``amax``
    of the result receives this call's max|y|."""
    shape = x.shape
    m, k = shape
    if out is None:
        out = empty_tensor_rmsnorm(m, k, fmt, rows, cols, residual is not None, y, x.device)
    args = _norm_args(x, shape, gamma, eps, fmt, residual, out)
    assert amax_in.dtype is _f32 and amax_in.numel() == 1 and amax_in.is_cuda
    qr = qc = scale = spare = None
    if out.rows is not None:
        qr, scale = _codes(out.rows, fmt, m, k), _ptr(out.rows.scale)
    if out.cols is not None:
        qc = _codes(out.cols, fmt, k, m)
        assert scale in (None, out.cols.scale.data_ptr()), "both orientations share one scale"
        scale = _ptr(out.cols.scale)
    if scale is None:  # only the bf16 form was asked for
        spare = torch.empty((1,), dtype=_f32, device=x.device)
        scale = spare.data_ptr()
    _check(lib().fp8_tensor_rmsnorm_quantize(*args, amax_in.data_ptr(), *_norm_outs(shape, out), qr, qc, scale,
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
    shape = h.shape
    rows, cols = shape
    r = residual_grad
    ldd, ldh, ldr = _rows(dy, shape), _rows(h, shape), 0 if r is None else _rows(r, shape)
    if out is None:
        out = torch.empty((rows, cols), dtype=_bf16, device=h.device)
    if dgamma is None:
        assert not accumulate, "accumulate needs dgamma"
        dgamma = torch.empty((cols,), dtype=_f32, device=h.device)
    if workspace is None:
        workspace = rmsnorm_workspace(rows, cols, h.device)
    assert workspace.is_contiguous() and workspace.is_cuda
    _check(lib().fp8_rmsnorm_backward(dy.data_ptr(), h.data_ptr(), _packed(gamma, _bf16, (cols,)),
                                      _packed(rstd, _f32, (rows,)), _ptr(r), rows, cols, ldd, ldh, ldr,
                                      _packed(out, _bf16, shape), _packed(dgamma, _f32, (cols,)), int(accumulate),
                                      workspace.data_ptr(), workspace.nbytes, _stream()),
           "fp8_rmsnorm_backward")
    return out, dgamma


# ----------------------------------------------------------------- product ----

def _linear_args(A, W, scales, bias, act, residual, out, aux, want_aux):
    """(Y, Z, the arguments in front of the operands, behind them, the outputs)"""
    (M, K), (N, KW) = A.q.shape, W.q.shape
    assert K == KW
    assert A.q.is_cuda and W.q.is_cuda and scales[0].is_cuda and scales[1].is_cuda
    if out is None:
        out = torch.empty((M, N), dtype=_bf16, device=A.q.device)
    if aux is None and want_aux:
        assert act == ACT_GELU, "only an activation has a pre-activation to keep"
        aux = torch.empty((M, N), dtype=_bf16, device=A.q.device)
    shape = (M, N)
    return (out, aux, (M, N, K), (_packed(bias, _bf16, (N,)), act, _ptr(residual),
                       0 if residual is None else _rows(residual, shape)),
            (_packed(out, _bf16, shape), _packed(aux, _bf16, shape)))


def gemm_linear(A: Fp8Tensor, W: Fp8Tensor, bias: Optional[torch.Tensor] = None, act: int = ACT_NONE,
                residual: Optional[torch.Tensor] = None, acc: int = ACC_FULL, out: Optional[torch.Tensor] = None,
                aux: Optional[torch.Tensor] = None, want_aux: bool = False):
    """Y (bf16 [M][N]) = act(A W^T + bias) + residual, rounded once; returns (Y,
    Z-or-None), Z = A W^T + bias with ``want_aux`` or ``aux`` (GELU only).
    ``out`` may be the residual itself.  Few rows run a kernel of their own."""
    out, aux, sizes, args, dst = _linear_args(A, W, (A.scale, W.scale), bias, act, residual, out, aux, want_aux)
    oa, ob = A.operand(), W.operand()
    _check(lib().fp8_gemm_linear(*sizes, ctypes.byref(oa), ctypes.byref(ob), *args, int(acc), *dst, _stream()),
           "fp8_gemm_linear")
    return out, aux


def mx_gemm_linear(A: Fp8MxTensor, W: Fp8MxTensor, bias: Optional[torch.Tensor] = None, act: int = ACT_NONE,
                   residual: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                   aux: Optional[torch.Tensor] = None, want_aux: bool = False):
    """``gemm_linear`` on MXFP8 operands."""
    out, aux, sizes, args, dst = _linear_args(A, W, (A.sf, W.sf), bias, act, residual, out, aux, want_aux)
    oa, ob = A.operand(), W.operand()
    _check(lib().fp8_mx_gemm_linear(*sizes, ctypes.byref(oa), ctypes.byref(ob), *args, *dst, _stream()),
           "fp8_mx_gemm_linear")
    return out, aux


def tensor_gemm_linear(A: Fp8TensorScaled, W: Fp8TensorScaled, bias: Optional[torch.Tensor] = None,
                       act: int = ACT_NONE, residual: Optional[torch.Tensor] = None,
                       out: Optional[torch.Tensor] = None, aux: Optional[torch.Tensor] = None,
                       want_aux: bool = False):
    """``gemm_linear`` on per-tensor scaled operands."""
    out, aux, sizes, args, dst = _linear_args(A, W, (A.scale, W.scale), bias, act, residual, out, aux, want_aux)
    oa, ob = A.operand(), W.operand()
    _check(lib().fp8_tensor_gemm_linear(*sizes, ctypes.byref(oa), ctypes.byref(ob), *args, *dst, _stream()),
           "fp8_tensor_gemm_linear")
    return out, aux


# ---------------------------------------------------------------- clipping ----

class GradList:
    """The gradient tensors of a model (fp32 or bf16, contiguous), with where
    their clipped values go (``out``: the tensors themselves by default), the
    norm's place on the device (``norm``, overwritten by each call) and the
    workspace: built once, used every step, by one call at a time.  It holds the
    tensors and their memory; what they contain is read at each call."""

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
        # the memory that the table points to stays allocated as long as the list,
        # whatever becomes of the tensors
        self._storages = [t.untyped_storage() for t in self.grads + self.out + [self.norm, self.workspace]]
        self._apart = self._outputs_apart()
        self._on_gpu = device.type == "cuda"  # all are on the device of the first
        self._tail = (self.norm.data_ptr(), self.workspace.data_ptr(), self.workspace.numel() * 4)

    def _outputs_apart(self) -> bool:
        # every place that clipping writes is apart from every other tensor of the
        # list (one listed twice would be scaled twice, in no certain order)
        spans = []
        for g, o in zip(self.grads, self.out):
            size = g.numel() * g.element_size()
            if size == 0:
                continue
            spans.append((o.data_ptr(), o.data_ptr() + size, True))
            if o.data_ptr() != g.data_ptr():
                spans.append((g.data_ptr(), g.data_ptr() + size, False))
        end, written = 0, 0  # of all spans so far, of those written to
        for lo, hi, writes in sorted(spans):
            if lo < (end if writes else written):
                return False
            end, written = max(end, hi), max(written, hi) if writes else written
        return True


def grad_norm(grads) -> torch.Tensor:
    """The L2 norm over all elements of all tensors (a ``GradList`` or a
    sequence of tensors), as a 1-element fp32 device tensor."""
    g = grads if isinstance(grads, GradList) else GradList(grads)
    assert g._on_gpu, "grad_norm: the tensors are not on the GPU"
    _check(lib().fp8_grad_norm(len(g.grads), g.table, *g._tail, _stream()), "fp8_grad_norm")
    return g.norm


def clip_grads(grads, max_norm: float) -> torch.Tensor:
    """Scales every tensor by min(1, max_norm / (norm + 1e-6)), norm the L2 norm
    over all of them, and returns the norm (device, 1 element).  No tensor may
    overlap another that is written to: a shared one is listed once."""
    g = grads if isinstance(grads, GradList) else GradList(grads)
    assert g._apart, "clip_grads: a tensor of the list overlaps another"
    assert g._on_gpu, "clip_grads: the tensors are not on the GPU"
    _check(lib().fp8_clip_grads(len(g.grads), g.table, float(max_norm), *g._tail, _stream()), "fp8_clip_grads")
    return g.norm
