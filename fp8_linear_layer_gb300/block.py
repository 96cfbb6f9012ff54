"""The operators of a pre-norm residual block around the FP8 linear layer:
RMS and layer norm with the residual's addition and an fp8 output, their backward
passes, dropout on the way into the residual stream, the matrix product with bias,
activation and residual, the gated product and its data gradient, and gradient
clipping.

Argument marshalling only, as in ``binding``: every computation happens in the
CUDA library, on torch's current stream.
"""
import ctypes
from dataclasses import dataclass
from typing import Optional, Sequence, Union

import torch

from . import binding as B
from .binding import (ACC_FULL, ACT_GELU, ACT_NONE, ACT_SILU, Fp8MxTensor, Fp8Tensor, Fp8TensorScaled, _check, empty_fp8,
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


# What the calls of the layer norm, of dropout and of the gated product check of a
# tensor: that it is on torch's current device, whose stream the call uses, its type
# and its size.  One pass over each tensor: a call of few tokens is bound by it.

def _current(t: torch.Tensor) -> int:
    """The current device, on which t is."""
    here = t.get_device()
    assert here >= 0 and here == _C._cuda_getDevice(), "the tensors are not on the current GPU"
    return here


def _vector(t, dtype, n, here):
    """Address of a contiguous tensor of n elements (or none)."""
    if t is None:
        return None
    assert t.numel() == n and t.dtype is dtype and t.is_contiguous() and t.get_device() == here
    return t.data_ptr()


def _matrix(t, dtype, shape, here):
    """Address of a contiguous tensor of this shape (or none)."""
    if t is None:
        return None
    assert t.shape == shape and t.dtype is dtype and t.is_contiguous() and t.get_device() == here
    return t.data_ptr()


def _strided(t, shape, here):
    """Address and leading dimension of a bf16 matrix with packed rows (or none)."""
    if t is None:
        return None, 0
    ld, one = t.stride()
    assert t.shape == shape and t.dtype is _bf16 and (one == 1 or shape[1] == 1) and t.get_device() == here
    return t.data_ptr(), ld if shape[0] > 1 else shape[1]


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


# -------------------------------------------------------------- layer norm ----

@dataclass
class LayerNorm(RmsNorm):
    """What a layer norm leaves: as ``RmsNorm``, and ``mean`` [rows]."""
    mean: Optional[torch.Tensor] = None


def _with_mean(n: RmsNorm) -> LayerNorm:
    return LayerNorm(n.h, n.rstd, n.rows, n.cols, n.y, n.amax, torch.empty_like(n.rstd))


def empty_layernorm(rows: int, cols: int, fmt: int, rows_too: bool = True, cols_too: bool = False,
                    residual: bool = False, y: bool = False, device="cuda") -> LayerNorm:
    """Outputs of ``layernorm_quantize``, to be used call after call."""
    return _with_mean(empty_rmsnorm(rows, cols, fmt, rows_too, cols_too, residual, y, device))


def empty_mx_layernorm(rows: int, cols: int, fmt: int, rows_too: bool = True, cols_too: bool = False,
                       residual: bool = False, y: bool = False, device="cuda") -> LayerNorm:
    """Outputs of ``mx_layernorm_quantize``."""
    return _with_mean(empty_mx_rmsnorm(rows, cols, fmt, rows_too, cols_too, residual, y, device))


def empty_tensor_layernorm(rows: int, cols: int, fmt: int, rows_too: bool = True, cols_too: bool = False,
                           residual: bool = False, y: bool = False, device="cuda") -> LayerNorm:
    """Outputs of ``tensor_layernorm_quantize``: both orientations share one scale."""
    return _with_mean(empty_tensor_rmsnorm(rows, cols, fmt, rows_too, cols_too, residual, y, device))


def _layernorm_args(x, gamma, beta, eps, fmt, residual, out):
    """(the current device, rows, columns, the arguments that the three recipes share, in front and behind)"""
    here, shape = _current(x), x.shape
    m, k = shape
    xp, ldx = _strided(x, shape, here)
    rp, ldr = _strided(residual, shape, here)
    assert residual is None or out.h is not None, "the sum x + residual needs its place (h)"
    return (here, m, k, (xp, rp, _vector(gamma, _bf16, k, here), _vector(beta, _bf16, k, here), m, k, ldx, ldr, eps, fmt),
            (_matrix(out.h, _bf16, shape, here), _vector(out.mean, _f32, m, here), _vector(out.rstd, _f32, m, here),
             _matrix(out.y, _bf16, shape, here)))


def _block_codes(t, fmt, shape, here):
    """(codes, scales, the scales' leading dimension) of an operand that a cast writes, or of none."""
    if t is None:
        return None, None, 0
    scale = t.scale
    (kb, rows), (ld, one) = scale.shape, scale.stride()
    assert t.fmt == fmt and scale.dtype is _f32 and one == 1 and kb == shape[1] // 128 and rows >= shape[0]
    assert scale.get_device() == here
    return _matrix(t.q, _u8, shape, here), scale.data_ptr(), ld


def _mx_bytes(rows, k):
    """``mx_sf_bytes`` of valid sizes, without a call into the library."""
    return k // 128 * (-(-rows // 256) * 1024)


def _mx_codes(t, fmt, shape, here):
    if t is None:
        return None, None
    assert t.fmt == fmt
    rows, k = shape
    return _matrix(t.q, _u8, shape, here), _vector(t.sf, _u8, _mx_bytes(rows, k), here)


def layernorm_quantize(x: torch.Tensor, gamma: torch.Tensor, beta: Optional[torch.Tensor], eps: float, fmt: int,
                       residual: Optional[torch.Tensor] = None, out: Optional[LayerNorm] = None, rows: bool = True,
                       cols: bool = False, y: bool = False) -> LayerNorm:
    """h = x + residual (bf16), then its layer norm y = (h - mean) rstd gamma + beta
    cast from fp32, as ``rmsnorm_quantize`` casts its output."""
    if out is None:
        out = empty_layernorm(*x.shape, fmt, rows, cols, residual is not None, y, x.device)
    here, m, k, args, outs = _layernorm_args(x, gamma, beta, eps, fmt, residual, out)
    _check(lib().fp8_layernorm_quantize(*args, *outs, *_block_codes(out.rows, fmt, (m, k), here),
                                        *_block_codes(out.cols, fmt, (k, m), here), _stream()),
           "fp8_layernorm_quantize")
    return out


def mx_layernorm_quantize(x: torch.Tensor, gamma: torch.Tensor, beta: Optional[torch.Tensor], eps: float, fmt: int,
                          residual: Optional[torch.Tensor] = None, out: Optional[LayerNorm] = None, rows: bool = True,
                          cols: bool = False, y: bool = False) -> LayerNorm:
    """``layernorm_quantize`` with MXFP8 operands (one power-of-two scale per 32 elements)."""
    if out is None:
        out = empty_mx_layernorm(*x.shape, fmt, rows, cols, residual is not None, y, x.device)
    here, m, k, args, outs = _layernorm_args(x, gamma, beta, eps, fmt, residual, out)
    _check(lib().fp8_mx_layernorm_quantize(*args, *outs, *_mx_codes(out.rows, fmt, (m, k), here),
                                           *_mx_codes(out.cols, fmt, (k, m), here), _stream()),
           "fp8_mx_layernorm_quantize")
    return out


def tensor_layernorm_quantize(x: torch.Tensor, gamma: torch.Tensor, beta: Optional[torch.Tensor], eps: float, fmt: int,
                              amax_in: torch.Tensor, residual: Optional[torch.Tensor] = None,
                              out: Optional[LayerNorm] = None, rows: bool = True, cols: bool = False,
                              y: bool = False) -> LayerNorm:
    """``layernorm_quantize`` with one scale for the tensor, made of ``amax_in`` (a
    1-element device tensor: the largest amax of earlier steps); ``amax`` of the
    result receives this call's max|y|."""
    if out is None:
        out = empty_tensor_layernorm(*x.shape, fmt, rows, cols, residual is not None, y, x.device)
    here, m, k, args, outs = _layernorm_args(x, gamma, beta, eps, fmt, residual, out)
    qr = qc = scale = None
    if out.rows is not None:
        assert out.rows.fmt == fmt
        qr, scale = _matrix(out.rows.q, _u8, (m, k), here), _vector(out.rows.scale, _f32, 1, here)
    if out.cols is not None:
        assert out.cols.fmt == fmt
        qc, other = _matrix(out.cols.q, _u8, (k, m), here), _vector(out.cols.scale, _f32, 1, here)
        assert scale in (None, other), "both orientations share one scale"
        scale = other
    if scale is None:  # only the bf16 form was asked for
        spare = torch.empty((1,), dtype=_f32, device=x.device)
        scale = spare.data_ptr()
    _check(lib().fp8_tensor_layernorm_quantize(*args, _vector(amax_in, _f32, 1, here), *outs, qr, qc, scale,
                                               _vector(out.amax, _f32, 1, here), _stream()),
           "fp8_tensor_layernorm_quantize")
    return out


def layernorm_workspace(rows: int, cols: int, device="cuda") -> torch.Tensor:
    """Workspace of ``layernorm_backward``."""
    return torch.empty((int(lib().fp8_layernorm_workspace_size(int(rows), int(cols))) // 4,), dtype=torch.float32,
                       device=device)


def layernorm_backward(dy: torch.Tensor, h: torch.Tensor, gamma: torch.Tensor, mean: torch.Tensor, rstd: torch.Tensor,
                       residual_grad: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                       dgamma: Optional[torch.Tensor] = None, dbeta: Optional[torch.Tensor] = None, bias: bool = True,
                       accumulate: bool = False, workspace: Optional[torch.Tensor] = None):
    """(dx, dgamma, dbeta) of y = (h - mean) rstd gamma + beta: dx (bf16) is the
    gradient of h, with the gradient that reaches h around the norm
    (``residual_grad``) added; dgamma and dbeta (fp32) are written, or added to
    with ``accumulate``.  Without ``bias`` the norm has no beta, and dbeta is None."""
    shape = h.shape
    rows, cols = shape
    r = residual_grad
    assert bias or dbeta is None, "a norm without bias has no dbeta"
    assert not accumulate or (dgamma is not None and (dbeta is not None or not bias)), "accumulate needs dgamma and dbeta"
    if out is None:
        out = torch.empty((rows, cols), dtype=_bf16, device=h.device)
    if dgamma is None:
        dgamma = torch.empty((cols,), dtype=_f32, device=h.device)
    if dbeta is None and bias:
        dbeta = torch.empty((cols,), dtype=_f32, device=h.device)
    if workspace is None:
        workspace = layernorm_workspace(rows, cols, h.device)
    here = _current(h)
    (hp, ldh), (dp, ldd), (rp, ldr) = _strided(h, shape, here), _strided(dy, shape, here), _strided(r, shape, here)
    assert workspace.is_contiguous() and workspace.get_device() == here
    _check(lib().fp8_layernorm_backward(dp, hp, _vector(gamma, _bf16, cols, here), _vector(mean, _f32, rows, here),
                                        _vector(rstd, _f32, rows, here), rp, rows, cols, ldd, ldh, ldr,
                                        _matrix(out, _bf16, shape, here), _vector(dgamma, _f32, cols, here),
                                        _vector(dbeta, _f32, cols, here), int(accumulate), workspace.data_ptr(),
                                        workspace.nbytes, _stream()), "fp8_layernorm_backward")
    return out, dgamma, dbeta


# ----------------------------------------------------------------- dropout ----

def dropout(x: torch.Tensor, p: float, seed: int, site: int = 0, step: Union[int, torch.Tensor] = 0,
            residual: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """residual + dropout(x) (bf16 [rows][cols]): an element of x is dropped with
    probability p, else scaled by 1 / (1 - p).  The mask is a function of the
    element's place in the matrix, of ``seed`` (of a run, 64 bits), ``site``
    (which dropout of the model, 32 bits) and ``step`` (64 bits; an int, or a
    1-element int64 device tensor that a captured step counts up), and is never
    stored: the gradient of x is this call on the output's gradient, with the same
    numbers and no residual.  ``out`` may be x or the residual itself."""
    here, shape = _current(x), x.shape
    rows, cols = shape
    (xp, ldx), (rp, ldr) = _strided(x, shape, here), _strided(residual, shape, here)
    assert 0 <= seed < 1 << 64 and 0 <= site < 1 << 32
    if out is None:
        out = torch.empty((rows, cols), dtype=_bf16, device=x.device)
    counter = None
    if isinstance(step, torch.Tensor):
        counter, step = _vector(step, torch.int64, 1, here), 0
    else:
        assert -(1 << 63) <= step < 1 << 63
    _check(lib().fp8_dropout(xp, rp, rows, cols, ldx, ldr, p, seed, site, step, counter,
                             _matrix(out, _bf16, shape, here), _stream()), "fp8_dropout")
    return out


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


# ----------------------------------------------------------- gated product ----

def _operand(t, kind, here):
    """(rows, K, the C struct) of an operand of the gated products."""
    assert type(t) is kind
    q = t.q
    (rows, k), (ld, one) = q.shape, q.stride()
    assert one == 1 and q.dtype is _u8 and q.get_device() == here
    if kind is Fp8Tensor:
        scale = t.scale
        (kb, n), (sld, one) = scale.shape, scale.stride()
        assert kb * 128 >= k and n >= rows and one == 1 and scale.dtype is _f32 and scale.get_device() == here
        return rows, k, B.OperandStruct(q.data_ptr(), scale.data_ptr(), ld, sld, t.fmt, 0)
    if kind is Fp8MxTensor:
        sf = t.sf
        assert sf.numel() >= _mx_bytes(rows, k) and sf.dtype is _u8 and sf.is_contiguous()
        assert sf.get_device() == here
        return rows, k, B.MxOperandStruct(q.data_ptr(), sf.data_ptr(), ld, t.fmt, 0)
    return rows, k, B.TensorOperandStruct(q.data_ptr(), _vector(t.scale, _f32, 1, here), ld, t.fmt, 0)


def _gated(kind, call, A, W, bias, act, acc, out, aux, want_aux):
    here = _current(A.q)
    (M, K, a), (R, KW, w) = _operand(A, kind, here), _operand(W, kind, here)
    N = R // 2
    assert K == KW and R == 2 * N, "W holds the gate's rows, then as many of the up projection"
    if out is None:
        out = torch.empty((M, N), dtype=_bf16, device=A.q.device)
    if aux is None and want_aux:
        aux = torch.empty((M, R), dtype=_bf16, device=A.q.device)
    _check(getattr(lib(), call)(M, N, K, ctypes.byref(a), ctypes.byref(w), _vector(bias, _bf16, R, here), act, *acc,
                                _matrix(out, _bf16, (M, N), here), _matrix(aux, _bf16, (M, R), here), _stream()), call)
    return out, aux


def gemm_gated(A: Fp8Tensor, W: Fp8Tensor, bias: Optional[torch.Tensor] = None, act: int = ACT_SILU,
               acc: int = ACC_FULL, out: Optional[torch.Tensor] = None, aux: Optional[torch.Tensor] = None,
               want_aux: bool = False):
    """Y (bf16 [M][N]) = act(Z[:, :N]) Z[:, N:] with Z = A W^T + bias [M][2 N], both
    projections in one kernel; W [2 N][K] holds the gate's rows, then the up
    projection's.  Returns (Y, Z-or-None), Z (bf16) with ``want_aux`` or ``aux`` for
    the backward pass.  act: ACT_SILU or ACT_GELU.  Few rows run a kernel of their own."""
    return _gated(Fp8Tensor, "fp8_gemm_gated", A, W, bias, act, (int(acc),), out, aux, want_aux)


def mx_gemm_gated(A: Fp8MxTensor, W: Fp8MxTensor, bias: Optional[torch.Tensor] = None, act: int = ACT_SILU,
                  out: Optional[torch.Tensor] = None, aux: Optional[torch.Tensor] = None, want_aux: bool = False):
    """``gemm_gated`` on MXFP8 operands."""
    return _gated(Fp8MxTensor, "fp8_mx_gemm_gated", A, W, bias, act, (), out, aux, want_aux)


def tensor_gemm_gated(A: Fp8TensorScaled, W: Fp8TensorScaled, bias: Optional[torch.Tensor] = None,
                      act: int = ACT_SILU, out: Optional[torch.Tensor] = None, aux: Optional[torch.Tensor] = None,
                      want_aux: bool = False):
    """``gemm_gated`` on per-tensor scaled operands."""
    return _gated(Fp8TensorScaled, "fp8_tensor_gemm_gated", A, W, bias, act, (), out, aux, want_aux)


def _gated_dgrad(kind, call, A, W, aux, act, acc, out):
    here = _current(A.q)
    (M, K, a), (N, KW, w) = _operand(A, kind, here), _operand(W, kind, here)
    assert K == KW
    if out is None:
        out = torch.empty((M, 2 * N), dtype=_bf16, device=A.q.device)
    _check(getattr(lib(), call)(M, N, K, ctypes.byref(a), ctypes.byref(w), _matrix(aux, _bf16, (M, 2 * N), here), act,
                                *acc, _matrix(out, _bf16, (M, 2 * N), here), _stream()), call)
    return out


def gemm_gated_dgrad(A: Fp8Tensor, W: Fp8Tensor, aux: torch.Tensor, act: int = ACT_SILU, acc: int = ACC_FULL,
                     out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """dZ (bf16 [M][2 N]), the gradient of ``gemm_gated``'s Z = ``aux``, from the
    gradient of its output, C = A W^T [M][N] (W: the second product's weight
    transposed): dZ[:, :N] = C Z[:, N:] act'(Z[:, :N]), dZ[:, N:] = C act(Z[:, :N]).
    ``out`` may be ``aux`` itself."""
    return _gated_dgrad(Fp8Tensor, "fp8_gemm_gated_dgrad", A, W, aux, act, (int(acc),), out)


def mx_gemm_gated_dgrad(A: Fp8MxTensor, W: Fp8MxTensor, aux: torch.Tensor, act: int = ACT_SILU,
                        out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """``gemm_gated_dgrad`` on MXFP8 operands."""
    return _gated_dgrad(Fp8MxTensor, "fp8_mx_gemm_gated_dgrad", A, W, aux, act, (), out)


def tensor_gemm_gated_dgrad(A: Fp8TensorScaled, W: Fp8TensorScaled, aux: torch.Tensor, act: int = ACT_SILU,
                            out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """``gemm_gated_dgrad`` on per-tensor scaled operands."""
    return _gated_dgrad(Fp8TensorScaled, "fp8_tensor_gemm_gated_dgrad", A, W, aux, act, (), out)


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
