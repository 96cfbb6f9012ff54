"""No write outside the outputs of the residual block's calls: each output is a
window into a larger allocation whose guards hold a sentinel, on ragged sizes
and through every kernel a size can reach."""
import pytest
import torch

import workloads
from test_gpu_canary import Guarded

pytestmark = pytest.mark.gpu
E4M3 = 0
RECIPES = ["block", "mx", "tensor"]


def operand(fp8, recipe, rows, k, scale=None):
    """An empty guarded operand with its guards."""
    q = Guarded((rows, k), torch.uint8)
    if recipe == "block":
        s = Guarded((k // 128, fp8.scale_ld(rows)), torch.float32)
        return fp8.Fp8Tensor(q.view, s.view, E4M3), [q, s]
    if recipe == "mx":
        s = Guarded((fp8.mx_sf_bytes(rows, k),), torch.uint8)
        return fp8.Fp8MxTensor(q.view, s.view, E4M3), [q, s]
    s = scale or Guarded((1,), torch.float32)
    return fp8.Fp8TensorScaled(q.view, s.view, E4M3), [q, s]


@pytest.mark.parametrize("recipe", RECIPES)
@pytest.mark.parametrize("rows,cols", [(1, 128), (5, 896), (131, 1152), (384, 384), (128, 4224), (3, 14336), (2, 32768)])
@pytest.mark.parametrize("y", [False, True])
def test_norm(fp8, recipe, rows, cols, y):
    x = workloads.normal_bf16((rows, cols), 710, "x").cuda()
    r = workloads.normal_bf16((rows, cols), 710, "r").cuda()
    gamma = workloads.normal_bf16((cols,), 710, "gamma").cuda()
    h, rstd = Guarded((rows, cols), torch.bfloat16), Guarded((rows,), torch.float32)
    guards = [h, rstd]
    scale = Guarded((1,), torch.float32)
    row_form, g = operand(fp8, recipe, rows, cols, scale)
    guards += g
    col_form = bf16 = amax = None
    if rows % 128 == 0:
        col_form, g = operand(fp8, recipe, cols, rows, scale)
        guards += g
    if y:
        bf16 = Guarded((rows, cols), torch.bfloat16)
        guards.append(bf16)
    out = fp8.RmsNorm(h.view, rstd.view, row_form, col_form, bf16.view if y else None)
    if recipe == "tensor":
        amax = Guarded((1,), torch.float32)
        guards.append(amax)
        out.amax = amax.view
        fp8.tensor_rmsnorm_quantize(x, gamma, 1e-6, E4M3, torch.tensor([4.0], device="cuda"), residual=r, out=out)
    else:
        call = fp8.rmsnorm_quantize if recipe == "block" else fp8.mx_rmsnorm_quantize
        call(x, gamma, 1e-6, E4M3, residual=r, out=out)
    assert all(v.intact() for v in guards)


@pytest.mark.parametrize("rows,cols", [(1, 8), (5, 264), (131, 1000), (700, 2056), (33, 8200), (9, 32768)])
def test_norm_backward(fp8, rows, cols):
    dy, h, res = (workloads.normal_bf16((rows, cols), 711, n).cuda() for n in ("dy", "h", "res"))
    gamma = workloads.normal_bf16((cols,), 711, "gamma").cuda()
    rstd = torch.ones(rows, device="cuda")
    dx, dgamma = Guarded((rows, cols), torch.bfloat16), Guarded((cols,), torch.float32)
    work = Guarded((fp8.rmsnorm_workspace(rows, cols).numel(),), torch.float32)
    for r in (None, res):
        fp8.rmsnorm_backward(dy, h, gamma, rstd, r, out=dx.view, dgamma=dgamma.view, workspace=work.view)
        assert dx.intact() and dgamma.intact() and work.intact()


@pytest.mark.parametrize("recipe", RECIPES)
@pytest.mark.parametrize("M,N,K", [(1, 13, 256), (5, 264, 1024), (31, 1001, 384), (65, 520, 1024), (129, 257, 128),
                                   (300, 520, 384), (600, 1023, 1024), (1000, 2110, 1664), (257, 1032, 2176)])
def test_linear_gemm(fp8, recipe, M, N, K):
    x = workloads.normal_bf16((M, K), 712, "x").cuda()
    w = workloads.normal_bf16((N, K), 712, "w", std=0.05).cuda()
    bias = workloads.normal_bf16((N,), 712, "b").cuda()
    res = workloads.normal_bf16((M, N), 712, "res").cuda()
    if recipe == "tensor":
        amax = torch.tensor([6.0], device="cuda")
        A, W = fp8.tensor_quantize(x, E4M3, amax)[0], fp8.tensor_quantize(w, E4M3, amax)[0]
        call = fp8.tensor_gemm_linear
    else:
        make, call = ((fp8.quantize, fp8.gemm_linear) if recipe == "block" else (fp8.mx_quantize, fp8.mx_gemm_linear))
        A, W = make(x, E4M3), make(w, E4M3)
    for act in (fp8.ACT_NONE, fp8.ACT_GELU):
        for r in (None, res):
            Y = Guarded((M, N), torch.bfloat16)
            Z = Guarded((M, N), torch.bfloat16) if act else None
            call(A, W, bias, act, r, out=Y.view, aux=Z.view if act else None)
            assert Y.intact() and (Z is None or Z.intact())
    assert fp8.device_status() == 0


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_clipping(fp8, dtype):
    sizes = (1, 7, 8193, 100003)
    grads, outs = [Guarded((n,), dtype) for n in sizes], [Guarded((n,), dtype) for n in sizes]
    for g in grads:
        g.view.fill_(0.5)
    plan = fp8.GradList([g.view for g in grads], [o.view for o in outs])
    fp8.clip_grads(plan, 1.0)
    assert all(v.intact() for v in grads + outs)
    fp8.clip_grads([g.view for g in grads], 1.0)
    assert all(g.intact() for g in grads)
