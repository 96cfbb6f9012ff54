"""The norm of rows that hold nothing, without eps: zeros with scale 1, and a
backward pass that such rows leave alone."""
import numpy as np
import pytest
import torch

import block_reference as ref
from block_reference import U, f64
from test_gpu_rmsnorm import check_backward, gradients, rstd_bound, scales, stream

pytestmark = pytest.mark.gpu
CALLS = {"block": "rmsnorm_quantize", "mx": "mx_rmsnorm_quantize", "tensor": "tensor_rmsnorm_quantize"}


def norm(fp8, recipe, x, gamma, eps, fmt, residual=None, **kw):
    amax = (torch.tensor([9.0], device="cuda"),) if recipe == "tensor" else ()
    return getattr(fp8, CALLS[recipe])(x, gamma, eps, fmt, *amax, residual=residual, **kw)


def reference(x, residual, gamma):
    """The 64-bit norm with eps = 0, a row of zeros staying zeros."""
    h = f64(x if residual is None else (x.float() + residual.float()).bfloat16())
    ms = (h * h).mean(1)
    rstd = np.where(ms > 0, 1.0 / np.sqrt(np.where(ms > 0, ms, 1.0)), 0.0)
    return rstd, h * rstd[:, None] * f64(gamma)


@pytest.mark.parametrize("recipe", ["block", "mx", "tensor"])
@pytest.mark.parametrize("cols", [128, 1152, 4096, 7168, 32768])
@pytest.mark.parametrize("with_residual", [False, True])
def test_zero_rows_without_eps(fp8, recipe, cols, with_residual):
    rows, fmt = 128, (cols // 128) % 2
    x, gamma = stream(rows, cols, cols), scales(cols, 1)
    x[5] = 0.0
    x[9] = -0.0
    r = None
    if with_residual:
        r = stream(rows, cols, cols + 1)
        r[5], r[9], r[rows // 2] = 0.0, 0.0, 0.0
        r[77] = -x[77]  # cancels
    empty = [5, 9, rows // 2] + ([77] if with_residual else [])
    got = norm(fp8, recipe, x, gamma, 0.0, fmt, r, cols=True, y=True)
    torch.cuda.synchronize()
    rstd, y = reference(x, r, gamma)
    rel = rstd_bound(cols) + 2 * U
    assert bool((got.rstd[empty] == 0).all())
    assert np.all(np.abs(f64(got.rstd) - rstd) <= rel * rstd)
    assert np.all(np.abs(f64(got.y) - y) <= (2.0 ** -8 + rel) * np.abs(y))
    ref.check_operand(got.rows, recipe, y, rel, "rows", amax=9.0)
    ref.check_operand(got.cols, recipe, y.T, rel, "columns", amax=9.0)
    assert not bool((got.rows.q[empty] & 0x7F).any()) and not bool((got.cols.q[:, empty] & 0x7F).any())
    # the backward pass: such a row has the residual's gradient alone and adds nothing to dgamma
    h = x if r is None else got.h
    dy, res = gradients(rows, cols, 3), gradients(rows, cols, 4)
    dx, dgamma = fp8.rmsnorm_backward(dy, h, gamma, got.rstd, res)
    torch.cuda.synchronize()
    assert torch.equal(dx[empty], res[empty])
    check_backward(dx, dgamma, dy, h, gamma, got.rstd, res)


@pytest.mark.parametrize("recipe", ["block", "mx", "tensor"])
def test_squares_that_vanish_in_fp32(fp8, recipe):
    x, gamma = stream(4, 256, 1), scales(256, 2)
    x[2] = 2.0 ** -76  # squares below half of the smallest fp32
    got = norm(fp8, recipe, x, gamma, 0.0, fp8.E4M3, y=True)
    torch.cuda.synchronize()
    assert got.rstd[2].item() == 0.0 and not bool((got.rows.q[2] & 0x7F).any()) and not bool(got.y[2].any())
    assert bool(torch.isfinite(got.y.float()).all())


def test_a_nan_row_stays_one_without_eps(fp8):
    x, gamma = stream(4, 256, 1), scales(256, 2)
    x[1, 7] = float("nan")
    got = fp8.rmsnorm_quantize(x, gamma, 0.0, fp8.E4M3, y=True)
    assert bool(got.rstd[1].isnan()) and bool(got.y[1].isnan().all()) and bool(torch.isfinite(got.y[2].float()).all())
