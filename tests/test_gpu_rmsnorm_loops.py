"""The norm's persistent loops: more rows than CTAs run at once, more tiles than
the column kernel's CTAs, in every kernel that a width reaches.  Neighbouring
rows differ in size, so that one row's sums or loads in another's place show."""
import numpy as np
import pytest
import torch

import block_reference as ref
from block_reference import U, f64
from test_gpu_rmsnorm import EPS, call, gradients, rstd_bound, scales, stream

pytestmark = pytest.mark.gpu


def uneven(rows, cols, seed, ld=None):
    x = stream(rows, cols, seed, ld)
    i = torch.arange(rows, device="cuda")
    x *= torch.exp2(((i * 5) % 11 - 5).float()).bfloat16()[:, None]  # exact; 5 i mod 11 differs by any step below 11
    return x


# one warp a row; a row per CTA with one, two and four vectors a thread; more than 512 threads
FORWARD = [(9733, 256), (2437, 1024), (1829, 2048), (917, 4096), (917, 7168), (309, 14336), (309, 32768)]


@pytest.mark.parametrize("recipe", ["block", "mx", "tensor"])
@pytest.mark.parametrize("rows,cols", FORWARD)
def test_rows(fp8, recipe, rows, cols):
    fmt = cols // 1024 % 2
    x, gamma = uneven(rows, cols, 31, cols + 8), scales(cols, 32)
    r = uneven(rows, cols, 33) if cols % 512 == 0 else None
    amax = torch.tensor([8.0], device="cuda")
    got = call(fp8, recipe, x, gamma, fmt, r, amax, y=True)
    torch.cuda.synchronize()
    h, rstd, y = ref.norm(x, r, gamma, EPS)
    if r is not None:
        assert torch.equal(got.h, (x.float() + r.float()).bfloat16())
    b = rstd_bound(cols)
    assert np.all(np.abs(f64(got.rstd) - rstd) <= b * rstd)
    rel = b + 2 * U
    assert np.all(np.abs(f64(got.y) - y) <= (2.0 ** -8 + rel) * np.abs(y))
    ref.check_operand(got.rows, recipe, y, rel, "rows", amax=8.0)
    if recipe == "tensor":
        assert abs(got.amax.item() - np.abs(y).max()) <= rel * np.abs(y).max()


@pytest.mark.parametrize("recipe", ["block", "mx", "tensor"])
@pytest.mark.parametrize("rows,cols", [(17 * 128, 4096), (17 * 128, 7168), (157 * 128, 1024), (9 * 128, 14336)])
def test_columns(fp8, recipe, rows, cols):
    fmt = rows // 128 % 3 == 0
    x, gamma = uneven(rows, cols, 41), scales(cols, 42)
    r = uneven(rows, cols, 43, cols + 16) if cols == 4096 else None
    amax = torch.tensor([8.0], device="cuda")
    got = call(fp8, recipe, x, gamma, int(fmt), r, amax, rows=False, cols=True)
    torch.cuda.synchronize()
    _, _, y = ref.norm(x, r, gamma, EPS)
    ref.check_operand(got.cols, recipe, np.ascontiguousarray(y.T), rstd_bound(cols) + 2 * U, "columns", amax=8.0)
    if recipe == "tensor":
        assert abs(got.amax.item() - np.abs(y).max()) <= (rstd_bound(cols) + 2 * U) * np.abs(y).max()


# rows, columns, rows of one CTA at a time (half a warp, a warp, a CTA each), CTAs per SM
BACKWARD = [(20001, 128, 16, 4), (10000, 256, 8, 4), (6000, 504, 8, 2), (3001, 1000, 8, 1), (1501, 2048, 1, 4),
            (701, 4096, 1, 2), (600, 7168, 1, 1), (401, 8200, 1, 1), (400, 14336, 1, 1), (401, 16392, 1, 1),
            (400, 32768, 1, 1)]


@pytest.mark.parametrize("rows,cols,per_cta,per_sm", BACKWARD)
def test_backward(fp8, rows, cols, per_cta, per_sm):
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    ctas = min(sms * per_sm, -(-rows // per_cta))
    assert rows > ctas * per_cta  # a second row for some
    pad = 8 if rows % 2 else 0
    h, gamma, dy = uneven(rows, cols, 51, cols + pad), scales(cols, 52), gradients(rows, cols, 53)
    res = gradients(rows, cols, 54, cols + 2 * pad) if cols % 1000 else None
    rstd = torch.rsqrt(h.float().square().mean(1) + EPS)
    before = torch.randn(cols, device="cuda", generator=torch.Generator(device="cuda").manual_seed(5))
    dgamma = before.clone()
    dx, _ = fp8.rmsnorm_backward(dy, h, gamma, rstd, res, dgamma=dgamma, accumulate=True)
    torch.cuda.synchronize()
    want, size, dg, dg_size = ref.norm_backward(dy, h, gamma, rstd, res)
    # the mean: at most 64 terms follow one another, ten levels; a handful of products and sums around it
    err, bound = np.abs(f64(dx) - want), 2.0 ** -8 * np.abs(want) + (2.0 ** -8 + 1) * 96 * U * size + 2.0 ** -134
    assert np.all(err <= bound), float((err / bound).max())
    # dgamma: a thread's rows one after another, the CTA's sums, every 32nd band, 32 of these sums; the product and
    # the sum with what was there round too
    steps = -(-rows // (ctas * per_cta)) + per_cta + -(-ctas // 32) + 32 + 4
    dg, dg_size = dg + f64(before), dg_size + np.abs(f64(before))
    err = np.abs(f64(dgamma) - dg)
    assert np.all(err <= steps * U * dg_size), float((err / (steps * U * dg_size)).max())
    again = before.clone()
    dx2, _ = fp8.rmsnorm_backward(dy, h, gamma, rstd, res, dgamma=again, accumulate=True)
    assert torch.equal(dx, dx2) and torch.equal(dgamma, again)
