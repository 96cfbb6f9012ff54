"""RMS norm with the residual's addition and an fp8 output, and its backward
pass, against plain 64-bit forms."""
import numpy as np
import pytest
import torch

import block_reference as ref
from block_reference import U, f64

pytestmark = pytest.mark.gpu
EPS = 1e-6


def stream(rows, cols, seed, ld=None):
    """bf16 rows with a few large channels; an empty row where there are several."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, cols, generator=g)
    x[:, torch.randint(0, cols, (2,), generator=g)] *= 20.0
    if rows > 4:
        x[rows // 2] = 0.0
    x = x.bfloat16().cuda()
    if ld is not None:
        wide = torch.full((rows, ld), float("nan"), dtype=torch.bfloat16, device="cuda")
        wide[:, :cols] = x
        x = wide[:, :cols]
    return x


def scales(cols, seed):
    g = torch.Generator().manual_seed(seed)
    return (1.0 + 0.3 * torch.randn(cols, generator=g)).bfloat16().cuda()


def rstd_bound(cols):
    # squares and products round once each; at most ceil(cols / 8 / 32) * 8 terms follow one another in a thread and
    # ten shuffle levels add the threads: half of it is left by the root; the division, the sum with eps and the
    # reciprocal root (2 ulp) follow
    return ((min(cols, 64) + 12) / 2 + 2 + 4) * U


def call(f, recipe, x, gamma, fmt, residual, amax=None, **kw):
    if recipe == "tensor":
        return f.tensor_rmsnorm_quantize(x, gamma, EPS, fmt, amax, residual=residual, **kw)
    return (f.rmsnorm_quantize if recipe == "block" else f.mx_rmsnorm_quantize)(x, gamma, EPS, fmt, residual=residual,
                                                                               **kw)


SIZES = [(1, 128), (1, 4096), (3, 256), (5, 896), (130, 1152), (300, 4096), (77, 7168), (9, 14336), (2, 32768)]


@pytest.mark.parametrize("recipe", ["block", "mx", "tensor"])
@pytest.mark.parametrize("rows,cols", SIZES)
@pytest.mark.parametrize("with_residual", [False, True])
def test_row_codes(fp8, recipe, rows, cols, with_residual):
    fmt = rows % 2  # both formats
    x, gamma = stream(rows, cols, rows + cols, cols + 8 if rows % 3 == 0 else None), scales(cols, 1)
    r = stream(rows, cols, rows + cols + 1, cols + 64 if rows % 3 == 0 else None) if with_residual else None
    amax = torch.tensor([7.5], device="cuda")
    got = call(fp8, recipe, x, gamma, fmt, r, amax, y=True)
    torch.cuda.synchronize()
    h, rstd, y = ref.norm(x, r, gamma, EPS)
    if with_residual:
        assert torch.equal(got.h, (x.float() + r.float()).bfloat16())
    b = rstd_bound(cols)
    assert np.all(np.abs(f64(got.rstd) - rstd) <= b * rstd)
    rel = b + 2 * U  # two products
    ref.check_operand(got.rows, recipe, y, rel, "rows", amax=7.5)
    yb = f64(got.y)
    assert np.all(np.abs(yb - y) <= (2.0 ** -8 + rel) * np.abs(y))
    if recipe == "tensor":
        assert abs(got.amax.item() - np.abs(y).max()) <= rel * np.abs(y).max()


@pytest.mark.parametrize("recipe", ["block", "mx", "tensor"])
@pytest.mark.parametrize("rows,cols", [(128, 128), (256, 640), (384, 4096), (128, 14336)])
@pytest.mark.parametrize("with_residual", [False, True])
def test_both_orientations(fp8, recipe, rows, cols, with_residual):
    fmt = (cols // 128) % 2
    x, gamma = stream(rows, cols, 7, cols + 16 if rows == 256 else None), scales(cols, 2)
    r = stream(rows, cols, 8) if with_residual else None
    amax = torch.tensor([5.0], device="cuda")
    got = call(fp8, recipe, x, gamma, fmt, r, amax, cols=True)
    alone = call(fp8, recipe, x, gamma, fmt, r, amax, rows=False, cols=True)
    torch.cuda.synchronize()
    _, _, y = ref.norm(x, r, gamma, EPS)
    rel = rstd_bound(cols) + 2 * U
    ref.check_operand(got.rows, recipe, y, rel, "rows", amax=5.0)
    ref.check_operand(got.cols, recipe, y.T, rel, "columns", amax=5.0)
    assert torch.equal(alone.cols.q, got.cols.q) and alone.rows is None


def test_codes_are_the_cast_of_the_same_values(fp8):
    # the row codes of a norm whose fp32 output happens to be exact in bf16 are the cast kernel's codes
    x = torch.ones(4, 256, dtype=torch.bfloat16, device="cuda")
    gamma = torch.arange(1, 257, device="cuda").bfloat16()
    got = fp8.rmsnorm_quantize(x, gamma, 0.0, fp8.E4M3, y=True)
    cast = fp8.quantize(got.y, fp8.E4M3)
    assert torch.equal(got.y.float(), gamma.float().expand(4, 256)) and torch.equal(got.rows.q, cast.q)
    assert torch.equal(got.rows.scale[:, :4], cast.scale[:, :4])


@pytest.mark.parametrize("recipe", ["block", "mx", "tensor"])
def test_rstd_at_any_element(fp8, recipe):
    # rstd needs no more than its own alignment
    x, gamma, amax = stream(256, 384, 3), scales(384, 4), torch.tensor([6.0], device="cuda")
    want = call(fp8, recipe, x, gamma, 0, None, amax, cols=True)
    make = {"block": fp8.empty_rmsnorm, "mx": fp8.empty_mx_rmsnorm, "tensor": fp8.empty_tensor_rmsnorm}[recipe]
    out = make(256, 384, 0, cols_too=True)
    out.rstd = torch.zeros(259, device="cuda")[3:]
    got = call(fp8, recipe, x, gamma, 0, None, amax, out=out)
    dx, _ = fp8.rmsnorm_backward(x, x, gamma, out.rstd)
    want_dx, _ = fp8.rmsnorm_backward(x, x, gamma, want.rstd)
    torch.cuda.synchronize()
    assert torch.equal(got.rstd, want.rstd) and torch.equal(got.rows.q, want.rows.q)
    assert torch.equal(got.cols.q, want.cols.q) and torch.equal(dx, want_dx)


@pytest.mark.parametrize("onto", ["x", "residual"])
def test_stream_in_place(fp8, onto):
    x, r, gamma = stream(37, 1024, 3), stream(37, 1024, 4), scales(1024, 5)
    want = fp8.rmsnorm_quantize(x, gamma, EPS, fp8.E4M3, residual=r)
    out = fp8.empty_rmsnorm(37, 1024, fp8.E4M3, residual=True)
    x2, r2 = x.clone(), r.clone()
    out.h = x2 if onto == "x" else r2
    got = fp8.rmsnorm_quantize(x2, gamma, EPS, fp8.E4M3, residual=r2, out=out)
    assert torch.equal(got.h, want.h) and torch.equal(got.rows.q, want.rows.q)
    assert torch.equal(got.rstd, want.rstd) and torch.equal(r2 if onto == "x" else x2, r if onto == "x" else x)


def test_rows_with_nan_and_infinity_stay_alone(fp8):
    rows, cols = 40, 2048
    x, gamma = stream(rows, cols, 11), scales(cols, 12)
    clean = fp8.rmsnorm_quantize(x, gamma, EPS, fp8.E4M3)
    bad = x.clone()
    bad[3, 17], bad[9, 2000] = float("nan"), float("inf")
    got = fp8.rmsnorm_quantize(bad, gamma, EPS, fp8.E4M3)
    keep = [i for i in range(rows) if i not in (3, 9)]
    assert torch.equal(got.rows.q[keep], clean.rows.q[keep]) and torch.equal(got.rstd[keep], clean.rstd[keep])
    assert bool(got.rstd[3].isnan()) and got.rstd[9].item() == 0.0
    v = got.rows.q.view(torch.float8_e4m3fn).float()
    assert bool(v[3].isnan().all()) and bool(v[9, 2000].isnan()) and bool((v[9, :2000] == 0).all())


def test_empty_and_other_streams(fp8):
    gamma = scales(256, 1)
    none = fp8.rmsnorm_quantize(torch.empty(0, 256, dtype=torch.bfloat16, device="cuda"), gamma, EPS, fp8.E4M3)
    assert none.rows.q.shape == (0, 256)
    x = stream(512, 256, 2)
    want = fp8.rmsnorm_quantize(x, gamma, EPS, fp8.E4M3, cols=True)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        late = torch.zeros_like(x)
        torch.cuda._sleep(20_000_000)  # the input is written behind a wait of this stream
        late.copy_(x)
        got = fp8.rmsnorm_quantize(late, gamma, EPS, fp8.E4M3, cols=True)
    s.synchronize()
    assert torch.equal(got.rows.q, want.rows.q) and torch.equal(got.cols.q, want.cols.q)


def test_more_than_two_to_the_31_elements(fp8):
    rows, cols = 65664, 32768  # 2^31 and 4 Mi elements
    gamma = scales(cols, 1)
    x = torch.zeros(rows, cols, dtype=torch.bfloat16, device="cuda")
    tail = stream(128, cols, 5)
    x[-128:] = tail
    got = fp8.rmsnorm_quantize(x, gamma, EPS, fp8.E4M3, cols=True)
    want = fp8.rmsnorm_quantize(tail, gamma, EPS, fp8.E4M3, cols=True)
    torch.cuda.synchronize()
    assert torch.equal(got.rows.q[-128:], want.rows.q) and torch.equal(got.cols.q[:, -128:], want.cols.q)
    assert torch.equal(got.rows.scale[:, rows - 128:rows], want.rows.scale[:, :128])
    assert torch.equal(got.cols.scale[-1], want.cols.scale[0]) and not bool((got.rows.q[:-128] & 0x7F).any())
    dx, dgamma = fp8.rmsnorm_backward(x, x, gamma, got.rstd)
    wx, wg = fp8.rmsnorm_backward(tail, tail, gamma, want.rstd)
    torch.cuda.synchronize()
    assert torch.equal(dx[-128:], wx)
    assert torch.allclose(dgamma, wg, rtol=200 * U, atol=200 * U * float(wg.abs().max()))


# ---------------------------------------------------------------- backward --

def gradients(rows, cols, seed, ld=None):
    g = torch.Generator().manual_seed(seed)
    t = (0.01 * torch.randn(rows, ld or cols, generator=g)).bfloat16().cuda()
    return t[:, :cols]


def check_backward(got_dx, got_dg, dy, h, gamma, rstd, res, before=None):
    rows, cols = h.shape
    dx, size, dg, dg_size = ref.norm_backward(dy, h, gamma, rstd, res)
    # the mean: at most 64 terms follow one another, ten levels; a handful of products and sums around it
    bound = 2.0 ** -8 * np.abs(dx) + (2.0 ** -8 + 1) * 96 * U * size
    err = np.abs(f64(got_dx) - dx)
    assert np.all(err <= bound + 2.0 ** -134), float((err / (bound + 2.0 ** -134)).max())
    if before is not None:
        dg, dg_size = dg + f64(before), dg_size + np.abs(f64(before))
    # no order of adding `rows` products has more than rows + 2 roundings on a term's way
    assert np.all(np.abs(f64(got_dg) - dg) <= (rows + 4) * U * dg_size + 1e-40)


@pytest.mark.parametrize("rows,cols", [(1, 8), (1, 4096), (2, 24), (7, 520), (333, 1000), (1000, 2048), (64, 7168),
                                       (5, 14336), (3, 16392), (4, 32768), (2500, 136), (5001, 128),
                                       (700, 504), (31, 1024), (33, 8192), (9, 8200)])
@pytest.mark.parametrize("with_residual", [False, True])
def test_backward(fp8, rows, cols, with_residual):
    pad = 8 if rows % 2 else 0
    h, gamma = stream(rows, cols, 21, cols + pad if pad else None), scales(cols, 22)
    dy = gradients(rows, cols, 23, cols + 2 * pad)
    res = gradients(rows, cols, 24, cols + 3 * pad) if with_residual else None
    rstd = torch.rsqrt(h.float().square().mean(1) + EPS)
    dx, dg = fp8.rmsnorm_backward(dy, h, gamma, rstd, res)
    dx2, dg2 = fp8.rmsnorm_backward(dy, h, gamma, rstd, res)
    torch.cuda.synchronize()
    check_backward(dx, dg, dy, h, gamma, rstd, res)
    assert torch.equal(dx, dx2) and torch.equal(dg, dg2)  # the same order every time


def test_backward_accumulates_and_works_in_place(fp8):
    rows, cols = 200, 1024
    h, gamma, dy, res = stream(rows, cols, 1), scales(cols, 2), gradients(rows, cols, 3), gradients(rows, cols, 4)
    rstd = torch.rsqrt(h.float().square().mean(1) + EPS)
    want, _ = fp8.rmsnorm_backward(dy, h, gamma, rstd, res)
    before = torch.randn(cols, device="cuda")
    dg = before.clone()
    on_res, on_dy = res.clone(), dy.clone()
    fp8.rmsnorm_backward(dy, h, gamma, rstd, on_res, out=on_res, dgamma=dg, accumulate=True)
    fp8.rmsnorm_backward(on_dy, h, gamma, rstd, res, out=on_dy)
    torch.cuda.synchronize()
    assert torch.equal(on_res, want) and torch.equal(on_dy, want)
    check_backward(on_res, dg, dy, h, gamma, rstd, res, before)


def test_backward_of_no_rows(fp8):
    e = torch.empty(0, 256, dtype=torch.bfloat16, device="cuda")
    dg = torch.full((256,), 3.0, device="cuda")
    ws = torch.empty(4, device="cuda")
    fp8.rmsnorm_backward(e, e, scales(256, 1), torch.empty(0, device="cuda"), dgamma=dg, accumulate=True, workspace=ws)
    assert bool((dg == 3.0).all())
    fp8.rmsnorm_backward(e, e, scales(256, 1), torch.empty(0, device="cuda"), dgamma=dg, workspace=ws)
    assert bool((dg == 0.0).all())


def test_backward_against_differences(fp8):
    # sum(dy y(h)) in 64 bits, moved by a small step in h and in gamma
    rows, cols = 3, 256
    x, gamma, dy = stream(rows, cols, 31), scales(cols, 32), gradients(rows, cols, 33)
    fwd = fp8.rmsnorm_quantize(x, gamma, EPS, fp8.E4M3)
    dx, dg = fp8.rmsnorm_backward(dy, x, gamma, fwd.rstd)
    torch.cuda.synchronize()
    h, g, d = f64(x), f64(gamma), f64(dy)

    def loss(h, g):
        return float((d * h / np.sqrt((h * h).mean(1, keepdims=True) + EPS) * g).sum())

    t = 1e-5
    top = float(np.abs(f64(dx)).max())
    for i, j in [(0, 0), (1, 77), (2, 255), (0, 128)]:
        e = np.zeros_like(h)
        e[i, j] = t
        want = (loss(h + e, g) - loss(h - e, g)) / (2 * t)
        # central differences: t^2 of the third derivative and 1e-16 / t of the loss; the output is bf16
        assert abs(f64(dx)[i, j] - want) <= 2.0 ** -8 * abs(want) + 1e-6 * top
        e = np.zeros_like(g)
        e[j] = t
        want = (loss(h, g + e) - loss(h, g - e)) / (2 * t)
        assert abs(f64(dg)[j] - want) <= 1e-5 * abs(want) + 1e-8
