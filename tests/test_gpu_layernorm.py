"""Layer norm with the residual's addition and an fp8 output, and its backward
pass, against plain 64-bit forms."""
import numpy as np
import pytest
import torch

import layernorm_reference as ref
from block_reference import U, f64

pytestmark = pytest.mark.gpu
EPS = 1e-5


def stream(rows, cols, seed, ld=None, centre=2.0):
    """bf16 rows off centre with a few large channels; an empty row and a constant one where there are several."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, cols, generator=g) + centre * torch.randn(rows, 1, generator=g)
    x[:, torch.randint(0, cols, (2,), generator=g)] *= 20.0
    if rows > 4:
        x[rows // 2] = 0.0
        x[rows // 3] = 1.2890625
    x = x.bfloat16().cuda()
    if ld is not None:
        wide = torch.full((rows, ld), float("nan"), dtype=torch.bfloat16, device="cuda")
        wide[:, :cols] = x
        x = wide[:, :cols]
    return x


def weights(cols, seed):
    g = torch.Generator().manual_seed(seed)
    return (1.0 + 0.3 * torch.randn(cols, generator=g)).bfloat16().cuda(), \
        (0.3 * torch.randn(cols, generator=g)).bfloat16().cuda()


def call(f, recipe, x, gamma, beta, fmt, residual, amax=None, eps=EPS, **kw):
    if recipe == "tensor":
        return f.tensor_layernorm_quantize(x, gamma, beta, eps, fmt, amax, residual=residual, **kw)
    return (f.layernorm_quantize if recipe == "block" else f.mx_layernorm_quantize)(x, gamma, beta, eps, fmt,
                                                                                   residual=residual, **kw)


SIZES = [(1, 128), (1, 4096), (3, 256), (5, 896), (130, 1152), (300, 4096), (77, 7168), (9, 14336), (2, 28672),
         (700, 2176), (3, 16512)]


@pytest.mark.parametrize("recipe", ["block", "mx", "tensor"])
@pytest.mark.parametrize("rows,cols", SIZES)
@pytest.mark.parametrize("with_residual", [False, True])
def test_row_codes(fp8, recipe, rows, cols, with_residual):
    fmt = rows % 2  # both formats
    x, (gamma, beta) = stream(rows, cols, rows + cols, cols + 8 if rows % 3 == 0 else None), weights(cols, 1)
    beta = beta if cols % 256 else None
    r = stream(rows, cols, rows + cols + 1, cols + 64 if rows % 3 == 0 else None) if with_residual else None
    amax = torch.tensor([7.5], device="cuda")
    got = call(fp8, recipe, x, gamma, beta, fmt, r, amax, y=True)
    torch.cuda.synchronize()
    h, mean, rstd, y, dmean, drstd, dy = ref.norm(x, r, gamma, beta, EPS)
    if with_residual:
        assert torch.equal(got.h, (x.float() + r.float()).bfloat16())
    assert np.all(np.abs(f64(got.mean) - mean) <= dmean)
    assert np.all(np.abs(f64(got.rstd) - rstd) <= drstd * rstd)
    ref.check_operand(got.rows, recipe, y, dy, "rows", amax=7.5)
    assert np.all(np.abs(f64(got.y) - y) <= 2.0 ** -8 * np.abs(y) + 1.01 * dy)
    if recipe == "tensor":
        assert abs(got.amax.item() - np.abs(y).max()) <= dy.max()


@pytest.mark.parametrize("recipe", ["block", "mx", "tensor"])
@pytest.mark.parametrize("rows,cols", [(128, 128), (256, 640), (384, 4096), (128, 14336), (1152, 384)])
@pytest.mark.parametrize("with_residual", [False, True])
def test_both_orientations(fp8, recipe, rows, cols, with_residual):
    fmt = (cols // 128) % 2
    x, (gamma, beta) = stream(rows, cols, 7, cols + 16 if rows == 256 else None), weights(cols, 2)
    gamma[5], beta[5], gamma[9] = 0.0, 0.0, -1.5
    r = stream(rows, cols, 8) if with_residual else None
    amax = torch.tensor([5.0], device="cuda")
    got = call(fp8, recipe, x, gamma, beta, fmt, r, amax, cols=True)
    alone = call(fp8, recipe, x, gamma, beta, fmt, r, amax, rows=False, cols=True)
    torch.cuda.synchronize()
    y, dy = ref.norm(x, r, gamma, beta, EPS)[3::3]
    ref.check_operand(got.rows, recipe, y, dy, "rows", amax=5.0)
    ref.check_operand(got.cols, recipe, y.T, dy.T, "columns", amax=5.0)
    assert torch.equal(alone.cols.q, got.cols.q) and alone.rows is None


@pytest.mark.parametrize("recipe", ["block", "mx", "tensor"])
def test_column_scales_are_those_of_the_values(fp8, recipe):
    # the columns' maxima come from the largest and smallest normalised value: the same as of all values, whatever the
    # signs of gamma and beta, and with NaN in gamma or beta
    rows, cols = 256, 384
    x, (gamma, beta) = stream(rows, cols, 3), weights(cols, 4)
    gamma[::3] *= -1
    beta *= 10
    gamma[7], beta[11], beta[12], gamma[13] = float("nan"), float("nan"), float("inf"), float("-inf")
    got = call(fp8, recipe, x, gamma, beta, 0, None, torch.tensor([4.0], device="cuda"), y=True, cols=True)
    # y is that fp32 value's bf16: as rows of the transpose, its own cast's maxima are within its rounding
    again = fp8.quantize(got.y.t().contiguous(), 0) if recipe == "block" else \
        fp8.mx_quantize(got.y.t().contiguous(), 0) if recipe == "mx" else None
    torch.cuda.synchronize()
    keep = [c for c in range(cols) if c not in (7, 11, 12, 13)]
    if recipe == "block":
        a, b = got.cols.scale[:, :cols], again.scale[:, :cols]
        assert torch.allclose(a[:, keep], b[:, keep], rtol=2.0 ** -8 + 8 * U)
        assert torch.equal(a[:, [7, 11, 12, 13]], b[:, [7, 11, 12, 13]])
    elif recipe == "mx":
        assert int((got.cols.sf.int() - again.sf.int()).abs().max()) <= 1
        byte = lambda sf, c: [sf.view(rows // 128, 4, 32, 4, 4)[k, c // 128, c % 32, c % 128 // 32].tolist()  # noqa: E731
                              for k in range(rows // 128)]
        for c in (7, 11, 12, 13):
            assert byte(got.cols.sf, c) == byte(again.sf, c)
    rows_q, cols_q = got.rows.q.view(torch.float8_e4m3fn).float(), got.cols.q.view(torch.float8_e4m3fn).float()
    if recipe == "tensor":  # one scale: the same codes in both orientations
        assert torch.equal(got.rows.q.t()[keep], got.cols.q[keep])
    assert bool(cols_q[7].isnan().all()) and bool(rows_q[:, 7].isnan().all())


@pytest.mark.parametrize("cols", [128, 1152, 4096, 14336])
@pytest.mark.parametrize("centre", [0.0, 100.0, 3e4])
def test_a_mean_far_from_zero(fp8, cols, centre):
    rows = 33
    x = (torch.randn(rows, cols, generator=torch.Generator().manual_seed(5)) * max(1.0, centre / 50) + centre).bfloat16()
    x, (gamma, beta) = x.cuda(), weights(cols, 6)
    got = fp8.layernorm_quantize(x, gamma, beta, EPS, fp8.E4M3, y=True)
    torch.cuda.synchronize()
    h, mean, rstd, y, dmean, drstd, dy = ref.norm(x, None, gamma, beta, EPS)
    assert np.all(np.abs(f64(got.mean) - mean) <= dmean) and np.all(np.abs(f64(got.rstd) - rstd) <= drstd * rstd)
    assert np.all(np.abs(f64(got.y) - y) <= 2.0 ** -8 * np.abs(y) + 1.01 * dy)
    ref.check_operand(got.rows, "block", y, dy, "rows")


def test_constant_rows_without_eps_give_beta(fp8):
    x = torch.full((6, 384), 3.140625, device="cuda").bfloat16()
    x[2] = 0.0
    gamma, beta = weights(384, 1)
    got = fp8.layernorm_quantize(x, gamma, beta, 0.0, fp8.E4M3, y=True)
    dx, dg, db = fp8.layernorm_backward(x, x, gamma, got.mean, got.rstd)
    torch.cuda.synchronize()
    assert torch.equal(got.y, beta.expand(6, 384)) and bool((got.rstd == 0).all()) and torch.equal(got.mean, x[:, 0].float())
    assert bool((dx == 0).all()) and bool((dg == 0).all()) and torch.equal(db, x.float().sum(0))


@pytest.mark.parametrize("recipe", ["block", "mx", "tensor"])
def test_statistics_at_any_element(fp8, recipe):
    x, (gamma, beta), amax = stream(256, 384, 3), weights(384, 4), torch.tensor([6.0], device="cuda")
    want = call(fp8, recipe, x, gamma, beta, 0, None, amax, cols=True)
    make = {"block": fp8.empty_layernorm, "mx": fp8.empty_mx_layernorm, "tensor": fp8.empty_tensor_layernorm}[recipe]
    out = make(256, 384, 0, cols_too=True)
    out.rstd, out.mean = torch.zeros(259, device="cuda")[3:], torch.zeros(257, device="cuda")[1:]
    got = call(fp8, recipe, x, gamma, beta, 0, None, amax, out=out)
    a = fp8.layernorm_backward(x, x, gamma, out.mean, out.rstd)
    b = fp8.layernorm_backward(x, x, gamma, want.mean, want.rstd)
    torch.cuda.synchronize()
    assert torch.equal(got.rstd, want.rstd) and torch.equal(got.mean, want.mean)
    assert torch.equal(got.rows.q, want.rows.q) and torch.equal(got.cols.q, want.cols.q)
    assert all(torch.equal(u, v) for u, v in zip(a, b))


@pytest.mark.parametrize("onto", ["x", "residual"])
def test_stream_in_place(fp8, onto):
    x, r, (gamma, beta) = stream(37, 1024, 3), stream(37, 1024, 4), weights(1024, 5)
    want = fp8.layernorm_quantize(x, gamma, beta, EPS, fp8.E4M3, residual=r)
    out = fp8.empty_layernorm(37, 1024, fp8.E4M3, residual=True)
    x2, r2 = x.clone(), r.clone()
    out.h = x2 if onto == "x" else r2
    got = fp8.layernorm_quantize(x2, gamma, beta, EPS, fp8.E4M3, residual=r2, out=out)
    assert torch.equal(got.h, want.h) and torch.equal(got.rows.q, want.rows.q) and torch.equal(got.mean, want.mean)
    assert torch.equal(got.rstd, want.rstd) and torch.equal(r2 if onto == "x" else x2, r if onto == "x" else x)


@pytest.mark.parametrize("rows,cols", [(702, 7168), (1300, 4096), (330, 16384)])
def test_more_rows_than_run_at_once(fp8, rows, cols):
    # wide rows, whose inputs are asked for ahead: packed, with gaps, and with the stream in the place of x
    x, r, (gamma, beta) = stream(rows, cols, 13), stream(rows, cols, 14), weights(cols, 15)
    parts = [fp8.layernorm_quantize(x[i:i + 97], gamma, beta, EPS, fp8.E4M3, residual=r[i:i + 97])
             for i in range(0, rows, 97)]
    room = torch.full((rows, cols + 8), float("nan"), dtype=torch.bfloat16, device="cuda")
    room[:, :cols] = x
    place = x.clone()
    out = fp8.empty_layernorm(rows, cols, fp8.E4M3, residual=True)
    out.h = place
    for got in (fp8.layernorm_quantize(x, gamma, beta, EPS, fp8.E4M3, residual=r),
                fp8.layernorm_quantize(room[:, :cols], gamma, beta, EPS, fp8.E4M3, residual=r),
                fp8.layernorm_quantize(place, gamma, beta, EPS, fp8.E4M3, residual=r, out=out)):
        torch.cuda.synchronize()
        for name in ("h", "mean", "rstd"):
            assert torch.equal(getattr(got, name), torch.cat([getattr(p, name) for p in parts])), name
        assert torch.equal(got.rows.q, torch.cat([p.rows.q for p in parts]))
        assert torch.equal(got.rows.scale[:, :rows], torch.cat([p.rows.scale[:, :len(p.mean)] for p in parts], 1))


@pytest.mark.parametrize("cols", [128, 896, 2048, 4096])
def test_rows_with_nan_and_infinity_stay_alone(fp8, cols):
    rows = 640
    x, (gamma, beta) = stream(rows, cols, 11), weights(cols, 12)
    clean = fp8.layernorm_quantize(x, gamma, beta, EPS, fp8.E4M3)
    bad = x.clone()
    bad[3, 17], bad[9, 100] = float("nan"), float("inf")
    got = fp8.layernorm_quantize(bad, gamma, beta, EPS, fp8.E4M3)
    keep = [i for i in range(rows) if i not in (3, 9)]
    assert torch.equal(got.rows.q[keep], clean.rows.q[keep]) and torch.equal(got.rstd[keep], clean.rstd[keep])
    assert bool(got.rstd[3].isnan()) and bool(got.rstd[9].isnan())
    assert bool(got.rows.q.view(torch.float8_e4m3fn).float()[[3, 9]].isnan().all())


def test_many_rows_through_few_blocks(fp8):
    # every block walks several rows, with the next one on its way: narrow, middling and wide rows
    for rows, cols in [(9000, 256), (5000, 2048), (3000, 5120), (1500, 12288)]:
        x, r, (gamma, beta) = stream(rows, cols, rows), stream(rows, cols, rows + 1), weights(cols, 2)
        got = fp8.layernorm_quantize(x, gamma, beta, EPS, fp8.E4M3, residual=r, y=True)
        part = fp8.layernorm_quantize(x[rows - 37:], gamma, beta, EPS, fp8.E4M3, residual=r[rows - 37:], y=True)
        torch.cuda.synchronize()
        assert torch.equal(got.y[-37:], part.y) and torch.equal(got.rows.q[-37:], part.rows.q)
        assert torch.equal(got.mean[-37:], part.mean) and torch.equal(got.rstd[-37:], part.rstd)
        h = (x.double() + r.double()).float().bfloat16().double()
        want = torch.nn.functional.layer_norm(h, (cols,), gamma.double(), beta.double(), EPS)
        # the bound of the tests above with its worst row: mean |h| rstd stays below 40 here but for the rows without
        # deviations, and 3e-5 of gamma covers 90 roundings of it
        err = (got.y.double() - want).abs()
        assert bool((err <= 2.0 ** -8 * want.abs() + 2e-4 * (gamma.double().abs() + want.abs())).all())


def test_empty_and_other_streams(fp8):
    gamma, beta = weights(256, 1)
    none = fp8.layernorm_quantize(torch.empty(0, 256, dtype=torch.bfloat16, device="cuda"), gamma, beta, EPS, fp8.E4M3)
    assert none.rows.q.shape == (0, 256) and none.mean.shape == (0,)
    x = stream(512, 256, 2)
    want = fp8.layernorm_quantize(x, gamma, beta, EPS, fp8.E4M3, cols=True)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        late = torch.zeros_like(x)
        torch.cuda._sleep(20_000_000)  # the input is written behind a wait of this stream
        late.copy_(x)
        got = fp8.layernorm_quantize(late, gamma, beta, EPS, fp8.E4M3, cols=True)
    s.synchronize()
    assert torch.equal(got.rows.q, want.rows.q) and torch.equal(got.cols.q, want.cols.q)


def test_more_than_two_to_the_31_elements(fp8):
    rows, cols = 78976, 27264  # 2^31 and 5 Mi elements
    gamma, beta = weights(cols, 1)
    x = torch.zeros(rows, cols, dtype=torch.bfloat16, device="cuda")
    tail = stream(128, cols, 5)
    x[-128:] = tail
    got = fp8.layernorm_quantize(x, gamma, beta, EPS, fp8.E4M3, cols=True)
    want = fp8.layernorm_quantize(tail, gamma, beta, EPS, fp8.E4M3, cols=True)
    torch.cuda.synchronize()
    assert torch.equal(got.rows.q[-128:], want.rows.q) and torch.equal(got.cols.q[:, -128:], want.cols.q)
    assert torch.equal(got.rows.scale[:, rows - 128:rows], want.rows.scale[:, :128])
    assert torch.equal(got.cols.scale[-1], want.cols.scale[0])
    assert torch.equal(got.rows.q[0], got.rows.q[-200]) and bool((got.mean[:-128] == 0).all())
    dx = fp8.layernorm_backward(x, x, gamma, got.mean, got.rstd)[0]
    wx = fp8.layernorm_backward(tail, tail, gamma, want.mean, want.rstd)[0]
    torch.cuda.synchronize()
    assert torch.equal(dx[-128:], wx) and not bool(dx[:-128].any())


# ---------------------------------------------------------------- backward --

def gradients(rows, cols, seed, ld=None):
    g = torch.Generator().manual_seed(seed)
    t = (0.01 * torch.randn(rows, ld or cols, generator=g) + 0.002).bfloat16().cuda()
    return t[:, :cols]


def statistics(h):
    d = h.double()
    mean = d.mean(1)
    return mean.float(), torch.rsqrt((d - mean[:, None]).square().mean(1) + EPS).float()


def check_backward(got, dy, h, gamma, mean, rstd, res, before=None):
    rows = h.shape[0]
    dx, size, dg, dg_size, db, db_size = ref.norm_backward(dy, h, gamma, mean, rstd, res)
    # the means: at most 64 terms follow one another, ten levels; a handful of products and sums around them
    bound = 2.0 ** -8 * np.abs(dx) + (2.0 ** -8 + 1) * 96 * U * size
    err = np.abs(f64(got[0]) - dx)
    assert np.all(err <= bound + 2.0 ** -134), float((err / (bound + 2.0 ** -134)).max())
    if before is not None:
        dg, dg_size = dg + f64(before[0]), dg_size + np.abs(f64(before[0]))
        db, db_size = db + f64(before[1]), db_size + np.abs(f64(before[1]))
    # no order of adding `rows` terms has more than rows + 2 roundings on a term's way; a product's own three
    assert np.all(np.abs(f64(got[1]) - dg) <= (rows + 5) * U * dg_size + 1e-40)
    if got[2] is not None:
        assert np.all(np.abs(f64(got[2]) - db) <= (rows + 2) * U * db_size + 1e-40)


@pytest.mark.parametrize("rows,cols", [(1, 8), (1, 4096), (2, 24), (7, 520), (333, 1000), (1000, 2048), (64, 7168),
                                       (5, 14336), (3, 16392), (4, 28672), (2500, 136), (5001, 128),
                                       (700, 504), (31, 1024), (33, 8192), (9, 8200), (1300, 5000), (1520, 1280),
                                       (1531, 2048)])
@pytest.mark.parametrize("with_residual", [False, True])
def test_backward(fp8, rows, cols, with_residual):
    pad = 8 if rows % 2 else 0
    h, (gamma, _) = stream(rows, cols, 21, cols + pad if pad else None), weights(cols, 22)
    dy = gradients(rows, cols, 23, cols + 2 * pad)
    res = gradients(rows, cols, 24, cols + 3 * pad) if with_residual else None
    mean, rstd = statistics(h)
    got = fp8.layernorm_backward(dy, h, gamma, mean, rstd, res)
    again = fp8.layernorm_backward(dy, h, gamma, mean, rstd, res)
    bare = fp8.layernorm_backward(dy, h, gamma, mean, rstd, res, bias=False)
    torch.cuda.synchronize()
    check_backward(got, dy, h, gamma, mean, rstd, res)
    assert all(torch.equal(a, b) for a, b in zip(got, again))  # the same order every time
    assert torch.equal(bare[0], got[0]) and torch.equal(bare[1], got[1]) and bare[2] is None


def test_backward_accumulates_and_works_in_place(fp8):
    rows, cols = 200, 1024
    h, (gamma, _), dy, res = stream(rows, cols, 1), weights(cols, 2), gradients(rows, cols, 3), gradients(rows, cols, 4)
    mean, rstd = statistics(h)
    want = fp8.layernorm_backward(dy, h, gamma, mean, rstd, res)[0]
    before = torch.randn(2, cols, device="cuda")
    dg, db = before.clone()
    on_res, on_dy = res.clone(), dy.clone()
    fp8.layernorm_backward(dy, h, gamma, mean, rstd, on_res, out=on_res, dgamma=dg, dbeta=db, accumulate=True)
    fp8.layernorm_backward(on_dy, h, gamma, mean, rstd, res, out=on_dy)
    torch.cuda.synchronize()
    assert torch.equal(on_res, want) and torch.equal(on_dy, want)
    check_backward((on_res, dg, db), dy, h, gamma, mean, rstd, res, before)


def test_backward_of_no_rows(fp8):
    e, none = torch.empty(0, 256, dtype=torch.bfloat16, device="cuda"), torch.empty(0, device="cuda")
    gamma, ws = weights(256, 1)[0], torch.empty(4, device="cuda")
    dg, db = torch.full((2, 256), 3.0, device="cuda")
    fp8.layernorm_backward(e, e, gamma, none, none, dgamma=dg, dbeta=db, accumulate=True, workspace=ws)
    assert bool((dg == 3.0).all()) and bool((db == 3.0).all())
    fp8.layernorm_backward(e, e, gamma, none, none, dgamma=dg, dbeta=db, workspace=ws)
    assert bool((dg == 0.0).all()) and bool((db == 0.0).all())


def test_backward_against_differences(fp8):
    # sum(dy y(h)) in 64 bits, moved by a small step in h, gamma and beta
    rows, cols = 3, 256
    x, (gamma, beta), dy = stream(rows, cols, 31), weights(cols, 32), gradients(rows, cols, 33)
    fwd = fp8.layernorm_quantize(x, gamma, beta, EPS, fp8.E4M3)
    dx, dg, db = fp8.layernorm_backward(dy, x, gamma, fwd.mean, fwd.rstd)
    torch.cuda.synchronize()
    h, g, b, d = f64(x), f64(gamma), f64(beta), f64(dy)

    def loss(h, g, b):
        c = h - h.mean(1, keepdims=True)
        return float((d * (c / np.sqrt((c * c).mean(1, keepdims=True) + EPS) * g + b)).sum())

    t = 1e-5
    top = float(np.abs(f64(dx)).max())
    for i, j in [(0, 0), (1, 77), (2, 255), (0, 128)]:
        e = np.zeros_like(h)
        e[i, j] = t
        want = (loss(h + e, g, b) - loss(h - e, g, b)) / (2 * t)
        # central differences: t^2 of the third derivative and 1e-16 / t of the loss; the output is bf16
        assert abs(f64(dx)[i, j] - want) <= 2.0 ** -8 * abs(want) + 1e-6 * top
        e = np.zeros_like(g)
        e[j] = t
        for got, want in ((dg, loss(h, g + e, b) - loss(h, g - e, b)), (db, loss(h, g, b + e) - loss(h, g, b - e))):
            assert abs(f64(got)[j] - want / (2 * t)) <= 1e-5 * abs(want / (2 * t)) + 1e-8
