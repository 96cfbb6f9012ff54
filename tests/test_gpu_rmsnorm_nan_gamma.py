"""Columns whose gamma is NaN or infinite: the column codes' scales are those of
the cast of the same values, which leaves NaN out of a maximum."""
import pytest
import torch

import block_reference as ref
from test_gpu_rmsnorm import EPS, call, scales, stream

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("recipe", ["block", "mx", "tensor"])
@pytest.mark.parametrize("fmt", [0, 1])
def test_column_scales(fp8, recipe, fmt):
    rows, cols = 256, 384
    x, gamma, amax = stream(rows, cols, 3), scales(cols, 4), torch.tensor([6.0], device="cuda")
    x[:, 200] = 0.0
    clean = call(fp8, recipe, x, gamma, fmt, None, amax, cols=True)
    gamma = gamma.clone()
    gamma[7], gamma[200] = float("nan"), float("inf")  # a column of NaN, and zeros times infinity
    got = call(fp8, recipe, x, gamma, fmt, None, amax, cols=True, y=True)
    torch.cuda.synchronize()
    bad = [7, 200]
    keep = [i for i in range(cols) if i not in bad]
    assert bool(got.y[:, bad].isnan().all())
    v = got.cols.q.view(torch.float8_e4m3fn if fmt == 0 else torch.float8_e5m2).float()
    assert bool(v[bad].isnan().all()) and torch.equal(got.cols.q[keep], clean.cols.q[keep])
    if recipe == "block":
        assert bool((got.cols.scale[:, bad] == 1.0).all())
        assert torch.equal(got.cols.scale[:, keep], clean.cols.scale[:, keep])
    elif recipe == "mx":
        cast = fp8.mx_quantize(got.y, fmt, transpose=True)
        b, c = (ref.mx_bytes(t.sf, cols, rows) for t in (got.cols, cast))
        assert (b[bad] == 127).all() and (c[bad] == 127).all()
        assert (b[keep] == ref.mx_bytes(clean.cols.sf, cols, rows)[keep]).all()
