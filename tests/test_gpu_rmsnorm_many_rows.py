"""Column codes of a norm with more than 65535 bands of 128 rows."""
import pytest
import torch

import block_reference as ref
from test_gpu_rmsnorm import call, scales, stream

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("recipe", ["block", "mx", "tensor"])
def test_column_codes_of_many_rows(fp8, recipe):
    rows, cols = 65537 * 128, 128
    gamma, amax = scales(cols, 1), torch.tensor([6.0], device="cuda")
    x = torch.zeros(rows, cols, dtype=torch.bfloat16, device="cuda")
    ends = stream(256, cols, 5)
    x[:128], x[-128:] = ends[:128], ends[128:]
    got = call(fp8, recipe, x, gamma, 0, None, amax, cols=True)
    want = call(fp8, recipe, ends, gamma, 0, None, amax, cols=True)
    torch.cuda.synchronize()
    for mine, theirs in ((slice(0, 128), slice(0, 128)), (slice(-128, None), slice(128, None))):
        assert torch.equal(got.rows.q[mine], want.rows.q[theirs])
        assert torch.equal(got.cols.q[:, mine], want.cols.q[:, theirs])
    assert not bool((got.cols.q[:, 128:-128] & 0x7F).any())
    if recipe == "block":
        assert torch.equal(got.cols.scale[[0, -1]], want.cols.scale) and bool((got.cols.scale[1:-1] == 1.0).all())
    elif recipe == "mx":
        a, b = ref.mx_bytes(got.cols.sf, cols, rows), ref.mx_bytes(want.cols.sf, cols, 256)
        assert (a[:, :4] == b[:, :4]).all() and (a[:, -4:] == b[:, 4:]).all() and (a[:, 4:-4] == 127).all()
    else:
        assert torch.equal(got.amax, want.amax)
