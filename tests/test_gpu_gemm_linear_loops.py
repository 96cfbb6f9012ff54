"""The linear GEMM with more output tiles than run at once: a persistent CTA or
CTA pair takes a second tile, on aligned, even and odd widths."""
import pytest
import torch

import workloads
from test_gpu_gemm_linear import RECIPES, check, operands, product

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("recipe", RECIPES)
@pytest.mark.parametrize("M,N,K", [(2560, 2304, 512), (2550, 2302, 256), (2550, 2303, 256)])
def test_more_tiles_than_ctas(fp8, recipe, M, N, K):
    a = workloads.normal_bf16((M, K), 61, "a")
    b = workloads.normal_bf16((N, K), 61, "b", std=0.05)
    bias = workloads.normal_bf16((N,), 61, "bias").cuda()
    res = workloads.normal_bf16((M, N), 61, "res", std=3.0).cuda()
    A, B, acc, S = operands(fp8, recipe, a, b, 0, 0)
    for act, bi, r in ((fp8.ACT_NONE, None, res), (fp8.ACT_GELU, bias, res), (fp8.ACT_GELU, bias, None)):
        y, z = product(fp8, recipe)(A, B, bi, act, r, want_aux=act == fp8.ACT_GELU)
        torch.cuda.synchronize()
        check(y, z, acc, S, bi, act, r)
        if r is not None:  # in the residual's place
            on = r.clone()
            product(fp8, recipe)(A, B, bi, act, on, out=on)
            assert torch.equal(on, y)
    assert fp8.device_status() == 0
