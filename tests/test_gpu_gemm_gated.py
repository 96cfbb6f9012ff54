"""The gated product and its data gradient, in the three recipes, against the
oracle's fp64 product."""
import dataclasses

import numpy as np
import pytest
import torch

import workloads
from helpers import FULL_C, assert_within, bf16_to_f64, bf16_ulp, dgelu_eval_bound
from test_gpu_gemm_linear import RECIPES, operands

pytestmark = pytest.mark.gpu
E4M3, E5M2 = 0, 1
SLOPE = 1.13  # of either activation, at most
EVAL = 1e-5   # relative error of an activation: the fast exponential's 96 ulp, the approximate division's 2


def forward(fp8, recipe):
    return {"block": fp8.gemm_gated, "mx": fp8.mx_gemm_gated, "tensor": fp8.tensor_gemm_gated}[recipe]


def gradient(fp8, recipe):
    return {"block": fp8.gemm_gated_dgrad, "mx": fp8.mx_gemm_gated_dgrad, "tensor": fp8.tensor_gemm_gated_dgrad}[recipe]


def logistic(x):
    return 1.0 / (1.0 + np.exp(-np.clip(x, -700, 700)))


def gate(z, act):
    """(act(z), act'(z))"""
    c = 2 * np.sqrt(2 / np.pi)
    x, dx = (z, 1.0) if act == 2 else (c * (z + 0.044715 * z ** 3), c * (1 + 3 * 0.044715 * z * z))
    s = logistic(x)
    return z * s, s + z * dx * s * logistic(-x)


def whole(got, want, extra=0.0):
    # the outputs' rounding alone leaves at most 2^-8 of the norm; the fp32 sums a small part of that
    assert np.linalg.norm(got - want) <= (2.0 ** -8 + 2e-4) * np.linalg.norm(want) + extra


def check_forward(y, z, acc, S, bias, act):
    """The bounds of the linear product's tests (c S for a product, fp32 roundings), through the gate."""
    N = acc.shape[1] // 2
    zo = acc + (bf16_to_f64(bias) if bias is not None else 0.0)
    dz = FULL_C * S + 2.0 ** -23 * np.abs(zo)
    g, u, dg, du = zo[:, :N], zo[:, N:], dz[:, :N], dz[:, N:]
    a, _ = gate(g, act)
    want, got = a * u, bf16_to_f64(y)
    err = SLOPE * dg * (np.abs(u) + du) + np.abs(a) * du + (EVAL + 2.0 ** -22) * np.abs(want) + 1e-30
    assert_within(got, want, err + bf16_ulp(np.maximum(np.abs(got), np.abs(want))), "Y")
    whole(got, want)
    if z is not None:
        gz = bf16_to_f64(z)
        assert_within(gz, zo, dz + bf16_ulp(np.maximum(np.abs(gz), np.abs(zo))), "Z")
        whole(gz, zo)


def weights(N, K, seed, std=0.05):
    return workloads.normal_bf16((2 * N, K), seed, "b", std=std)


# few tokens in every tile width and split of K; more, by the rows' kernel; whole tiles, split in two and in four;
# more tiles than run at once
SHAPES = [(1, 128, 128), (1, 256, 4096), (2, 384, 256), (3, 128, 896), (8, 640, 1280), (9, 128, 2048), (16, 512, 7168),
          (17, 384, 384), (33, 1152, 512), (64, 128, 1024), (50, 256, 4096), (100, 256, 640), (129, 128, 256),
          (300, 512, 384), (150, 256, 4096), (257, 128, 2048), (128, 1024, 4096), (800, 2176, 256), (1000, 1920, 128),
          (1000, 896, 2048), (900, 1152, 4096), (650, 1408, 2304), (2600, 1792, 384)]
# gradients of whole tiles, on both sides of the sum's length at which B's rows are ordered
WHOLE = [(1300, 2176, 2944), (1250, 2176, 3200)]


@pytest.mark.parametrize("recipe", RECIPES)
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_forward(fp8, recipe, M, N, K):
    seed = M + N + K
    fa, fb = E5M2 if M % 3 == 0 else E4M3, E5M2 if N % 5 == 0 else E4M3
    bias = workloads.normal_bf16((2 * N,), seed, "bias").cuda()
    A, B, acc, S = operands(fp8, recipe, workloads.normal_bf16((M, K), seed, "a"), weights(N, K, seed), fa, fb)
    for act in (fp8.ACT_SILU, fp8.ACT_GELU):
        for b in (None, bias):
            seen = []
            for aux in (False, True):
                out = torch.full((M, N), float("nan"), dtype=torch.bfloat16, device="cuda")
                y, z = forward(fp8, recipe)(A, B, b, act, out=out, want_aux=aux)
                torch.cuda.synchronize()
                assert fp8.device_status() == 0 and (z is not None) == aux
                seen.append(y)
            check_forward(y, z, acc, S, b, act)
            assert torch.equal(*seen)  # what is kept changes nothing


@pytest.mark.parametrize("recipe", RECIPES)
@pytest.mark.parametrize("M,N,K", [s for s in SHAPES if s[0] > 8 or s[0] == 1] + WHOLE)
def test_gradient(fp8, recipe, M, N, K):
    seed = M + N + K
    A, B, acc, S = operands(fp8, recipe, workloads.normal_bf16((M, K), seed, "a", std=0.02),
                            workloads.normal_bf16((N, K), seed, "b", std=0.05), E5M2, E4M3 if N % 5 else E5M2)
    z = workloads.normal_bf16((M, 2 * N), seed, "z", std=2.0).cuda()
    z[0, :4] = torch.tensor([0.0, -30.0, 30.0, -300.0]).bfloat16()  # far out on both sides
    zo = bf16_to_f64(z)
    g, u = zo[:, :N], zo[:, N:]
    for act in (fp8.ACT_SILU, fp8.ACT_GELU):
        out = torch.full((M, 2 * N), float("nan"), dtype=torch.bfloat16, device="cuda")
        dz = gradient(fp8, recipe)(A, B, z, act, out=out)
        on_z = z.clone()
        same = gradient(fp8, recipe)(A, B, on_z, act, out=on_z)
        torch.cuda.synchronize()
        assert fp8.device_status() == 0 and torch.equal(dz, same) and same.data_ptr() == on_z.data_ptr()
        a, d = gate(g, act)
        got = bf16_to_f64(dz)
        # the derivative's evaluation as for the GELU epilogue; SiLU's terms are no larger
        ev = dgelu_eval_bound(g) if act == fp8.ACT_GELU else 2.0 ** -16 * (1 + np.abs(g)) * logistic(g) + 1e-30
        for part, factor, eval_err in ((slice(0, N), u * d, np.abs(u) * ev), (slice(N, None), a, EVAL * np.abs(a) + 1e-30)):
            want = acc * factor
            err = FULL_C * S * (np.abs(factor) + eval_err) + np.abs(acc) * eval_err + 2.0 ** -22 * np.abs(want)
            assert_within(got[:, part], want, err + bf16_ulp(np.maximum(np.abs(got[:, part]), np.abs(want))) + 2.0 ** -133, "dZ")
            whole(got[:, part], want)


@pytest.mark.parametrize("recipe", RECIPES)
@pytest.mark.parametrize("M,N,K", [(1, 1152, 256), (40, 384, 1024), (700, 640, 256), (300, 256, 4096)])
def test_neighbours_are_left_alone(fp8, recipe, M, N, K):
    A, B, acc, S = operands(fp8, recipe, workloads.normal_bf16((M, K), 1, "a"), weights(N, K, 1), E4M3, E4M3)
    room = torch.full((M * N + 256,), 7.0, dtype=torch.bfloat16, device="cuda")
    zroom = torch.full((2 * M * N + 256,), 7.0, dtype=torch.bfloat16, device="cuda")
    out, aux = room[128:128 + M * N].view(M, N), zroom[128:128 + 2 * M * N].view(M, 2 * N)
    forward(fp8, recipe)(A, B, None, fp8.ACT_SILU, out=out, aux=aux)
    torch.cuda.synchronize()
    check_forward(out, aux, acc, S, None, fp8.ACT_SILU)
    for r in (room, zroom):
        assert bool((r[:128] == 7).all()) and bool((r[-128:] == 7).all())
    A, B, acc, S = operands(fp8, recipe, workloads.normal_bf16((M, K), 1, "a"), workloads.normal_bf16((N, K), 1, "b"),
                            E4M3, E4M3)
    zroom.fill_(float("nan"))  # no output is one
    gradient(fp8, recipe)(A, B, aux.clone().fill_(0.5), fp8.ACT_SILU, out=aux)
    torch.cuda.synchronize()
    assert bool(zroom[:128].isnan().all()) and bool(zroom[-128:].isnan().all()) and not bool(aux.isnan().any())


def test_columns_of_one_projection_come_from_its_rows(fp8):
    # weights that name their row: every output knows which gate and which up row made it, in every kernel
    for M, N, K in ((5, 1152, 128), (200, 1152, 128), (700, 1152, 128), (300, 384, 2048)):
        x = torch.zeros(M, K, dtype=torch.bfloat16, device="cuda")
        x[:, 0] = 1.0
        w = torch.zeros(2 * N, K, dtype=torch.bfloat16, device="cuda")
        w[:N, 0] = 100.0                                              # silu(100) = 100
        w[N:, 0] = (torch.arange(N, device="cuda") % 16).bfloat16()   # exact in e4m3 times a power of two
        w[:, 1] = 448.0                                               # one scale for all rows: 1
        want = (torch.arange(N, device="cuda") % 16).float()
        for recipe in RECIPES:
            if recipe == "block":
                A, B = fp8.quantize(x, E4M3), fp8.quantize(w, E4M3)
            elif recipe == "mx":
                A, B = fp8.mx_quantize(x, E4M3), fp8.mx_quantize(w, E4M3)
            else:
                A = fp8.tensor_quantize(x, E4M3, fp8.tensor_amax(x))[0]
                B = fp8.tensor_quantize(w, E4M3, fp8.tensor_amax(w))[0]
            y, z = forward(fp8, recipe)(A, B, None, fp8.ACT_SILU, want_aux=True)
            torch.cuda.synchronize()
            g, u = z[:, :N].float(), z[:, N:].float()
            assert bool(((g - 100.0).abs() <= 4.0).all())  # 100 as e4m3: 96 or 104
            assert torch.equal(u, want.expand(M, N)), recipe
            assert bool(((y.float() - g * u).abs() <= 2.0 ** -7 * (g * u).abs()).all())


@pytest.mark.parametrize("recipe", RECIPES)
def test_infinities_and_nan_stay_in_their_outputs(fp8, recipe):
    # fp8 codes of NaN in one token and in one gate row
    M, N, K = 150, 256, 256
    A, B, _, _ = operands(fp8, recipe, workloads.normal_bf16((M, K), 3, "a"), weights(N, K, 3), E4M3, E4M3)
    clean = forward(fp8, recipe)(A, B)[0].clone()
    A.q[7, 5], B.q[130, 9] = 0x7F, 0x7F
    y = forward(fp8, recipe)(A, B)[0]
    torch.cuda.synchronize()
    bad = torch.zeros(M, N, dtype=torch.bool, device="cuda")
    bad[7], bad[:, 130] = True, True
    assert bool(y[bad].isnan().all()) and torch.equal(y[~bad], clean[~bad])


def test_gradient_far_out(fp8):
    # the limits of both activations and of their slopes, and NaN where Z holds it
    M, N, K = 130, 256, 256
    A, B, acc, _ = operands(fp8, "block", workloads.normal_bf16((M, K), 3, "a"), workloads.normal_bf16((N, K), 3, "b"),
                            E5M2, E4M3)
    far = torch.tensor([-3e38, -1e30, -1e5, -100.0, 100.0, 1e5, 1e30, float("nan")]).bfloat16()
    z = torch.ones(M, 2 * N, dtype=torch.bfloat16, device="cuda")
    z[:, :N] = far.repeat(N // 8).cuda()
    for act in (fp8.ACT_SILU, fp8.ACT_GELU):
        dz = fp8.gemm_gated_dgrad(A, B, z, act).float()
        torch.cuda.synchronize()
        c = torch.from_numpy(acc).cuda()
        slope = torch.tensor([0.0, 0.0, 0.0, 0.0, 1.0, 1.0, 1.0, float("nan")], dtype=torch.float64, device="cuda").repeat(N // 8)
        top = far.double().clamp(min=0).cuda().repeat(N // 8)
        for got, want in ((dz[:, :N], c * slope), (dz[:, N:], c * top)):
            finite = want.abs() < 3e38
            assert torch.equal(got.isnan(), want.isnan())
            assert torch.allclose(got[finite].double(), want[finite], rtol=2.0 ** -7, atol=1e-30)


@pytest.mark.parametrize("recipe", RECIPES)
def test_kernels_for_few_and_for_many_rows_agree(fp8, recipe):
    # the same rows alone, in a batch for the split kernels, and in one for whole tiles: sums in another order only
    N, K = 384, 1024
    x, w = workloads.normal_bf16((3000, K), 1, "a").cuda(), weights(N, K, 1).cuda()

    def cast(t):
        if recipe == "block":
            return fp8.quantize(t, E4M3)
        if recipe == "mx":
            return fp8.mx_quantize(t, E4M3)
        return fp8.tensor_quantize(t, E4M3, torch.tensor([6.0], device="cuda"))[0]

    W = cast(w)
    many = forward(fp8, recipe)(cast(x), W)[0]
    for n in (1, 5, 30, 64, 100, 130, 500):
        few = forward(fp8, recipe)(cast(x[:n]), W)[0]
        torch.cuda.synchronize()
        scale = many[:n].float().abs().max()
        assert bool(((few.float() - many[:n].float()).abs() <= 2.0 ** -7 * many[:n].float().abs() + 1e-4 * scale).all())


@pytest.mark.parametrize("recipe", RECIPES)
def test_streams_and_graphs(fp8, recipe):
    M, N, K = 20, 256, 512
    A, B, acc, S = operands(fp8, recipe, workloads.normal_bf16((M, K), 1, "a"), weights(N, K, 1), E4M3, E4M3)
    call = forward(fp8, recipe)
    out, aux = torch.empty(M, N, dtype=torch.bfloat16, device="cuda"), torch.empty(M, 2 * N, dtype=torch.bfloat16, device="cuda")
    want = call(A, B)[0]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(A, B, None, fp8.ACT_SILU, out=out, aux=aux)
    out.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    codes, late = A.q.clone(), A.q
    s = torch.cuda.Stream()
    late.zero_()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        torch.cuda._sleep(20_000_000)  # the codes are written behind a wait of this stream
        late.copy_(codes)
        y = call(A, B)[0]
    s.synchronize()
    assert torch.equal(y, want)


def test_more_than_two_to_the_31_outputs(fp8):
    M, N, K = 72000, 16384, 128  # 2^31 and more of Z and of Y's gradient
    x, w = torch.zeros(M, K, dtype=torch.bfloat16, device="cuda"), weights(N, K, 1).cuda()
    x[-100:] = workloads.normal_bf16((100, K), 1, "a").cuda()
    W = fp8.mx_quantize(w, E4M3)
    y, z = fp8.mx_gemm_gated(fp8.mx_quantize(x, E4M3), W, want_aux=True)
    ty, tz = fp8.mx_gemm_gated(fp8.mx_quantize(x[-356:], E4M3), W, want_aux=True)
    torch.cuda.synchronize()
    assert torch.equal(y[-100:], ty[-100:]) and torch.equal(z[-100:], tz[-100:])
    assert not bool(y[:100].any()) and not bool(z[-200:-100].any())
    del y
    back = fp8.quantize(workloads.normal_bf16((M, K), 2, "d").cuda(), E5M2)
    T = fp8.quantize(workloads.normal_bf16((N, K), 2, "t").cuda(), E4M3)
    dz = fp8.gemm_gated_dgrad(back, T, z, out=z.clone())
    tail = fp8.Fp8Tensor(back.q[-356:].clone(), back.scale[:, -356:].clone(), E5M2)
    td = fp8.gemm_gated_dgrad(tail, T, tz)
    torch.cuda.synchronize()
    assert torch.equal(dz[-100:], td[-100:])


@pytest.mark.parametrize("recipe", RECIPES)
@pytest.mark.parametrize("M,grad", [(4, False), (300, False), (300, True)])
def test_a_starved_pipeline_reports_and_returns(fp8, recipe, M, grad):
    N, K = 256, 512
    A, B, acc, S = operands(fp8, recipe, workloads.normal_bf16((M, K), 1, "a"),
                            weights(N // 2 if grad else N, K, 1), E4M3, E4M3)
    out = torch.full((M, 2 * N if grad else N), 7.0, dtype=torch.bfloat16, device="cuda")
    z = torch.zeros(M, 2 * N, dtype=torch.bfloat16, device="cuda")
    torch.cuda.synchronize()
    fp8.debug_starve_next_gemm(5)
    if grad:
        gradient(fp8, recipe)(A, B, z, out=out)
    else:
        forward(fp8, recipe)(A, B, out=out)
    assert fp8.device_status() == fp8.binding.ERR_TIMEOUT and bool((out == 7).all())
    if not grad:
        y, _ = forward(fp8, recipe)(A, B)
        torch.cuda.synchronize()
        check_forward(y, None, acc, S, None, fp8.ACT_SILU)


def cast(fp8, recipe, x, fmt):
    if recipe == "tensor":
        return fp8.tensor_quantize(x, fmt, fp8.tensor_amax(x))[0]
    return (fp8.quantize if recipe == "block" else fp8.mx_quantize)(x, fmt)


def spaced(t):
    """The operand with NaN codes between its rows and NaN scales between those of its K blocks."""
    rows, k = t.q.shape
    q = torch.full((rows, k + 128), 0x7F, dtype=torch.uint8, device="cuda")  # NaN in both formats
    q[:, :k] = t.q
    scale = {}
    if hasattr(t, "scale") and t.scale.dim() == 2:
        kb, n = t.scale.shape
        wide = torch.full((kb, n + 68), float("nan"), device="cuda")
        wide[:, :n] = t.scale
        scale = {"scale": wide[:, :n]}
    return dataclasses.replace(t, q=q[:, :k], **scale)


# few rows; tiles; tiles of which K is split; more tiles than run at once
@pytest.mark.parametrize("recipe", RECIPES)
@pytest.mark.parametrize("M,N,K", [(3, 384, 512), (50, 256, 4096), (300, 512, 384), (257, 128, 2048), (1300, 2176, 384)])
def test_forward_of_operands_with_gaps(fp8, recipe, M, N, K):
    A = cast(fp8, recipe, workloads.normal_bf16((M, K), 3, "a").cuda(), E4M3)
    W = cast(fp8, recipe, weights(N, K, 3).cuda(), E4M3)
    want = forward(fp8, recipe)(A, W, want_aux=True)
    for a, w in ((spaced(A), W), (A, spaced(W)), (spaced(A), spaced(W))):
        for got, packed in zip(forward(fp8, recipe)(a, w, want_aux=True), want):
            assert torch.equal(got, packed) and not bool(got.isnan().any())


# B's rows ordered (1x128: over 384) and not; K split
@pytest.mark.parametrize("recipe", RECIPES)
@pytest.mark.parametrize("M,N,K", [(1300, 2176, 384), (1250, 2176, 3200), (300, 384, 384), (300, 512, 2048), (1000, 896, 1024)])
def test_gradient_of_operands_with_gaps(fp8, recipe, M, N, K):
    A = cast(fp8, recipe, workloads.normal_bf16((M, K), 4, "a", std=0.02).cuda(), E5M2)
    W = cast(fp8, recipe, workloads.normal_bf16((N, K), 4, "b", std=0.05).cuda(), E4M3)
    z = workloads.normal_bf16((M, 2 * N), 4, "z").cuda()
    want = gradient(fp8, recipe)(A, W, z)
    for a, w in ((spaced(A), W), (A, spaced(W)), (spaced(A), spaced(W))):
        got = gradient(fp8, recipe)(a, w, z)
        assert torch.equal(got, want) and not bool(got.isnan().any())
