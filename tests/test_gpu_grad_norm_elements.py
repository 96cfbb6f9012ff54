"""Every element of a gradient counts once in the norm: single elements at the
edges of rows of vectors, of chunks and of the tensors, whose norm is exact, and
a set larger than what stays in L2, to the sum's own rounding."""
import numpy as np
import pytest
import torch

from block_reference import U, f64

pytestmark = pytest.mark.gpu
CHUNK = 8192  # elements that a CTA takes at a time
SINGLE = 1216 * CHUNK  # eight CTAs on each of 152 SMs take one chunk each


def edges(n):
    at = {0, 1, 2, 3, 7, 8, 9, 15, 16, n // 2}
    for k in (CHUNK, 2 * CHUNK, SINGLE, 2 * SINGLE):
        at |= {k - 9, k - 8, k - 1, k, k + 1, k + 8}
    at |= {n - 1 - i for i in range(18)}
    return sorted(i for i in at if 0 <= i < n)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("n", [1, 5, 13, 8191, 8192, 8193, 20011, 2 * SINGLE + 12347])
def test_one_element(fp8, dtype, n):
    base = torch.zeros(n + 8, dtype=dtype, device="cuda")
    other = torch.zeros(100, device="cuda")
    for off in range(8) if n < SINGLE else (0, 3):
        t = base[off:off + n]
        plan = fp8.GradList([other, t, other[:7]])
        at = edges(n)
        got = torch.zeros(len(at), device="cuda")
        for k, i in enumerate(at):
            t[i] = -3.0
            got[k:k + 1] = fp8.grad_norm(plan)
            t[i] = 0.0
        assert bool((got == 3.0).all()), [i for k, i in enumerate(at) if got[k].item() != 3.0]


def test_one_element_of_each_of_many_tensors(fp8):
    for full in (64, 65, 1000, 1001, 2003):
        base = torch.zeros(full, 12, device="cuda")
        plan = fp8.GradList([base[i, :5 + i % 7] for i in range(full)])
        at = sorted({0, 1, 63, 64, 65, 998, 999, 1000, 1001, 1999, 2000, 2001, full - 1} & set(range(full)))
        for i in at:
            base[i, 4 + i % 7] = 5.0
            norm = fp8.clip_grads(plan, 2.5)
            # 5 / 2: the sum with 1e-6 and the division round once each, the product is by 5
            v = base[i, 4 + i % 7].item()
            assert norm.item() == 5.0 and abs(v - 12.5 / 5.000001) <= 2.0 ** -21 * v
            base[i, 4 + i % 7] = 0.0
        base[:] = 1.0
        total = sum(5 + i % 7 for i in range(full))
        assert abs(fp8.grad_norm(plan).item() - total ** 0.5) <= 2.0 ** -23 * total ** 0.5  # whole numbers: exact sum


def test_more_than_stays_in_l2(fp8):
    g = torch.Generator(device="cuda").manual_seed(3)
    sizes = [(9_000_011, torch.float32), (4097, torch.bfloat16), (12_345_677, torch.bfloat16), (11_000_003, torch.float32),
             (77, torch.float32), (9_999_999, torch.bfloat16)]
    grads = [(torch.randn(n, generator=g, device="cuda") * 10.0 ** (-2 - i % 3)).to(t) for i, (n, t) in enumerate(sizes)]
    want = float(np.sqrt(sum(float(v.double().square().sum()) for v in grads)))
    chunks = sum(-(-n // CHUNK) for n, _ in sizes)
    # the longest way of a square: eight of a vector, two joins of four vectors, a thread's two sums and two loose
    # elements per chunk, a warp's five and a CTA's seven, the partial sums of a thread, five and seven again; a tree of
    # d roundings is off by d U of a sum of squares, half of it is left by the root, which rounds once
    per_cta = -(-chunks // 1216)
    depth = 8 + 2 + 4 * per_cta + 5 + 7 + 8 + 5 + 7
    rel = (depth / 2 + 1) * U
    norm = fp8.grad_norm(grads)
    assert abs(norm.item() - want) <= rel * want
    out = [torch.full_like(v, float("nan")) for v in grads]
    top = want / 3
    again = fp8.clip_grads(fp8.GradList(grads, out), top)
    assert again.item() == norm.item()
    f = top / (want + 1e-6)
    for o, v in zip(out, grads):
        exact = v.double() * f
        rounding = 2.0 ** -8 if v.dtype == torch.bfloat16 else U
        assert bool(((o.double() - exact).abs() <= (rel + 6 * U + rounding) * exact.abs() + 2.0 ** -134).all())
    kept = [v.clone() for v in grads]
    fp8.clip_grads(grads, top)  # in place
    assert all(torch.equal(a, b) for a, b in zip(grads, out))
    fp8.clip_grads(kept, 10 * want)  # unchanged
    assert abs(fp8.grad_norm(kept).item() - want) <= rel * want
