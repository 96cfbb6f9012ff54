"""Global gradient norm and clipping against plain 64-bit forms."""
import numpy as np
import pytest
import torch

from block_reference import U, f64

pytestmark = pytest.mark.gpu


def tensors(sizes, seed, std=1e-2):
    """Sizes with their type: "f" fp32, "b" bf16."""
    g = torch.Generator().manual_seed(seed)
    return [(std * torch.randn(n, generator=g)).to(torch.float32 if t == "f" else torch.bfloat16).cuda()
            for n, t in sizes]


def norm64(ts):
    return float(np.sqrt(sum((f64(t) ** 2).sum() for t in ts)))


def norm_bound(ts):
    # a thread adds the squares of its share one after the other, in groups of 32 at the shortest; the shares are at
    # most total / (32 threads) plus one chunk's; then 16 levels and the root, which halves what is left
    n = sum(t.numel() for t in ts)
    return (min(n, n / 32 + 64) / 2 + 16) * U


def check_scaled(out, grads, norm, max_norm, rel):
    f = min(1.0, max_norm / (norm + 1e-6))
    for o, g in zip(out, grads):
        want = f64(g) * f
        rounding = 2.0 ** -8 if g.dtype == torch.bfloat16 else U
        # the factor: its norm's error, a sum, a division; then the product
        assert np.all(np.abs(f64(o) - want) <= (rel + 6 * U + rounding) * np.abs(want) + 2.0 ** -134)


SETS = [[(1, "f")], [(1, "b")], [(3, "b"), (0, "f"), (5, "f")], [(8192, "f"), (8193, "b"), (8191, "f")],
        [(100003, "f"), (77777, "b"), (16, "f"), (33, "b")], [(1000, "fb"[i % 2]) for i in range(130)],
        [(17 + i % 5, "fb"[i % 2]) for i in range(2100)]]


@pytest.mark.parametrize("sizes", SETS, ids=lambda s: "%d tensors" % len(s))
@pytest.mark.parametrize("max_norm", [1e-3, 1e9])
def test_norm_and_clip(fp8, sizes, max_norm):
    grads = tensors(sizes, len(sizes))
    want = norm64(grads)
    kept = [g.clone() for g in grads]
    got = fp8.grad_norm(grads)
    assert abs(got.item() - want) <= norm_bound(grads) * want
    out = [torch.full_like(g, float("nan")) for g in grads]
    plan = fp8.GradList(grads, out)
    again = fp8.clip_grads(plan, max_norm)
    torch.cuda.synchronize()
    assert again.item() == got.item()  # the same partial sums in the same order
    assert all(torch.equal(a, b) for a, b in zip(grads, kept))
    check_scaled(out, grads, want, max_norm, norm_bound(grads))
    fp8.clip_grads(grads, max_norm)  # in place
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(grads, out))
    if max_norm == 1e9:
        assert all(torch.equal(a, b) for a, b in zip(grads, kept))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("a,b", [(0, 1), (1, 0), (3, 3), (1, 2), (5, 1)])
def test_any_alignment(fp8, dtype, a, b):
    n = 20011
    g = torch.Generator().manual_seed(5)
    base = torch.randn(n + 8, generator=g).to(dtype).cuda()
    grads, out = base[a:a + n], torch.full((n + 8,), 7.0, dtype=dtype, device="cuda")
    norm = fp8.clip_grads(fp8.GradList([grads], [out[b:b + n]]), 1.0)
    torch.cuda.synchronize()
    want = norm64([grads])
    assert abs(norm.item() - want) <= norm_bound([grads]) * want
    check_scaled([out[b:b + n]], [grads], want, 1.0, norm_bound([grads]))
    assert bool((out[:b] == 7.0).all()) and bool((out[b + n:] == 7.0).all())  # nothing beside it


def test_a_plan_reads_the_values_of_each_call(fp8):
    grads = tensors([(5000, "f"), (300, "b")], 1)
    plan = fp8.GradList(grads)
    first = fp8.grad_norm(plan).item()
    for g in grads:
        g.mul_(2.0)
    assert abs(fp8.grad_norm(plan).item() - 2 * first) <= 8 * U * first


def test_nothing_and_not_finite(fp8):
    assert fp8.grad_norm([]).item() == 0.0 and fp8.clip_grads([], 1.0).item() == 0.0
    zero = [torch.zeros(100, device="cuda"), torch.empty(0, device="cuda")]
    assert fp8.clip_grads(zero, 1.0).item() == 0.0 and bool((zero[0] == 0).all())
    g = torch.ones(10000, device="cuda")
    g[77] = float("nan")
    assert np.isnan(fp8.clip_grads([g], 1.0).item()) and bool(g.isnan().all())
    g = torch.ones(10000, device="cuda")
    g[77] = float("inf")
    assert fp8.clip_grads([g], 1.0).item() == float("inf")
    assert bool(g[77].isnan()) and bool((g[:77] == 0).all())
    g = torch.ones(64, device="cuda")
    assert fp8.clip_grads([g], 0.0).item() == 8.0 and bool((g == 0).all())


def test_more_than_two_to_the_31_elements(fp8):
    n = 2 ** 31 + 4099
    g = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    g[-3:] = torch.tensor([1.0, 2.0, 2.0], device="cuda").bfloat16()
    g[2 ** 31 - 1] = 4.0
    norm = fp8.clip_grads([g], 2.5)
    torch.cuda.synchronize()
    assert norm.item() == 5.0
    assert torch.equal(g[-3:].float().cpu(), torch.tensor([0.5, 1.0, 1.0])) and g[2 ** 31 - 1].item() == 2.0


def test_after_another_streams_work(fp8):
    grads = tensors([(200000, "f")], 3)
    want = fp8.grad_norm(grads).item()
    s = torch.cuda.Stream()
    late = torch.zeros_like(grads[0])
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        torch.cuda._sleep(20_000_000)
        late.copy_(grads[0])
        got = fp8.clip_grads([late], 1.0)
    s.synchronize()
    assert got.item() == want


def test_refuses_what_it_cannot_clip(fp8):
    with pytest.raises(AssertionError):
        fp8.GradList([torch.zeros(4, 4, device="cuda").t()[:, :2]])
    with pytest.raises(AssertionError):
        fp8.GradList([torch.zeros(4, dtype=torch.float16, device="cuda")])
    with pytest.raises(fp8.Fp8Error):
        fp8.clip_grads([torch.zeros(4, device="cuda")], float("nan"))
