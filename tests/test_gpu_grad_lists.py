"""Gradient lists whose tensors do not fill the last launch: one launch takes up
to 1000 tensors that are not empty."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("full,empty", [(1000, 1), (1000, 70), (2000, 1), (999, 1), (1000, 0), (1001, 3), (64, 2)])
@pytest.mark.parametrize("in_place", [True, False])
def test_empty_tensors_behind_a_whole_launch(fp8, full, empty, in_place):
    base = torch.ones(full * 8, device="cuda")
    grads = [base[8 * i:8 * i + 4] for i in range(full)] + [torch.empty(0, device="cuda") for _ in range(empty)]
    out = None if in_place else [torch.full_like(g, 7.0) for g in grads]
    norm = fp8.clip_grads(fp8.GradList(grads, out), 0.5)
    torch.cuda.synchronize()
    # 4 full squares of one: the sum is exact, its root and the factor round once each, as the product and the sum
    # with 1e-6 do
    want = (4.0 * full) ** 0.5
    assert abs(norm.item() - want) <= 2.0 ** -23 * want
    f = 0.5 / (want + 1e-6)
    for g in (grads if in_place else out)[:full]:
        assert bool(((g - f).abs() <= 2.0 ** -21 * f).all())
    assert bool((base.view(full, 8)[:, 4:] == 1.0).all())  # nothing beside them
    if not in_place:
        assert bool((base == 1.0).all())


def test_empty_tensors_between_launches(fp8):
    # 2500 tensors in three launches, empty ones at the ends of the first and the second
    base = torch.ones(2500 * 4, device="cuda")
    grads = []
    for i in range(2500):
        if i in (1000, 2000):
            grads += [torch.empty(0, device="cuda")] * 5
        grads.append(base[4 * i:4 * i + 4])
    norm = fp8.clip_grads(grads, 10.0)
    torch.cuda.synchronize()
    assert norm.item() == 100.0 and bool(((base - 0.1).abs() <= 2.0 ** -21 * 0.1).all())
