"""Dropout from the counter-based generator, added to a residual stream: masks
word for word against the published generator, values against 64 bits."""
import numpy as np
import pytest
import torch

import layernorm_reference as ref
from block_reference import U, f64

pytestmark = pytest.mark.gpu


def matrix(rows, cols, seed, ld=None, offset=0):
    """bf16 [rows][cols], rows ld apart, `offset` elements into its memory; NaN in between."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, cols, generator=g).bfloat16()
    ld = ld or cols
    flat = torch.full((rows * ld + offset,), float("nan"), dtype=torch.bfloat16, device="cuda")
    out = flat[offset:].view(rows, ld)[:, :cols]
    out.copy_(x)
    return out


def check(got, x, res, p, seed, site, step):
    kept = ref.philox_words(x.numel(), seed, site, step).reshape(tuple(x.shape)) >= np.uint64(int(p * 2 ** 32))
    want = np.where(kept, f64(x) / (1 - p), 0.0)
    # the factor's rounding and the fused product and sum's, then the output's
    err = U * np.abs(want)
    if res is not None:
        want = want + f64(res)
    assert np.all(np.abs(f64(got) - want) <= (2.0 ** -8 + 2 * U) * np.abs(want) + 1.01 * err)
    dropped = f64(got)[~kept]
    assert np.array_equal(dropped, f64(res)[~kept] if res is not None else np.zeros_like(dropped))


def test_published_vectors():
    # the generator's known answers for counters and keys of all zeros and all ones (the reference's own check)
    zero = ref.philox_words(4, 0, 0, 0)
    assert [hex(int(v)) for v in zero] == ["0x6627e8d5", "0xe169c58d", "0xbc57ac4c", "0x9b00dbd8"]


SIZES = [(1, 1), (1, 3), (1, 7), (1, 8), (3, 5), (2, 4), (7, 129), (129, 1001), (64, 1024), (1000, 2048), (33, 4096),
         (2500, 2048)]


@pytest.mark.parametrize("rows,cols", SIZES)
@pytest.mark.parametrize("with_residual", [False, True])
@pytest.mark.parametrize("p", [0.0, 0.1, 0.5, 0.9])
def test_masks_and_values(fp8, rows, cols, with_residual, p):
    seed, site, step = 0x123456789ABCDEF0 + rows, 3 + cols, (1 << 35) + 17
    x, res = matrix(rows, cols, 1), matrix(rows, cols, 2) if with_residual else None
    got = fp8.dropout(x, p, seed, site, step, residual=res)
    check(got, x, res, p, seed, site, step)


@pytest.mark.parametrize("rows,cols,ldx,ldr", [(5, 9, 9, 17), (33, 256, 264, 256), (33, 256, 256, 288), (33, 256, 257, 256),
                                               (40, 250, 256, 512), (1, 1000, 1003, 1001), (300, 4096, 4104, 4104),
                                               (1300, 1024, 1032, 1024)])
@pytest.mark.parametrize("offset", [0, 1, 8])
def test_any_layout_draws_the_same_mask(fp8, rows, cols, ldx, ldr, offset):
    x, res = matrix(rows, cols, 1, ldx, offset), matrix(rows, cols, 2, ldr, offset)
    plain = fp8.dropout(x.contiguous(), 0.3, 99, 4, 5, residual=res.contiguous())
    room = torch.full((rows * cols + 64,), 7.0, dtype=torch.bfloat16, device="cuda")
    out = room[offset:offset + rows * cols].view(rows, cols)
    got = fp8.dropout(x, 0.3, 99, 4, 5, residual=res, out=out)
    torch.cuda.synchronize()
    check(plain, x, res, 0.3, 99, 4, 5)
    assert torch.equal(got, plain) and got.data_ptr() == out.data_ptr()
    assert bool((room[:offset] == 7).all()) and bool((room[offset + rows * cols:] == 7).all())  # left as it was


def test_in_place(fp8):
    x, res = matrix(65, 1000, 1), matrix(65, 1000, 2)
    want = fp8.dropout(x, 0.2, 1, residual=res)
    for on in (0, 1):
        a, b = x.clone(), res.clone()
        got = fp8.dropout(a, 0.2, 1, residual=b, out=(a, b)[on])
        torch.cuda.synchronize()
        assert torch.equal(got, want) and torch.equal((b, a)[on], (res, x)[on])


def test_a_dropped_element_counts_as_zero_whatever_it_holds(fp8):
    x, res = matrix(64, 512, 1), matrix(64, 512, 2)
    words = ref.philox_words(x.numel(), 7, 0, 0).reshape(64, 512)
    dropped = torch.from_numpy(words < np.uint64(2 ** 31)).cuda()
    x[dropped] = float("nan")
    x[3, :8] = float("inf")
    for r in (None, res):
        got = fp8.dropout(x, 0.5, 7, residual=r)
        assert torch.equal(got[dropped], r[dropped] if r is not None else torch.zeros_like(got[dropped]))
        assert not bool(got.isnan().any()) and bool(got[3, :8][~dropped[3, :8]].isinf().all())


def test_seed_site_and_step_matter_and_nothing_else(fp8):
    x = torch.ones(64, 1024, dtype=torch.bfloat16, device="cuda")
    base = fp8.dropout(x, 0.5, 1, 2, 3)
    for other in ((2, 2, 3), (1 + (1 << 32), 2, 3), (1, 3, 3), (1, 2, 4), (1, 2, 3 + (1 << 32)), (1, 3, 2)):
        got = fp8.dropout(x, 0.5, *other)
        same = float((got == base).float().mean())
        assert abs(same - 0.5) < 6 * 0.5 / 256  # six deviations of 65536 fair coins
        check(got, x, None, 0.5, *other)
    assert torch.equal(fp8.dropout(x.mul(-1), 0.5, 1, 2, 3), -base)
    check(fp8.dropout(x, 0.5, (1 << 64) - 1, (1 << 32) - 1, -1), x, None, 0.5, (1 << 64) - 1, (1 << 32) - 1, -1)


@pytest.mark.parametrize("p", [1e-3, 0.1, 0.5, 0.99])
def test_how_many_are_dropped(fp8, p):
    n = 1 << 24
    got = fp8.dropout(torch.ones(4096, 4096, dtype=torch.bfloat16, device="cuda"), p, 12345, 1, 1)
    dropped = int((got == 0).sum())
    assert abs(dropped - p * n) <= 6 * (n * p * (1 - p)) ** 0.5


def test_the_gradient_is_the_same_call(fp8):
    # out = res + m x: against differences of sum(dy out), which is linear in x
    rows, cols, p, key = 9, 130, 0.25, (11, 1, 2)
    x, dy = matrix(rows, cols, 1), matrix(rows, cols, 3)
    dx = fp8.dropout(dy, p, *key)
    step = torch.zeros_like(x)
    for i, j in [(0, 0), (4, 77), (8, 129), (3, 5)]:
        step.zero_()
        step[i, j] = 1.0
        slope = f64(fp8.dropout(step, p, *key))[i, j] * f64(dy)[i, j]
        assert abs(f64(dx)[i, j] - slope) <= 2.0 ** -7 * abs(slope) + 0.0
    check(dx, dy, None, p, *key)


def test_step_on_the_device_counts_through_replays(fp8):
    x, res = matrix(40, 512, 1), matrix(40, 512, 2)
    step, out = torch.zeros(1, dtype=torch.int64, device="cuda"), torch.empty_like(x)
    fp8.dropout(x, 0.4, 5, 6, step, residual=res, out=out)  # first use outside the capture
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fp8.dropout(x, 0.4, 5, 6, step, residual=res, out=out)
        step.add_(1)
    for i in range(3):
        graph.replay()
        torch.cuda.synchronize()
        check(out, x, res, 0.4, 5, 6, i)
    step.fill_((1 << 40) + 3)
    x.mul_(2)
    graph.replay()
    check(out, x, res, 0.4, 5, 6, (1 << 40) + 3)


def test_empty_and_other_streams(fp8):
    assert fp8.dropout(torch.empty(0, 16, dtype=torch.bfloat16, device="cuda"), 0.5, 1).shape == (0, 16)
    x = matrix(512, 256, 2)
    want = fp8.dropout(x, 0.5, 1)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        late = torch.zeros_like(x)
        torch.cuda._sleep(20_000_000)  # the input is written behind a wait of this stream
        late.copy_(x)
        got = fp8.dropout(late, 0.5, 1)
    s.synchronize()
    assert torch.equal(got, want)


def test_more_than_two_to_the_31_elements(fp8):
    rows, cols = 1 << 16, (1 << 15) + 8  # 2^31 and 2^19 elements
    x = torch.ones(rows, cols, dtype=torch.bfloat16, device="cuda")
    got = fp8.dropout(x, 0.5, 21, 1, 1)
    gaps = torch.ones(rows, cols + 8, dtype=torch.bfloat16, device="cuda")[:, :cols]
    assert torch.equal(fp8.dropout(gaps, 0.5, 21, 1, 1), got)
    # the words of the last elements, their groups counted from the start
    first = rows * cols - 4096
    words = torch.from_numpy(last_words(first, 4096, 21, 1, 1) >= np.uint64(2 ** 31)).cuda()
    assert torch.equal(got.view(-1)[-4096:] != 0, words)


def test_rows_of_more_than_two_to_the_32_columns_with_gaps(fp8):
    rows, cols, tail = 2, (1 << 32) + 8, 64
    room = torch.zeros(rows, cols + 8, dtype=torch.bfloat16, device="cuda")  # 17 GB
    x, res = room[:, :cols], room[:, 8:]  # each row of the residual lies 8 elements behind the row of x
    room[:, -tail:] = matrix(rows, tail, 1)
    got = fp8.dropout(x, 0.5, 21, 1, 1, residual=res)
    for r in range(rows):
        first = r * cols + cols - tail
        kept = torch.from_numpy(last_words(first, tail, 21, 1, 1) >= np.uint64(2 ** 31)).cuda()
        want = torch.where(kept, 2 * x[r, -tail:].float(), 0.0) + res[r, -tail:].float()  # p = 1/2: one rounding
        assert torch.equal(got[r, -tail:], want.bfloat16())


def last_words(first, n, seed, site, step):
    """Words first .. first + n - 1 (first a multiple of 4) without those before."""
    low, half = np.uint64(0xFFFFFFFF), np.uint64(32)
    c = [np.arange(first // 4, (first + n) // 4, dtype=np.uint64), np.uint64(site), np.uint64(step), np.uint64(0)]
    k = [seed, 0]
    for _ in range(10):
        p0, p1 = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        c = [(p1 >> half) ^ c[1] ^ np.uint64(k[0]), p1 & low, (p0 >> half) ^ c[3] ^ np.uint64(k[1]), p0 & low]
        k = [(k[0] + 0x9E3779B9) & 0xFFFFFFFF, (k[1] + 0xBB67AE85) & 0xFFFFFFFF]
    return np.stack(np.broadcast_arrays(*c), 1).reshape(-1)
