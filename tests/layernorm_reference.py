"""Plain 64-bit forms of the layer norm, its backward pass and the dropout's
generator, and what their rounded outputs may be off by.  Nothing here uses the
library."""
import numpy as np

from block_reference import FMAX, U, block_amax, f64, mx_bytes, step


def levels(cols):
    """Roundings on the way of a term into a row's sum: at most 64 terms follow one another in a thread, and ten levels
    of shuffles add the threads."""
    return min(cols, 64) + 12


def norm(x, residual, gamma, beta, eps):
    """In 64 bits: h (rounded to bf16), mean, rstd, y, and what the kernel's may be off by: mean, rstd (relative), y."""
    h = f64(x if residual is None else (x.float() + residual.float()).bfloat16())
    n, g = levels(h.shape[1]), f64(gamma)
    mean = h.mean(1)
    c = h - mean[:, None]
    rstd = 1.0 / np.sqrt((c * c).mean(1) + eps)
    xhat = c * rstd[:, None]
    y = xhat * g + (f64(beta) if beta is not None else 0.0)
    # the sum's roundings and the division's
    dmean = (n + 1) * U * np.abs(h).mean(1)
    # squares of deviations that are off by their own rounding and by dmean, which adds its square (the deviations add
    # up to 0); half of that is left by the root.  The division, the sum with eps and the reciprocal root follow.
    off = dmean * rstd
    drstd = ((n + 3) / 2 + 6) * U + 0.5 * off * off + U * off
    # the difference and its product with rstd round once each, the fused product and sum once
    dy = 1.01 * np.abs(g) * (np.abs(xhat) * (drstd + 2 * U)[:, None] + off[:, None]) + U * np.abs(y)
    return h, mean, rstd, y, dmean, drstd, dy


def check_codes(codes, scale, y, err, fmt, what):
    """codes (bytes) stand for y / scale, y known to within err: half a step, and three roundings of the factor."""
    import torch
    got = f64(codes.view(torch.float8_e4m3fn if fmt == 0 else torch.float8_e5m2))
    want = np.clip(y / scale, -FMAX[fmt], FMAX[fmt])
    slack = err / scale + 8 * U * np.abs(want)
    # where the value may lie on either side of a power of two the larger spacing counts
    bad = ~(np.abs(got - want) <= 0.5 * step(np.abs(want) + slack, fmt) * (1 + 1e-6) + slack)
    assert not bad.any(), "%s: %d codes off, first at %s: %r for %r" % (
        what, bad.sum(), np.argwhere(bad)[0], got[bad][0], want[bad][0])


def check_operand(t, recipe, y, err, what, amax=None):
    """An operand's codes and scales against y [rows][k] in 64 bits, known to within err."""
    rows, k = y.shape
    top = FMAX[t.fmt]
    if recipe == "block":
        s = f64(t.scale)[:, :rows].T
        a, e = block_amax(y, 128), block_amax(err, 128)
        assert np.all(np.abs(s - np.where(a > 0, a / top, 1.0)) <= e / top + 4 * U * s), what + ": scales"
        check_codes(t.q, np.repeat(s, 128, 1), y, err, t.fmt, what)
    elif recipe == "mx":
        b = mx_bytes(t.sf, rows, k)
        assert np.all(b[rows:] == 127), what + ": padding"
        a, d = block_amax(y, 32), block_amax(err, 32)
        e = b[:rows].astype(np.int64) - 127
        # the smallest exponent that holds the block
        assert np.all(a - d <= top * np.exp2(e)), what + ": a block saturates"
        assert np.all((a == 0) | (e == -127) | (a + d > top * np.exp2(e - 1.0))), what + ": scales too large"
        check_codes(t.q, np.repeat(np.exp2(e), 32, 1), y, err, t.fmt, what)
    else:
        s = float(t.scale.item())
        assert abs(s - amax / top) <= 2 * U * s
        check_codes(t.q, s, y, err, t.fmt, what)


def norm_backward(dy, h, gamma, mean, rstd, res):
    """In 64 bits: dx, the magnitude that its rounding errors scale with, dgamma, dbeta and their sums of magnitudes."""
    dy, c, g, r = f64(dy), f64(h) - f64(mean)[:, None], f64(gamma), f64(rstd)[:, None]
    xhat, d = c * r, dy * g
    m0, m = d.mean(1, keepdims=True), (d * xhat).mean(1, keepdims=True)
    dx = r * (d - m0 - xhat * m)
    size = np.abs(r) * (np.abs(d) + np.abs(d).mean(1, keepdims=True)
                        + np.abs(xhat) * np.abs(d * xhat).mean(1, keepdims=True))
    if res is not None:
        dx, size = dx + f64(res), size + np.abs(f64(res))
    return dx, size, (dy * xhat).sum(0), np.abs(dy * xhat).sum(0), dy.sum(0), np.abs(dy).sum(0)


def philox_words(n, seed, site, step):
    """The words of elements 0 .. n - 1: Philox4x32-10 as published (Salmon, Moraes, Dror and Shaw, 2011)."""
    low = np.uint64(0xFFFFFFFF)
    groups = -(-n // 4)
    step %= 1 << 64
    c = [np.arange(groups, dtype=np.uint64), np.full(groups, site, np.uint64),
         np.full(groups, step & 0xFFFFFFFF, np.uint64), np.full(groups, step >> 32, np.uint64)]
    k = [seed & 0xFFFFFFFF, seed >> 32]
    for _ in range(10):
        p0, p1 = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        c = [(p1 >> np.uint64(32)) ^ c[1] ^ np.uint64(k[0]), p1 & low,
             (p0 >> np.uint64(32)) ^ c[3] ^ np.uint64(k[1]), p0 & low]
        k = [(k[0] + 0x9E3779B9) & 0xFFFFFFFF, (k[1] + 0xBB67AE85) & 0xFFFFFFFF]
    return np.stack(c, 1).reshape(-1)[:n]
