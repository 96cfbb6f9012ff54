"""Plain 64-bit forms of the residual block's operators, and what an fp8 code
may be off by, for the tests.  Nothing here uses the library."""
import numpy as np
import torch

FMAX = {0: 448.0, 1: 57344.0}
U = 2.0 ** -24  # half an fp32 ulp, relative


def f64(t):
    return t.detach().cpu().double().numpy() if t.dtype == torch.float64 else t.detach().float().cpu().double().numpy()


def norm(x, residual, gamma, eps):
    """(h rounded to bf16, rstd, y) in 64 bits."""
    h = x if residual is None else (x.float() + residual.float()).bfloat16()
    h = f64(h)
    rstd = 1.0 / np.sqrt((h * h).mean(1) + eps)
    return h, rstd, h * rstd[:, None] * f64(gamma)


def norm_backward(dy, h, gamma, rstd, res):
    dy, h, g, r = f64(dy), f64(h), f64(gamma), f64(rstd)[:, None]
    xhat, d = h * r, dy * g
    m = (d * xhat).mean(1, keepdims=True)
    dx = r * (d - xhat * m)
    # every term of the sums above in magnitude: what the rounding errors scale with
    size = np.abs(r) * (np.abs(d) + np.abs(xhat) * np.abs(d * xhat).mean(1, keepdims=True))
    if res is not None:
        dx, size = dx + f64(res), size + np.abs(f64(res))
    return dx, size, (dy * xhat).sum(0), np.abs(dy * xhat).sum(0)


def step(v, fmt):
    """Spacing of the fp8 format at |v| (subnormal spacing below the normal range)."""
    bits, low = (3, -6) if fmt == 0 else (2, -14)
    _, e = np.frexp(np.abs(v))
    return np.ldexp(1.0, np.maximum(e - 1, low) - bits)


def check_codes(codes, scale, y, fmt, rel, what):
    """codes (bytes) stand for y / scale: each within half a step of it, or of a value `rel` away from it."""
    got = codes.view(torch.float8_e4m3fn if fmt == 0 else torch.float8_e5m2)
    got = f64(got)
    want = np.clip(y / scale, -FMAX[fmt], FMAX[fmt])
    bound = 0.5 * step(want, fmt) * (1 + 1e-6) + rel * np.abs(want)
    # at a power of two the spacing below is half of the one above: both sides are covered by the larger
    bad = ~(np.abs(got - want) <= bound)
    assert not bad.any(), "%s: %d codes off, first at %s: %r for %r" % (
        what, bad.sum(), np.argwhere(bad)[0], got[bad][0], want[bad][0])


def block_amax(y, width):
    return np.abs(y.reshape(y.shape[0], -1, width)).max(2)


def mx_bytes(sf, rows, k):
    """Scale bytes in the GEMM's order -> [padded rows][k / 32]."""
    groups = 2 * -(-rows // 256)
    return sf.cpu().numpy().reshape(k // 128, groups, 32, 4, 4).transpose(1, 3, 2, 0, 4).reshape(groups * 128, k // 32)


def check_operand(t, recipe, y, rel, what, amax=None):
    """An operand's codes and scales against y [rows][k] in 64 bits."""
    rows, k = y.shape
    if recipe == "block":
        s = f64(t.scale)[:, :rows].T
        a = block_amax(y, 128)
        want = np.where(a > 0, a / FMAX[t.fmt], 1.0)
        assert np.all(np.abs(s - want) <= (rel + 4 * U) * want), what + ": scales"
        check_codes(t.q, np.repeat(s, 128, 1), y, t.fmt, rel + 8 * U, what)
    elif recipe == "mx":
        b = mx_bytes(t.sf, rows, k)
        assert np.all(b[rows:] == 127), what + ": padding"
        a = block_amax(y, 32)
        e = b[:rows].astype(np.int64) - 127
        top = FMAX[t.fmt]
        # the smallest exponent that holds the block, of an amax up to `rel` away
        assert np.all(a * (1 - rel) <= top * np.exp2(e)), what + ": a block saturates"
        assert np.all((a == 0) | (e == -127) | (a * (1 + rel) > top * np.exp2(e - 1.0))), what + ": scales too large"
        assert np.all(e[a == 0] == 0), what + ": empty blocks"
        check_codes(t.q, np.repeat(np.exp2(e), 32, 1), y, t.fmt, rel + 4 * U, what)
    else:
        s = float(t.scale.item())
        assert abs(s - amax / FMAX[t.fmt]) <= U * 2 * s
        check_codes(t.q, s, y, t.fmt, rel + 8 * U, what)
