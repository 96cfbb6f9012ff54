"""Refusals of the residual block's calls: bad arguments are settled on the
host before any device work.  CPU only: no call here reaches a GPU."""
import ctypes

import pytest

vp = ctypes.c_void_p
X, R, G, H, RS, Y, QR, SR, QC, SC = (vp(0x1000000 * i) for i in range(1, 11))


@pytest.fixture(scope="module")
def f():
    import fp8_linear_layer_gb300.build as b
    b.build()
    import fp8_linear_layer_gb300 as f
    f.lib()
    return f


NORM = dict(x=X, r=R, g=G, rows=256, cols=512, ldx=512, ldr=512, eps=1e-6, fmt=0, h=H, rstd=RS, y=Y, qr=QR, sr=SR,
            sldr=256, qc=QC, sc=SC, sldc=512)


def block_norm(f, **k):
    a = dict(NORM, **k)
    return f.lib().fp8_rmsnorm_quantize(*a.values(), None)


@pytest.mark.parametrize("bad", [
    dict(fmt=2), dict(rows=-1), dict(cols=500, ldx=512, ldr=512), dict(cols=32896, ldx=32896, ldr=32896, sldc=32896),
    dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")),
    dict(x=None), dict(x=vp(0x1000008)), dict(ldx=504), dict(ldx=516), dict(r=vp(0x2000002)), dict(ldr=500),
    dict(h=None), dict(h=vp(0x4000002)), dict(g=None), dict(g=vp(0x3000004)), dict(rstd=None), dict(rstd=vp(0x5000002)),
    dict(y=vp(0x6000001)), dict(y=None, qr=None, qc=None), dict(rows=100, sldr=100), dict(qr=vp(0x7000008)),
    dict(sr=None), dict(sldr=255), dict(sldr=252), dict(sc=None), dict(sldc=508), dict(sldc=514),
    dict(h=vp(0x1000010)),                       # h over x, not on it
    dict(h=X, ldx=520), dict(h=R, ldr=520),      # h on x or the residual, which are not packed
    dict(y=vp(0x1000000 + 256 * 512 * 2 - 16)),  # y over x's end
    dict(qr=vp(0x4000000 + 256 * 512 * 2 - 16)),  # codes over h's end
    dict(sr=vp(0x9000010)),                      # scales inside the column codes
    dict(rstd=vp(0x3000000 + 1020)),             # rstd over gamma's end
])
def test_norm_refusals(f, bad):
    assert block_norm(f, **bad) == f.binding.ERR_INVALID_ARG


def test_norm_of_nothing_is_a_no_op(f):
    assert block_norm(f, rows=0) == 0
    assert block_norm(f, cols=0) == 0


def test_mx_and_tensor_norm_refusals(f):
    E = f.binding.ERR_INVALID_ARG
    L = f.lib()
    head = (X, R, G, 256, 512, 512, 512, 1e-6, 0)
    mx = L.fp8_mx_rmsnorm_quantize
    assert mx(*head, H, RS, Y, QR, None, QC, SC, None) == E           # no scale bytes
    assert mx(*head, H, RS, Y, QR, vp(0x8000008), QC, SC, None) == E  # misaligned
    assert mx(*head, H, RS, Y, QR, SR, QC, vp(0x8000010), None) == E  # both scale arrays in one place
    ts = L.fp8_tensor_rmsnorm_quantize
    am, sc, ao = vp(0xB000000), vp(0xC000000), vp(0xD000000)
    assert ts(*head, None, H, RS, Y, QR, QC, sc, ao, None) == E
    assert ts(*head, am, H, RS, Y, QR, QC, None, ao, None) == E
    assert ts(*head, am, H, RS, Y, QR, QC, am, ao, None) == E         # the scale on the amax it is made of
    assert ts(*head, am, H, RS, Y, QR, QC, sc, am, None) == E
    assert ts(*head, am, H, RS, Y, QR, QC, sc, sc, None) == E
    assert ts(*head, vp(0xB000002), H, RS, Y, QR, QC, sc, ao, None) == E


BACK = dict(dy=X, h=H, g=G, rstd=RS, res=R, rows=100, cols=520, lddy=520, ldh=520, ldres=520, dx=Y, dgamma=SR,
            acc=0, ws=QC, bytes=1 << 30)


@pytest.mark.parametrize("bad,code", [
    (dict(cols=516), "E"), (dict(cols=32776), "E"), (dict(rows=-1), "E"), (dict(acc=2), "E"), (dict(dgamma=None), "E"),
    (dict(dgamma=vp(0x8000008)), "E"), (dict(dy=None), "E"), (dict(dy=vp(0x1000008)), "E"), (dict(lddy=512), "E"),
    (dict(lddy=524), "E"), (dict(ldh=512), "E"), (dict(ldres=516), "E"), (dict(rstd=None), "E"), (dict(dx=None), "E"),
    (dict(dx=vp(0x6000008)), "E"), (dict(dx=H), "E"), (dict(dx=X, lddy=528), "E"), (dict(dx=R, ldres=528), "E"),
    (dict(dgamma=G), "E"), (dict(ws=X), "E"), (dict(ws=vp(0x8000010)), "E"),
    (dict(ws=None), "WS"), (dict(bytes=100 * 520 * 4 - 4), "WS"), (dict(ws=vp(0x9000008)), "WS"),
])
def test_norm_backward_refusals(f, bad, code):
    want = f.binding.ERR_INVALID_ARG if code == "E" else f.binding.ERR_WORKSPACE
    assert f.lib().fp8_rmsnorm_backward(*dict(BACK, **bad).values(), None) == want


def test_norm_backward_workspace(f):
    ws = f.lib().fp8_rmsnorm_workspace_size
    assert ws(0, 128) == 0 and ws(5, 0) == 0 and ws(5, 1 << 20) == 0
    assert ws(3, 256) == 3 * 256 * 4
    assert ws(1 << 20, 256) == ws(1 << 21, 256)  # partial sums do not grow with the rows for ever
    assert f.lib().fp8_rmsnorm_backward(*dict(BACK, cols=0).values(), None) == 0


def test_gradient_list_refusals(f):
    E, WS = f.binding.ERR_INVALID_ARG, f.binding.ERR_WORKSPACE
    L, S = f.lib(), f.binding.GradStruct
    need = L.fp8_grad_norm_workspace_size(2)
    norm, ws = vp(0x10000), vp(0x20000)

    def call(entries, max_norm=1.0, norm=norm, ws=ws, bytes=need, count=None):
        t = (S * len(entries))(*[S(*e) for e in entries])
        return L.fp8_clip_grads(len(entries) if count is None else count, t, max_norm, norm, ws, bytes, None)

    ok = (0x1000000, 0x2000000, 100, 0, 0)
    assert call([ok], count=-1) == E
    assert call([ok], max_norm=-1.0) == E and call([ok], max_norm=float("nan")) == E
    assert call([ok], norm=None) == E and call([ok], norm=vp(0x10002)) == E
    assert call([(None, 0x2000000, 100, 0, 0)]) == E
    assert call([(0x1000000, None, 100, 0, 0)]) == E
    assert call([(0x1000002, 0x2000000, 100, 0, 0)]) == E      # fp32 on a 2-byte boundary
    assert call([(0x1000001, 0x2000000, 100, 1, 0)]) == E
    assert call([(0x1000000, 0x2000000, -1, 0, 0)]) == E
    assert call([(0x1000000, 0x2000000, 100, 2, 0)]) == E      # type
    assert call([(0x1000000, 0x1000000 + 16, 100, 0, 0)]) == E  # out over its own gradient, not on it
    assert call([(0x10000 - 16, 0x2000000, 100, 0, 0)]) == E   # the norm inside a gradient
    assert call([(0x1000000, 0x20000, 100, 0, 0)]) == E        # out inside the workspace
    assert call([ok, (0x3000000, 0x4000000, 1 << 41, 0, 0)]) == E
    assert call([ok], bytes=need - 4 - L.fp8_grad_norm_workspace_size(2) + L.fp8_grad_norm_workspace_size(1)) == WS
    assert call([ok], ws=None) == WS and call([ok], ws=vp(0x20008)) == WS
    assert L.fp8_grad_norm_workspace_size(-1) == 0
    assert L.fp8_grad_norm_workspace_size(5000) > L.fp8_grad_norm_workspace_size(500) > 0


def test_extents_beyond_64_bits_are_refused(f):
    E = f.binding.ERR_INVALID_ARG
    far = (1 << 36) - 8
    many = dict(rows=(1 << 31) - 1, qc=None, sc=None, sldr=1 << 31)
    assert block_norm(f, **dict(many, ldx=far)) == E
    assert block_norm(f, **dict(many, ldr=far)) == E
    for ld in ("lddy", "ldh", "ldres"):
        assert f.lib().fp8_rmsnorm_backward(*dict(BACK, **{"rows": (1 << 31) - 1, ld: far}).values(), None) == E


@pytest.mark.parametrize("views,apart", [
    ([(0, 100), (100, 200)], True),
    ([(0, 100), (0, 100)], False),             # a shared weight listed twice
    ([(0, 100), (99, 120)], False),
    ([(0, 300), (20, 40)], False),             # one inside another
    ([(0, 10), (50, 50), (10, 20)], True),     # an empty one
])
def test_overlapping_gradients(f, views, apart):
    torch = pytest.importorskip("torch")
    t = torch.zeros(300)
    g = f.GradList([t[a:b] for a, b in views])
    assert g._apart is apart
    # with outputs elsewhere the gradients may overlap, the outputs may not
    o = [torch.zeros(b - a) for a, b in views]
    assert f.GradList([t[a:b] for a, b in views], o)._apart is True
    assert f.GradList(o, [t[a:b] for a, b in views])._apart is apart
    if not apart:
        with pytest.raises(AssertionError, match="overlaps"):
            f.clip_grads(g, 1.0)


def test_output_over_another_gradient(f):
    torch = pytest.importorskip("torch")
    a, b = torch.zeros(64), torch.zeros(64)
    assert f.GradList([a, b], [torch.zeros(64), a])._apart is False
    assert f.GradList([a, b], [a, b])._apart is True
    assert f.GradList([a, b], [b, a])._apart is False
