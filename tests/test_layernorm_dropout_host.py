"""Refusals of the layer norm's and the dropout's calls: bad arguments are
settled on the host before any device work.  CPU only: no call here reaches a GPU."""
import ctypes

import pytest
import torch

vp = ctypes.c_void_p
X, R, G, BE, H, MU, RS, Y, QR, SR, QC, SC = (vp(0x1000000 * i) for i in range(1, 13))


@pytest.fixture(scope="module")
def f():
    import fp8_linear_layer_gb300.build as b
    b.build()
    import fp8_linear_layer_gb300 as f
    f.lib()
    return f


NORM = dict(x=X, r=R, g=G, b=BE, rows=256, cols=512, ldx=512, ldr=512, eps=1e-6, fmt=0, h=H, mean=MU, rstd=RS, y=Y,
            qr=QR, sr=SR, sldr=256, qc=QC, sc=SC, sldc=512)


def block_norm(f, **k):
    return f.lib().fp8_layernorm_quantize(*dict(NORM, **k).values(), None)


@pytest.mark.parametrize("bad", [
    dict(fmt=2), dict(rows=-1), dict(cols=500, ldx=512, ldr=512), dict(cols=28800, ldx=28800, ldr=28800, sldc=28800),
    dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")),
    dict(x=None), dict(x=vp(0x1000008)), dict(ldx=504), dict(ldx=516), dict(r=vp(0x2000002)), dict(ldr=500),
    dict(h=None), dict(h=vp(0x5000002)), dict(g=None), dict(g=vp(0x3000004)), dict(b=vp(0x4000008)),
    dict(mean=None), dict(mean=vp(0x6000002)), dict(rstd=None), dict(rstd=vp(0x7000002)),
    dict(y=vp(0x8000001)), dict(y=None, qr=None, qc=None), dict(rows=100, sldr=100), dict(qr=vp(0x9000008)),
    dict(sr=None), dict(sldr=255), dict(sldr=252), dict(sc=None), dict(sldc=508), dict(sldc=514),
    dict(h=vp(0x1000010)),                        # h over x, not on it
    dict(h=X, ldx=520), dict(h=R, ldr=520),       # h on x or the residual, which are not packed
    dict(y=vp(0x1000000 + 256 * 512 * 2 - 16)),   # y over x's end
    dict(mean=vp(0x7000000 + 4 * 255)),           # mean over rstd's end
    dict(mean=vp(0x4000000 + 1020)),              # mean over beta's end
    dict(rstd=vp(0x3000000 + 1020)),              # rstd over gamma's end
    dict(sr=vp(0xB000010)),                       # scales inside the column codes
])
def test_norm_refusals(f, bad):
    assert block_norm(f, **bad) == f.binding.ERR_INVALID_ARG


def test_norm_of_nothing_is_a_no_op(f):
    assert block_norm(f, rows=0) == 0
    assert block_norm(f, cols=0) == 0


def test_mx_and_tensor_norm_refusals(f):
    E = f.binding.ERR_INVALID_ARG
    head = (X, R, G, BE, 256, 512, 512, 512, 1e-6, 0)
    mx = f.lib().fp8_mx_layernorm_quantize
    assert mx(*head, H, MU, RS, Y, QR, None, QC, SC, None) == E           # no scale bytes
    assert mx(*head, H, MU, RS, Y, QR, vp(0xA000008), QC, SC, None) == E  # misaligned
    assert mx(*head, H, MU, RS, Y, QR, SR, QC, vp(0xA000010), None) == E  # both scale arrays in one place
    assert mx(*head, H, None, RS, Y, QR, SR, QC, SC, None) == E
    ts = f.lib().fp8_tensor_layernorm_quantize
    am, sc, ao = vp(0xD000000), vp(0xE000000), vp(0xF000000)
    assert ts(*head, None, H, MU, RS, Y, QR, QC, sc, ao, None) == E
    assert ts(*head, am, H, MU, RS, Y, QR, QC, None, ao, None) == E
    assert ts(*head, am, H, MU, RS, Y, QR, QC, am, ao, None) == E         # the scale on the amax it is made of
    assert ts(*head, am, H, MU, RS, Y, QR, QC, sc, am, None) == E
    assert ts(*head, am, H, MU, RS, Y, QR, QC, sc, sc, None) == E
    assert ts(*head, am, H, am, RS, Y, QR, QC, sc, ao, None) == E         # the mean on the amax that is read
    assert ts(*head, vp(0xD000002), H, MU, RS, Y, QR, QC, sc, ao, None) == E


DG, DB, WS = vp(0xA000000), vp(0xB000000), vp(0xC000000)
BACK = dict(dy=X, h=H, g=G, mean=MU, rstd=RS, res=R, rows=100, cols=520, lddy=520, ldh=520, ldres=520, dx=Y, dgamma=DG,
            dbeta=DB, acc=0, ws=WS, bytes=1 << 30)


@pytest.mark.parametrize("bad,code", [
    (dict(cols=516), "E"), (dict(cols=28680), "E"), (dict(rows=-1), "E"), (dict(acc=2), "E"), (dict(dgamma=None), "E"),
    (dict(dgamma=vp(0xA000008)), "E"), (dict(dbeta=vp(0xB000008)), "E"), (dict(dy=None), "E"),
    (dict(dy=vp(0x1000008)), "E"), (dict(lddy=512), "E"), (dict(lddy=524), "E"), (dict(ldh=512), "E"),
    (dict(ldres=516), "E"), (dict(mean=None), "E"), (dict(rstd=None), "E"), (dict(dx=None), "E"),
    (dict(dx=vp(0x8000008)), "E"), (dict(dx=H), "E"), (dict(dx=X, lddy=528), "E"), (dict(dx=R, ldres=528), "E"),
    (dict(dgamma=G), "E"), (dict(dbeta=DG), "E"), (dict(dbeta=MU), "E"), (dict(dbeta=vp(0xA000000 + 2064)), "E"),
    (dict(ws=X), "E"), (dict(ws=vp(0xB000010)), "E"), (dict(rows=0, dbeta=DG), "E"),
    (dict(ws=None), "WS"), (dict(bytes=100 * 2 * 520 * 4 - 4), "WS"), (dict(ws=vp(0xC000008)), "WS"),
])
def test_backward_refusals(f, bad, code):
    want = f.binding.ERR_INVALID_ARG if code == "E" else f.binding.ERR_WORKSPACE
    assert f.lib().fp8_layernorm_backward(*dict(BACK, **bad).values(), None) == want


def test_workspace_size(f):
    size = f.lib().fp8_layernorm_workspace_size
    assert size(100, 520) == 100 * 2 * 520 * 4 and size(1 << 20, 4096) == 1024 * 2 * 4096 * 4
    assert size(0, 8) == size(8, 0) == size(8, 28680) == 0


DROP = dict(x=X, r=R, rows=100, cols=500, ldx=500, ldr=500, p=0.1, seed=1, site=2, step=3, step_dev=G, out=Y)


@pytest.mark.parametrize("bad", [
    dict(rows=-1), dict(cols=-1), dict(p=-0.1), dict(p=1.0), dict(p=float("nan")), dict(p=float("inf")),
    dict(x=None), dict(x=vp(0x1000001)), dict(r=vp(0x2000001)), dict(out=None), dict(out=vp(0x8000001)),
    dict(ldx=499), dict(ldr=499), dict(step_dev=vp(0x3000004)), dict(rows=1 << 20, cols=1 << 14, ldx=1 << 14, ldr=1 << 14),
    dict(rows=1 << 40, cols=1 << 40, ldx=1 << 40, ldr=1 << 40), dict(rows=1, cols=1 << 34, ldx=1 << 34, ldr=1 << 34),
    dict(ldx=1 << 36), dict(rows=1 << 33, cols=1, ldx=1 << 30, ldr=1),
    dict(out=vp(0x1000002)), dict(out=X, ldx=504), dict(out=R, ldr=504), dict(out=vp(0x2000000 + 100 * 500 * 2 - 2)),
    dict(step_dev=vp(0x8000000 + 8)),  # the counter inside the output
])
def test_dropout_refusals(f, bad):
    assert f.lib().fp8_dropout(*dict(DROP, **bad).values(), None) == f.binding.ERR_INVALID_ARG


def test_dropout_of_nothing_is_a_no_op(f):
    assert f.lib().fp8_dropout(*dict(DROP, rows=0).values(), None) == 0
    assert f.lib().fp8_dropout(*dict(DROP, cols=0).values(), None) == 0


class Placed(torch.Tensor):
    """A CPU tensor that says it is on GPU `where`."""
    is_cuda = True
    where = 0

    def get_device(self):
        return self.where


class Elsewhere(Placed):
    where = 1


@pytest.fixture
def spied(f, monkeypatch):
    from fp8_linear_layer_gb300 import block
    calls = []

    class Library:
        def __getattr__(self, name):
            return lambda *a: calls.append(name) or 0

    monkeypatch.setattr(block, "lib", lambda lib=Library(): lib)
    monkeypatch.setattr(block, "_stream", lambda: 0)
    monkeypatch.setattr(block, "_C", type("C", (), {"_cuda_getDevice": staticmethod(lambda: 0)}))
    return f, calls


U8, F32, I64 = torch.uint8, torch.float32, torch.int64
M, K = 128, 256


def tensors():
    z = lambda *s, t=torch.bfloat16: torch.zeros(*s, dtype=t)  # noqa: E731
    return dict(x=z(M, K), r=z(M, K), gamma=z(K), beta=z(K), h=z(M, K), y=z(M, K), mean=z(M, t=F32), rstd=z(M, t=F32),
                q=z(M, K, t=U8), q_c=z(K, M, t=U8), scale=z(2, M, t=F32), scale_c=z(1, K, t=F32), sf=z(2048, t=U8),
                sf_c=z(1024, t=U8), one=z(1, t=F32), amax=z(1, t=F32), amax_out=z(1, t=F32), dy=z(M, K),
                dgamma=z(K, t=F32), dbeta=z(K, t=F32), work=z(1 << 10, t=F32), step=z(1, t=I64), out=z(M, K))


def norm(recipe):
    def call(f, t):
        if recipe == "block":
            codes = f.Fp8Tensor(t["q"], t["scale"], 0), f.Fp8Tensor(t["q_c"], t["scale_c"], 0)
        elif recipe == "mx":
            codes = f.Fp8MxTensor(t["q"], t["sf"], 0), f.Fp8MxTensor(t["q_c"], t["sf_c"], 0)
        else:
            codes = f.Fp8TensorScaled(t["q"], t["one"], 0), f.Fp8TensorScaled(t["q_c"], t["one"], 0)
        out = f.LayerNorm(t["h"], t["rstd"], *codes, t["y"], t["amax_out"] if recipe == "tensor" else None, t["mean"])
        name = {"block": "layernorm_quantize", "mx": "mx_layernorm_quantize", "tensor": "tensor_layernorm_quantize"}
        amax = (t["amax"],) if recipe == "tensor" else ()
        getattr(f, name[recipe])(t["x"], t["gamma"], t["beta"], 1e-6, 0, *amax, residual=t["r"], out=out)
    return call


def backward(f, t):
    f.layernorm_backward(t["dy"], t["x"], t["gamma"], t["mean"], t["rstd"], t["r"], out=t["h"], dgamma=t["dgamma"],
                         dbeta=t["dbeta"], workspace=t["work"])


def drop(f, t):
    f.dropout(t["x"], 0.5, 1, 2, t["step"], residual=t["r"], out=t["out"])


NORM_USES = ["x", "r", "gamma", "beta", "h", "y", "mean", "rstd", "q", "q_c"]
USES = [(norm("block"), NORM_USES + ["scale", "scale_c"]), (norm("mx"), NORM_USES + ["sf", "sf_c"]),
        (norm("tensor"), NORM_USES + ["one", "amax", "amax_out"]),
        (backward, ["dy", "x", "gamma", "mean", "rstd", "r", "h", "dgamma", "dbeta", "work"]),
        (drop, ["x", "r", "step", "out"])]


@pytest.mark.parametrize("call,used", USES)
def test_tensors_off_the_current_device_are_refused(spied, call, used):
    f, calls = spied
    here = {k: v.as_subclass(Placed) for k, v in tensors().items()}
    call(f, here)
    assert len(calls) == 1
    for name in used:
        for elsewhere in (tensors()[name], tensors()[name].as_subclass(Elsewhere)):
            with pytest.raises(AssertionError):
                call(f, dict(here, **{name: elsewhere}))
    with pytest.raises(AssertionError):  # all together on another device than the current one
        call(f, {k: v.as_subclass(Elsewhere) for k, v in tensors().items()})
    assert len(calls) == 1


@pytest.mark.parametrize("call,used", USES)
def test_tensors_of_another_type_or_shape_are_refused(spied, call, used):
    f, calls = spied
    here = {k: v.as_subclass(Placed) for k, v in tensors().items()}
    for name in used:
        if name == "work":  # of any type: only its bytes count
            continue
        t = tensors()[name]
        for other in (t.to(torch.float64), t[:-1] if t.numel() > 1 else t.expand(2).contiguous()):
            with pytest.raises(AssertionError):
                call(f, dict(here, **{name: other.as_subclass(Placed)}))
    assert not calls


def test_the_layer_knows_how_many_scale_bytes_there_are(f):
    from fp8_linear_layer_gb300.block import _mx_bytes
    for rows in (1, 127, 128, 255, 256, 257, 1000):
        for k in (128, 384, 4096):
            assert _mx_bytes(rows, k) == f.mx_sf_bytes(rows, k)


def test_dropout_numbers_are_checked(spied):
    f, calls = spied
    x = torch.zeros(4, 8, dtype=torch.bfloat16).as_subclass(Placed)
    for bad in ((-1, 0, 0), (1 << 64, 0, 0), (0, -1, 0), (0, 1 << 32, 0), (0, 0, 1 << 63), (0, 0, -(1 << 63) - 1)):
        with pytest.raises(AssertionError):
            f.dropout(x, 0.5, *bad)
    assert not calls


def test_accumulate_and_bias_are_checked(spied):
    f, calls = spied
    t = {k: v.as_subclass(Placed) for k, v in tensors().items()}
    args = (t["dy"], t["x"], t["gamma"], t["mean"], t["rstd"])
    for bad in (dict(accumulate=True, dbeta=t["dbeta"]), dict(accumulate=True, dgamma=t["dgamma"]),
                dict(bias=False, dbeta=t["dbeta"])):
        with pytest.raises(AssertionError):
            f.layernorm_backward(*args, out=t["h"], workspace=t["work"], **bad)
    assert not calls
