"""Refusals of the gated product's calls: bad arguments are settled on the host
before any device work.  CPU only: no call here reaches a GPU."""
import ctypes

import pytest
import torch

vp = ctypes.c_void_p
Q, SC, QB, SB, BIAS, OUT, AUX = (0x1000000 * i for i in range(1, 8))
RECIPES = ["block", "mx", "tensor"]


@pytest.fixture(scope="module")
def f():
    import fp8_linear_layer_gb300.build as b
    b.build()
    import fp8_linear_layer_gb300 as f
    f.lib()
    return f


def call(f, recipe, grad, M=100, N=256, K=512, a=None, b=None, bias=BIAS, act=2, acc=0, out=OUT, aux=AUX):
    B = f.binding
    rows_b = N if grad else 2 * N
    if recipe == "block":
        ops = [B.OperandStruct(Q, SC, 512, 100, 0, 0), B.OperandStruct(QB, SB, 512, max(rows_b, 4), 0, 0)]
    elif recipe == "mx":
        ops = [B.MxOperandStruct(Q, SC, 512, 0, 0), B.MxOperandStruct(QB, SB, 512, 0, 0)]
    else:
        ops = [B.TensorOperandStruct(Q, SC, 512, 0, 0), B.TensorOperandStruct(QB, SB, 512, 0, 0)]
    for op, change in zip(ops, (a, b)):
        for k, v in (change or {}).items():
            setattr(op, k, v)
    name = {"block": "fp8_", "mx": "fp8_mx_", "tensor": "fp8_tensor_"}[recipe] + "gemm_gated" + ("_dgrad" if grad else "")
    args = [M, N, K, ctypes.byref(ops[0]), ctypes.byref(ops[1]), vp(aux) if grad else vp(bias), act]
    if recipe == "block":
        args.append(acc)
    args.append(vp(out))
    if not grad:
        args.append(vp(aux))
    return getattr(f.lib(), name)(*args, None)


BOTH = [dict(M=0), dict(M=-1), dict(N=0), dict(N=-128), dict(N=64), dict(N=200), dict(N=257), dict(K=0), dict(K=64),
        dict(K=500), dict(K=1 << 31), dict(N=1 << 31), dict(act=0), dict(act=3), dict(act=-1),
        dict(out=None), dict(out=OUT + 8), dict(aux=AUX + 8), dict(aux=OUT + 16), dict(out=AUX + 100 * 256 * 4 - 16),
        dict(a=dict(q=None)), dict(a=dict(q=Q + 8)), dict(a=dict(ld_q=496)), dict(a=dict(ld_q=520)), dict(a=dict(fmt=2)),
        dict(b=dict(q=None)), dict(b=dict(q=QB + 4)), dict(b=dict(ld_q=500)), dict(b=dict(fmt=-1))]


@pytest.mark.parametrize("recipe", RECIPES)
@pytest.mark.parametrize("grad", [False, True])
@pytest.mark.parametrize("bad", BOTH)
def test_refusals(f, recipe, grad, bad):
    assert call(f, recipe, grad, **bad) == f.binding.ERR_INVALID_ARG


@pytest.mark.parametrize("recipe", RECIPES)
def test_refusals_of_one_direction(f, recipe):
    E = f.binding.ERR_INVALID_ARG
    scale = "sf" if recipe == "mx" else "scale"
    assert call(f, recipe, False, bias=BIAS + 8) == E
    assert call(f, recipe, False, aux=OUT) == E                             # Z on Y
    assert call(f, recipe, False, bias=OUT + 512) == E                      # the bias inside Y
    assert call(f, recipe, False, bias=AUX + 512) == E                      # the bias inside Z
    assert call(f, recipe, True, aux=None) == E
    assert call(f, recipe, False, b={scale: None}) == E
    assert call(f, recipe, True, a={scale: SC + 2}) == E
    if recipe == "block":
        assert call(f, recipe, False, acc=2) == E and call(f, recipe, True, acc=-1) == E
        assert call(f, recipe, False, b=dict(scale_ld=508)) == E            # fewer scales than both projections' rows
        assert call(f, recipe, True, b=dict(scale_ld=252)) == E


def test_the_linear_product_takes_no_gate(f):
    B = f.binding
    a, b = B.OperandStruct(Q, SC, 512, 100, 0, 0), B.OperandStruct(QB, SB, 512, 256, 0, 0)
    assert f.lib().fp8_gemm_linear(100, 256, 512, ctypes.byref(a), ctypes.byref(b), None, B.ACT_SILU, None, 0, 0, vp(OUT),
                                   None, None) == B.ERR_INVALID_ARG


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


M, N, K = 100, 256, 512


def tensors(recipe, grad):
    z = lambda *s, t=torch.bfloat16: torch.zeros(*s, dtype=t)  # noqa: E731
    rows = N if grad else 2 * N
    if recipe == "block":
        sa, sb = z(K // 128, M, t=torch.float32), z(K // 128, rows, t=torch.float32)
    elif recipe == "mx":
        sa, sb = z(8 * K, t=torch.uint8), z(8 * K * -(-rows // 256), t=torch.uint8)
    else:
        sa, sb = z(1, t=torch.float32), z(1, t=torch.float32)
    t = dict(a=z(M, K, t=torch.uint8), sa=sa, b=z(rows, K, t=torch.uint8), sb=sb, aux=z(M, 2 * N))
    return dict(t, out=z(M, 2 * N)) if grad else dict(t, bias=z(2 * N), out=z(M, N))


def python_call(f, recipe, grad, t):
    kind = {"block": f.Fp8Tensor, "mx": f.Fp8MxTensor, "tensor": f.Fp8TensorScaled}[recipe]
    name = {"block": "", "mx": "mx_", "tensor": "tensor_"}[recipe] + ("gemm_gated_dgrad" if grad else "gemm_gated")
    a, b = kind(t["a"], t["sa"], 0), kind(t["b"], t["sb"], 0)
    if grad:
        return getattr(f, name)(a, b, t["aux"], out=t["out"])
    return getattr(f, name)(a, b, t["bias"], out=t["out"], aux=t["aux"])


@pytest.mark.parametrize("recipe", RECIPES)
@pytest.mark.parametrize("grad", [False, True])
def test_tensors_elsewhere_or_of_another_kind_are_refused(spied, recipe, grad):
    f, calls = spied
    here = {k: v.as_subclass(Placed) for k, v in tensors(recipe, grad).items()}
    python_call(f, recipe, grad, here)
    assert len(calls) == 1
    for name, t in tensors(recipe, grad).items():
        others = [t, t.as_subclass(Elsewhere), t.to(torch.float64).as_subclass(Placed)]
        others.append((t[:-1] if t.shape[0] > 1 else t.expand(2).contiguous()).as_subclass(Placed))
        if name == "a":
            others.pop()  # fewer tokens are another call, which the outputs' shapes refuse
        for other in others:
            with pytest.raises(AssertionError):
                python_call(f, recipe, grad, dict(here, **{name: other}))
    assert len(calls) == 1


def test_operands_of_another_recipe_are_refused(spied):
    f, calls = spied
    t = {k: v.as_subclass(Placed) for k, v in tensors("block", False).items()}
    mixed = f.Fp8Tensor(t["a"], t["sa"], 0), f.Fp8MxTensor(t["b"], t["sb"], 0)
    for fn in (f.gemm_gated, f.mx_gemm_gated, f.tensor_gemm_gated):
        with pytest.raises(AssertionError):
            fn(*mixed)
    odd = f.Fp8Tensor(t["b"][:511], t["sb"], 0)
    with pytest.raises(AssertionError):
        f.gemm_gated(f.Fp8Tensor(t["a"], t["sa"], 0), odd)
    assert not calls
