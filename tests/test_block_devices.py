"""The residual block's calls take tensors on the GPU alone: an address of host
memory never reaches a kernel.  CPU only: the library is a stand-in that says
whether it was called."""
import pytest

torch = pytest.importorskip("torch")


class OnGpu(torch.Tensor):
    """A CPU tensor that says it is on the GPU."""
    is_cuda = True


def gpu(*shape, dtype=torch.bfloat16):
    return torch.zeros(*shape, dtype=dtype).as_subclass(OnGpu)


@pytest.fixture
def f(monkeypatch):
    import fp8_linear_layer_gb300 as f
    from fp8_linear_layer_gb300 import block

    class Library:
        calls = 0

        def __getattr__(self, name):
            def call(*args):
                Library.calls += 1
                return 0
            return call

    monkeypatch.setattr(block, "lib", lambda lib=Library(): lib)
    monkeypatch.setattr(block, "_stream", lambda: 0)
    f.calls = lambda: Library.calls
    yield f
    del f.calls


U8, F32 = torch.uint8, torch.float32
M, K, N = 128, 256, 384


def norm(f, recipe, t):
    kind, name = {"block": (f.Fp8Tensor, "rmsnorm_quantize"), "mx": (f.Fp8MxTensor, "mx_rmsnorm_quantize"),
                  "tensor": (f.Fp8TensorScaled, "tensor_rmsnorm_quantize")}[recipe]
    scale_c = t["scale"] if recipe == "tensor" else t["scale_c"]
    out = f.RmsNorm(t["h"], t["rstd"], kind(t["q"], t["scale"], 0), kind(t["q_c"], scale_c, 0), t["y"],
                    t["amax_out"] if recipe == "tensor" else None)
    amax = (t["amax"],) if recipe == "tensor" else ()
    getattr(f, name)(t["x"], t["gamma"], 1e-6, 0, *amax, residual=t["r"], out=out)


def backward(f, recipe, t):
    f.rmsnorm_backward(t["dy"], t["x"], t["gamma"], t["rstd"], t["r"], out=t["h"], dgamma=t["dgamma"],
                       workspace=t["work"])


def product(f, recipe, t):
    kind, name = {"block": (f.Fp8Tensor, "gemm_linear"), "mx": (f.Fp8MxTensor, "mx_gemm_linear"),
                  "tensor": (f.Fp8TensorScaled, "tensor_gemm_linear")}[recipe]
    getattr(f, name)(kind(t["q"], t["scale"], 0), kind(t["w"], t["scale_w"], 0), t["bias"], f.ACT_GELU, t["res"],
                     out=t["out"], aux=t["aux"])


def tensors():
    return dict(x=gpu(M, K), r=gpu(M, K), gamma=gpu(K), h=gpu(M, K), y=gpu(M, K), dy=gpu(M, K),
                rstd=gpu(M, dtype=F32), dgamma=gpu(K, dtype=F32), work=gpu(M * K, dtype=F32),
                q=gpu(M, K, dtype=U8), q_c=gpu(K, M, dtype=U8), scale=gpu(2, M, dtype=F32), scale_c=gpu(1, K, dtype=F32),
                amax=gpu(1, dtype=F32), amax_out=gpu(1, dtype=F32), w=gpu(N, K, dtype=U8),
                scale_w=gpu(2, N, dtype=F32), bias=gpu(N), res=gpu(M, N), out=gpu(M, N), aux=gpu(M, N))


NORM = ["x", "r", "gamma", "h", "rstd", "y", "q", "q_c", "scale"]
CASES = [(norm, "block", NORM + ["scale_c"]), (norm, "mx", NORM + ["scale_c"]),
         (norm, "tensor", NORM + ["amax", "amax_out"]),
         (backward, None, ["dy", "x", "gamma", "rstd", "r", "h", "dgamma", "work"])]
CASES += [(product, r, ["q", "scale", "w", "scale_w", "bias", "res", "out", "aux"]) for r in ("block", "mx", "tensor")]


@pytest.mark.parametrize("call,recipe,names", CASES)
def test_every_tensor_is_on_the_gpu(f, call, recipe, names):
    call(f, recipe, tensors())
    assert f.calls() == 1
    for name in names:
        t = tensors()
        t[name] = torch.zeros(t[name].shape, dtype=t[name].dtype)
        with pytest.raises(AssertionError):
            call(f, recipe, t)
    assert f.calls() == 1


def test_gradients_off_the_gpu(f):
    for grads in ([torch.zeros(5)], f.GradList([torch.zeros(5), torch.zeros(0)])):
        made = f.calls()  # a list asks for the size of its workspace
        with pytest.raises(AssertionError, match="not on the GPU"):
            f.clip_grads(grads, 1.0)
        with pytest.raises(AssertionError, match="not on the GPU"):
            f.grad_norm(grads)
        assert f.calls() - made <= 2
