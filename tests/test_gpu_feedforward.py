"""The residual feed-forward block: the norm, the products with their epilogues,
the norm's backward pass and the clipping strung together, against autograd of the same
block in fp32.

What fp8 operands leave: an e4m3 element is off by at most 2^-4 of itself (rms
2^-4 / sqrt(3) = 3.6%), an e5m2 one by 2^-3 (7.2%).  In a product's result, a sum
of many terms, the relative error in the 2-norm is that of its operands, added in
squares: Y's branch sqrt(4) x 3.6% at most (two products), the gradients of W2
sqrt(7.2^2 + 3.6^2), those of W1 and x behind one more product of each kind."""
import pytest
import torch

pytestmark = pytest.mark.gpu
M, K, N = 512, 384, 1024


def normal(g, *shape, std=1.0):
    return (std * torch.randn(*shape, generator=g)).bfloat16().cuda()


@pytest.fixture(scope="module")
def made(fp8):
    from fp8_linear_layer_gb300.feedforward import FeedForwardBlock
    g = torch.Generator().manual_seed(3)
    params = (1 + normal(g, K, std=0.2), normal(g, N, K, std=0.05), normal(g, N, std=0.2),
              normal(g, K, N, std=0.05), normal(g, K, std=0.2))
    block = FeedForwardBlock(M, K, N)
    block.load(*params)
    return block, params, (normal(g, M, K), normal(g, M, K, std=2.0), normal(g, M, K, std=1e-2))


def reference(params, x, r, dY):
    p = [t.float().requires_grad_() for t in params]
    gamma, W1, b1, W2, b2 = p
    h = (x.float() + r.float()).bfloat16().float().requires_grad_()
    y = h * torch.rsqrt(h.square().mean(1, keepdim=True) + 1e-6) * gamma
    u = torch.nn.functional.gelu(y @ W1.t() + b1, approximate="tanh")
    out = u @ W2.t() + b2 + h
    out.backward(dY.float())
    return h.detach(), out.detach(), h.grad, dict(zip(("dgamma", "dW1", "db1", "dW2", "db2"), (t.grad for t in p)))


def off(got, want):
    return float((got.float() - want).norm() / want.norm())


def test_a_training_step(fp8, made):
    block, params, (x, r, dY) = made
    block.zero_grad()
    Y = block.forward(x, r)
    dX = block.backward(dY)
    torch.cuda.synchronize()
    h, want, dh, grads = reference(params, x, r, dY)
    assert torch.equal(block.norm.h.float(), h)
    assert off(Y.float() - h, want - h) < 0.075  # the branch without the stream
    assert off(block.dW2, grads["dW2"]) < 0.1 and off(block.db2, grads["db2"]) < 2e-3
    assert off(block.dW1, grads["dW1"]) < 0.15 and off(block.db1, grads["db1"]) < 0.15
    assert off(dX.float() - dY.float(), dh - dY.float()) < 0.15 and off(block.dgamma, grads["dgamma"]) < 0.15
    # a second micro-batch adds up
    first = block.dW1.clone()
    block.forward(x, r)
    block.backward(dY)
    torch.cuda.synchronize()
    assert off(block.dW1, 2 * first) < 1e-6 and off(block.dgamma, 2 * grads["dgamma"]) < 0.15
    total = torch.stack([g.double().norm() for g in block.grads.grads]).norm()
    kept = block.dW2.clone()
    norm = block.clip(0.5 * float(total))
    torch.cuda.synchronize()
    assert abs(norm.item() - float(total)) < 1e-5 * float(total)
    assert off(block.dW2, 0.5 * kept) < 1e-5
    assert fp8.device_status() == 0


@pytest.mark.parametrize("tokens", [1, 7, 100])
def test_a_few_tokens_get_what_the_training_step_gives(fp8, made, tokens):
    block, params, (x, r, _) = made
    Y = block.forward(x, r).clone()
    got, h = block.decode(x[:tokens].contiguous(), r[:tokens].contiguous())
    torch.cuda.synchronize()
    # the same codes; sums in another order may move a GELU output to the neighbouring bf16, and that a code by a
    # step (2^-3 of it at the most) before the second product
    assert torch.equal(h, block.norm.h[:tokens])
    assert off(got.float() - h.float(), (Y[:tokens] - h).float()) < 2e-2


def test_a_step_in_a_graph(fp8, made):
    block, params, (x, r, dY) = made
    block.zero_grad()
    block.forward(x, r)
    block.backward(dY)
    block.clip(1e9)
    torch.cuda.synchronize()
    want = [g.clone() for g in block.grads.grads]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        block.forward(x, r)
        block.backward(dY)
        block.clip(1e9)
    block.zero_grad()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(block.grads.grads, want)) and fp8.device_status() == 0


def test_bias_gradients_add_up(fp8, made):
    block, _, (x, r, dY) = made
    block.zero_grad()
    block.forward(x, r)
    block.backward(dY)
    torch.cuda.synchronize()
    first = [block.db1.clone(), block.db2.clone()]
    block.forward(x, r)
    block.backward(dY)
    torch.cuda.synchronize()
    # twice the same sums: doubling is exact
    assert torch.equal(block.db1, 2 * first[0]) and torch.equal(block.db2, 2 * first[1])
    assert float(first[0].abs().max()) > 0 and float(first[1].abs().max()) > 0
