"""The gated feed-forward block: dropout into the stream, layer norm, the gated
product, its data gradient and the layer norm's backward pass strung together, against
autograd of the same block in fp32.

What fp8 operands leave: an e4m3 element is off by at most 2^-4 of itself (rms
2^-4 / sqrt(3) = 3.6%), an e5m2 one by 2^-3 (7.2%).  In a product's result, a sum
of many terms, the relative error in the 2-norm is that of its operands, added in
squares: sqrt(2) x 3.6% = 5.1% for each projection, which the gate multiplies, and one
more e4m3 operand pair behind them: Y's branch 5.1% x sqrt(2) and 5.1%, 8.9%.  The
gradient at Z comes of an e5m2 and an e4m3 operand (8.0%) and of the rounded Z of
5.1% in both factors (7.2%), 10.8%, and is cast to e5m2 for what is behind it: 13%,
with the other operand's 3.6% 13.5%, in each of two products' worth 14%."""
import numpy as np
import pytest
import torch

import layernorm_reference as ref

pytestmark = pytest.mark.gpu
M, K, N, P, SEED, SITE = 512, 384, 640, 0.3, 1234567890123, 9


def normal(g, *shape, std=1.0):
    return (std * torch.randn(*shape, generator=g)).bfloat16().cuda()


@pytest.fixture(scope="module", params=["silu", "gelu"])
def made(fp8, request):
    from fp8_linear_layer_gb300.feedforward import GatedFeedForwardBlock
    g = torch.Generator().manual_seed(3)
    params = (1 + normal(g, K, std=0.2), normal(g, K, std=0.2), normal(g, 2 * N, K, std=0.05), normal(g, 2 * N, std=0.2),
              normal(g, K, N, std=0.05), normal(g, K, std=0.2))
    block = GatedFeedForwardBlock(M, K, N, p=P, act=fp8.ACT_SILU if request.param == "silu" else fp8.ACT_GELU, seed=SEED,
                                  site=SITE)
    block.load(*params)
    return block, params, (normal(g, M, K), normal(g, M, K, std=2.0), normal(g, M, K, std=1e-2)), request.param


def kept(step):
    return torch.from_numpy(ref.philox_words(M * K, SEED, SITE, step).reshape(M, K) >= np.uint64(int(P * 2 ** 32))).cuda()


def branch(act, h, gamma, beta, W1, b1, W2, b2):
    z = torch.nn.functional.layer_norm(h, (K,), gamma, beta, 1e-5) @ W1.t() + b1
    gate = torch.nn.functional.silu(z[:, :N]) if act == "silu" else torch.nn.functional.gelu(z[:, :N], approximate="tanh")
    return (gate * z[:, N:]) @ W2.t() + b2


def reference(act, params, x, r, dY, mask):
    p = [t.float().requires_grad_() for t in params]
    x, r = x.float().requires_grad_(), r.float().requires_grad_()
    h = torch.where(mask, x / (1 - P), torch.zeros_like(x)) + r
    h = h + (h.bfloat16().float() - h).detach()  # the stream's rounding, which passes gradients on
    out = branch(act, h, *p) + h
    out.backward(dY.float())
    return h.detach(), out.detach(), x.grad, r.grad, dict(zip(("dgamma", "dbeta", "dW1", "db1", "dW2", "db2"),
                                                              (t.grad for t in p)))


def off(got, want):
    return float((got.float() - want).norm() / want.norm())


def test_a_training_step(fp8, made):
    block, params, (x, r, dY), act = made
    block.zero_grad()
    block.step.fill_(5)
    Y = block.forward(x, r)
    dX, dh = block.backward(dY)
    torch.cuda.synchronize()
    h, want, dx, dr, grads = reference(act, params, x, r, dY, kept(5))
    # the stream: one rounding of the fused sum where torch's fp32 has three, a bf16 neighbour at a few elements
    assert off(block.h, h) < 2.0 ** -9 and float((block.h.float() != h).float().mean()) < 1e-3
    assert off(Y.float() - block.h.float(), want - h) < 0.09
    assert off(block.dW2, grads["dW2"]) < 0.13 and off(block.db2, grads["db2"]) < 2e-3
    assert off(block.dW1, grads["dW1"]) < 0.15 and off(block.db1, grads["db1"]) < 0.15
    assert off(dh.float() - dY.float(), dr - dY.float()) < 0.15
    assert off(block.dgamma, grads["dgamma"]) < 0.15 and off(block.dbeta, grads["dbeta"]) < 0.15
    # the same mask in both directions
    assert torch.equal(dX != 0, kept(5) & (dh != 0)) and off(dX, torch.where(kept(5), dh.float() / (1 - P), 0.0)) < 2.0 ** -8
    assert int(block.step) == 6
    # a second micro-batch has another mask, and its gradients add up
    first = {n: getattr(block, n).clone() for n in grads}
    block.forward(x, r)
    block.backward(dY)
    torch.cuda.synchronize()
    h2, _, _, _, more = reference(act, params, x, r, dY, kept(6))
    assert off(block.h, h2) < 2.0 ** -9 and not torch.equal(h2, h)
    for n in grads:
        assert off(getattr(block, n) - first[n], more[n]) < 0.15, n
    total = torch.stack([g.double().norm() for g in block.grads.grads]).norm()
    kept_grad = block.dW2.clone()
    norm = block.clip(0.5 * float(total))
    torch.cuda.synchronize()
    assert abs(norm.item() - float(total)) < 1e-5 * float(total) and off(block.dW2, 0.5 * kept_grad) < 1e-5
    assert fp8.device_status() == 0


@pytest.mark.parametrize("tokens", [1, 7, 100, 300])
def test_a_few_tokens_get_what_a_step_without_dropout_gives(fp8, made, tokens):
    block, params, (x, r, _), act = made
    block.p = 0.0
    Y = block.forward(x, r).clone()
    block.p = P
    got, h = block.decode(x[:tokens].contiguous(), r[:tokens].contiguous())
    torch.cuda.synchronize()
    # the same codes; sums in another order may move an output of the gate to the neighbouring bf16, and that a code by
    # a step (2^-3 of it at the most) before the second product
    assert torch.equal(h, block.h[:tokens])
    assert off(got.float() - h.float(), (Y[:tokens] - h).float()) < 2e-2


def test_a_step_in_a_graph(fp8, made):
    block, params, (x, r, dY), act = made
    want = []
    for step in (0, 1):
        block.step.fill_(step)
        block.zero_grad()
        block.forward(x, r)
        dX, dh = block.backward(dY)
        block.clip(1e9)
        torch.cuda.synchronize()
        want.append([t.clone() for t in [dX, dh] + block.grads.grads])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        block.forward(x, r)
        block.backward(dY)
        block.clip(1e9)
    block.step.zero_()
    for step in (0, 1):  # the captured step counts: each replay has its own mask
        block.zero_grad()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip([block.dX, block.dh] + block.grads.grads, want[step]))
    assert fp8.device_status() == 0 and not torch.equal(want[0][0], want[1][0])
