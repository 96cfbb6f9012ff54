"""Pre-norm residual feed-forward blocks on the FP8 linear layer's GEMMs: one
training step's forward and backward pass with gradient clipping, and the same
block on a few tokens.  ``FeedForwardBlock``, with RMS norm and GELU:

    h = x + r                                              (the residual stream)
    N = rmsnorm(h) gamma        --cast from fp32: rows and columns, e4m3-->
    Z = N W1^T + b1,  U = gelu(Z)    --rows and columns, e4m3-->
    Y = U W2^T + b2 + h                                    (one epilogue)

    dY --one read: rows, columns (e5m2), db2-->
    dW2 += dY^T U
    dZ = (dY W2) gelu'(Z)  --one read: rows, columns (e5m2), db1-->
    dW1 += dZ^T N
    dN = dZ W1
    dh = rmsnorm'(dN) + dY,  dgamma                        (dh: the gradient of x and of r)

``GatedFeedForwardBlock``, with dropout on the way into the stream, layer norm and a
gate (W1 holds the gate's n rows, then the up projection's):

    h = r + dropout(x)
    N = layernorm(h) gamma + beta   --cast from fp32: rows and columns, e4m3-->
    Z = N W1^T + b1 [m][2 n],  U = act(Z[:, :n]) Z[:, n:]      (one kernel)
    Y = U W2^T + b2 + h

    dY, dW2, db2 as above
    dZ = (dY W2) through the gate [m][2 n]                     (one kernel)
    dZ's casts, db1, dW1, dN as above, with 2 n features
    dh = layernorm'(dN) + dY,  dgamma, dbeta                   (dh: the gradient of r)
    dx = dropout(dh), the mask drawn again

No arithmetic here but the bias gradients' sum over calls and the dropout's
count of steps: every step is a library kernel.  Run as a module for the time of a step: ``python -m
fp8_linear_layer_gb300.feedforward``.
"""
import torch

from . import binding as B
from . import block as K


class FeedForwardBlock:
    """tokens m, width k, hidden width n, in the 1x128 recipe; m, k and n multiples
    of 128.  Gradients accumulate in fp32 over calls of ``backward`` until
    ``zero_grad``; ``clip`` scales them in place."""

    def __init__(self, m: int, k: int, n: int, eps: float = 1e-6, device="cuda"):
        assert m % 128 == 0 and k % 128 == 0 and n % 128 == 0
        self.m, self.k, self.n, self.eps = m, k, n, eps
        dev = torch.device(device)

        def bf16(*shape):
            return torch.empty(shape, dtype=torch.bfloat16, device=dev)

        def f32(*shape):
            return torch.zeros(shape, dtype=torch.float32, device=dev)

        # weights, by rows for the forward products and down their columns for the gradients'
        self.W1q, self.W1Tq = B.empty_fp8(n, k, B.E4M3, dev), B.empty_fp8(k, n, B.E4M3, dev)
        self.W2q, self.W2Tq = B.empty_fp8(k, n, B.E4M3, dev), B.empty_fp8(n, k, B.E4M3, dev)
        self.norm = K.empty_rmsnorm(m, k, B.E4M3, cols_too=True, residual=True, device=dev)
        self.Z, self.U = bf16(m, n), bf16(m, n)
        self.Uq, self.UTq = B.empty_fp8(m, n, B.E4M3, dev), B.empty_fp8(n, m, B.E4M3, dev)
        self.Y = bf16(m, k)
        self.dYq, self.dYTq = B.empty_fp8(m, k, B.E5M2, dev), B.empty_fp8(k, m, B.E5M2, dev)
        self.dZ = bf16(m, n)
        self.dZq, self.dZTq = B.empty_fp8(m, n, B.E5M2, dev), B.empty_fp8(n, m, B.E5M2, dev)
        self.dN, self.dX = bf16(m, k), bf16(m, k)
        self.dW1, self.dW2 = f32(n, k), f32(k, n)
        self.db1, self.db2, self.dgamma = f32(n), f32(k), f32(k)
        self.db1_new, self.db2_new = f32(n), f32(k)  # one call's
        self.grads = K.GradList([self.dW1, self.dW2, self.db1, self.db2, self.dgamma])
        self.cast_work = torch.empty((B.workspace_size(m, max(k, n)) // 4,), dtype=torch.float32, device=dev)
        self.norm_work = K.rmsnorm_workspace(m, k, dev)

    def load(self, gamma, W1, b1, W2, b2):
        """Take the parameters (bf16: gamma [k], W1 [n][k], b1 [n], W2 [k][n], b2 [k])
        and cast the weights; again after every optimizer step."""
        self.gamma, self.b1, self.b2 = gamma, b1, b2
        B.quantize_dual(W1, B.E4M3, out=self.W1q, out_t=self.W1Tq)
        B.quantize_dual(W2, B.E4M3, out=self.W2q, out_t=self.W2Tq)

    def zero_grad(self):
        for g in self.grads.grads:
            g.zero_()

    def forward(self, x, residual):
        """Y [m][k] from x and the residual stream that it joins."""
        K.rmsnorm_quantize(x, self.gamma, self.eps, B.E4M3, residual=residual, out=self.norm)
        K.gemm_linear(self.norm.rows, self.W1q, self.b1, B.ACT_GELU, out=self.U, aux=self.Z)
        B.quantize_dual(self.U, B.E4M3, out=self.Uq, out_t=self.UTq)
        K.gemm_linear(self.Uq, self.W2q, self.b2, B.ACT_NONE, self.norm.h, out=self.Y)
        return self.Y

    def backward(self, dY):
        """The gradient of x (and of the residual) from that of Y; the parameters'
        gradients are added up."""
        B.quantize_dbias(dY, B.E5M2, out_t=self.dYTq, out=self.dYq, dbias=self.db2_new, workspace=self.cast_work)
        self.db2.add_(self.db2_new)
        B.gemm_wgrad(self.dYTq, self.UTq, self.dW2)
        B.gemm_dgrad(self.dYq, self.W2Tq, self.Z, B.EPI_DGELU, out=self.dZ)
        B.quantize_dbias(self.dZ, B.E5M2, out_t=self.dZTq, out=self.dZq, dbias=self.db1_new, workspace=self.cast_work)
        self.db1.add_(self.db1_new)
        B.gemm_wgrad(self.dZTq, self.norm.cols, self.dW1)
        K.gemm_linear(self.dZq, self.W1Tq, out=self.dN)
        K.rmsnorm_backward(self.dN, self.norm.h, self.gamma, self.norm.rstd, residual_grad=dY, out=self.dX,
                           dgamma=self.dgamma, accumulate=True, workspace=self.norm_work)
        return self.dX

    def clip(self, max_norm: float):
        """Scale all gradients so that their norm is at most max_norm; returns the
        norm before (device, 1 element)."""
        return K.clip_grads(self.grads, max_norm)

    def decode(self, x, residual):
        """(Y, h) for any number of tokens (a few: the products' kernel for few rows)."""
        norm = K.rmsnorm_quantize(x, self.gamma, self.eps, B.E4M3, residual=residual)
        U, _ = K.gemm_linear(norm.rows, self.W1q, self.b1, B.ACT_GELU)
        Y, _ = K.gemm_linear(B.quantize(U, B.E4M3), self.W2q, self.b2, B.ACT_NONE, norm.h)
        return Y, norm.h


class GatedFeedForwardBlock:
    """tokens m, width k, hidden width n, in the 1x128 recipe; m, k and n multiples
    of 128.  act: B.ACT_SILU or B.ACT_GELU.  p: the probability with which an element
    of x is dropped, by masks of ``seed`` (of the run) and ``site`` (this block's
    number in the model: blocks with the same seed and site, the defaults among them,
    draw the same mask, so each block of a model needs a site of its own); ``step``
    (int64, on the device) counts the calls of ``backward``, so a forward pass and its
    backward pass draw the same mask, and the replays of a captured step different
    ones.  Without dropout: ``decode``, or ``p`` set to 0.  Gradients accumulate in fp32
    over calls of ``backward`` until ``zero_grad``; ``clip`` scales them in place."""

    def __init__(self, m: int, k: int, n: int, p: float = 0.1, act: int = B.ACT_SILU, eps: float = 1e-5, seed: int = 0,
                 site: int = 0, device="cuda"):
        assert m % 128 == 0 and k % 128 == 0 and n % 128 == 0
        self.m, self.k, self.n, self.p, self.act, self.eps = m, k, n, p, act, eps
        self.seed, self.site = seed, site
        dev = torch.device(device)

        def bf16(*shape):
            return torch.empty(shape, dtype=torch.bfloat16, device=dev)

        def f32(*shape):
            return torch.zeros(shape, dtype=torch.float32, device=dev)

        self.step = torch.zeros((1,), dtype=torch.int64, device=dev)
        self.W1q, self.W1Tq = B.empty_fp8(2 * n, k, B.E4M3, dev), B.empty_fp8(k, 2 * n, B.E4M3, dev)
        self.W2q, self.W2Tq = B.empty_fp8(k, n, B.E4M3, dev), B.empty_fp8(n, k, B.E4M3, dev)
        self.h = bf16(m, k)
        self.norm = K.empty_layernorm(m, k, B.E4M3, cols_too=True, device=dev)
        self.Z, self.U = bf16(m, 2 * n), bf16(m, n)
        self.Uq, self.UTq = B.empty_fp8(m, n, B.E4M3, dev), B.empty_fp8(n, m, B.E4M3, dev)
        self.Y = bf16(m, k)
        self.dYq, self.dYTq = B.empty_fp8(m, k, B.E5M2, dev), B.empty_fp8(k, m, B.E5M2, dev)
        self.dZ = bf16(m, 2 * n)
        self.dZq, self.dZTq = B.empty_fp8(m, 2 * n, B.E5M2, dev), B.empty_fp8(2 * n, m, B.E5M2, dev)
        self.dN, self.dh, self.dX = bf16(m, k), bf16(m, k), bf16(m, k)
        self.dW1, self.dW2 = f32(2 * n, k), f32(k, n)
        self.db1, self.db2, self.dgamma, self.dbeta = f32(2 * n), f32(k), f32(k), f32(k)
        self.db1_new, self.db2_new = f32(2 * n), f32(k)  # one call's
        self.grads = K.GradList([self.dW1, self.dW2, self.db1, self.db2, self.dgamma, self.dbeta])
        self.cast_work = torch.empty((B.workspace_size(m, max(k, 2 * n)) // 4,), dtype=torch.float32, device=dev)
        self.norm_work = K.layernorm_workspace(m, k, dev)

    def load(self, gamma, beta, W1, b1, W2, b2):
        """Take the parameters (bf16: gamma [k], beta [k], W1 [2 n][k], b1 [2 n],
        W2 [k][n], b2 [k]) and cast the weights; again after every optimizer step."""
        self.gamma, self.beta, self.b1, self.b2 = gamma, beta, b1, b2
        B.quantize_dual(W1, B.E4M3, out=self.W1q, out_t=self.W1Tq)
        B.quantize_dual(W2, B.E4M3, out=self.W2q, out_t=self.W2Tq)

    def zero_grad(self):
        for g in self.grads.grads:
            g.zero_()

    def forward(self, x, residual):
        """Y [m][k] from x and the residual stream that it joins."""
        K.dropout(x, self.p, self.seed, self.site, self.step, residual=residual, out=self.h)
        K.layernorm_quantize(self.h, self.gamma, self.beta, self.eps, B.E4M3, out=self.norm)
        K.gemm_gated(self.norm.rows, self.W1q, self.b1, self.act, out=self.U, aux=self.Z)
        B.quantize_dual(self.U, B.E4M3, out=self.Uq, out_t=self.UTq)
        K.gemm_linear(self.Uq, self.W2q, self.b2, B.ACT_NONE, self.h, out=self.Y)
        return self.Y

    def backward(self, dY):
        """(The gradient of x, that of the residual) from that of Y; the parameters'
        gradients are added up."""
        B.quantize_dbias(dY, B.E5M2, out_t=self.dYTq, out=self.dYq, dbias=self.db2_new, workspace=self.cast_work)
        self.db2.add_(self.db2_new)
        B.gemm_wgrad(self.dYTq, self.UTq, self.dW2)
        K.gemm_gated_dgrad(self.dYq, self.W2Tq, self.Z, self.act, out=self.dZ)
        B.quantize_dbias(self.dZ, B.E5M2, out_t=self.dZTq, out=self.dZq, dbias=self.db1_new, workspace=self.cast_work)
        self.db1.add_(self.db1_new)
        B.gemm_wgrad(self.dZTq, self.norm.cols, self.dW1)
        K.gemm_linear(self.dZq, self.W1Tq, out=self.dN)
        K.layernorm_backward(self.dN, self.h, self.gamma, self.norm.mean, self.norm.rstd, residual_grad=dY,
                             out=self.dh, dgamma=self.dgamma, dbeta=self.dbeta, accumulate=True,
                             workspace=self.norm_work)
        K.dropout(self.dh, self.p, self.seed, self.site, self.step, out=self.dX)
        self.step.add_(1)
        return self.dX, self.dh

    def clip(self, max_norm: float):
        """Scale all gradients so that their norm is at most max_norm; returns the
        norm before (device, 1 element)."""
        return K.clip_grads(self.grads, max_norm)

    def decode(self, x, residual):
        """(Y, h) for any number of tokens (a few: the products' kernels for few
        rows), without dropout."""
        norm = K.layernorm_quantize(x, self.gamma, self.beta, self.eps, B.E4M3, residual=residual)
        U, _ = K.gemm_gated(norm.rows, self.W1q, self.b1, self.act)
        Y, _ = K.gemm_linear(B.quantize(U, B.E4M3), self.W2q, self.b2, B.ACT_NONE, norm.h)
        return Y, norm.h


def _time(fn, n):
    for _ in range(3):
        fn()
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    torch.cuda.synchronize()
    start.record()
    for _ in range(n):
        fn()
    end.record()
    torch.cuda.synchronize()
    return start.elapsed_time(end) / n


def main():
    m, k, n = 8192, 4096, 14336  # the linear layer's training step
    g = torch.Generator(device="cuda").manual_seed(0)

    def normal(*shape, std=1.0):
        return torch.randn(*shape, generator=g, device="cuda").mul_(std).bfloat16()

    x, r, dY = normal(m, k), normal(m, k), normal(m, k, std=1e-3)
    plain = FeedForwardBlock(m, k, n)
    plain.load(1 + normal(k, std=0.1), normal(n, k, std=0.02), normal(n, std=0.1), normal(k, n, std=0.02),
               normal(k, std=0.1))
    gated = GatedFeedForwardBlock(m, k, n)
    gated.load(1 + normal(k, std=0.1), normal(k, std=0.1), normal(2 * n, k, std=0.02), normal(2 * n, std=0.1),
               normal(k, n, std=0.02), normal(k, std=0.1))
    for name, block, products in (("block", plain, 2), ("gated block", gated, 3)):
        def step():
            block.forward(x, r)
            block.backward(dY)
            block.clip(1.0)

        ms = _time(step, 10)
        print("%s of %d tokens, %d to %d: forward, backward and clipping %.3f ms (%.0f TFLOP/s)"
              % (name, m, k, n, ms, 3 * products * 2 * m * k * n / ms / 1e9))
        for tokens in (1, 16, 64):
            xt, rt = x[:tokens].clone(), r[:tokens].clone()
            eager = _time(lambda: block.decode(xt, rt), 50)
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                block.decode(xt, rt)
            print("%3d tokens: %.1f us, %.1f us as a graph" % (tokens, 1e3 * eager, 1e3 * _time(graph.replay, 50)))


if __name__ == "__main__":
    main()
