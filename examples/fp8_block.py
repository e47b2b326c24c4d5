"""One block on FP8 weights, served and trained, with the operators around the products together.

    python examples/fp8_block.py                 # 2048 channels, 64 experts, 1 to 4096 tokens

    h, n = norm(y, residual)              residual_norm: the block before's output, its norm and gate, the residual sum
    logits = gate(n)                      fp8_linear
    ids, weights = router(logits)         moe_topk; in training also moe_balance_loss
    m = W2 (silu(g) * u), g | u = W1 n    fp8_linear twice
    few tokens, served:                   residual_norm_fp8 hands the rows to fp8_gemm in 8 bits, and moe_fp8_layer
                                          adds the experts that the router chose

A training step quantizes the weights in both orientations (``fp8_quantize_weight_device``), and its gradients come from
``fp8_linear_backward``, ``moe_router_backward`` and ``residual_norm_backward``.  Weights are random.
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import fp8_block_scaled_amd as gfg  # noqa: E402

ALPHA = 0.01       # of the balance loss


class Linear:
    """w [N, K] float32, the master copy; its FP8 codes in both orientations, and its gradient."""

    def __init__(self, w):
        self.w, self.grad = w, torch.zeros_like(w)
        self.quantize()

    def quantize(self):
        self.q, self.s, self.qt, self.st = gfg.fp8_quantize_weight_device(self.w, transposed=True)

    def __call__(self, x):
        return gfg.fp8_linear(x, self.q, self.s, torch.empty(x.shape[0], self.w.shape[0], dtype=x.dtype, device=x.device))

    def on_codes(self, q, scale, dtype):
        d = torch.empty(q.shape[0], self.w.shape[0], dtype=dtype, device=q.device)
        return gfg.fp8_gemm(q, scale, self.q, self.s, d)

    def backward(self, dy, x):
        """dx; the weight's gradient is added to ``grad``."""
        dx = torch.empty_like(x)
        gfg.fp8_linear_backward(dy, x, self.qt, self.st, dx=dx, dw=self.grad, accumulate=True)
        return dx


def silu_mul(gu):
    g, u = gu.float().chunk(2, dim=-1)
    return (torch.nn.functional.silu(g) * u).to(gu.dtype)


def silu_mul_backward(gu, dh):
    g, u = gu.float().chunk(2, dim=-1)
    s, dh = torch.sigmoid(g), dh.float()
    return torch.cat([dh * u * s * (1 + g * (1 - s)), dh * g * s], dim=-1).to(gu.dtype)


class FP8Block:
    """norm [H]; post norm and gate of the block before [H]; router weight [E, H], E a multiple of 16; w1 [2I, H] (gate rows, then up rows);
    w2 [H, I]; experts: (w1, s1, w2, s2) of ``moe_fp8_layer``, or None."""

    def __init__(self, norm, post, gate, router, w1, w2, top_k, experts=None):
        self.norm, self.post, self.gate, self.top_k, self.experts = norm, post, gate, top_k, experts
        self.router, self.w1, self.w2 = Linear(router), Linear(w1), Linear(w2)
        self.norm_grad, self.post_grad, self.gate_grad = (torch.zeros_like(t) for t in (norm, post, gate))

    def choose(self, logits):
        T, dev = logits.shape[0], logits.device
        ids = torch.empty(T, self.top_k, dtype=torch.int32, device=dev)
        return gfg.moe_topk(logits, ids, torch.empty(T, self.top_k, device=dev))

    def serve(self, y, residual):
        """(the residual stream, this block's output)."""
        out, q, scale, _ = gfg.residual_norm_fp8(y, residual, self.norm, post_weight=self.post, gate=self.gate)
        m = self.w2(silu_mul(self.w1.on_codes(q, scale, y.dtype)))
        if self.experts is not None:
            _, n, _ = gfg.residual_norm(None, out, self.norm, normed=torch.empty_like(y))
            ids, weights = self.choose(self.router(n))
            m = m + gfg.moe_fp8_layer(n, ids, weights, *self.experts, torch.empty_like(n))
        return out, m

    def forward(self, y, residual):
        stats = torch.empty(2, y.shape[0], device=y.device)
        out, n, _ = gfg.residual_norm(y, residual, self.norm, post_weight=self.post, gate=self.gate, stats=stats)
        logits = self.router(n)
        ids, weights = self.choose(logits)
        loss, counts, factors = gfg.moe_balance_loss(logits, ids, alpha=ALPHA)
        gu = self.w1(n)
        h = silu_mul(gu)
        return out, self.w2(h), weights, loss, (y, out, stats, n, logits, ids, factors, gu, h)

    def backward(self, dout, dm, dweights, saved):
        """(dy, dresidual) from the gradients of out, the output and the router's weights; the loss counts once."""
        y, out, stats, n, logits, ids, factors, gu, h = saved
        dn = self.w1.backward(silu_mul_backward(gu, self.w2.backward(dm, h)), n).float()
        dlogits = gfg.moe_router_backward(logits, ids, torch.empty_like(logits), dweights=dweights, factors=factors,
                                          dloss=torch.ones((), device=y.device))
        dn += self.router.backward(dlogits, n).float()
        dy, dresidual = torch.empty_like(y), torch.empty_like(out)
        gfg.residual_norm_backward(dout, dn.to(n.dtype), out, y, stats, self.norm, post_weight=self.post, gate=self.gate,
                                   dresidual=dresidual, dy=dy, dweight=self.norm_grad, dpost_weight=self.post_grad,
                                   dgate=self.gate_grad, accumulate=True)
        return dy, dresidual


def random_block(E, k, H, I, seed=0, device="cuda", with_experts=False):
    gen = torch.Generator(device=device)
    gen.manual_seed(seed)

    def weight(*shape):
        return torch.randn(*shape, generator=gen, device=device).mul_(shape[-1] ** -0.5)

    vector = lambda: 1 + 0.1 * torch.randn(H, generator=gen, device=device)  # noqa: E731
    experts = None
    if with_experts:
        experts = (*gfg.fp8_quantize_weight_device(weight(E, 2 * I, H)), *gfg.fp8_quantize_weight_device(weight(E, H, I)))
    return FP8Block(vector(), vector(), vector(), weight(E, H), weight(2 * I, H), weight(H, I), k, experts)


def main():
    E, k, H, I = 64, 6, 2048, 1408
    block = random_block(E, k, H, I, with_experts=True)
    for T in (1, 16, 128, 1024, 4096):
        y, r = (torch.randn(T, H, device="cuda").to(torch.bfloat16) for _ in range(2))

        def serve():
            return block.serve(y, r)

        def train():
            out, m, weights, loss, saved = block.forward(y, r)
            return block.backward(out, m, weights, saved)

        line = f"{T:5d} tokens"
        for name, step in (("served", serve), ("a training step", train)):
            if name == "served" and T * k > 1024:
                continue
            for _ in range(3):
                step()
            begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            begin.record()
            for _ in range(10):
                got = step()
            end.record()
            torch.cuda.synchronize()
            line += f"  {name} {begin.elapsed_time(end) / 10 * 1e3:8.1f} us (|.| = {float(got[0].float().norm()):.3g})"
        print(line, flush=True)


if __name__ == "__main__":
    main()
