"""One mixture-of-experts block served from int8 weights, with the framework's serving operators together.

    python examples/moe_block.py                 # 64 experts, 6 a token, 1 to 4096 tokens

    logits = gate(x)                       int8_linear
    ids, weights = router(logits)          moe_topk
    few tokens:   y = experts(x, ids)      moe_int8_layer: reads each chosen expert's weights once
    many tokens:  y = experts(x, ids)      int8_quantize_token_device and grouped_int8_gemm_contiguous, on the
                                           same weights, over the pairs sorted by expert
    y + shared(x)                          int8_linear twice: an expert that every token passes

Weights are random; ``quantize_weight`` is how a user's own become int8.
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import fp8_block_scaled_amd as gfg  # noqa: E402

TILE = 128         # rows of one expert come in tiles of this many in the contiguous layout
FEW_PAIRS = 1024   # pairs (token, expert) that the expert layer takes


def quantize_weight(w):
    """[..., N, K] -> int8 codes with one scale per output channel (the token quantizer, on the weight's rows)."""
    return gfg.int8_quantize_token_device(w.contiguous())


def silu_mul(gu):
    g, u = gu.float().chunk(2, dim=-1)
    return (torch.nn.functional.silu(g) * u).to(gu.dtype)


class MoEBlock:
    """gate [E, H]; w1 [E, 2I, H] (gate rows, then up rows); w2 [E, H, I]; shared1 [2S, H]; shared2 [H, S]."""

    def __init__(self, gate, w1, w2, shared1, shared2, top_k, score="softmax"):
        self.gate, self.w1, self.w2 = quantize_weight(gate), quantize_weight(w1), quantize_weight(w2)
        self.shared1, self.shared2 = quantize_weight(shared1), quantize_weight(shared2)
        self.top_k, self.score = top_k, score
        self.E, self.H, self.I = w2.shape

    def _linear(self, x, weight):
        q, scale = weight
        return gfg.int8_linear(x, q, scale, torch.empty(x.shape[0], q.shape[0], dtype=x.dtype, device=x.device))

    def route(self, x):
        T = x.shape[0]
        ids = torch.empty(T, self.top_k, dtype=torch.int32, device=x.device)
        weights = torch.empty(T, self.top_k, dtype=torch.float32, device=x.device)
        return gfg.moe_topk(self._linear(x, self.gate), ids, weights, score=self.score)

    def experts_few(self, x, ids, weights):
        return gfg.moe_int8_layer(x, ids, weights, *self.w1, *self.w2, torch.empty_like(x))

    def experts_many(self, x, ids, weights):
        T, E, dev = x.shape[0], self.E, x.device
        # the pairs in expert order, each expert's rows from a multiple of TILE on; pairs of no expert come last,
        # into the tiles that nothing computes.  Sizes depend on the shapes alone, so nothing waits for the GPU.
        expert = torch.where((ids >= 0) & (ids < E), ids, E).flatten().long()
        order = torch.argsort(expert, stable=True)
        counts = torch.zeros(E + 1, dtype=torch.long, device=dev).index_add_(0, expert, torch.ones_like(expert))
        padded = (counts + TILE - 1) // TILE * TILE
        start, first = padded.cumsum(0) - padded, counts.cumsum(0) - counts
        sorted_expert = expert[order]
        row = start[sorted_expert] + torch.arange(expert.numel(), device=dev) - first[sorted_expert]
        M = (expert.numel() + TILE - 1) // TILE * TILE + (E + 1) * TILE
        layout = torch.full((M,), -1, dtype=torch.int32, device=dev)
        layout[row] = torch.where(sorted_expert < E, sorted_expert, -1).int()
        token = order // self.top_k

        q, s = gfg.int8_quantize_token_device(x)
        a = torch.zeros(M, self.H, dtype=torch.int8, device=dev)
        sa = torch.zeros(M, device=dev)
        a[row], sa[row] = q[token], s[token]
        gu = torch.zeros(M, 2 * self.I, dtype=x.dtype, device=dev)
        gfg.grouped_int8_gemm_contiguous(a, sa, *self.w1, layout, gu)
        h, sh = gfg.int8_quantize_token_device(silu_mul(gu))
        d = torch.zeros(M, self.H, dtype=x.dtype, device=dev)
        gfg.grouped_int8_gemm_contiguous(h, sh, *self.w2, layout, d)
        y = torch.empty(T * self.top_k, self.H, dtype=x.dtype, device=dev)
        y[order] = d[row]
        return (y.view(T, self.top_k, self.H).float() * weights[:, :, None]).sum(1).to(x.dtype)

    def experts(self, x, ids, weights):
        few = ids.numel() <= FEW_PAIRS and self.H % 128 == 0 and self.I % 128 == 0
        return (self.experts_few if few else self.experts_many)(x, ids, weights)

    def shared(self, x):
        return self._linear(silu_mul(self._linear(x, self.shared1)), self.shared2)

    def __call__(self, x):
        ids, weights = self.route(x)
        return self.experts(x, ids, weights) + self.shared(x)


def random_block(E, k, H, I, S, seed=0, device="cuda"):
    gen = torch.Generator(device=device)
    gen.manual_seed(seed)

    def weight(*shape):
        return torch.randn(*shape, generator=gen, device=device, dtype=torch.float32).mul_(shape[-1] ** -0.5)

    return MoEBlock(weight(E, H), weight(E, 2 * I, H), weight(E, H, I), weight(2 * S, H), weight(H, S), k)


def main():
    E, k, H, I, S = 64, 6, 2048, 1408, 2816
    block = random_block(E, k, H, I, S)
    for T in (1, 5, 32, 128, 1024, 4096):
        x = torch.randn(T, H, device="cuda").to(torch.bfloat16)
        for _ in range(3):
            y = block(x)
        begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        begin.record()
        for _ in range(10):
            y = block(x)
        end.record()
        torch.cuda.synchronize()
        path = "expert layer" if T * k <= FEW_PAIRS else "grouped products"
        line = f"{T:5d} tokens  {begin.elapsed_time(end) / 10 * 1e3:8.1f} us a block  ({path})"
        if T * k <= FEW_PAIRS:
            ids, weights = block.route(x)
            few, many = block.experts_few(x, ids, weights).float(), block.experts_many(x, ids, weights).float()
            line += f"  the two paths differ by {float((few - many).norm() / few.norm()):.1%} (tokens in 16 or 8 bits)"
        print(line + f"  |y| = {float(y.float().norm()):.3g}", flush=True)


if __name__ == "__main__":
    main()
