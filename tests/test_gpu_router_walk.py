"""The router's training over more tokens than one turn of its workgroups takes: gradients of tokens whose operands were
loaded a turn ahead, ranges of the loss of several turns, a last turn that is not full.

A gradient's launch has at most 2048 workgroups of 4 waves, and a wave 1 to 8 tokens at a time, so it walks above 8192
tokens of more than 256 experts, 65536 of up to 64.  Tolerances are those of the smaller sizes: 2^-13 of the terms' size
(chains of 2^11 additions at most) and one rounding of the output.
"""
import numpy as np
import pytest
import torch

import fp8_block_scaled_amd as gfg
from oracle import layers_oracle as lo

HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
REL = 2.0 ** -13


def spans(T, offsets):
    return [(0, T)] if offsets is None else list(zip(offsets[:-1], offsets[1:]))


def definition(logits, ids, dw, score, renormalize, scale, alpha, z, dloss, offsets):
    """The definitions of the 64-bit oracle for all tokens at once: (loss, counts, factors, dlogits, the terms' size)."""
    T, E = logits.shape
    k, here = ids.shape[1], (ids >= 0) & (ids < E)
    at = np.where(here, ids, 0)
    sc, p, soft, lse = lo._scores(logits, score)
    counted, S = here.any(1), len(spans(T, offsets))
    counts, factors, loss = np.zeros((S, E), np.int64), np.zeros((S, E + 1)), 0.0
    d, size = np.zeros((T, E)), np.zeros((T, E))
    slope = sc if score == "softmax" else sc * (1 - sc) / np.where(sc.sum(1) > 0, sc.sum(1), 1.0)[:, None]
    for s, (a, b) in enumerate(spans(T, offsets)):
        c = counted[a:b]
        n = int(c.sum())
        if not n:
            continue
        counts[s] = np.bincount(ids[a:b][here[a:b]], minlength=E)
        f = counts[s] * E / (k * n)
        loss += (alpha * (f * p[a:b][c].mean(0)).sum() + z * (lse[a:b][c] ** 2).mean()) / S
        factors[s, :E], factors[s, E] = alpha * f / (S * n), 2 * z / (S * n)
        f = factors[s, :E]
        inner = f - (f * p[a:b]).sum(1, keepdims=True)
        d[a:b] = dloss * c[:, None] * (slope[a:b] * inner + factors[s, E] * lse[a:b, None] * soft[a:b])
        size[a:b] = dloss * (p[a:b] * (f + (f * p[a:b]).sum(1, keepdims=True)) + factors[s, E] * np.abs(lse[a:b, None]) * soft[a:b])
    v = np.where(here, np.take_along_axis(sc, at, 1), 0.0)
    total = v.sum(1, keepdims=True)
    one = np.where(total > 0, v / np.where(total > 0, total, 1.0), 0.0) if renormalize else v
    g = scale * np.where(here, dw.astype(np.float64), 0.0)
    each = one * (np.abs(g) + (2 * np.abs(g).max(1, keepdims=True) if renormalize else 0.0))     # (less the first one's, less their mean)
    g = (g - (g * one).sum(1, keepdims=True)) * one if renormalize else g * one
    rows = np.repeat(np.arange(T)[:, None], k, 1)
    add = lambda to, w: np.add.at(to, (rows[here], at[here]), w[here])  # noqa: E731
    if score == "sigmoid":
        add(d, g * (1 - np.take_along_axis(sc, at, 1)))
    else:
        add(d, g)
        d -= soft * g.sum(1, keepdims=True)
        size += soft * each.sum(1, keepdims=True)
    add(size, each)
    return loss, counts, factors, d, size


def drawn(T, E, k, dtype, seed):
    r = np.random.default_rng(seed)
    logits = torch.from_numpy(2 * r.standard_normal((T, E)).astype(np.float32)).to(dtype).double().numpy()
    logits[:, 0] = np.where(r.random(T) < 0.1, -np.inf, logits[:, 0])
    ids = r.integers(0, E, (T, k))                             # the same id twice here and there
    ids[r.random((T, k)) < 0.1] = -1
    ids[r.random(T) < 0.05] = -1                               # padding
    ids[r.random((T, k)) < 0.02] = E + 3
    return logits, ids, r.standard_normal((T, k)).astype(np.float32)


@pytest.mark.parametrize("score,renormalize", [("softmax", True), ("softmax", False), ("sigmoid", True), ("sigmoid", False)])
def test_the_definition_for_all_tokens_at_once(score, renormalize):
    logits, ids, dw = drawn(60, 13, 4, torch.float32, 1)
    offsets = [0, 7, 7, 40, 60]
    loss, counts, factors, d, _ = definition(logits, ids, dw, score, renormalize, 2.5, 0.3, 0.02, 1.7, offsets)
    want = lo.balance(logits, ids, score, 0.3, 0.02, offsets)
    assert np.isclose(loss, want[0], rtol=1e-12) and np.array_equal(counts, want[1]) and np.allclose(factors, want[2], rtol=1e-12, atol=0)
    assert np.allclose(d, lo.router_backward(logits, ids, dw, score, renormalize, 2.5, factors, 1.7, offsets), rtol=1e-9, atol=1e-15)


@pytest.mark.gpu
@pytest.mark.parametrize("T,E,k,dtype,score,renormalize,z,offsets", [
    (8197, 385, 9, torch.bfloat16, "sigmoid", True, 0.0, [0, 1000, 1000, 4099, 8190, 8197]),
    (20011, 385, 9, torch.float32, "sigmoid", True, 0.02, [0, 3, 9000, 20011]),
    (20011, 300, 8, torch.float16, "softmax", True, 0.0, None),
    (32768, 385, 9, torch.bfloat16, "sigmoid", False, 0.0, [4096 * s for s in range(9)]),
    (8300, 1000, 64, torch.float32, "softmax", False, 0.02, None),
    (16390, 200, 6, torch.bfloat16, "softmax", False, 0.02, [0, 16390]),
    (32800, 128, 2, torch.float32, "sigmoid", True, 0.0, None),
    (65600, 40, 2, torch.bfloat16, "softmax", True, 0.02, [0, 60000, 65000, 65600]),
    (140003, 24, 8, torch.float32, "sigmoid", True, 0.0, None),
    (66000, 7, 3, torch.float32, "softmax", True, 0.0, None),
])
def test_many_tokens(T, E, k, dtype, score, renormalize, z, offsets):
    logits, ids, dw = drawn(T, E, k, dtype, T)
    dev = lambda x: torch.from_numpy(np.ascontiguousarray(x)).cuda()  # noqa: E731
    l, i, off = dev(logits).to(dtype), dev(ids.astype(np.int32)), None if offsets is None else dev(np.asarray(offsets, np.int32))
    loss, counts, factors = gfg.moe_balance_loss(l, i, score=score, alpha=0.3, z=z, seq_offsets=off)
    d = torch.full((T, E), 9.0, dtype=dtype, device="cuda")
    gfg.moe_router_backward(l, i, d, dweights=dev(dw), score=score, renormalize=renormalize, scale=2.5, factors=factors,
                            dloss=torch.tensor(1.75, device="cuda"), seq_offsets=off)
    rl, rc, rf, rd, size = definition(logits, ids, dw, score, renormalize, 2.5, 0.3, z, 1.75, offsets)
    assert np.array_equal(counts.cpu().numpy(), rc) and abs(float(loss) - rl) <= REL * rl
    assert np.allclose(factors.cpu().numpy(), rf, rtol=2.0 ** -20, atol=0)
    got = d.double().cpu().numpy()
    least = 2.0 ** -25 if dtype == torch.float16 else 0.0      # half of f16's smallest step
    off_by = np.abs(got - rd) - (HALF[dtype] * np.abs(rd) + REL * size + least) * 1.01
    assert np.isfinite(got).all() and off_by.max() <= 0, (off_by.max(), np.unravel_index(off_by.argmax(), off_by.shape))
