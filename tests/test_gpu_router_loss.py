"""The router's balance loss, counts and gradient against 64-bit definitions.

Tolerances: an exponential of the native instruction has a relative error of (|x| + 2) 2^-23 for its argument x, here
below 32: 2^-18; sums of up to 1024 experts and the chains over tokens (below 2^11 additions) add 2^-13 at worst in a
bound, of the terms' size.  16-bit gradients are rounded once.
"""
import numpy as np
import pytest
import torch

import fp8_block_scaled_amd as gfg
from oracle import layers_oracle as lo
from oracle import serving_oracle as so

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
HALF = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11, "f32": 2.0 ** -24}
REL = 2.0 ** -13


def dev(x, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(x)).cuda()
    return t if dtype is None else t.to(dtype)


def case(T, E, k, dt, offsets=None, seed=0):
    r = np.random.default_rng(seed + T + E)
    logits = dev((r.standard_normal((T, E)) * 2).astype(np.float32), DT[dt]).double().cpu().numpy()
    logits[:, 0] = np.where(r.random(T) < 0.1, -np.inf, logits[:, 0])      # an expert masked for some tokens
    ids = so.topk(logits, k)[0]
    ids[r.random(T) < 0.1] = -1                                            # padding
    if T > 3:
        ids[1, :] = 10 ** 6                                                # another rank's experts only
        ids[2, 0] = E
        ids[3, :] = ids[3, 0]                                              # the same one k times
    return logits, ids, r


def check(logits, ids, r, dt, score, renormalize, z, offsets):
    T, E = logits.shape
    k = ids.shape[1]
    S = 1 if offsets is None else len(offsets) - 1
    off = None if offsets is None else dev(np.asarray(offsets, np.int32))
    l, i = dev(logits, DT[dt]), dev(ids.astype(np.int32))
    loss, counts, factors = gfg.moe_balance_loss(l, i, score=score, alpha=0.3, z=z, seq_offsets=off)
    rl, rc, rf = lo.balance(logits, ids, score, 0.3, z, offsets)
    assert counts.shape == (S, E) and np.array_equal(counts.cpu().numpy(), rc)
    assert abs(float(loss) - rl) <= REL * abs(rl), (float(loss), rl)
    assert np.allclose(factors.cpu().numpy(), rf, rtol=2.0 ** -20, atol=0)
    dw, dloss = r.standard_normal((T, k)).astype(np.float32), np.float32(1.7)
    for parts in ("both", "loss", "weights"):
        d = torch.full((T, E), 9.0, dtype=DT[dt], device="cuda")
        args = {}
        if parts != "weights":
            args.update(factors=factors, dloss=torch.tensor(float(dloss), device="cuda"), seq_offsets=off)
        if parts != "loss":
            args.update(dweights=dev(dw))
        gfg.moe_router_backward(l, i, d, score=score, renormalize=renormalize, scale=2.5, **args)
        ref = lo.router_backward(logits, ids, dw if parts != "loss" else None, score, renormalize, 2.5,
                                 factors.double().cpu().numpy() if parts != "weights" else None, float(dloss), offsets)
        # the terms' sizes: a gradient of softmax or normalized scores is a difference of terms of that size
        sc, p, soft, lse = lo._scores(logits, score)
        size = np.abs(ref)
        if parts != "weights":
            for s, (a, b) in enumerate(lo._sequences(T, offsets)):
                f = np.abs(rf[s, :E])
                size[a:b] += float(dloss) * (p[a:b] * (f + (f * p[a:b]).sum(1, keepdims=True)) + rf[s, E] * np.abs(lse[a:b, None]) * soft[a:b])
        if parts != "loss":
            wts = np.abs(lo.topk_weights(logits, ids, score, renormalize, 2.5))
            mass = np.zeros((T, E))
            here = (ids >= 0) & (ids < E)
            for t in range(T):
                np.add.at(mass[t], ids[t][here[t]], (np.abs(dw[t]) * wts[t])[here[t]])
            part = wts / np.maximum(wts.sum(1, keepdims=True), 1e-300)
            each = np.zeros((T, E))
            for t in range(T):
                np.add.at(each[t], ids[t][here[t]], (wts[t] * (np.abs(dw[t]) * part[t]).sum())[here[t]] if renormalize else 0 * wts[t][here[t]])
            size += mass + each + (soft * mass.sum(1, keepdims=True) if score == "softmax" else 0)
        g = d.double().cpu().numpy()
        least = 2.0 ** -25 if dt == "f16" else 0.0                          # half of f16's smallest step
        bad = np.abs(g - ref) - (HALF[dt] * np.abs(ref) + REL * size + least) * 1.01
        assert np.isfinite(g).all() and bad.max() <= 0, (parts, bad.max(), np.unravel_index(bad.argmax(), bad.shape))


@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 256, 8), (5, 64, 6), (77, 65, 3), (200, 128, 2), (300, 385, 9), (64, 1000, 64), (40, 1024, 4), (2100, 24, 2)])
@pytest.mark.parametrize("dt", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("score,renormalize,z", [("softmax", True, 0.0), ("softmax", False, 0.02), ("sigmoid", True, 0.02), ("sigmoid", False, 0.0)])
def test_against_the_definition(T, E, k, dt, score, renormalize, z):
    check(*case(T, E, k, dt), dt, score, renormalize, z, None)


# sequences that start and end inside a workgroup's tokens, empty ones, one token, tokens before the first and behind the last
@pytest.mark.parametrize("T,offsets", [(100, [0, 100]), (100, [0, 1, 1, 1, 37, 64, 100]), (100, [0] * 40 + [100]), (100, [0, 100] + [100] * 9),
                                       (1700, [0, 5, 16, 17, 900, 1700]), (9, list(range(10))), (60, [7, 20, 20, 41])])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_sequences(T, offsets, score):
    check(*case(T, 40, 3, "f32", seed=1), "f32", score, True, 0.02, offsets)


def test_no_token_counts():
    """All padding, and no tokens at all: loss, counts and gradient are zero, not NaN."""
    l, ids = torch.randn(20, 30, device="cuda"), torch.full((20, 2), -1, dtype=torch.int32, device="cuda")
    loss, counts, factors = gfg.moe_balance_loss(l, ids, z=1.0)
    assert float(loss) == 0 and not bool(counts.any()) and not bool(factors.any())
    d = torch.full((20, 30), 9.0, device="cuda")
    gfg.moe_router_backward(l, ids, d, dweights=torch.randn(20, 2, device="cuda"), factors=factors, dloss=torch.ones((), device="cuda"))
    assert not bool(d.any())
    loss, counts, factors = gfg.moe_balance_loss(l[:0], ids[:0], z=1.0, loss=torch.ones((), device="cuda"))
    assert float(loss) == 0 and not bool(counts.any()) and not bool(factors.any())
    gfg.moe_router_backward(l[:0], ids[:0], d[:0], dweights=torch.randn(0, 2, device="cuda"))


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_masked_logits(score):
    """Tokens with every expert masked, NaN among the masks, and the type's lowest value: no NaN comes out."""
    l = torch.randn(8, 12, device="cuda")
    l[0] = -float("inf")
    l[1, :11] = -float("inf")
    l[2] = float("nan")
    l[3] = torch.finfo(torch.float32).min
    l[4, 3] = torch.finfo(torch.float32).min
    l[5] = 80.0
    l[6] = -80.0
    ids = torch.zeros(8, 2, dtype=torch.int32, device="cuda")
    ids[:, 1] = 11
    loss, counts, factors = gfg.moe_balance_loss(l, ids, score=score)
    assert bool(torch.isfinite(loss)) and counts[0, 0] == 8 and counts[0, 11] == 8
    for renormalize in (True, False):
        d = torch.empty_like(l)
        gfg.moe_router_backward(l, ids, d, dweights=torch.randn(8, 2, device="cuda"), score=score, renormalize=renormalize, factors=factors,
                                dloss=torch.ones((), device="cuda"))
        assert bool(torch.isfinite(d).all())
        assert not bool(d[0].any()) and not bool(d[2].any()) and not bool(d[1, :11].any())


@pytest.mark.parametrize("E,k", [(8, 1), (64, 4), (100, 9), (300, 3), (600, 40)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_equal_gradients_of_normalized_weights_give_zero(E, k, score):
    """Normalized weights add up to one whatever the logits, so equal gradients of them (one choice above all) have no
    gradient, exactly, and nothing of it is left beside a far smaller one of the loss."""
    torch.manual_seed(E)
    l = torch.randn(200, E, device="cuda") * 3
    ids = torch.topk(l, k)[1].int()
    ids[::3, 0] = -1                                       # padding before the choices that are there
    dw = torch.randn(200, 1, device="cuda").expand(200, k).contiguous()
    d = torch.full_like(l, 9.0)
    gfg.moe_router_backward(l, ids, d, dweights=dw, score=score, renormalize=True)
    assert not bool(d.any())
    factors, e = torch.randn(1, E + 1, device="cuda") * 1e-9, torch.empty_like(l)
    one = torch.ones((), device="cuda")
    gfg.moe_router_backward(l, ids, d, dweights=dw, score=score, renormalize=True, factors=factors, dloss=one)
    gfg.moe_router_backward(l, ids, e, score=score, factors=factors, dloss=one)
    assert torch.equal(d, e) and bool(d.any())


def test_gradient_against_differences():
    """Differences of the calls themselves: moe_topk's weights and the loss, along one direction, step 2^-7 (fp32 noise of
    2^-21 over the step for each of T k weights, and the change of the difference between two steps)."""
    torch.manual_seed(1)
    T, E, k = 33, 20, 4
    # every token's logits a quarter apart, so that the choice stays as the steps move them (by at most 2^-8 * 5 here)
    l = torch.rand(T, E, device="cuda").argsort(-1) * 0.25 - 2.0
    new = lambda t, *s: torch.empty(*s, dtype=t, device="cuda")  # noqa: E731
    ids, _ = gfg.moe_topk(l, new(torch.int32, T, k), new(torch.float32, T, k))
    dw, dloss = torch.randn(T, k, device="cuda"), torch.tensor(3.0, device="cuda")
    top = torch.zeros(T, E, device="cuda").scatter_(1, ids.long(), 1.0).bool()
    way = torch.where(top, torch.randn(T, E, device="cuda"), 0.0)

    def loss(v):
        i, w = gfg.moe_topk(v, new(torch.int32, T, k), new(torch.float32, T, k), scale=2.0)
        same = (i[:, :, None] == ids[:, None, :])
        w = (w[:, :, None] * same).sum(1)                  # in the first call's order
        value, _, _ = gfg.moe_balance_loss(v, ids, alpha=0.5, z=0.01)
        return float((w.double() * dw).sum() + dloss.double() * value), bool(same.any(1).all())

    _, _, factors = gfg.moe_balance_loss(l, ids, alpha=0.5, z=0.01)
    d = gfg.moe_router_backward(l, ids, torch.empty_like(l), dweights=dw, scale=2.0, factors=factors, dloss=dloss)
    said = float((d.double() * way).sum())

    def at(h):
        (a, ok1), (b, ok2) = loss(l + h * way), loss(l - h * way)
        keep = ok1 and ok2
        return (a - b) / (2 * h), keep

    (d1, ok1), (d2, ok2) = at(2.0 ** -9), at(2.0 ** -8)
    assert ok1 and ok2
    assert abs(said - d1) <= 2.0 ** -21 * 2.0 ** 9 * np.sqrt(T * k) * 2 + abs(d2 - d1), (said, d1, d2)


def test_two_calls_give_the_same_bytes():
    torch.manual_seed(2)
    l, ids = torch.randn(3000, 100, device="cuda"), torch.randint(0, 100, (3000, 4), device="cuda", dtype=torch.int32)
    off = torch.tensor([0, 700, 701, 3000], dtype=torch.int32, device="cuda")
    runs = [gfg.moe_balance_loss(l, ids, z=0.1, seq_offsets=off) for _ in range(4)]
    assert all(torch.equal(a, b) for r in runs[1:] for a, b in zip(runs[0], r))
