"""The router's gradient where the scores are small: chosen sigmoids near the end of fp32's normal range, choices (by a
selection bias, say) far below a token's largest logit, and tokens whose experts are all that small.

Their weights and their normalized scores are ordinary numbers, and so are the gradients.  Tolerance: an exponential of
the native instruction has a relative error of (|x| + 2) 2^-23, here below 92 2^-23 < 2^-16; a gradient has at most six
such factors and two sums of up to 64 terms, 2^-13 of its terms' size in all.  The 64-bit definition itself subtracts the
mean of centred gradients, which is zero but for its rounding: 64 terms, each off by 2^-52 of the largest gradient, below
2^-45 of it on any expert (the kernel gives exactly zero to an expert that is not chosen).
"""
import numpy as np
import pytest
import torch

import fp8_block_scaled_amd as gfg
from oracle import layers_oracle as lo

pytestmark = pytest.mark.gpu

REL = 2.0 ** -13


def dev(x):
    return torch.from_numpy(np.ascontiguousarray(x)).cuda()


def weights_gradient(logits, ids, dw, score, scale=1.0):
    d = torch.full(logits.shape, 9.0, device="cuda")
    gfg.moe_router_backward(dev(logits), dev(ids), d, dweights=dev(dw), score=score, renormalize=True, scale=scale)
    ref = lo.router_backward(logits, ids, dw, score, True, scale)
    part = lo.topk_weights(logits, ids, score, True, 1.0)
    size = np.zeros(logits.shape)
    np.put_along_axis(size, ids, scale * part * (2 * np.abs(dw) + 2 * np.abs(dw).max(1, keepdims=True)), 1)
    return d.double().cpu().numpy(), ref, REL * size + 2.0 ** -45 * scale * np.abs(dw).max(1, keepdims=True)


def drawn(T, E, k, seed):
    r = np.random.default_rng(seed)
    ids = np.stack([r.permutation(E)[:k] for _ in range(T)]).astype(np.int32)
    return r, ids


@pytest.mark.parametrize("E,k", [(8, 2), (40, 4), (100, 9), (385, 9), (600, 40)])
@pytest.mark.parametrize("dweight", [1.0, 1e4])
@pytest.mark.parametrize("low,high", [(-87.0, -84.0), (-87.0, -78.0), (-62.0, -58.0)])
def test_small_chosen_sigmoids(E, k, dweight, low, high):
    r, ids = drawn(37, E, k, E + k)
    logits = r.uniform(-100, -90, (37, E)).astype(np.float32)
    np.put_along_axis(logits, ids, r.uniform(low, high, ids.shape).astype(np.float32), 1)
    dw = (dweight * r.standard_normal(ids.shape)).astype(np.float32)
    got, ref, bound = weights_gradient(logits, ids, dw, "sigmoid", 2.5)
    assert np.isfinite(got).all() and (np.abs(got - ref) <= bound).all()


@pytest.mark.parametrize("E,k", [(8, 2), (40, 4), (100, 9), (385, 9), (600, 40)])
@pytest.mark.parametrize("below", [(75, 80), (80, 88), (86, 100)])
def test_choices_far_below_the_largest_logit(E, k, below):
    r, ids = drawn(37, E, k, E + 2 * k)
    logits = r.uniform(-1, 0, (37, E)).astype(np.float32)
    np.put_along_axis(logits, ids, -r.uniform(*below, ids.shape).astype(np.float32), 1)
    logits[np.arange(37), [next(e for e in range(E) if e not in row) for row in ids]] = 0.5
    dw = r.standard_normal(ids.shape).astype(np.float32)
    got, ref, bound = weights_gradient(logits, ids, dw, "softmax")
    assert np.isfinite(got).all() and (np.abs(got - ref) <= bound).all()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("k", [1, 5])
def test_equal_gradients_of_small_scores_give_zero(score, k):
    """Scores down to where moe_topk's become zero, and choices among them that are masked."""
    r, ids = drawn(64, 40, k, k)
    logits = r.uniform(-2, 0, (64, 40)).astype(np.float32)
    np.put_along_axis(logits, ids, -r.uniform(80, 110, ids.shape).astype(np.float32), 1)
    logits[::5, ids[0, 0]] = -np.inf
    dw = np.repeat(r.standard_normal((64, 1)), k, 1).astype(np.float32)
    got = weights_gradient(logits, ids, dw, score)[0]
    assert not got.any()


def test_weights_of_zero_have_no_gradient():
    """Choices whose scores are zero in fp32 have weights of zero, whatever the definition in 64 bits makes of them."""
    logits, ids = np.full((3, 12), -1.0, np.float32), np.asarray([[2, 5, 9]] * 3, np.int32)
    logits[:, [2, 5, 9]] = [-200.0, -201.0, -202.0]
    dw = np.asarray([[1.0, -2.0, 3.0]] * 3, np.float32)
    i, w = dev(ids), torch.empty(3, 3, device="cuda")
    for score in ("softmax", "sigmoid"):
        d = torch.full((3, 12), 9.0, device="cuda")
        gfg.moe_router_backward(dev(logits), i, d, dweights=dev(dw), score=score, renormalize=True)
        assert not bool(d.any())
        bias = torch.zeros(12, device="cuda")
        bias[[2, 5, 9]] = 10.0
        chosen, _ = gfg.moe_topk(dev(logits), torch.empty_like(i), w, score=score, bias=bias)
        assert sorted(chosen[0].tolist()) == [2, 5, 9] and not bool(w.any())


@pytest.mark.parametrize("E,k", [(8, 2), (64, 6), (385, 9), (600, 40)])
@pytest.mark.parametrize("dloss", [1.0, 2.0 ** 16])
@pytest.mark.parametrize("alpha", [0.01, 1e-6])
def test_loss_of_tokens_with_small_sigmoids_alone(E, k, alpha, dloss):
    r, ids = drawn(50, E, k, E)
    logits = r.uniform(-86, -78, (50, E)).astype(np.float32)
    l, i = dev(logits), dev(ids)
    loss, _, factors = gfg.moe_balance_loss(l, i, score="sigmoid", alpha=alpha)
    want = lo.balance(logits, ids, "sigmoid", alpha)[0]
    assert abs(float(loss) - want) <= REL * want
    d = torch.full((50, E), 9.0, device="cuda")
    gfg.moe_router_backward(l, i, d, score="sigmoid", factors=factors, dloss=torch.tensor(dloss, device="cuda"))
    f = factors.double().cpu().numpy()
    ref = lo.router_backward(logits, ids, None, "sigmoid", True, 1.0, f, dloss)
    p = lo._scores(logits, "sigmoid")[1]
    size = dloss * p * (f[0, :E] + (f[0, :E] * p).sum(1, keepdims=True))
    got = d.double().cpu().numpy()
    assert np.isfinite(got).all() and (np.abs(got - ref) <= REL * size).all()


@pytest.mark.parametrize("E,k", [(7, 2), (40, 4), (100, 9), (200, 6), (385, 9), (600, 40)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_small_scores_beside_ordinary_ones(E, k, score):
    """Tokens that share a wave with others of either kind get the gradients that they have alone."""
    r, ids = drawn(96, E, k, E + 3)
    logits = r.standard_normal((96, E)).astype(np.float32)
    small = r.random(96) < 0.5
    if score == "sigmoid":
        logits[small] = r.uniform(-86, -78, (int(small.sum()), E))
    else:
        low = logits.copy()
        np.put_along_axis(low, ids, -r.uniform(75, 100, ids.shape).astype(np.float32), 1)
        logits[small] = low[small]
    dw = r.standard_normal(ids.shape).astype(np.float32)
    factors = torch.rand(1, E + 1, device="cuda") * 1e-5

    def gradient(rows):
        d = torch.full((len(rows), E), 9.0, device="cuda")
        gfg.moe_router_backward(dev(logits[rows]), dev(ids[rows]), d, dweights=dev(dw[rows]), score=score, factors=factors,
                                dloss=torch.tensor(2.0 ** 16, device="cuda"))
        return d

    every = gradient(np.arange(96))
    assert bool(torch.isfinite(every).all()) and bool((every != 0).any(1).all())
    for rows in (np.flatnonzero(small), np.flatnonzero(~small), np.arange(95, -1, -1)):
        assert torch.equal(gradient(rows), every[torch.from_numpy(rows.copy()).cuda()])
