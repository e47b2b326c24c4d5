"""The router's choice under a selection bias, and its softmax weights at the bound that their roundings allow.

A weight may differ from the 64-bit one by (|l - max| + 24) * 2^-23 relative for the softmax, (|l| + 24) * 2^-23 for
the sigmoid: the rounding of the exponential's argument acts on the exponent, the sums and quotients are the 24.
A selection value score + bias has an error below 2^-20 (scores in [0, 1], biases below 1), so the inputs keep
different values 2^-16 apart, and the 64-bit order is the only right one.
"""
import numpy as np
import pytest
import torch

import fp8_block_scaled_amd as gfg
from oracle import serving_oracle as so

pytestmark = pytest.mark.gpu


def route(logits, k, **kw):
    l = torch.from_numpy(logits).cuda()
    bias = kw.pop("bias", None)
    ids = torch.full((l.shape[0], k), -9, dtype=torch.int32, device="cuda")
    w = torch.full((l.shape[0], k), -9.0, device="cuda")
    gfg.moe_topk(l, ids, w, bias=None if bias is None else torch.from_numpy(bias).cuda(), **kw)
    return ids.cpu().numpy(), w.cpu().numpy().astype(np.float64)


def scores(logits, score):
    l = logits.astype(np.float64)
    if score == "sigmoid":
        return 1.0 / (1.0 + np.exp(-l))
    e = np.exp(l - l.max(1, keepdims=True))
    return e / e.sum(1, keepdims=True)


def separated(rng, T, E, score):
    """Logits and a bias of about the scores' own size whose selection values are 2^-16 apart in every row."""
    spread = 0.5 if score == "sigmoid" else 2.0 / E
    bias = (rng.uniform(-0.5, 0.5, E) * spread).astype(np.float32)
    rows = []
    while len(rows) < T:
        l = (rng.standard_normal((1, E)) * 1.5).astype(np.float32)
        s = np.sort((scores(l, score) + bias)[0])
        if np.diff(s).min() > 2.0 ** -16:
            rows.append(l)
    return np.concatenate(rows), bias


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,E,k", [(1, 64, 6), (9, 24, 4), (300, 48, 8), (5, 65, 9)])
def test_scores_and_bias_choose_together(T, E, k, score):
    rng = np.random.default_rng(T + E)
    logits, bias = separated(rng, T, E, score)
    p = scores(logits, score)
    order = np.argsort(-(p + bias), axis=1, kind="stable")[:, :k]
    # neither alone chooses like that
    by_bias = np.argsort(-bias, kind="stable")[:k]
    by_score = np.argsort(-p, axis=1, kind="stable")[:, :k]
    assert all(set(o) != set(by_bias) for o in order) and sum(set(o) != set(b) for o, b in zip(order, by_score)) * 2 >= T
    gap = np.abs(logits) if score == "sigmoid" else logits.max(1, keepdims=True) - logits
    for renormalize in (False, True):
        ids, w = route(logits, k, score=score, bias=bias, renormalize=renormalize, scale=1.5)
        assert np.array_equal(ids, order)
        want = np.take_along_axis(p, order, 1)             # the weights are the scores, without the bias
        if renormalize:
            want = want / want.sum(1, keepdims=True)
        bound = (np.take_along_axis(gap, order, 1).max(1, keepdims=True) + 24) * 2.0 ** -23
        assert (np.abs(w - 1.5 * want) <= bound * 1.5 * want).all()


def test_bias_of_many_experts_and_equal_sums():
    """385 experts, sigmoid, k = 9: equal logits under equal biases go to the lowest index."""
    E, k = 385, 9
    logits = np.zeros((3, E), np.float32)
    bias = np.zeros(E, np.float32)
    bias[[384, 130, 7, 200]] = 0.25
    logits[1, 300] = -np.inf
    logits[2, [384, 7]] = -8.0                             # their scores fall by 0.4997: behind the experts without a bias
    ids, w = route(logits, k, score="sigmoid", bias=bias, renormalize=True)
    assert ids[0].tolist() == [7, 130, 200, 384, 0, 1, 2, 3, 4] and ids[1].tolist() == ids[0].tolist()
    assert ids[2].tolist() == [130, 200, 0, 1, 2, 3, 4, 5, 6]
    assert np.abs(w - 1 / 9).max() <= 24 * 2.0 ** -23


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_rows_of_the_lowest_value_share_their_softmax(dtype):
    low = torch.finfo(dtype).min
    l = torch.full((2, 200), low, dtype=dtype, device="cuda")
    l[1, 150] = 3.0                                        # beside it the others have no weight
    for renormalize, each in ((True, 1 / 5), (False, 1 / 200)):
        ids = torch.zeros(2, 5, dtype=torch.int32, device="cuda")
        w = torch.zeros(2, 5, device="cuda")
        gfg.moe_topk(l, ids, w, renormalize=renormalize)
        assert ids.tolist() == [[0, 1, 2, 3, 4], [150, 0, 1, 2, 3]]
        assert np.abs(w[0].cpu().numpy().astype(np.float64) - each).max() <= 24 * 2.0 ** -23 * each
        assert w[1].tolist() == [1.0, 0.0, 0.0, 0.0, 0.0]


@pytest.mark.parametrize("T,E,k", [(3, 64, 64), (130, 385, 9), (4, 513, 33), (1000, 8, 2)])
@pytest.mark.parametrize("renormalize", [False, True])
def test_softmax_weights_far_from_zero(T, E, k, renormalize):
    """Logits around 80: the bound goes by the distance from the largest, not by the logits' size."""
    rng = np.random.default_rng(T * 3 + E)
    logits = (80 + rng.standard_normal((T, E)) * 2).astype(np.float32)
    ids, w = route(logits, k, renormalize=renormalize)
    want_ids, want = so.topk(logits, k, renormalize=renormalize)
    assert np.array_equal(ids, want_ids)
    gap = logits.max(1, keepdims=True) - np.take_along_axis(logits, ids, 1)
    assert (np.abs(w - want) <= (gap.max(1, keepdims=True) + 24) * 2.0 ** -23 * want).all()
