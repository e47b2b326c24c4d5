"""The serving operators together, as examples/moe_block.py runs them, against float64."""
import os
import sys

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import moe_block as mb  # noqa: E402
from oracle import serving_oracle as so  # noqa: E402


def dequant(w):
    q, s = w
    return so.dequantize_int8(q.cpu().numpy(), s.cpu().numpy())


def swiglu(gu):
    g, u = np.split(gu, 2, axis=-1)
    return g / (1.0 + np.exp(-g)) * u


def norm_error(got, ref):
    got = got.float().cpu().numpy().astype(np.float64)
    assert np.all(np.isfinite(got))
    return float(np.linalg.norm(got - ref) / np.linalg.norm(ref))


# Bounds.  A row of n values rounded to 8 bits carries an error of amax / 127 /
# sqrt(12) per value: relative to the row's norm 0.0023 * amax / rms.  amax / rms
# is about 4 for normal values and below 10 for silu(g) * u, so two roundings in
# turn leave less than sqrt(0.009^2 + 0.023^2) = 0.025 of the norm; twice that is
# allowed.  Without them (the expert layer) only the output's bf16 rounding, at
# most 2^-8 of a value, and less than 2^-12 of the sums are left.
EIGHT_BITS, SIXTEEN_BITS = 0.05, 2.0 ** -8 + 2.0 ** -12


@pytest.mark.parametrize("T,E,k,H,I,S", [(1, 8, 2, 256, 128, 128), (37, 16, 4, 512, 384, 256), (130, 5, 3, 384, 256, 640)])
def test_block(T, E, k, H, I, S):
    block = mb.random_block(E, k, H, I, S, seed=T)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(T)
    x = torch.randn(T, H, generator=gen, device="cuda").to(torch.bfloat16)
    x64 = x.float().cpu().numpy().astype(np.float64)
    ids, weights = block.route(x)
    logits = block._linear(x, block.gate)
    assert norm_error(logits, x64 @ dequant(block.gate).T) < EIGHT_BITS
    ref_ids, ref_w = so.topk(logits.float().cpu().numpy(), k)
    assert np.array_equal(ids.cpu().numpy(), ref_ids)
    ref = so.layer(x64, ids.cpu().numpy(), weights.cpu().numpy(), dequant(block.w1), dequant(block.w2))
    assert norm_error(block.experts_few(x, ids, weights), ref) < SIXTEEN_BITS
    assert norm_error(block.experts_many(x, ids, weights), ref) < EIGHT_BITS
    shared = swiglu(x64 @ dequant(block.shared1).T) @ dequant(block.shared2).T
    assert norm_error(block.shared(x), shared) < EIGHT_BITS
    assert norm_error(block(x), ref + shared) < EIGHT_BITS


def test_block_pairs_of_no_expert_in_both_paths():
    T, E, k, H, I = 20, 6, 3, 256, 256
    block = mb.random_block(E, k, H, I, 128, seed=3)
    x = torch.randn(T, H, device="cuda").to(torch.bfloat16)
    ids, weights = block.route(x)
    ids[::2, 1] = -1
    ids[3] = E                                            # every choice of token 3 is another rank's
    ref = so.layer(x.float().cpu().numpy(), ids.cpu().numpy(), weights.cpu().numpy(), dequant(block.w1), dequant(block.w2))
    for path, bound in ((block.experts_few, SIXTEEN_BITS), (block.experts_many, EIGHT_BITS)):
        y = path(x, ids, weights)
        assert norm_error(y, ref) < bound
        assert not y[3].any()


def test_block_many_pairs_take_the_grouped_products():
    T, E, k, H, I = 600, 8, 2, 256, 128                   # 1200 pairs: past the expert layer's 1024
    block = mb.random_block(E, k, H, I, 128, seed=4)
    x = torch.randn(T, H, device="cuda").to(torch.bfloat16)
    ids, weights = block.route(x)
    ref = so.layer(x.float().cpu().numpy(), ids.cpu().numpy(), weights.cpu().numpy(), dequant(block.w1), dequant(block.w2))
    assert norm_error(block.experts(x, ids, weights), ref) < EIGHT_BITS
