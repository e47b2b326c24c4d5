"""CPU tests of the serving operators: what their entry points refuse, with the documented status codes and before
anything touches a GPU, and the 64-bit definitions against worked examples.  Pointers are made-up aligned addresses:
no call here reaches a launch."""
import os

import numpy as np
import pytest
import torch

import fp8_block_scaled_amd as gfg
from oracle import serving_oracle as so

EINVAL, EUNSUPPORTED = 1, 2
P = 1 << 20            # an aligned made-up address


def lib():
    return gfg.load_library()


def last():
    return lib().grouped_fp8_last_error().decode()


QUANT = dict(x=P, dt=0, M=4, K=64, q=P, scale=P)


@pytest.mark.parametrize("change,code", [
    (dict(dt=3), EINVAL), (dict(dt=-1), EINVAL), (dict(M=-1), EINVAL), (dict(K=0), EINVAL), (dict(K=-16), EINVAL),
    (dict(K=24), EUNSUPPORTED), (dict(K=1 << 17), EUNSUPPORTED), (dict(M=1 << 31), EUNSUPPORTED), (dict(x=None), EINVAL),
    (dict(q=None), EINVAL), (dict(scale=None), EINVAL), (dict(x=P + 8), EINVAL), (dict(q=P + 4), EINVAL),
    (dict(scale=P + 2), EINVAL),
])
def test_quantizer_refuses(change, code):
    a = {**QUANT, **change}
    assert lib().int8_quantize_token_device(a["x"], a["dt"], a["M"], a["K"], a["q"], a["scale"], None) == code
    assert "int8_quantize_token_device" in last()


GEMM = dict(a=P, sa=P, b=P, sb=P, bias=None, d=P, M=4, N=5, K=64, out=0)


@pytest.mark.parametrize("change,code", [
    (dict(out=2), EINVAL), (dict(M=-1), EINVAL), (dict(N=0), EINVAL), (dict(K=0), EINVAL), (dict(K=40), EUNSUPPORTED),
    (dict(K=1 << 17), EUNSUPPORTED), (dict(N=(1 << 30) + 1), EUNSUPPORTED), (dict(M=128 * 65535 + 1), EUNSUPPORTED),
    (dict(a=None), EINVAL), (dict(sa=None), EINVAL), (dict(b=None), EINVAL), (dict(sb=None), EINVAL), (dict(d=None), EINVAL),
    (dict(a=P + 8), EINVAL), (dict(b=P + 1), EINVAL), (dict(sa=P + 1), EINVAL), (dict(sb=P + 2), EINVAL),
    (dict(bias=P + 2), EINVAL), (dict(d=P + 4), EINVAL),
])
def test_product_refuses(change, code):
    a = {**GEMM, **change}
    assert lib().int8_gemm(a["a"], a["sa"], a["b"], a["sb"], a["bias"], a["d"], a["M"], a["N"], a["K"], a["out"], None) == code
    assert "int8_gemm" in last()


def test_large_tile_refuses_wide_outputs():
    gfg.set_tile_shape(gfg.TILE_256x256)
    try:
        assert lib().int8_gemm(P, P, P, P, None, P, 4, (1 << 22) + 8, 64, 0, None) == EUNSUPPORTED
    finally:
        gfg.set_tile_shape(gfg.TILE_AUTO)


@pytest.mark.parametrize("change,code", [
    (dict(M=1 << 62), EUNSUPPORTED), (dict(dt=5), EINVAL), (dict(ws=None), EINVAL), (dict(ws=P + 8), EINVAL), (dict(bytes=4 * 68 - 1), EINVAL), (dict(x=None), EINVAL),
    (dict(K=24), EUNSUPPORTED), (dict(out=9), EINVAL), (dict(b=None), EINVAL), (dict(d=P + 2), EINVAL), (dict(x=P + 4), EINVAL),
])
def test_linear_refuses(change, code):
    a = {**GEMM, "x": P, "dt": 1, "ws": P, "bytes": 4 * 68, **change}
    assert lib().int8_linear(a["x"], a["dt"], a["b"], a["sb"], a["bias"], a["d"], a["M"], a["N"], a["K"], a["out"], a["ws"],
                             a["bytes"], None) == code
    assert "int8_linear" in last()


@pytest.mark.parametrize("change,code", [
    (dict(G=0), EINVAL), (dict(G=65536), EINVAL), (dict(meta=None), EINVAL), (dict(meta=P + 1), EINVAL), (dict(K=8), EUNSUPPORTED),
    (dict(M=4096 * 128 + 1), EUNSUPPORTED), (dict(N=-4), EINVAL), (dict(out=-1), EINVAL),
])
@pytest.mark.parametrize("masked", [False, True])
def test_grouped_refuses(change, code, masked):
    a = {**GEMM, "G": 1, "meta": P, **change}
    ops = (a["a"], a["sa"], a["b"], a["sb"], a["meta"], a["d"])
    if masked:
        rc = lib().grouped_int8_gemm_masked(*ops, a["G"], a["M"], a["N"], a["K"], a["out"], None)
    else:
        rc = lib().grouped_int8_gemm_contiguous(*ops, a["M"], a["N"], a["K"], a["G"], a["out"], None)
    assert rc == code and "grouped_int8_gemm" in last()


TOPK = dict(l=P, dt=0, bias=None, ids=P, w=P, T=3, E=8, k=2, score=0)


@pytest.mark.parametrize("change,code", [
    (dict(dt=7), EINVAL), (dict(score=2), EINVAL), (dict(T=-1), EINVAL), (dict(E=0), EINVAL), (dict(k=0), EINVAL),
    (dict(k=9), EINVAL), (dict(E=1025), EUNSUPPORTED), (dict(E=100, k=65), EUNSUPPORTED), (dict(T=1 << 31), EUNSUPPORTED),
    (dict(l=None), EINVAL), (dict(ids=None), EINVAL), (dict(w=None), EINVAL), (dict(l=P + 2), EINVAL), (dict(ids=P + 2), EINVAL),
    (dict(bias=P + 1), EINVAL), (dict(dt=1, l=P + 1), EINVAL),
])
def test_topk_refuses(change, code):
    a = {**TOPK, **change}
    assert lib().moe_topk(a["l"], a["dt"], a["bias"], a["ids"], a["w"], a["T"], a["E"], a["k"], a["score"], 1, 1.0, None) == code
    assert "moe_topk" in last()


LAYER = dict(x=P, dt=0, ids=P, w=P, w1=P, s1=P, w2=P, s2=P, out=P, T=2, k=3, E=4, H=256, I=128, ws=P, bytes=2 * 3 * 384 * 4)


@pytest.mark.parametrize("change,code", [
    (dict(dt=2), EINVAL), (dict(T=-1), EINVAL), (dict(k=0), EINVAL), (dict(E=0), EINVAL), (dict(H=0), EINVAL), (dict(I=-128), EINVAL),
    (dict(E=1025), EUNSUPPORTED), (dict(T=342), EUNSUPPORTED), (dict(T=1 << 40, k=1 << 40), EUNSUPPORTED), (dict(H=192), EUNSUPPORTED),
    (dict(I=64), EUNSUPPORTED), (dict(H=65664), EUNSUPPORTED), (dict(H=32384), EUNSUPPORTED), (dict(I=32384), EUNSUPPORTED), (dict(x=None), EINVAL), (dict(ids=None), EINVAL), (dict(w=None), EINVAL),
    (dict(w1=None), EINVAL), (dict(s1=None), EINVAL), (dict(w2=None), EINVAL), (dict(s2=None), EINVAL), (dict(out=None), EINVAL),
    (dict(x=P + 8), EINVAL), (dict(w1=P + 8), EINVAL), (dict(out=P + 2), EINVAL), (dict(ids=P + 2), EINVAL), (dict(ws=None), EINVAL),
    (dict(ws=P + 4), EINVAL), (dict(bytes=2 * 3 * 384 * 4 - 1), EINVAL),
])
@pytest.mark.parametrize("weight", ["fp8", "int8"])
def test_layer_refuses(change, code, weight):
    a = {**LAYER, **change}
    entry = lib().moe_fp8_layer if weight == "fp8" else lib().moe_int8_layer
    assert entry(*(a[n] for n in ("x", "dt", "ids", "w", "w1", "s1", "w2", "s2", "out", "T", "k", "E", "H", "I", "ws", "bytes")),
                 None) == code
    assert f"moe_{weight}_layer" in last()


def test_nothing_to_do_is_no_error():
    """No rows: success without a launch, whatever the pointers."""
    n = None
    assert lib().int8_quantize_token_device(n, 0, 0, 64, n, n, n) == 0
    assert lib().int8_gemm(n, n, n, n, n, n, 0, 5, 64, 0, n) == 0
    assert lib().int8_linear(n, 1, n, n, n, n, 0, 5, 64, 0, n, 0, n) == 0
    assert lib().grouped_int8_gemm_contiguous(n, n, n, n, n, n, 0, 5, 64, 2, 0, n) == 0
    assert lib().grouped_int8_gemm_masked(n, n, n, n, n, n, 2, 0, 5, 64, 0, n) == 0
    assert lib().moe_topk(n, 0, n, n, n, 0, 8, 2, 0, 1, 1.0, n) == 0
    assert lib().moe_fp8_layer(n, 0, n, n, n, n, n, n, n, 0, 3, 4, 256, 128, n, 0, n) == 0


def test_workspace_sizes():
    assert gfg.int8_linear_workspace_bytes(7, 64) == 7 * 68 and gfg.int8_linear_workspace_bytes(0, 64) == 0
    assert gfg.moe_layer_workspace_bytes(2, 3, 256, 128) == 2 * 3 * 384 * 4 and gfg.moe_layer_workspace_bytes(0, 3, 256, 128) == 0


def test_bindings_refuse_what_is_not_on_a_gpu():
    z = torch.zeros
    i8, i32 = torch.int8, torch.int32
    d = z(2, 4, dtype=torch.bfloat16)
    for call in (
        lambda: gfg.int8_quantize_token_device(z(2, 16)),
        lambda: gfg.int8_gemm(z(2, 16, dtype=i8), z(2), z(4, 16, dtype=i8), z(4), d),
        lambda: gfg.int8_linear(z(2, 16), z(4, 16, dtype=i8), z(4), d),
        lambda: gfg.grouped_int8_gemm_contiguous(z(2, 16, dtype=i8), z(2), z(1, 4, 16, dtype=i8), z(1, 4), z(2, dtype=i32), d),
        lambda: gfg.grouped_int8_gemm_masked(z(1, 2, 16, dtype=i8), z(1, 2), z(1, 4, 16, dtype=i8), z(1, 4), z(1, dtype=i32), d[None]),
        lambda: gfg.moe_topk(z(2, 8), z(2, 2, dtype=i32), z(2, 2)),
        lambda: gfg.moe_int8_layer(z(2, 128, dtype=torch.bfloat16), z(2, 1, dtype=i32), z(2, 1), z(1, 256, 128, dtype=i8), z(1, 256),
                                   z(1, 128, 128, dtype=i8), z(1, 128), z(2, 128, dtype=torch.bfloat16)),
    ):
        with pytest.raises(ValueError, match="must be on a GPU"):
            call()


# ------------------------------------------------------------------ the definitions
def test_quantizer_definition_examples():
    q, s = so.quantize_token(np.array([[127.0, -127.0, 0.5, 1.5], [0, 0, 0, 0], [1, np.nan, 0, 0]], np.float32))
    assert q.tolist() == [[127, -127, 0, 2], [0] * 4, [0] * 4]
    assert s[0] == 1.0 and s[1] == np.float32(2.0 ** -100) / np.float32(127) and np.isnan(s[2])


def test_topk_definition_examples():
    ids, w = so.topk([[0.0, np.log(3.0), 0.0, -np.inf]], 3)
    assert ids.tolist() == [[1, 0, 2]] and np.allclose(w, [[0.6, 0.2, 0.2]])
    ids, w = so.topk([[0.0, np.nan, 0.0]], 3, score="sigmoid", renormalize=False, scale=2.0)
    assert ids.tolist() == [[0, 2, -1]] and np.allclose(w, [[1.0, 1.0, 0.0]])
    ids, _ = so.topk([[4.0, 0.0, 0.0]], 1, bias=[0.0, 0.0, 5.0])
    assert ids.tolist() == [[2]]


def test_layer_definition_example():
    """One channel each way: silu(2) * 3 * 0.5 + nothing from a foreign expert."""
    w1 = np.array([[[2.0], [3.0]]])
    w2 = np.array([[[1.0]]])
    out = so.layer(np.array([[1.0]]), [[0, 7]], [[0.5, 9.0]], w1, w2)
    assert np.allclose(out, 0.5 * 3 * 2 / (1 + np.exp(-2.0)))
