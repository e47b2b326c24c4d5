"""The first norm of a network on a 32-bit residual stream: no y, the normed rows in 16 bits for the block behind it."""
import os
import sys

import numpy as np
import pytest
import torch

import fp8_block_scaled_amd as gfg
import test_gpu_norm as norm
from oracle import layers_oracle as lo
from test_layers_host import bf16, f32, t, u8, world  # noqa: F401

f16 = torch.float16


@pytest.mark.parametrize("dtype", [bf16, f16, f32])
def test_normed_decides_the_type_of_the_rows(dtype, world):  # noqa: F811
    library, _ = world
    got = gfg.residual_norm(None, t(f32, 5, 33), t(f32, 33), normed=t(dtype, 5, 33))
    assert got[0] is None and got[1].dtype == dtype and [name for name, *_ in library.seen] == ["residual_norm"]


def test_without_normed_the_rows_are_like_the_residual(world):  # noqa: F811
    for dtype in (bf16, f16, f32):
        assert gfg.residual_norm(None, t(dtype, 5, 33), t(f32, 33))[1].dtype == dtype


@pytest.mark.parametrize("y,residual,normed", [(None, bf16, f32), (None, bf16, f16), (None, f32, u8), (bf16, f32, f16), (bf16, f32, f32)])
def test_other_types_are_refused(y, residual, normed, world):  # noqa: F811
    with pytest.raises(TypeError, match="normed has dtype"):
        gfg.residual_norm(None if y is None else t(y, 5, 33), t(residual, 5, 33), t(f32, 33), normed=t(normed, 5, 33))
    assert not world[0].seen


@pytest.mark.gpu
@pytest.mark.parametrize("M,H", [(1, 7168), (5, 33), (333, 2049), (300, 16384)])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_rows_of_16_bits_from_a_residual_of_32(M, H, dtype):
    a = norm.inputs(M, H, dtype, "f32", False, "none", 8)
    r, w = norm.dev(a["residual"]), norm.dev(a["weight"])
    normed = torch.full((M, H), 9.0, dtype=norm.DT[dtype], device="cuda")
    stats = torch.empty(2, M, device="cuda")
    gfg.residual_norm(None, r, w, normed=normed, stats=stats)
    want = lo.residual_norm(None, a["residual"], a["weight"])
    norm.close(normed, want[1], 2 * np.abs(want[1]), norm.DT[dtype], "normed")
    # and its gradients, in the residual's type
    dz, dr, dw = torch.randn(M, H, device="cuda").to(norm.DT[dtype]), torch.empty_like(r), torch.empty_like(w)
    gfg.residual_norm_backward(None, dz, r, None, stats, w, dresidual=dr, dweight=dw)
    ro, dz = norm.host(stats)[1][:, None], norm.host(dz)
    ref = lo.residual_norm_backward(None, dz, a["residual"], None, None, ro, a["weight"])
    zh, h = np.abs(a["residual"] * ro), np.abs(dz * a["weight"])
    norm.close(dr, ref[0], ro * (h + zh * (h * zh).mean(1, keepdims=True)), torch.float32, "dresidual")
    norm.close(dw, ref[2], (np.abs(dz) * zh).sum(0), torch.float32, "dweight")


@pytest.mark.gpu
def test_the_example_serves_on_a_residual_of_32_bits():
    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
    import fp8_block as ex
    block = ex.random_block(16, 2, 256, 128, with_experts=True)
    y, r = torch.randn(9, 256, device="cuda").to(torch.bfloat16), torch.randn(9, 256, device="cuda")
    out, m = block.serve(y, r)
    assert out.dtype == torch.float32 and m.dtype == torch.bfloat16 and bool(torch.isfinite(m).all()) and bool(torch.isfinite(out).all())
    # where the residual is one that 16 bits hold, only out's rounding differs
    r16 = r.to(torch.bfloat16)
    out16, m16 = block.serve(y, r16)
    out32, m32 = block.serve(y, r16.float())
    assert torch.equal(out32.to(torch.bfloat16), out16) and m32.shape == m16.shape
