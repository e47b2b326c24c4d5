"""Few tokens and an output wider than 32768, as a vocabulary's head has it: from 4 to 64 tokens on, more tiles of 128 x 128
than CUs, that is tiles of 256 x 256 most of whose rows are past the end.  Whole numbers: exact sums on every tile."""
import numpy as np
import pytest
import torch

import fp8_block_scaled_amd as gfg

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("N", [32752, 33024, 40001])
@pytest.mark.parametrize("bias", [True, False])
def test_products_of_few_tokens(N, bias):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(N)
    K = 272
    b = torch.randint(-8, 9, (N, K), generator=gen, device="cuda").float()
    qb, sb = gfg.fp8_quantize_weight_device(b)
    add = torch.randint(-64, 65, (N,), generator=gen, device="cuda").float() if bias else None
    b = b.double().t().contiguous()
    for M in (1, 3, 4, 5, 16, 17, 32, 33, 64, 130):
        x = torch.randint(-8, 9, (M, K), generator=gen, device="cuda").float()
        want = x.double() @ b + (0 if add is None else add.double())
        for dtype in (torch.bfloat16, torch.float16):
            d = torch.full((M + 1, N), 99.0, dtype=dtype, device="cuda")
            gfg.fp8_linear(x, qb, sb, d[:M], bias=add)
            assert torch.equal(d[:M], want.to(dtype)) and bool((d[M] == 99.0).all()), (M, dtype)


def test_norm_into_a_head():
    torch.manual_seed(0)
    M, H, N = 9, 272, 33001
    y, r, w = torch.randn(M, H, device="cuda").to(torch.bfloat16), torch.randn(M, H, device="cuda"), torch.rand(H, device="cuda") + 0.5
    _, q, s, _ = gfg.residual_norm_fp8(y, r, w)
    weight = torch.randn(N, H, device="cuda") * H ** -0.5
    qw, sw = gfg.fp8_quantize_weight_device(weight)
    d = gfg.fp8_gemm(q, s, qw, sw, torch.empty(M, N, dtype=torch.bfloat16, device="cuda"))
    pad = lambda t, f: t.repeat_interleave(f, -1)[..., :H]  # noqa: E731
    value = lambda b: torch.exp2(b.double() - 127)  # noqa: E731
    a = q.double() * pad(value(s).t(), 128)
    b = qw.double() * pad(value(sw), 128).repeat_interleave(128, 0)[:N]
    b = b.t().contiguous()
    # one rounding to bf16, and products 2^-14 below the largest of their group of 16 left out: 2^-10 of the products' sizes
    assert bool(((d.double() - a @ b).abs() <= 2.0 ** -8 * (a @ b).abs() + 2.0 ** -10 * (a.abs() @ b.abs())).all())
