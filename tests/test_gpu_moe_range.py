"""Hidden values at the end of fp32's range in the expert layer.

x = (1, -d, 0, ...), and an expert's rows pick g = (1 - d) 2^64 and u = +-2^64, so that h = silu(g) * u =
+-(1 - d) 2^128 exactly: finite in fp32, for d from 2^-8 (the largest bf16) to 2^-16, and for d < 2^-9 nearer to
2^128 than to any bf16 number.  Each output picks one hidden value and scales it by 2^-20.  The only errors left are
the hidden rows' 16 significant bits (2^-16 at this end of the range, where the high part is held down) and the
output's rounding, 2^-8, which act on the same value.
"""
import numpy as np
import pytest
import torch

import fp8_block_scaled_amd as gfg

pytestmark = pytest.mark.gpu


def expert_weights(weight, E, H, I):
    """Codes and scales of the rows above; the odd rows' up value is negative."""
    one = 0x38 if weight == "fp8" else 1                   # 1.0 in E4M3
    minus = 0xB8 if weight == "fp8" else 0xFF
    w1 = torch.zeros(E, 2 * I, H, dtype=torch.uint8, device="cuda")
    w1[:, :I, :2] = one                                    # gate: x0 + x1
    w1[:, I::2, 0] = one                                   # up: x0, -x0
    w1[:, I + 1::2, 0] = minus
    w2 = torch.zeros(E, H, I, dtype=torch.uint8, device="cuda")
    n = torch.arange(H, device="cuda")
    w2[:, n, n % I] = one
    if weight == "fp8":
        s1 = torch.full((E, 2 * I // 128, H // 128), 127 + 64, dtype=torch.uint8, device="cuda")
        s2 = torch.full((E, H // 128, I // 128), 127 - 20, dtype=torch.uint8, device="cuda")
        return w1, s1, w2, s2
    s1 = torch.full((E, 2 * I), 2.0 ** 64, device="cuda")
    s2 = torch.full((E, H), 2.0 ** -20, device="cuda")
    return w1.view(torch.int8), s1, w2.view(torch.int8), s2


# the last size's down projection runs by items that the waves share, the others' by 16 or 32 columns a workgroup
@pytest.mark.parametrize("weight", ["fp8", "int8"])
@pytest.mark.parametrize("T,E,k,H,I", [(1, 2, 1, 128, 128), (40, 2, 1, 256, 256), (100, 8, 1, 4096, 1792)])
def test_largest_hidden_values_stay_finite(weight, T, E, k, H, I):
    print(f"[moe] range {weight} T={T} H={H} I={I}", flush=True)
    ops = expert_weights(weight, E, H, I)
    d = 2.0 ** -(8.0 + (np.arange(T) + 2) % 9)             # bf16 holds these
    x = torch.zeros(T, H)
    x[:, 0], x[:, 1] = 1.0, torch.from_numpy(-d).float()
    x = x.to(torch.bfloat16).cuda()
    ids = (torch.arange(T * k, device="cuda", dtype=torch.int32) % E).view(T, k)
    out = torch.empty_like(x)
    layer = gfg.moe_fp8_layer if weight == "fp8" else gfg.moe_int8_layer
    layer(x, ids, torch.ones(T, k, device="cuda"), *ops, out)
    sign = np.where((np.arange(H) % I) % 2 == 0, 1.0, -1.0)
    want = (1 - d)[:, None] * sign[None] * 2.0 ** 108
    got = out.float().cpu().numpy().astype(np.float64)
    assert np.isfinite(got).all(), f"{np.isnan(got).sum()} NaNs, {np.isinf(got).sum()} infinities of {got.size}"
    assert (np.abs(got - want) <= (2.0 ** -8 + 2.0 ** -15) * np.abs(want)).all()
