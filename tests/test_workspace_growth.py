"""A workspace for the most tokens that a program has serves every smaller call too: no call's need falls as tokens are added."""
import pytest

import fp8_block_scaled_amd as gfg

EINVAL = 1
P = 1 << 20
COUNTS = sorted({*range(0, 300), *(n + d for n in (512, 768, 1024, 1280, 1536, 2048, 2560, 4096, 8192, 32768, 65536) for d in range(-2, 3)),
                 *range(300, 140000, 997)})


@pytest.mark.parametrize("need", [
    *(pytest.param(lambda M, H=H: gfg.residual_norm_backward_workspace_bytes(M, H), id=f"norm {H}") for H in (8, 64, 1030, 2049, 4104, 8192, 16384, 32768)),
    *(pytest.param(lambda T, E=E, S=S: gfg.moe_balance_workspace_bytes(T, E, S), id=f"balance {E} {S}") for E in (3, 64, 385, 1000) for S in (1, 7)),
    *(pytest.param(lambda M, K=K: gfg.fp8_linear_workspace_bytes(M, K), id=f"linear {K}") for K in (16, 2304)),
    *(pytest.param(lambda M, N=N: gfg.fp8_linear_backward_workspace_bytes(M, N, 272), id=f"backward {N}") for N in (48, 7168)),
    pytest.param(lambda M: gfg.int8_linear_workspace_bytes(M, 272), id="int8"),
    pytest.param(lambda T: gfg.moe_layer_workspace_bytes(T, 4, 512, 256), id="experts"),
])
def test_needs_do_not_fall(need):
    got = [need(n) for n in COUNTS]
    assert got == sorted(got)


@pytest.mark.parametrize("M", [1, 255, 256, 700, 1024])
def test_what_the_largest_call_needs_is_asked_of_no_smaller_one(M):
    """And the argument check asks for that need, not a byte less."""
    lib = gfg.load_library()
    H, most = 8192, gfg.residual_norm_backward_workspace_bytes(1025, 8192)
    short = gfg.residual_norm_backward_workspace_bytes(M, H)
    assert short <= most
    assert lib.residual_norm_backward(P, P, P, P, P, P, P, None, 0, 1.0, P, P, P, P, None, 0, M, H, 1, 1, P, short - 1, None) == EINVAL
    assert "workspace" in lib.grouped_fp8_last_error().decode()
