"""The widest outputs that the integer products take, at their documented limit (CPU: nothing is launched)."""
import pytest

import fp8_block_scaled_amd as gfg

P = 1 << 20            # an aligned made-up address


@pytest.mark.parametrize("entry", ["int8_gemm", "int8_linear", "grouped_int8_gemm_contiguous", "grouped_int8_gemm_masked"])
def test_outputs_wider_than_2_to_28(entry):
    lib, N = gfg.load_library(), (1 << 28) + 1

    def call(M, N):
        if entry == "int8_gemm":
            return lib.int8_gemm(P, P, P, P, None, P, M, N, 64, 0, None)
        if entry == "int8_linear":
            return lib.int8_linear(P, 1, P, P, None, P, M, N, 64, 0, P, 1 << 20, None)
        if entry == "grouped_int8_gemm_contiguous":
            return lib.grouped_int8_gemm_contiguous(P, P, P, P, P, P, M, N, 64, 1, 0, None)
        return lib.grouped_int8_gemm_masked(P, P, P, P, P, P, 1, M, N, 64, 0, None)

    assert call(4, N) == 2 and entry in lib.grouped_fp8_last_error().decode()      # GFG_EUNSUPPORTED
    assert call(0, N - 1) == 0                             # the limit itself is a size like others
