"""The hardware's scaled conversions, as the quantizers use them, give the nearest E4M3 code (ties to even) of value / scale
at every scale: all finite bit patterns of both 16-bit types, and of 32 bits the values around every border between two
codes, every code, and subnormal values.

A block of 128 x 128 is led by a value that gives it its scale and filled with values that this scale covers.  Both
orientations go through instructions of their own (pairs of a row, pairs of a column).
"""
import numpy as np
import pytest
import torch

import fp8_block_scaled_amd as gfg

pytestmark = pytest.mark.gpu

BLOCK = 128 * 128


def codes(v):
    """E4M3 codes of float64 values of at most 448."""
    a = np.abs(v)
    _, e = np.frexp(a)
    step = np.ldexp(1.0, np.maximum(e - 1, -6) - 3)
    r = np.rint(a / step) * step
    _, e = np.frexp(r)
    e = np.where(r >= 2.0 ** -6, e - 1, -6)
    mant = np.rint(np.ldexp(r, 3 - e)).astype(np.int64)        # 8 to 15 in the normal range, 0 to 7 below
    code = np.where(r >= 2.0 ** -6, ((e + 7) << 3) + mant - 8, mant)
    return (code | np.where(np.signbit(v), 0x80, 0)).astype(np.uint8)


def check(values, scales, dtype):
    """values(t): ascending magnitudes (float64) that the type holds, up to 448 2^t."""
    blocks, bytes_ = [], []
    for t in scales:
        v = values(t)
        if not len(v) or v[-1] <= 448.0 * 2.0 ** (t - 1):      # nothing gives this scale
            continue
        v = np.concatenate([v, -v])
        lead = np.abs(v).max()
        for i in range(0, len(v), BLOCK - 1):
            part = v[i:i + BLOCK - 1]
            blocks.append(np.concatenate([[lead], part, np.zeros(BLOCK - 1 - len(part))]))
            bytes_.append(t + 127)
    assert len(bytes_) > 30
    for i in range(0, len(blocks), 256):
        some = np.stack(blocks[i:i + 256])
        w = torch.from_numpy(some).to(dtype).view(-1, 128, 128)
        assert torch.equal(w.double().view(len(some), -1), torch.from_numpy(some))          # (the type holds them)
        q, s, q_t, s_t = gfg.fp8_quantize_weight_device(w.cuda(), transposed=True)
        assert s.flatten().tolist() == bytes_[i:i + 256] == s_t.flatten().tolist()
        want = torch.from_numpy(codes(some * np.exp2(127.0 - np.asarray(bytes_[i:i + 256], np.float64))[:, None])).view(-1, 128, 128)
        assert torch.equal(q.view(torch.uint8).cpu(), want) and torch.equal(q_t.view(torch.uint8).cpu(), want.transpose(1, 2))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_every_pattern_of_16_bits(dtype):
    every = torch.arange(1 << 15, dtype=torch.int32).to(torch.int16).view(dtype).double().numpy()
    every = np.sort(every[np.isfinite(every)])
    check(lambda t: every[:np.searchsorted(every, 448.0 * 2.0 ** t, "right")], range(-127, 121), dtype)


def test_borders_of_32_bits():
    grid = np.unique(np.concatenate([m * 2.0 ** e for e in range(-9, 9) for m in [np.arange(8, 16) / 8.0]] + [np.arange(0, 8) * 2.0 ** -9]))
    grid = grid[grid <= 448]
    at = np.concatenate([grid, (grid[1:] + grid[:-1]) / 2]).astype(np.float32)
    rng = np.random.default_rng(1)
    near = np.concatenate([at, np.nextafter(at, np.float32(1e9)), np.nextafter(at, np.float32(0)), rng.uniform(0, 448, 3000).astype(np.float32),
                           np.exp2(rng.uniform(-30, 8.8, 3000)).astype(np.float32)]).astype(np.float64)

    def values(t):
        v = (near * 2.0 ** t).astype(np.float32).astype(np.float64)         # (rounded where they are subnormal)
        return np.unique(v[v <= 448.0 * 2.0 ** t])

    check(values, range(-127, 120), torch.float32)
