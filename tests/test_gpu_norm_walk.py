"""The norms over more rows than one turn of their workgroups takes, at every number of lanes a row: rows loaded a turn
ahead, the alternating buffers of the sums, sums over a workgroup's rows, in place while walking.

Forward walks above 4096 rows up to 1024 channels, 2048 up to 2048, 1024 up to 4096, 512 up to 8192 and 256 above; backward
from 256 of its turns on.  Checks and tolerances are those of the smaller sizes (a sum over rows is a chain of at most
five of a workgroup's, 16 of a lane's partial sums and 32 of the lanes').
"""
import numpy as np
import pytest
import torch

import fp8_block_scaled_amd as gfg
import test_gpu_norm as norm
from oracle import layers_oracle as lo

pytestmark = pytest.mark.gpu

# channels of whole and of partial chunks at 64, 128, 256, 512 and 1024 lanes, and at 1024 of four chunks, the last one of
# which is empty, partial or full
SIZES = [(4100, 64), (5300, 520), (2051, 1030), (1027, 2049), (1300, 2056), (600, 4104), (1100, 8191), (300, 8200), (520, 12288), (300, 16384),
         (3, 16385), (5, 24584), (260, 20001), (520, 17000), (258, 32768)]
KINDS = [("bf16", "f32", True, "channel"), ("f16", "f16", True, "token"), ("f32", "f32", False, "none")]


@pytest.mark.parametrize("M,H", SIZES)
@pytest.mark.parametrize("y,r,post,gate", KINDS)
def test_forward(M, H, y, r, post, gate):
    norm.test_forward(M, H, y, r, post, gate)


@pytest.mark.parametrize("M,H", SIZES)
@pytest.mark.parametrize("y,r,post,gate", KINDS)
def test_backward(M, H, y, r, post, gate):
    norm.test_backward(M, H, y, r, post, gate)


@pytest.mark.parametrize("M,H", [(4100, 64), (2051, 1040), (1027, 2064), (600, 4112), (300, 8208), (520, 16384), (260, 20000)])
def test_fp8_rows(M, H):
    norm.test_fp8_rows(M, H, "bf16", "f32")


@pytest.mark.parametrize("M,H", [(4100, 70), (2051, 1030), (1027, 2049), (600, 4104), (300, 8200), (260, 20001)])
@pytest.mark.parametrize("weight", [True, False])
def test_in_place(M, H, weight):
    """out may be the residual itself: the same bytes as in a tensor of its own."""
    a = norm.inputs(M, H, "bf16", "bf16", True, "channel", 5)
    y, r, w, p, g = (norm.dev(a[n], norm.DT[t]) for n, t in (("y", "bf16"), ("residual", "bf16"), ("weight", "f32"), ("post", "f32"), ("gate", "f32")))
    args = dict(post_weight=p, gate=g, alpha=0.75)
    out, normed, _ = gfg.residual_norm(y, r.clone(), w if weight else None, **args)
    same = r.clone()
    _, again, _ = gfg.residual_norm(y, same, w if weight else None, out=same, **args)
    assert torch.equal(same, out) and (not weight or torch.equal(again, normed))


@pytest.mark.parametrize("M,H", [(4100, 64), (1027, 2049), (600, 4104), (300, 16384), (260, 20001)])
def test_backward_adds_up_over_calls(M, H):
    """Two halves of the rows, the second one accumulated: the sums of all, to the rounding of a sum of two."""
    rng = np.random.default_rng(M)
    n = lambda *s: rng.standard_normal(s).astype(np.float32)  # noqa: E731
    dout, dz, out, y, w, p, g = n(M, H), n(M, H), n(M, H), n(M, H), 1 + 0.2 * n(H), 1 + 0.2 * n(H), n(H)
    stats = 1 / np.sqrt(np.stack([(y.astype(np.float64) ** 2).mean(1), (out.astype(np.float64) ** 2).mean(1)]))
    stats = stats.astype(np.float32)
    grads = [torch.full((H,), 7.0, device="cuda") for _ in range(3)]
    for rows, add in ((slice(0, M // 2 + 1), False), (slice(M // 2 + 1, M), True)):
        d = lambda v: norm.dev(v[rows])  # noqa: E731
        gfg.residual_norm_backward(d(dout), d(dz), d(out), d(y), norm.dev(stats[:, rows]), norm.dev(w), post_weight=norm.dev(p), gate=norm.dev(g),
                                   dweight=grads[0], dpost_weight=grads[1], dgate=grads[2], accumulate=add)
    ry, ro = stats[0][:, None].astype(np.float64), stats[1][:, None].astype(np.float64)
    ref = lo.residual_norm_backward(dout, dz, out, y, ry, ro, w, p, g)
    zh, h = np.abs(out * ro), np.abs(dz * w)
    G = np.abs(dout) + ro * (h + zh * (h * zh).mean(1, keepdims=True))
    yh = np.abs(y * ry)
    for got, want, size in zip(grads, ref[2:], ((np.abs(dz) * zh).sum(0), (np.abs(g) * G * yh).sum(0), (G * yh * np.abs(p)).sum(0))):
        norm.close(got, want, size, torch.float32, "sum")
