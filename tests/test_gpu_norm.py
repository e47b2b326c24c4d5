"""The norms around a block with gate and residual sum, and their gradients, against 64-bit definitions.

Tolerances: an output is rounded once (eps / 2 of the value); before that, in fp32, a sum of H squares has a relative
error of at most n 2^-24 with n the longest chain of additions (H / lanes + 20 < 96), rsqrt and the products add a few
2^-24 more: 2^-16 of the terms' size in all, which for a gradient are the sizes of its terms, and for a sum over rows
the sum of their sizes.  Below 2^-14 float16's step is 2^-24 whatever the value, so its rounding is 2^-25 there.
"""
import numpy as np
import pytest
import torch

import fp8_block_scaled_amd as gfg
from oracle import fp8_oracle as o
from oracle import layers_oracle as lo

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
HALF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
F32 = 2.0 ** -16
LEAST = {torch.float16: 2.0 ** -25}
TYPES = [("bf16", "bf16"), ("bf16", "f32"), ("f16", "f16"), ("f16", "f32"), ("f32", "f32")]
SIZES = [(1, 9), (1, 7168), (3, 8), (5, 33), (4, 15), (7, 1023), (8, 1025), (333, 2049), (17, 2048), (9, 4096), (4, 4104), (2, 8191), (3, 16384), (2, 32768), (1030, 64), (600, 300)]


def dev(x, dtype=torch.float32):
    return None if x is None else torch.from_numpy(np.ascontiguousarray(x)).cuda().to(dtype)


def host(t):
    return None if t is None else t.double().cpu().numpy()


def close(got, ref, size, dtype, what):
    g = host(got)
    off = np.abs(g - ref) - (HALF[dtype] * np.abs(ref) + F32 * size + LEAST.get(dtype, 0.0)) * (1 + 2.0 ** -10)
    assert np.isfinite(g).all() and off.max() <= 0, (what, off.max())


def inputs(M, H, y, r, post, gate, seed=0):
    rng = np.random.default_rng(seed + M + H)
    n = lambda *s: rng.standard_normal(s)  # noqa: E731
    held = lambda v, t: host(dev(v, DT[t]))  # noqa: E731     as the type holds it
    f = lambda v: held(v, "f32")  # noqa: E731
    return dict(y=held(n(M, H) * np.exp2(rng.integers(-4, 5, (M, 1))), y), residual=held(3 * n(M, H), r), weight=f(1 + 0.2 * n(H)),
                post=f(1 + 0.2 * n(H)) if post else None, gate={"none": None, "channel": f(n(H)), "token": f(n(M, 1))}[gate])


@pytest.mark.parametrize("M,H", SIZES)
@pytest.mark.parametrize("y,r", TYPES)
@pytest.mark.parametrize("post,gate", [(True, "channel"), (True, "token"), (False, "none"), (False, "channel")])
def test_forward(M, H, y, r, post, gate):
    a = inputs(M, H, y, r, post, gate)
    out, normed, stats = gfg.residual_norm(dev(a["y"], DT[y]), dev(a["residual"], DT[r]), dev(a["weight"]), post_weight=dev(a["post"]),
                                           gate=dev(a["gate"]), alpha=0.75, eps=1e-5, stats=torch.empty(2, M, device="cuda"))
    ro, rn, ry, rr = lo.residual_norm(a["y"], a["residual"], a["weight"], a["post"], a["gate"], 0.75, 1e-5)
    u = np.abs(ro - 0.75 * a["residual"])
    size = 0.75 * np.abs(a["residual"]) + u
    close(out, ro, size, DT[r], "out")
    close(normed, rn, np.abs(size * rr * a["weight"]) + np.abs(rn), DT[y], "normed")
    s = host(stats)
    assert np.allclose(s[0], ry[:, 0], rtol=F32, atol=0) and np.allclose(s[1], rr[:, 0], rtol=4 * F32, atol=0)


@pytest.mark.parametrize("M,H", SIZES)
@pytest.mark.parametrize("y,r", TYPES)
@pytest.mark.parametrize("post,gate", [(True, "channel"), (True, "token"), (True, "none"), (False, "none"), (False, "channel"), (False, "token")])
def test_backward(M, H, y, r, post, gate):
    a = inputs(M, H, y, r, post, gate, 1)
    rng = np.random.default_rng(M * H)
    dout, dz = host(dev(rng.standard_normal((M, H)), DT[r])), host(dev(rng.standard_normal((M, H)), DT[y]))
    out, _, ry, ro = lo.residual_norm(a["y"], a["residual"], None, a["post"], a["gate"], 0.75, 1e-5)
    out = host(dev(out, DT[r]))                            # as the forward call stored it
    stats = host(dev(np.concatenate([ry.T, ro.T])))
    ry, ro = stats[0][:, None], stats[1][:, None]
    new = lambda like, t: torch.full(like.shape, 9.0, dtype=t, device="cuda")  # noqa: E731
    g = dict(dresidual=new(out, DT[r]), dy=new(out, DT[y]), dweight=new(a["weight"], torch.float32),
             dpost_weight=new(a["weight"], torch.float32) if post else None, dgate=None if a["gate"] is None else new(a["gate"], torch.float32))
    gfg.residual_norm_backward(dev(dout, DT[r]), dev(dz, DT[y]), dev(out, DT[r]), dev(a["y"], DT[y]), dev(stats), dev(a["weight"]),
                               post_weight=dev(a["post"]), gate=dev(a["gate"]), alpha=0.75, **g)
    ref = lo.residual_norm_backward(dout, dz, out, a["y"], ry, ro, a["weight"], a["post"], a["gate"], 0.75)
    # the sizes of the terms
    zh, h = np.abs(out * ro), np.abs(dz * a["weight"])
    G = np.abs(dout) + ro * (h + zh * (h * zh).mean(1, keepdims=True))
    gate_ = 1.0 if a["gate"] is None else np.abs(a["gate"])
    yh = np.abs(a["y"] * (ry if post else 1.0))
    u = yh * (np.abs(a["post"]) if post else 1.0)
    v = gate_ * G * (np.abs(a["post"]) if post else 1.0)
    sy = (ry * (v + yh * (v * yh).mean(1, keepdims=True))) if post else v
    close(g["dresidual"], ref[0], 0.75 * G, DT[r], "dresidual")
    close(g["dy"], ref[1], sy, DT[y], "dy")
    close(g["dweight"], ref[2], (np.abs(dz) * zh).sum(0), torch.float32, "dweight")
    if post:
        close(g["dpost_weight"], ref[3], (gate_ * G * yh).sum(0), torch.float32, "dpost")
    if gate != "none":
        close(g["dgate"], ref[4], (G * u).sum(0) if gate == "channel" else (G * u).sum(1, keepdims=True), torch.float32, "dgate")


@pytest.mark.parametrize("M,H", [(1, 16), (1, 7168), (5, 144), (333, 1040), (6, 2048), (3, 4112), (2, 16384), (64, 300 * 16)])
@pytest.mark.parametrize("y,r", TYPES)
def test_fp8_rows(M, H, y, r):
    """The codes are the quantizer's of the 64-bit rows, but for values within 2^-13 of a border between two codes (a
    step then), and scales likewise."""
    a = inputs(M, H, y, r, True, "channel", 2)
    out, q, s, _ = gfg.residual_norm_fp8(dev(a["y"], DT[y]), dev(a["residual"], DT[r]), dev(a["weight"]), post_weight=dev(a["post"]),
                                         gate=dev(a["gate"]), alpha=0.75)
    ro, rn, _, rr = lo.residual_norm(a["y"], a["residual"], a["weight"], a["post"], a["gate"], 0.75)
    size = (0.75 * np.abs(a["residual"]) + np.abs(ro - 0.75 * a["residual"])) * rr * np.abs(a["weight"])
    got = o.dequantize_act(q.view(torch.uint8).cpu().numpy(), s.cpu().numpy())
    scale = o.e8m0_value(s.cpu().numpy()).T.repeat(128, 1)[:, :H]
    amax = np.pad(np.abs(rn), ((0, 0), (0, -H % 128))).reshape(M, -1, 128).max(2)
    fits = 448.0 * o.e8m0_value(s.cpu().numpy()).T / amax
    assert (fits >= 1 - 2.0 ** -14).all() and (fits <= 2 * (1 + 2.0 ** -14)).all()
    # nearest code: within half a step (2^-4 of the value, 2^-10 of the scale below the normal range) of the row
    assert (np.abs(got - rn) <= 2.0 ** -4 * np.abs(rn) + 2.0 ** -10 * scale + F32 * size).all()
    exact = o.decode_e4m3(o.encode_e4m3_rne(np.clip(rn / scale, -448, 448))) * scale
    differ = got != exact
    assert differ.mean() <= 2.0 ** -9                      # (2^-16 of a value is 2^-12 of a step, either side)
    assert np.allclose(host(out), ro, rtol=HALF[DT[r]] * 1.01, atol=F32 * 64)


def test_fp8_rows_feed_the_product():
    torch.manual_seed(3)
    M, H, N = 70, 528, 96
    y, r, w = torch.randn(M, H, device="cuda", dtype=torch.bfloat16), torch.randn(M, H, device="cuda"), torch.rand(H, device="cuda")
    wide = torch.full((5, 76), 255, dtype=torch.uint8, device="cuda")
    _, q, s, _ = gfg.residual_norm_fp8(y, r, w, scale=wide[:, :M])
    assert bool((wide[:, M:] == 255).all())
    qw, sw = gfg.fp8_quantize_weight_device(torch.randn(N, H, device="cuda"))
    d, e = (torch.empty(M, N, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    gfg.fp8_gemm(q, s, qw, sw, d)
    rows = torch.from_numpy(o.dequantize_act(q.view(torch.uint8).cpu().numpy(), s.cpu().numpy())).float().cuda()
    gfg.fp8_linear(rows, qw, sw, e)                        # values that are codes already: the same codes, or finer scales of them
    assert torch.allclose(d.float(), e.float(), rtol=2.0 ** -7, atol=2.0 ** -10 * 528)


def test_parts_may_be_left_out():
    torch.manual_seed(4)
    M, H = 21, 70
    y, r, w = torch.randn(M, H, device="cuda"), torch.randn(M, H, device="cuda"), torch.rand(H, device="cuda") + 0.5
    out, normed, _ = gfg.residual_norm(None, r, w)                          # the first norm of a network
    assert out is None
    want = lo.residual_norm(None, host(r), host(w))
    close(normed, want[1], 2 * np.abs(want[1]), torch.float32, "normed")
    out, normed, _ = gfg.residual_norm(y, r, None, gate=None, alpha=2.0)    # the last sum
    assert normed is None and torch.allclose(out, 2 * r + y, rtol=1e-6, atol=1e-6)
    same = r.clone()
    gfg.residual_norm(y, same, None, out=same)                              # in place
    assert torch.allclose(same, r + y, rtol=1e-6, atol=1e-6)
    # backward of each
    dz, g = torch.randn(M, H, device="cuda"), torch.empty(M, H, device="cuda")
    _, _, stats = gfg.residual_norm(None, r, w, stats=torch.empty(2, M, device="cuda"))
    dw = torch.full((H,), 3.0, device="cuda")
    gfg.residual_norm_backward(None, dz, r, None, stats, w, dresidual=g, dweight=dw, accumulate=True)
    ref = lo.residual_norm_backward(None, host(dz), host(r), None, None, host(stats)[1][:, None], host(w))
    assert np.allclose(host(g), ref[0], rtol=1e-5, atol=1e-5) and np.allclose(host(dw), ref[2] + 3, rtol=1e-5, atol=1e-4)
    dy = torch.empty(M, H, device="cuda")
    gfg.residual_norm_backward(dz, None, None, y, None, None, dy=dy, dresidual=g, alpha=2.0)
    assert torch.equal(dy, dz) and torch.equal(g, 2 * dz)


def test_no_rows():
    z = lambda *s: torch.empty(*s, device="cuda")  # noqa: E731
    gfg.residual_norm(z(0, 32), z(0, 32), z(32))
    grads = dict(dweight=torch.ones(32, device="cuda"), dpost_weight=torch.ones(32, device="cuda"), dgate=torch.ones(32, device="cuda"))
    gfg.residual_norm_backward(z(0, 32), z(0, 32), z(0, 32), z(0, 32), z(2, 0), z(32), post_weight=z(32), gate=z(32), accumulate=True, **grads)
    assert all(bool((g == 1).all()) for g in grads.values())
    gfg.residual_norm_backward(z(0, 32), z(0, 32), z(0, 32), z(0, 32), z(2, 0), z(32), post_weight=z(32), gate=z(32), **grads)
    assert all(not bool(g.any()) for g in grads.values())


def test_zero_rows_and_not_a_number():
    """A row of zeros divides by sqrt(eps); a row with a NaN or an infinity touches no other."""
    H = 528
    y = torch.randn(4, H, device="cuda")
    y[1] = 0
    y[2, 7] = float("nan")
    r = torch.zeros(4, H, device="cuda")
    w = torch.ones(H, device="cuda")
    out, normed, _ = gfg.residual_norm(y, r, w, post_weight=w)
    assert not bool(out[1].any()) and not bool(normed[1].any()) and bool(torch.isnan(normed[2]).all())
    assert bool(torch.isfinite(normed[[0, 3]]).all())
    _, q, s, _ = gfg.residual_norm_fp8(y, r, w, post_weight=w)
    assert bool((s[:, 2] == 255).all()) and bool((q.view(torch.uint8)[2] == 0x7F).all())
    assert bool((s[:, 1] == 127).all()) and not bool(q.view(torch.uint8)[1].any())


def test_gradients_against_differences():
    """Directional differences of the fp32 calls themselves, step 2^-7: their noise is 2^-22 of the outputs' size over
    the step, sqrt(values) of them; the curvature's share is checked to be small by a second step."""
    torch.manual_seed(6)
    M, H = 9, 120
    ins = dict(y=torch.randn(M, H, device="cuda"), residual=torch.randn(M, H, device="cuda"), weight=torch.rand(H, device="cuda") + 0.5,
               post_weight=torch.rand(H, device="cuda") + 0.5, gate=torch.randn(M, 1, device="cuda"))
    dout, dz = torch.randn(M, H, device="cuda"), torch.randn(M, H, device="cuda")

    def loss(v):
        out, z, _ = gfg.residual_norm(**v, alpha=0.75)
        return float((out.double() * dout).sum() + (z.double() * dz).sum())

    stats = torch.empty(2, M, device="cuda")
    out, _, _ = gfg.residual_norm(**ins, alpha=0.75, stats=stats)
    new = {k: torch.empty_like(v) for k, v in ins.items()}
    gfg.residual_norm_backward(dout, dz, out, ins["y"], stats, ins["weight"], post_weight=ins["post_weight"], gate=ins["gate"], alpha=0.75,
                               dresidual=new["residual"], dy=new["y"], dweight=new["weight"], dpost_weight=new["post_weight"], dgate=new["gate"])
    way = {k: torch.randn_like(v) for k, v in ins.items()}
    said = sum(float((new[k].double() * way[k]).sum()) for k in ins)
    at = lambda h: (loss({k: v + h * way[k] for k, v in ins.items()}) - loss({k: v - h * way[k] for k, v in ins.items()})) / (2 * h)  # noqa: E731
    d1, d2 = at(2.0 ** -7), at(2.0 ** -6)
    noise = 2.0 ** -22 * 2.0 ** 7 * 4 * np.sqrt(2 * M * H)
    assert abs(said - d1) <= noise + abs(d2 - d1), (said, d1, d2)


def test_two_calls_give_the_same_bytes():
    torch.manual_seed(7)
    M, H = 700, 528
    y, r = torch.randn(M, H, device="cuda", dtype=torch.bfloat16), torch.randn(M, H, device="cuda", dtype=torch.bfloat16)
    w, st = torch.rand(H, device="cuda"), torch.empty(2, M, device="cuda")
    out, z, _ = gfg.residual_norm(y, r, w, post_weight=w, gate=w, stats=st)
    runs = []
    for _ in range(3):
        g = [torch.empty_like(out), torch.empty_like(y)] + [torch.empty(H, device="cuda") for _ in range(3)]
        gfg.residual_norm_backward(r, z, out, y, st, w, post_weight=w, gate=w, dresidual=g[0], dy=g[1], dweight=g[2], dpost_weight=g[3], dgate=g[4])
        runs.append(g)
    assert all(torch.equal(a, b) for g in runs[1:] for a, b in zip(runs[0], g))
