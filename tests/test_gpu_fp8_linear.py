"""The FP8 linear layer, its gradients and the weight quantizer against 64-bit definitions.

Tolerance of a product: one rounding to the output type, at most eps / 2 of the value; and the matrix instruction's own
sums, inside which a product 2^-14 or more below the largest of its group of 16 may be dropped: at most 15 * 2^-14 of
that largest one, below 2^-10 of the group's sum of |products| (the fp32 additions of up to 2^7 blocks add 2^-17 of it
at most).  Operands of small whole numbers have no such products (ratios below 2^14, sums below 2^24), so those results
are exact up to the one rounding.  Below 2^-14 float16's step is 2^-24 whatever the value, so its rounding is 2^-25 there.
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
DROPPED = 2.0 ** -10
LEAST = {torch.float16: 2.0 ** -25}


@pytest.fixture(autouse=True)
def _restore_settings():
    yield
    gfg.set_tile_shape(gfg.TILE_AUTO)
    gfg.set_grid_limit(0)


def dev(x, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(x)).cuda()
    return t if dtype is None else t.to(dtype)


def host(t):
    return t.double().cpu().numpy()


def close(got, ref, size, dtype):
    """got within one rounding of ref and the dropped products of size = sum of |products|."""
    g = host(got)
    assert np.isfinite(g).all()
    off = np.abs(g - ref) - (HALF[dtype] * np.abs(ref) + DROPPED * size + LEAST.get(dtype, 0.0)) * (1 + 2.0 ** -10)
    assert off.max() <= 0, (off.max(), np.unravel_index(off.argmax(), off.shape))


def weight(rng, N, K):
    w = rng.standard_normal((N, K)).astype(np.float32) / np.float32(np.sqrt(K))
    q, s = o.quantize_weight_128x128(w[None])
    return q[0], s[0], o.dequantize_weight(q, s)[0]


def whole(rng, *shape):
    """Whole numbers up to 8: exact in E4M3 at any power-of-two scale that reaches 448."""
    return rng.integers(-8, 9, shape).astype(np.float32)


# rows from one on, odd and ragged in every direction; each kernel's tile and its edges
SHAPES = [(1, 1, 16), (1, 7168, 2304), (2, 33, 144), (3, 257, 1040), (5, 1003, 1072), (16, 130, 128), (17, 64, 272), (31, 500, 4096), (33, 129, 112),
          (77, 1003, 1072), (128, 128, 128), (129, 300, 528), (300, 2049, 640), (520, 4100, 400), (1500, 1999, 272), (2500, 2600, 144), (4200, 2200, 144)]


@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
def test_linear(M, N, K, dt):
    rng = np.random.default_rng(M + N + K)
    x = rng.standard_normal((M, K)).astype(np.float32) * np.exp2(rng.integers(-6, 7, (M, 1))).astype(np.float32)
    x = host(dev(x, DT[dt])).astype(np.float32)            # as the type holds it
    q, s, w = weight(rng, N, K)
    bias = rng.standard_normal(N).astype(np.float32) if N % 2 else None
    out = torch.float16 if dt == "f16" else torch.bfloat16
    d = torch.full((M, N), 99.0, dtype=out, device="cuda")
    got = gfg.fp8_linear(dev(x, DT[dt]), dev(q), dev(s), d, bias=None if bias is None else dev(bias))
    assert got is d
    close(d, lo.linear(x, w, bias), np.abs(lo.through_fp8(x)) @ np.abs(w).T, out)


@pytest.mark.parametrize("M,N,K", SHAPES)
def test_product_of_whole_numbers_is_exact(M, N, K):
    """The same sums in every tile, to the last bit; rows of scales at any distance and any alignment."""
    rng = np.random.default_rng(M * 3 + N)
    a, b = whole(rng, M, K), whole(rng, N, K)
    qa, sa = o.quantize_act_1x128(a)
    qb, sb = o.quantize_weight_128x128(b[None])
    ref = torch.from_numpy(a.astype(np.float64) @ b.astype(np.float64).T)
    for ld, first in ((M, 0), (M + 3, 1), ((M + 3) // 4 * 4 + 4, 0)):
        store = torch.full((sa.shape[0] * ld + 8,), 255, dtype=torch.uint8, device="cuda")
        view = store[first:first + sa.shape[0] * ld].view(sa.shape[0], ld)[:, :M]
        view.copy_(dev(sa))
        for shape in (gfg.TILE_AUTO, gfg.TILE_128x256, gfg.TILE_256x256):
            gfg.set_tile_shape(shape)
            d = torch.full((M + 1, N), 99.0, dtype=torch.bfloat16, device="cuda")
            gfg.fp8_gemm(dev(qa), view, dev(qb[0]), dev(sb[0]), d[:M])
            assert torch.equal(d[:M].cpu(), ref.to(torch.bfloat16)), (ld, first, shape)
            assert bool((d[M] == 99.0).all())              # the row behind the last is left alone


@pytest.mark.parametrize("M,N,K", [(5, 130, 272), (40, 96, 128), (300, 520, 400), (700, 1304, 528), (700, 1301, 272)])
@pytest.mark.parametrize("dt", ["bf16", "f16"])
def test_bias_in_every_tile(M, N, K, dt):
    """Also over several tiles a workgroup (the bias of the next one is loaded while one is stored)."""
    rng = np.random.default_rng(M + N)
    a, b, bias = whole(rng, M, K), whole(rng, N, K), whole(rng, N) * 16
    qa, sa = o.quantize_act_1x128(a)
    qb, sb = o.quantize_weight_128x128(b[None])
    ref = torch.from_numpy(a.astype(np.float64) @ b.astype(np.float64).T + bias).to(DT[dt])
    for shape in (gfg.TILE_AUTO, gfg.TILE_128x256, gfg.TILE_256x256):
        for limit in (0, 8):
            gfg.set_tile_shape(shape)
            gfg.set_grid_limit(limit)
            d = torch.full((M + 1, N), 99.0, dtype=DT[dt], device="cuda")
            gfg.fp8_gemm(dev(qa), dev(sa), dev(qb[0]), dev(sb[0]), d[:M], bias=dev(bias))
            assert torch.equal(d[:M].cpu(), ref) and bool((d[M] == 99.0).all()), (shape, limit)


@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("dwt", ["f32", "bf16"])
def test_weight_gradient_over_several_tiles(accumulate, dwt):
    if accumulate and dwt != "f32":
        pytest.skip("refused")
    rng = np.random.default_rng(8)
    M, N, K = 260, 1040, 784
    dy, x = whole(rng, M, N), whole(rng, M, K)
    ref = torch.from_numpy(dy.T.astype(np.float64) @ x + (3.0 if accumulate else 0.0)).to(DT[dwt])
    for shape in (gfg.TILE_AUTO, gfg.TILE_128x256, gfg.TILE_256x256):
        for limit in (0, 8):
            gfg.set_tile_shape(shape)
            gfg.set_grid_limit(limit)
            dw = torch.full((N, K), 3.0, dtype=DT[dwt], device="cuda")
            gfg.fp8_linear_backward(dev(dy), dev(x), None, None, dw=dw, accumulate=accumulate)
            assert torch.equal(dw.cpu(), ref), (shape, limit)


def test_scales_differ_by_block():
    """A scale of its own for every row and block of A and every block of B, the whole range that sums can take."""
    rng = np.random.default_rng(9)
    M, N, K = 70, 400, 656
    a, b = whole(rng, M, K), whole(rng, N, K)
    qa, qb = o.encode_e4m3_rne(a.astype(np.float64)), o.encode_e4m3_rne(b.astype(np.float64))
    sa = rng.integers(100, 140, (6, M)).astype(np.uint8)
    sb = rng.integers(120, 135, (4, 6)).astype(np.uint8)
    A, B = o.dequantize_act(qa, sa), o.dequantize_weight(qb[None], sb[None])[0]
    for rows in (M, 16, 3):
        d = torch.empty(rows, N, dtype=torch.bfloat16, device="cuda")
        gfg.fp8_gemm(dev(qa[:rows]), dev(sa[:, :rows]), dev(qb), dev(sb), d)
        close(d, A[:rows] @ B.T, np.abs(A[:rows]) @ np.abs(B).T, torch.bfloat16)


def test_linear_takes_the_quantizers_codes():
    """A layer from tokens is the product from the quantizer's codes: the same definition of a block's scale, zero
    blocks, subnormal values and the border of the ceil among them."""
    rng = np.random.default_rng(12)
    M, N, K = 40, 96, 512
    x = rng.standard_normal((M, K)).astype(np.float32)
    x[1, :128] = 0
    x[2] *= np.float32(1e-39)
    x[3] *= np.float32(2.0 ** 100)
    x[4, :128] = 0
    x[4, 5] = 448 * 2.0 ** 3                               # t = 3 exactly
    x[5, :128] = 0
    x[5, 6] = np.nextafter(np.float32(448 * 2.0 ** 3), np.float32(1e9))      # just past it: t = 4
    q, s, w = weight(rng, N, K)
    qa, sa = gfg.fp8_quantize_act_1x128(np.where(np.abs(x) < 1e-30, 0, x).astype(np.float32))
    for rows in (M, 6):
        d, e = torch.empty(rows, N, dtype=torch.bfloat16, device="cuda"), torch.empty(rows, N, dtype=torch.bfloat16, device="cuda")
        gfg.fp8_linear(dev(x[:rows]), dev(q), dev(s), d)
        gfg.fp8_gemm(dev(qa[:rows]), dev(sa[:, :rows]), dev(q), dev(s), e)
        keep = [i for i in range(rows) if i != 2]
        A = o.dequantize_act(qa, sa)[:rows]
        size = np.abs(A) @ np.abs(w).T
        a, b = host(d), host(e)
        assert (np.abs(a - b)[keep] <= (2 * HALF[torch.bfloat16] * np.abs(b) + 2 * DROPPED * size)[keep]).all()
        assert np.abs(a[2]).max() < 1e-36


def test_not_a_number_stays_in_its_row():
    rng = np.random.default_rng(13)
    for M in (3, 16, 40):
        x = rng.standard_normal((M, 272)).astype(np.float32)
        x[1, 260], x[2, 3] = np.nan, np.inf
        q, s, w = weight(rng, 64, 272)
        d = torch.empty(M, 64, dtype=torch.bfloat16, device="cuda")
        gfg.fp8_linear(dev(x), dev(q), dev(s), d)
        bad = torch.isnan(d).cpu()
        assert bool(bad[1:3].all()) and not bool(bad[0].any()) and not bool(bad[3:].any())


# ------------------------------------------------------------------ the weight quantizer
@pytest.mark.parametrize("dt", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("G,N,K", [(1, 16, 16), (1, 128, 128), (2, 272, 400), (3, 1003, 1072), (1, 2304, 1040)])
def test_weight_quantizer_is_the_host_quantizer(dt, G, N, K):
    rng = np.random.default_rng(N + K)
    w = rng.standard_normal((G, N, K)).astype(np.float32)
    w[0, :, :16] = 0
    w = host(dev(w, DT[dt])).astype(np.float32)
    q, s = gfg.fp8_quantize_weight_128x128(w)
    t = dev(w, DT[dt])
    both = N % 16 == 0
    got = gfg.fp8_quantize_weight_device(t if G > 1 else t[0], transposed=both)
    bytes_of = lambda v: v.view(torch.uint8).cpu().numpy().reshape((G,) + tuple(v.shape[-2:]))  # noqa: E731
    assert np.array_equal(bytes_of(got[0]), q) and np.array_equal(bytes_of(got[1]), s)
    if both:
        assert np.array_equal(bytes_of(got[2]), q.transpose(0, 2, 1)) and np.array_equal(bytes_of(got[3]), s.transpose(0, 2, 1))


def test_weight_quantizer_marks_blocks_without_a_scale():
    w = torch.randn(256, 256, device="cuda")
    w[130, 7] = float("nan")
    q, s, qt, st = gfg.fp8_quantize_weight_device(w, transposed=True)
    assert s.tolist()[1][0] == 255 and st.tolist()[0][1] == 255 and (s != 255).sum() == 3
    assert bool((q.view(torch.uint8)[128:, :128] == 0x7F).all()) and bool((qt.view(torch.uint8)[:128, 128:] == 0x7F).all())
    assert not bool(torch.isnan(q[:128].float()).any())


# ------------------------------------------------------------------ gradients
BACK = [(1, 16, 16), (2, 144, 48), (100, 16, 272), (127, 272, 128), (128, 128, 128), (129, 528, 1040), (300, 528, 1040), (257, 2048, 2112), (1000, 128, 384), (16, 4208, 2208), (2100, 48, 2112)]


def operands(rng, M, N, K, dtype, values=None):
    make = values or (lambda *shape: rng.standard_normal(shape).astype(np.float32) * np.exp2(rng.integers(-3, 4, (shape[0], 1))).astype(np.float32))
    dy, x = (host(dev(make(M, n), dtype)).astype(np.float32) for n in (N, K))
    w = whole(rng, N, K) if values else rng.standard_normal((N, K)).astype(np.float32)
    return dy, x, w


@pytest.mark.parametrize("M,N,K", BACK)
@pytest.mark.parametrize("dt,dwt", [("bf16", "bf16"), ("f16", "f32"), ("f32", "f16")])
def test_backward(M, N, K, dt, dwt):
    rng = np.random.default_rng(M + N + K)
    dy, x, w = operands(rng, M, N, K, DT[dt])
    q, s, qt, st = gfg.fp8_quantize_weight_device(dev(w), transposed=True)
    wd = o.dequantize_weight(q.view(torch.uint8).cpu().numpy()[None], s.cpu().numpy()[None])[0]
    out = torch.float16 if dt == "f16" else torch.bfloat16
    dx, dw, db = torch.empty(M, K, dtype=out, device="cuda"), torch.empty(N, K, dtype=DT[dwt], device="cuda"), torch.empty(N, device="cuda")
    gfg.fp8_linear_backward(dev(dy, DT[dt]), dev(x, DT[dt]), qt, st, dx=dx, dw=dw, dbias=db)
    rx, rw, rb = lo.linear_backward(dy, x, wd)
    close(dx, rx, np.abs(lo.through_fp8(dy)) @ np.abs(wd), out)
    close(dw, rw, np.abs(lo.through_fp8(dy.T)) @ np.abs(lo.through_fp8(x.T)).T, DT[dwt])
    # fp32 sums of M values: below 2^4 additions in a row each way
    assert (np.abs(host(db) - rb) <= 2.0 ** -24 * 64 * np.abs(dy).sum(0)).all()


@pytest.mark.parametrize("M,N,K", BACK)
@pytest.mark.parametrize("accumulate", [False, True])
def test_backward_of_whole_numbers_is_exact(M, N, K, accumulate):
    rng = np.random.default_rng(M * 5 + N)
    dy, x, w = operands(rng, M, N, K, torch.bfloat16, lambda *shape: whole(rng, *shape))
    _, _, qt, st = gfg.fp8_quantize_weight_device(dev(w), transposed=True)
    for shape, limit in ((gfg.TILE_AUTO, 0), (gfg.TILE_AUTO, 1 << 20), (gfg.TILE_AUTO, 5), (gfg.TILE_128x256, 0), (gfg.TILE_256x256, 0)):
        gfg.set_tile_shape(shape)
        gfg.set_grid_limit(limit)
        dx = torch.empty(M, K, dtype=torch.float16, device="cuda")
        dw, db = torch.full((N, K), 5.0, device="cuda"), torch.full((N,), -3.0, device="cuda")
        gfg.fp8_linear_backward(dev(dy, torch.bfloat16), dev(x, torch.bfloat16), qt, st, dx=dx, dw=dw, dbias=db, accumulate=accumulate)
        first = (5.0, -3.0) if accumulate else (0.0, 0.0)
        assert np.array_equal(host(dw), dy.T.astype(np.float64) @ x + first[0])
        assert np.array_equal(host(db), dy.sum(0) + first[1])
        assert torch.equal(dx.cpu(), torch.from_numpy(dy.astype(np.float64) @ w).to(torch.float16))


@pytest.mark.parametrize("want", [("dx",), ("dw",), ("dbias",), ("dx", "dbias"), ("dw", "dbias"), ("dx", "dw")])
def test_backward_computes_what_is_asked_for(want):
    rng = np.random.default_rng(1)
    M, N, K = 200, 144, 272
    dy, x, w = operands(rng, M, N, K, torch.bfloat16, lambda *shape: whole(rng, *shape))
    _, _, qt, st = gfg.fp8_quantize_weight_device(dev(w), transposed=True)
    outs = dict(dx=torch.empty(M, K, dtype=torch.bfloat16, device="cuda"), dw=torch.empty(N, K, device="cuda"), dbias=torch.empty(N, device="cuda"))
    outs = {n: v for n, v in outs.items() if n in want}
    gfg.fp8_linear_backward(dev(dy, torch.bfloat16), dev(x, torch.bfloat16) if "dw" in want else None, qt if "dx" in want else None,
                            st if "dx" in want else None, **outs)
    refs = dict(dx=torch.from_numpy(dy.astype(np.float64) @ w).to(torch.bfloat16).double(), dw=torch.from_numpy(dy.T.astype(np.float64) @ x),
                dbias=torch.from_numpy(dy.sum(0).astype(np.float64)))
    for n, v in outs.items():
        assert torch.equal(v.double().cpu(), refs[n]), n


def test_backward_of_no_tokens():
    dw, db = torch.full((32, 48), 7.0, dtype=torch.bfloat16, device="cuda"), torch.full((32,), 7.0, device="cuda")
    none = torch.empty(0, 32, dtype=torch.bfloat16, device="cuda"), torch.empty(0, 48, dtype=torch.bfloat16, device="cuda")
    gfg.fp8_linear_backward(*none, None, None, dw=dw, dbias=db)
    assert not bool(dw.any()) and not bool(db.any())
    dw = torch.full((32, 48), 7.0, device="cuda")
    gfg.fp8_linear_backward(*none, None, None, dw=dw, accumulate=True)
    assert bool((dw == 7.0).all())


def test_gradients_against_differences():
    """Where quantizing is exact the layer is linear, so a difference of the forward calls is the gradient: whole
    numbers, f16 outputs below 2^11."""
    rng = np.random.default_rng(2)
    M, N, K = 37, 48, 80
    small = lambda *shape: rng.integers(-1, 2, shape).astype(np.float32)  # noqa: E731
    x, w, dy = small(M, K), small(N, K), small(M, N)

    def loss(x, w):
        q, s = gfg.fp8_quantize_weight_device(dev(w))
        y = gfg.fp8_linear(dev(x), q, s, torch.empty(M, N, dtype=torch.float16, device="cuda"))
        return float((host(y) * dy).sum())

    _, _, qt, st = gfg.fp8_quantize_weight_device(dev(w), transposed=True)
    dx, dw = torch.empty(M, K, dtype=torch.float16, device="cuda"), torch.empty(N, K, device="cuda")
    gfg.fp8_linear_backward(dev(dy), dev(x), qt, st, dx=dx, dw=dw)
    for i, j in ((0, 0), (36, 79), (20, 33), (7, 64)):
        e = np.zeros_like(x)
        e[i, j] = 1
        assert (loss(x + e, w) - loss(x - e, w)) / 2 == float(dx[i, j])
        f = np.zeros_like(w)
        f[i, j] = 1
        assert (loss(x, w + f) - loss(x, w - f)) / 2 == float(dw[i, j])


def test_two_calls_give_the_same_bytes():
    torch.manual_seed(0)
    M, N, K = 300, 528, 1040
    x, dy = torch.randn(M, K, device="cuda", dtype=torch.bfloat16), torch.randn(M, N, device="cuda", dtype=torch.bfloat16)
    q, s, qt, st = gfg.fp8_quantize_weight_device(torch.randn(N, K, device="cuda"), transposed=True)
    runs = []
    for _ in range(3):
        y, dx, dw, db = (torch.empty(*n, device="cuda", dtype=t) for n, t in (((M, N), torch.bfloat16), ((M, K), torch.bfloat16), ((N, K), torch.float32), ((N,), torch.float32)))
        gfg.fp8_linear(x, q, s, y)
        gfg.fp8_linear_backward(dy, x, qt, st, dx=dx, dw=dw, dbias=db)
        runs.append((y, dx, dw, db))
    assert all(torch.equal(a, b) for r in runs[1:] for a, b in zip(runs[0], r))


@pytest.mark.parametrize("limit", [8, 24])
@pytest.mark.parametrize("M,N,K", [(16, 2000, 272), (30, 1500, 400), (100, 1999, 272), (600, 1900, 144), (1900, 1500, 272), (2100, 2050, 272)])
def test_grid_limit_changes_nothing(M, N, K, limit):
    rng = np.random.default_rng(M)
    a, b = whole(rng, M, K), whole(rng, N, K)
    qa, sa = o.quantize_act_1x128(a)
    qb, sb = o.quantize_weight_128x128(b[None])
    gfg.set_grid_limit(limit)
    d = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
    gfg.fp8_gemm(dev(qa), dev(sa), dev(qb[0]), dev(sb[0]), d)
    assert torch.equal(d.cpu(), torch.from_numpy(a.astype(np.float64) @ b.astype(np.float64).T).to(torch.bfloat16))
