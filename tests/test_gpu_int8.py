"""GPU parity of the 8-bit integer products and their token quantizer.

The quantizer is compared bit for bit.  The products' integer sums are exact,
so an output differs from the 64-bit value by at most one rounding to the
output type (unit roundoff u: 2^-8 for bf16, 2^-11 for f16, plus half of f16's
subnormal step 2^-24) and four fp32 roundings (sum to float, two scales, the
bias) of the scaled sum and the bias.
"""
import numpy as np
import pytest
import torch

import fp8_block_scaled_amd as gfg
from oracle import serving_oracle as so
from parity_utils import SENTINEL, bits, sentinel_bits, to_dev, torch_dtype

pytestmark = pytest.mark.gpu
U = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11}


def check(got, ref, out, size, what):
    """size: magnitude that the fp32 roundings act on, |scaled sum| + |bias|."""
    got = got.float().cpu().numpy().astype(np.float64)
    tol = U[out] * np.abs(ref) * 1.001 + 4 * 2.0 ** -24 * size * 1.01 + (2.0 ** -25 if out == "f16" else 0.0)
    err = np.abs(got - ref)
    worst = float(np.max(err - tol, initial=-1.0))
    print(f"[int8] {what}: worst error minus bound {worst:.3e}", flush=True)
    assert np.all(np.isfinite(got)) and worst <= 0.0, what


def codes(rng, shape):
    return np.clip(np.rint(rng.standard_normal(shape) * 32), -127, 127).astype(np.int8)


def scales(rng, shape, K):
    return (rng.uniform(0.5, 2.0, shape) / (32 * np.sqrt(K))).astype(np.float32)


# ------------------------------------------------------------------ quantizer
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("M,K", [(1, 16), (3, 128), (5, 2048), (2, 2064), (7, 7168), (4, 16400), (2, 131056), (1000, 272)])
def test_quantizer_bit_exact(M, K, dtype):
    print(f"[int8] quantizer {M} x {K} {dtype}", flush=True)
    rng = np.random.default_rng(M * 131 + K)
    x = rng.standard_normal((M, K)) * 2.0 ** rng.uniform(-8, 8, (M, 1))
    if M > 2:
        x[1] = 0.0                                       # a row of zeros
        x[2, :-1] = 0.0                                  # only the last element
        x[2, -1] = -3.0
    t = torch.from_numpy(x).to(dtype).cuda()
    q, s = gfg.int8_quantize_token_device(t)
    ref_q, ref_s = so.quantize_token(t.float().cpu().numpy())
    assert np.array_equal(s.cpu().numpy().view(np.int32), ref_s.view(np.int32))
    assert np.array_equal(q.cpu().numpy(), ref_q)


@pytest.mark.parametrize("M,K", [(9, 2576), (6, 3056), (5, 3088), (3, 8208), (2, 16384)])
def test_quantizer_of_every_row_split(M, K):
    for dtype in (torch.bfloat16, torch.float32):
        x = torch.randn(M, K, generator=torch.Generator().manual_seed(K)).to(dtype)
        x[0, K - 1] = 9.0                                # the maximum in the row's last chunk
        x[1, K // 2] = float("nan")
        q, s = gfg.int8_quantize_token_device(x.cuda())
        ref_q, ref_s = so.quantize_token(x.float().numpy())
        assert np.array_equal(q.cpu().numpy(), ref_q) and np.array_equal(s.cpu().numpy(), ref_s, equal_nan=True)


def test_quantizer_ties_extremes_and_non_finite_rows():
    K = 64
    x = np.zeros((9, K), np.float32)
    x[0, :4] = [127.0, 0.5, 1.5, -2.5]                   # factor 1: ties to even
    x[1, :] = np.float32(3.4e38)                         # near the largest float
    x[2, :] = np.float32(1e-38)                          # below the floor of amax
    x[3, 0] = np.nan
    x[4, 5] = np.inf
    x[5, 63] = -np.inf
    x[6, :2] = [np.float32(1e-45), -np.float32(1e-45)]   # subnormal
    x[7, :] = -1.0
    t = torch.from_numpy(x).cuda()
    q = torch.full((9, K), 7, dtype=torch.int8, device="cuda")
    s = torch.zeros(9, device="cuda")
    gfg.int8_quantize_token_device(t, q, s)
    ref_q, ref_s = so.quantize_token(x)
    assert np.array_equal(q.cpu().numpy(), ref_q)
    got = s.cpu().numpy()
    assert np.array_equal(np.isnan(got), np.isnan(ref_s)) and np.isnan(got[3:6]).all()
    assert np.array_equal(got[~np.isnan(got)], ref_s[~np.isnan(ref_s)])
    assert q.cpu().numpy()[0, :4].tolist() == [127, 0, 2, -2]


# ------------------------------------------------------------------ dense product
@pytest.fixture(params=[gfg.TILE_AUTO, gfg.TILE_128x256, gfg.TILE_256x256], ids=["auto", "small", "large"])
def tile(request):
    """Every product runs on the automatic choice and on each tile shape, forced."""
    gfg.set_tile_shape(request.param)
    yield request.param
    gfg.set_tile_shape(gfg.TILE_AUTO)


@pytest.mark.parametrize("M,N,K,out,bias", [
    (1, 1, 16, "bf16", False), (1, 128, 128, "f16", True), (1, 7168, 2304, "bf16", False), (2, 515, 1040, "bf16", True),
    (15, 33, 48, "f16", False), (16, 256, 256, "bf16", False), (17, 100, 112, "f16", True), (33, 1000, 7168, "bf16", False),
    (64, 384, 512, "bf16", True), (65, 129, 144, "f16", False), (77, 1003, 1072, "f16", True), (128, 128, 256, "bf16", False),
    (129, 130, 272, "bf16", True), (300, 770, 384, "f16", False), (513, 1024, 2048, "bf16", False),
    (1000, 517, 656, "f16", True), (2100, 2050, 400, "bf16", False), (700, 1501, 528, "bf16", True), (20, 90, 2000, "f16", True),
])
def test_dense(M, N, K, out, bias, tile):
    what = f"dense M={M} N={N} K={K} {out} bias={bias}"
    print(f"[int8] {what}", flush=True)
    rng = np.random.default_rng(M * 7 + N * 3 + K)
    a, b, sa, sb = codes(rng, (M, K)), codes(rng, (N, K)), scales(rng, M, 1), scales(rng, N, K)
    bi = rng.standard_normal(N).astype(np.float32) if bias else None
    # the output sits inside a larger buffer whose ends must stay untouched
    flat = torch.full((M * N + 128,), SENTINEL, dtype=torch_dtype(out), device="cuda")
    d = flat[64:64 + M * N].view(M, N)
    gfg.int8_gemm(to_dev(a), to_dev(sa), to_dev(b), to_dev(sb), d, bias=None if bi is None else to_dev(bi))
    prod = so.int8_product(a, sa, b, sb)
    ref = so.int8_product(a, sa, b, sb, bi)
    check(d, ref, out, np.abs(prod) + (0 if bi is None else np.abs(bi)), what)
    ends = bits(torch.cat([flat[:64], flat[-64:]]))
    assert np.all(ends == sentinel_bits(out)), f"{what}: written outside the output"
    again = torch.empty_like(d)
    gfg.int8_gemm(to_dev(a), to_dev(sa), to_dev(b), to_dev(sb), again, bias=None if bi is None else to_dev(bi))
    assert torch.equal(d, again)


@pytest.mark.parametrize("M", [2, 70, 300])
def test_dense_extreme_sums_are_exact(M, tile):
    """All products 127 * 127 or -128 * -128 at the largest K: sums near 2^31, and integer outputs."""
    K, N = 131056, 5
    a = np.full((M, K), -128, np.int8)
    b = np.full((N, K), -128, np.int8)
    b[1:3] = 127
    b[3, ::2] = 127
    one = np.ones(max(M, N), np.float32)
    d = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
    gfg.int8_gemm(to_dev(a), to_dev(one[:M]), to_dev(b), to_dev(one[:N]), d)
    ref = so.int8_product(a, one[:M], b, one[:N])
    check(d, ref, "bf16", np.abs(ref), f"extreme sums M={M}")


def test_dense_small_integers_bit_exact():
    rng = np.random.default_rng(3)
    a, b = rng.integers(-2, 3, (70, 48)).astype(np.int8), rng.integers(-2, 3, (50, 48)).astype(np.int8)
    d = torch.empty(70, 50, dtype=torch.float16, device="cuda")
    one = torch.ones(70, device="cuda")
    gfg.int8_gemm(to_dev(a), one, to_dev(b), one[:50].contiguous(), d)
    assert np.array_equal(d.float().cpu().numpy(), a.astype(np.float32) @ b.astype(np.float32).T)


@pytest.mark.parametrize("M", [1, 2, 3, 4, 5, 9, 40, 200])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
def test_linear_equals_quantizer_and_product(M, dtype):
    """int8_linear is the two calls, bit for bit, with a workspace of exactly the size it names."""
    N, K = (333, 2320) if M != 2 else (70, 16400)        # 2 x 16400: the longest rows quantized on the way
    rng = np.random.default_rng(M)
    x = torch.from_numpy(rng.standard_normal((M, K))).to(dtype).cuda()
    x[M // 2] = 0
    if M > 2:
        x[2, 7] = float("nan")
    b, sb = to_dev(codes(rng, (N, K))), to_dev(scales(rng, N, K))
    bias = torch.randn(N, device="cuda")
    q, s = gfg.int8_quantize_token_device(x)
    want = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
    gfg.int8_gemm(q, s, b, sb, want, bias=bias)
    need = gfg.int8_linear_workspace_bytes(M, K)
    flat = torch.full((need + 256,), 0x5A, dtype=torch.uint8, device="cuda")
    got = torch.empty_like(want)
    gfg.int8_linear(x, b, sb, got, bias=bias, workspace=flat[128:128 + need])
    assert np.array_equal(bits(got), bits(want))
    assert bool((flat[:128] == 0x5A).all()) and bool((flat[128 + need:] == 0x5A).all())
    if M > 2:
        assert bool(torch.isnan(got[2]).all()) and not bool(torch.isnan(got[:2]).any())
    again = torch.empty_like(want)
    gfg.int8_linear(x, b, sb, again, bias=bias)           # a workspace of its own
    assert np.array_equal(bits(again), bits(want))


def test_linear_without_rows_and_stream():
    d = torch.empty(0, 8, dtype=torch.bfloat16, device="cuda")
    b, sb = torch.ones(8, 16, dtype=torch.int8, device="cuda"), torch.ones(8, device="cuda")
    assert gfg.int8_linear(torch.empty(0, 16, device="cuda"), b, sb, d).shape == (0, 8)
    x = torch.ones(3, 16, device="cuda")
    d = torch.zeros(3, 8, dtype=torch.bfloat16, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    gfg.int8_linear(x, b, sb, d, workspace=torch.empty(1024, dtype=torch.uint8, device="cuda"), stream=s)
    s.synchronize()
    # codes 127 and scale 1/127: 16 * 127 * (1/127), one rounding short of 16 at most
    assert torch.equal(d, torch.full_like(d, 16.0))


# ------------------------------------------------------------------ grouped layouts
@pytest.mark.parametrize("m_per_group,N,K,out", [
    ([100, 1, 128, 129, 300], 256, 256, "bf16"), ([5, 250], 130, 400, "f16"), ([0, 128, 77], 384, 128, "bf16"),
    ([1000, 30], 641, 656, "bf16"), ([700, 0, 513, 256], 512, 1024, "f16"), ([1], 7, 16, "bf16"),
    ([1000, 900, 700], 700, 272, "bf16"), ([3000, 2000], 701, 144, "f16"),
])
def test_contiguous(m_per_group, N, K, out, tile):
    from fp8_block_scaled_amd import workloads as wl
    what = f"contiguous {m_per_group} N={N} K={K} {out}"
    print(f"[int8] {what}", flush=True)
    rng = np.random.default_rng(sum(m_per_group) + N + K)
    layout = wl.contiguous_layout(m_per_group)
    G, M = len(m_per_group), layout.size
    if len(m_per_group) > 3:
        layout[50] = -1                                   # a hole, and ids that name no expert or another one
        layout[51], layout[52] = G, -7
        layout[53] = 2
    a, b, sa, sb = codes(rng, (M, K)), codes(rng, (G, N, K)), scales(rng, M, 1), scales(rng, (G, N), K)
    d = torch.full((M, N), SENTINEL, dtype=torch_dtype(out), device="cuda")
    gfg.grouped_int8_gemm_contiguous(to_dev(a), to_dev(sa), to_dev(b), to_dev(sb), to_dev(layout), d)
    tile = layout[::128].repeat(128)
    live = (layout >= 0) & (layout < G) & (layout == tile)
    assert np.all(bits(d)[~live] == sentinel_bits(out)), f"{what}: rows of no expert were written"
    for g in range(G):
        rows = live & (layout == g)
        if rows.any():
            ref = so.int8_product(a[rows], sa[rows], b[g], sb[g])
            check(d[torch.from_numpy(rows).cuda()], ref, out, np.abs(ref), f"{what} expert {g}")


def test_contiguous_all_padding(tile):
    d = torch.full((256, 24), SENTINEL, dtype=torch.bfloat16, device="cuda")
    z = torch.zeros
    gfg.grouped_int8_gemm_contiguous(z(256, 64, dtype=torch.int8, device="cuda"), z(256, device="cuda"),
                                     z(2, 24, 64, dtype=torch.int8, device="cuda"), z(2, 24, device="cuda"),
                                     torch.full((256,), -1, dtype=torch.int32, device="cuda"), d)
    assert np.all(bits(d) == sentinel_bits("bf16"))


@pytest.mark.parametrize("masked_m,Mmax,N,K,out", [
    ([0, 64, 200], 256, 256, 384, "bf16"), ([512, 3, 129, 0], 512, 133, 272, "f16"), ([-5, 900, 37], 300, 512, 512, "bf16"),
    ([1], 1, 16, 16, "bf16"), ([600, 1024, 0, 257], 1024, 520, 1024, "bf16"),
    ([1000, 100, 300, 1024], 1024, 803, 144, "f16"), ([3, 0, 9, 16], 16, 200, 656, "bf16"), ([30, 17, 0], 32, 136, 528, "f16"),
])
def test_masked(masked_m, Mmax, N, K, out, tile):
    what = f"masked {masked_m} M_max={Mmax} N={N} K={K} {out}"
    print(f"[int8] {what}", flush=True)
    rng = np.random.default_rng(Mmax + N + K)
    G = len(masked_m)
    a, b = codes(rng, (G, Mmax, K)), codes(rng, (G, N, K))
    sa, sb = scales(rng, (G, Mmax), 1), scales(rng, (G, N), K)
    d = torch.full((G, Mmax, N), SENTINEL, dtype=torch_dtype(out), device="cuda")
    gfg.grouped_int8_gemm_masked(to_dev(a), to_dev(sa), to_dev(b), to_dev(sb), to_dev(np.asarray(masked_m, np.int32)), d)
    for g, mm in enumerate(masked_m):
        mm = min(max(mm, 0), Mmax)
        assert np.all(bits(d)[g, mm:] == sentinel_bits(out)), f"{what}: rows past the count were written"
        if mm:
            ref = so.int8_product(a[g, :mm], sa[g, :mm], b[g], sb[g])
            check(d[g, :mm], ref, out, np.abs(ref), f"{what} group {g}")


def test_large_product_on_both_tiles():
    """Several tiles for every workgroup of the 256 x 256 kernel, and both tiles bit for bit: the sums are exact."""
    rng = np.random.default_rng(21)
    M, N, K = 5000, 5128, 400
    a, b, sa, sb = codes(rng, (M, K)), codes(rng, (N, K)), scales(rng, M, 1), scales(rng, N, K)
    bias = to_dev(rng.standard_normal(N).astype(np.float32))
    ops = to_dev(a), to_dev(sa), to_dev(b), to_dev(sb)
    got = []
    try:
        for shape in (gfg.TILE_AUTO, gfg.TILE_128x256, gfg.TILE_256x256):
            gfg.set_tile_shape(shape)
            got.append(gfg.int8_gemm(*ops, torch.empty(M, N, dtype=torch.bfloat16, device="cuda"), bias=bias))
    finally:
        gfg.set_tile_shape(gfg.TILE_AUTO)
    assert torch.equal(got[0], got[1]) and torch.equal(got[1], got[2])
    rows = rng.permutation(M)[:64]
    prod = so.int8_product(a[rows], sa[rows], b, sb)
    bi = bias.cpu().numpy()
    check(got[0][torch.from_numpy(rows).cuda()], prod + bi, "bf16", np.abs(prod) + np.abs(bi), "large product")


def test_graph_replays_match_eager():
    rng = np.random.default_rng(11)
    M, N, K = 150, 260, 528
    x = torch.randn(M, K, device="cuda", dtype=torch.bfloat16)
    b, sb = to_dev(codes(rng, (N, K))), to_dev(scales(rng, N, K))
    d = torch.zeros(M, N, dtype=torch.bfloat16, device="cuda")
    one = torch.zeros(1, N, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(gfg.int8_linear_workspace_bytes(M, K), dtype=torch.uint8, device="cuda")
    ws1 = torch.empty(gfg.int8_linear_workspace_bytes(1, K), dtype=torch.uint8, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())

    def launches():
        gfg.int8_linear(x, b, sb, d, workspace=ws, stream=s)
        gfg.int8_linear(x[:1], b, sb, one, workspace=ws1, stream=s)

    with torch.cuda.stream(s):
        launches()
    torch.cuda.synchronize()
    want = d.clone(), one.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        launches()
    for r in range(4):
        d.fill_(3.0)
        one.fill_(3.0)
        ws.fill_(r)
        torch.cuda.synchronize()
        with torch.cuda.stream(s):
            g.replay()
        torch.cuda.synchronize()
        assert torch.equal(d, want[0]) and torch.equal(one, want[1]), f"replay {r}"


# ------------------------------------------------------------------ rows of the large tile
@pytest.fixture
def eight_workgroups():
    """Eight workgroups on the large tile: a few tiles are several rounds, which decide the tile's rows."""
    gfg.set_tile_shape(gfg.TILE_256x256)
    gfg.set_grid_limit(8)
    yield
    gfg.set_grid_limit(0)
    gfg.set_tile_shape(gfg.TILE_AUTO)


# 8 tiles of 256 rows are one round where 16 of 192 are two; 8 of 192 (rows up to 192) are as good as 8 of 256
@pytest.mark.parametrize("M,N,K", [(256, 2048, 272), (255, 2047, 272), (193, 2042, 400), (192, 2048, 400), (160, 1999, 144),
                                   (97, 1030, 2064), (700, 1500, 656), (510, 1028, 144), (576, 769, 1296)])
def test_dense_rows_of_the_large_tile(M, N, K, eight_workgroups):
    rng = np.random.default_rng(M + N + K)
    a, b, sa, sb = codes(rng, (M, K)), codes(rng, (N, K)), scales(rng, M, 1), scales(rng, N, K)
    bias = rng.standard_normal(N).astype(np.float32)
    flat = torch.full((M * N + 128,), SENTINEL, dtype=torch.float16, device="cuda")
    d = flat[64:64 + M * N].view(M, N)
    gfg.int8_gemm(to_dev(a), to_dev(sa), to_dev(b), to_dev(sb), d, bias=to_dev(bias))
    prod = so.int8_product(a, sa, b, sb)
    check(d, prod + bias, "f16", np.abs(prod) + np.abs(bias), f"rows of the large tile {M} {N} {K}")
    assert np.all(bits(torch.cat([flat[:64], flat[-64:]])) == sentinel_bits("f16"))


@pytest.mark.parametrize("masked_m,Mmax,N,K", [([256, 0, 256], 256, 1024, 272), ([192, 10, 0, 150], 400, 517, 400), ([600, 1, 193], 600, 770, 144),
                                               ([0, 0], 300, 256, 128), ([256] * 5, 256, 1000, 528), ([383, 385, 384], 385, 511, 272)])
def test_masked_rows_of_the_large_tile(masked_m, Mmax, N, K, eight_workgroups):
    rng = np.random.default_rng(sum(masked_m) + N + K)
    G = len(masked_m)
    a, b, sa, sb = codes(rng, (G, Mmax, K)), codes(rng, (G, N, K)), scales(rng, (G, Mmax), 1), scales(rng, (G, N), K)
    d = torch.full((G, Mmax, N), SENTINEL, dtype=torch.bfloat16, device="cuda")
    gfg.grouped_int8_gemm_masked(to_dev(a), to_dev(sa), to_dev(b), to_dev(sb), torch.tensor(masked_m, dtype=torch.int32, device="cuda"), d)
    for g, m in enumerate(masked_m):
        ref = so.int8_product(a[g, :m], sa[g, :m], b[g], sb[g])
        check(d[g, :m], ref, "bf16", np.abs(ref), f"masked rows of the large tile {g} {m}")
        assert np.all(bits(d[g, m:]) == sentinel_bits("bf16"))


# ------------------------------------------------------------------ offsets past 32 bits
def some_codes(seed, *shape):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    return torch.randint(-127, 128, shape, dtype=torch.int8, device="cuda", generator=gen)


def check_rows(d, a, sa, b, sb, rows, out, what):
    rows = torch.tensor(rows, device="cuda")
    got, pa, ps = d[rows], a[rows].cpu().numpy(), sa[rows].cpu().numpy()
    ref = so.int8_product(pa, ps, b.cpu().numpy(), sb.cpu().numpy())
    check(got, ref, out, np.abs(ref), what)


def test_dense_operands_past_4_gib(tile):
    M, N, K = 530_001, 72, 8208                           # A has 4.35e9 bytes
    a, b = some_codes(1, M, K), some_codes(2, N, K)
    sa, sb = torch.rand(M, device="cuda") + 0.5, (torch.rand(N, device="cuda") + 0.5) / 4096
    d = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
    print(f"[int8] A past 4 GiB, tile {tile}", flush=True)
    gfg.int8_gemm(a, sa, b, sb, d)
    check_rows(d, a, sa, b, sb, [0, 1, 261_632, 523_263, 523_264, 523_500, M - 1], "bf16", "A past 4 GiB")


def test_outputs_past_4_gib(tile):
    M, N, K = 33_000, 70_000, 32                          # D has 4.6e9 bytes
    a, b = some_codes(3, M, K), some_codes(4, N, K)
    sa, sb = torch.rand(M, device="cuda") + 0.5, (torch.rand(N, device="cuda") + 0.5) / 256
    d = torch.empty(M, N, dtype=torch.float16, device="cuda")
    print(f"[int8] D past 4 GiB, tile {tile}", flush=True)
    gfg.int8_gemm(a, sa, b, sb, d)
    check_rows(d, a, sa, b, sb, [0, 15_339, 15_340, 30_678, 30_679, M - 1], "f16", "D past 4 GiB")


@pytest.mark.parametrize("rows", [3, 300])
def test_grouped_weights_past_4_gib(rows, tile):
    G, N, K = 36, 8192, 16384                             # 134 MB an expert, 4.8e9 bytes
    b = some_codes(5, G, N, K)
    sb = (torch.rand(G, N, device="cuda") + 0.5) / 8192
    a, sa = some_codes(6, rows, K), torch.rand(rows, device="cuda") + 0.5
    print(f"[int8] B past 4 GiB, {rows} rows, tile {tile}", flush=True)
    for g in (0, 17, G - 1):
        d = torch.empty(rows, N, dtype=torch.bfloat16, device="cuda")
        gfg.grouped_int8_gemm_contiguous(a, sa, b, sb, torch.full((rows,), g, dtype=torch.int32, device="cuda"), d)
        ref = so.int8_product(a[:8].cpu().numpy(), sa[:8].cpu().numpy(), b[g].cpu().numpy(), sb[g].cpu().numpy())
        check(d[:8], ref, "bf16", np.abs(ref), f"expert {g}")
        assert torch.equal(d, gfg.int8_gemm(a, sa, b[g], sb[g], torch.empty_like(d)))


def test_quantizer_past_4_gib():
    M, K = 280_001, 8208                                  # x has 4.6e9 bytes
    x = (some_codes(7, M, K).to(torch.bfloat16) * 0.125)
    q, s = gfg.int8_quantize_token_device(x)
    rows = torch.tensor([0, 130_800, 261_632, 261_700, M - 1], device="cuda")
    ref_q, ref_s = so.quantize_token(x[rows].float().cpu().numpy())
    assert np.array_equal(q[rows].cpu().numpy(), ref_q) and np.array_equal(s[rows].cpu().numpy(), ref_s)


def test_quantizer_many_rows():
    """More rows than one launch has workgroups for, in both of the quantizer's forms."""
    for M, K in ((1 << 24) + 9, 16), ((1 << 22) + 3, 2064):
        x = some_codes(M, M, K).to(torch.float16)
        q, s = gfg.int8_quantize_token_device(x)
        rows = torch.tensor([0, 1 << 20, (1 << 22) - 1, 1 << 22, M - 1], device="cuda")
        ref_q, ref_s = so.quantize_token(x[rows].float().cpu().numpy())
        assert np.array_equal(q[rows].cpu().numpy(), ref_q) and np.array_equal(s[rows].cpu().numpy(), ref_s)
        del x, q, s
        torch.cuda.empty_cache()
