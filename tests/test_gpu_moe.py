"""GPU parity of the router and of the expert layer for a few tokens.

Router: ids equal the definition's; a weight may differ by the fp32 roundings
of its exponential, sums and quotients: (|l - max| + 24) * 2^-23 relative (the
rounding of l - max acts on the exponent, hence its size in the bound).

Layer: one rounding to the output type (unit roundoff u: 2^-8 bf16, 2^-11
f16), whose relative error is at most u and u / sqrt(3) in the root mean
square; the hidden rows' 16 significant bits and the fp32 sums add below 2^-12
of a row's largest output (2^-17 sqrt-summed over I, and sqrt(H) * 2^-24).
"""
import numpy as np
import pytest
import torch

import fp8_block_scaled_amd as gfg
from oracle import serving_oracle as so
from parity_utils import bits, to_dev, torch_dtype

pytestmark = pytest.mark.gpu
U = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11}


# ------------------------------------------------------------------ router
def run_topk(logits, k, **kw):
    T = logits.shape[0]
    flat_i = torch.full((T * k + 16,), 77, dtype=torch.int32, device="cuda")
    flat_w = torch.full((T * k + 16,), 77.0, device="cuda")
    ids, w = flat_i[8:8 + T * k].view(T, k), flat_w[8:8 + T * k].view(T, k)
    gfg.moe_topk(logits, ids, w, **kw)
    for f in (flat_i, flat_w):
        assert bool((f[:8] == 77).all()) and bool((f[8 + T * k:] == 77).all())
    return ids.cpu().numpy(), w.cpu().numpy().astype(np.float64)


def check_topk(logits, k, **kw):
    ids, w = run_topk(logits, k, **kw)
    l = logits.float().cpu().numpy()
    b = kw.pop("bias", None)
    ref_ids, ref_w = so.topk(l, k, bias=None if b is None else b.cpu().numpy(), **kw)
    assert np.array_equal(ids, ref_ids)
    with np.errstate(invalid="ignore"):
        clean = np.where(np.isnan(l), -np.inf, l)
        gap = np.abs(np.nan_to_num(np.take_along_axis(clean, np.maximum(ids, 0), 1) - clean.max(1, keepdims=True),
                                   nan=0.0, posinf=0.0, neginf=0.0))
    tol = np.abs(ref_w) * (np.maximum(gap, np.abs(np.nan_to_num(np.take_along_axis(clean, np.maximum(ids, 0), 1),
                                                                posinf=0.0, neginf=0.0))) + 24) * 2.0 ** -23 + 1e-37
    assert np.all(np.abs(w - ref_w) <= tol), np.max(np.abs(w - ref_w) / np.maximum(ref_w, 1e-30))
    return ids, w


@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 256, 8), (3, 64, 64), (5, 65, 7), (130, 385, 9), (2, 1024, 64),
                                   (7, 127, 1), (1000, 8, 2), (4, 513, 33)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("score,renormalize", [("softmax", True), ("softmax", False), ("sigmoid", True), ("sigmoid", False)])
def test_topk(T, E, k, dtype, score, renormalize):
    rng = np.random.default_rng(T + E + k)
    logits = torch.from_numpy(rng.standard_normal((T, E)) * 3).to(dtype).cuda()    # 16-bit logits hold many ties
    check_topk(logits, k, score=score, renormalize=renormalize, scale=2.5)


def test_topk_ties_masks_and_non_finite():
    inf, nan = float("inf"), float("nan")
    rows = torch.zeros(8, 200)
    rows[1] = -inf                                        # nothing to choose
    rows[2] = -inf
    rows[2, [190, 3, 64]] = torch.tensor([1.0, 1.0, 2.0])  # fewer than k
    rows[3] = nan
    rows[4, 7] = nan
    rows[4, 150] = 5.0
    rows[5, [10, 100]] = inf
    rows[6] = torch.finfo(torch.float32).min              # the type's lowest value is a number, not a mask
    rows[7] = torch.arange(200.0) * 30                    # all weight on one
    for score in ("softmax", "sigmoid"):
        for renormalize in (True, False):
            ids, w = check_topk(rows.cuda(), 5, score=score, renormalize=renormalize)
    assert ids[0].tolist() == [0, 1, 2, 3, 4] and ids[1].tolist() == [-1] * 5 and ids[3].tolist() == [-1] * 5
    assert ids[2].tolist() == [64, 3, 190, -1, -1] and ids[6].tolist() == [0, 1, 2, 3, 4]
    assert ids[5, :2].tolist() == [10, 100] and not np.isnan(w).any()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_topk_bias_selects_only(score):
    """Scores of a few well-separated values, so that fp32 and 64-bit sums order them alike."""
    rng = np.random.default_rng(5)
    E, T = 96, 40
    logits = np.stack([rng.permutation(E) / 8.0 - 6 for _ in range(T)]).astype(np.float32)
    bias = (rng.permutation(E) * 4.0).astype(np.float32)   # steps of 4 outweigh any score in [0, 1]
    bias[5] = -np.inf
    l = torch.from_numpy(logits).cuda()
    l[3, 17] = -float("inf")
    ids, _ = check_topk(l, 6, score=score, bias=to_dev(bias))
    want = [e for e in np.argsort(-bias, kind="stable") if e != 5][:6]
    assert ids[0].tolist() == [int(e) for e in want]


def test_topk_no_tokens():
    ids = torch.empty(0, 3, dtype=torch.int32, device="cuda")
    gfg.moe_topk(torch.empty(0, 8, device="cuda"), ids, torch.empty(0, 3, device="cuda"))


# ------------------------------------------------------------------ layer
def make(rng, weight, E, H, I):
    """(device w1, s1, w2, s2), (dequantized w1, w2)."""
    def fp8(N, K):
        x = torch.from_numpy((rng.standard_normal((E, N, K)) * 96).clip(-448, 448)).to(torch.float8_e4m3fn)
        t = 127 - int(round(np.log2(96 * np.sqrt(K))))
        s = rng.integers(t - 1, t + 2, (E, N // 128, K // 128)).astype(np.uint8)
        return x.cuda(), to_dev(s), so.dequantize_fp8(x.view(torch.uint8).numpy(), s)

    def int8(N, K):
        q = np.clip(np.rint(rng.standard_normal((E, N, K)) * 32), -128, 127).astype(np.int8)
        s = (rng.uniform(0.5, 2.0, (E, N)) / (32 * np.sqrt(K))).astype(np.float32)
        return to_dev(q), to_dev(s), so.dequantize_int8(q, s)

    f = fp8 if weight == "fp8" else int8
    (w1, s1, d1), (w2, s2, d2) = f(2 * I, H), f(H, I)
    return (w1, s1, w2, s2), (d1, d2)


def call(weight, x, ids, w, ops, out=None, **kw):
    out = torch.full_like(x, float("nan")) if out is None else out
    return (gfg.moe_fp8_layer if weight == "fp8" else gfg.moe_int8_layer)(x, ids, w, *ops, out, **kw)


def check_layer(got, ref, dt, what):
    got = got.float().cpu().numpy().astype(np.float64)
    assert np.all(np.isfinite(got)), what
    err = np.abs(got - ref)
    top = np.abs(ref).max(1, keepdims=True)
    tol = 1.01 * U[dt] * np.abs(ref) + 2.0 ** -12 * top + (2.0 ** -25 if dt == "f16" else 0)
    norm = float(np.linalg.norm(got - ref) / max(np.linalg.norm(ref), 1e-300))
    print(f"[moe] {what}: norm error {norm:.2e}, worst error minus bound {np.max(err - tol):.2e}", flush=True)
    assert np.all(err <= tol), what
    assert norm <= U[dt] / np.sqrt(3) * 1.1 + 2.0 ** -14, what


def choose(rng, T, E, k):
    return np.stack([rng.permutation(E)[:k] for _ in range(T)]).astype(np.int32)


@pytest.mark.parametrize("weight", ["fp8", "int8"])
@pytest.mark.parametrize("T,E,k,H,I,dt", [
    (1, 1, 1, 128, 128, "bf16"), (1, 8, 2, 256, 128, "f16"), (1, 16, 8, 1024, 512, "bf16"), (3, 4, 4, 384, 640, "f16"),
    (5, 6, 1, 128, 384, "bf16"), (17, 4, 2, 256, 256, "bf16"), (40, 3, 2, 640, 128, "f16"), (64, 40, 8, 128, 256, "bf16"),
    (100, 2, 1, 128, 128, "bf16"), (150, 2, 2, 256, 128, "f16"), (128, 8, 8, 128, 128, "bf16"), (1024, 1, 1, 128, 128, "bf16"),
    (16, 64, 64, 128, 128, "bf16"), (33, 5, 3, 2048, 1024, "f16"), (2, 1024, 6, 128, 128, "bf16"),
    (200, 4, 2, 256, 2048, "bf16"), (150, 6, 2, 384, 1536, "f16"), (90, 9, 3, 1152, 1408, "bf16"), (100, 8, 1, 128, 2048, "f16"),
])
def test_layer(weight, T, E, k, H, I, dt):
    what = f"{weight} T={T} E={E} k={k} H={H} I={I} {dt}"
    print(f"[moe] {what}", flush=True)
    rng = np.random.default_rng(T + E + k + H + I)
    ops, (d1, d2) = make(rng, weight, E, H, I)
    x = torch.from_numpy(rng.standard_normal((T, H))).to(torch_dtype(dt)).cuda()
    ids = choose(rng, T, E, k)
    w = rng.uniform(0.05, 1.0, (T, k)).astype(np.float32)
    need = gfg.moe_layer_workspace_bytes(T, k, H, I)
    flat = torch.full((need + 256,), 0xFF, dtype=torch.uint8, device="cuda")      # NaNs, if any were read
    out = call(weight, x, to_dev(ids), to_dev(w), ops, workspace=flat[128:128 + need])
    assert bool((flat[:128] == 0xFF).all()) and bool((flat[128 + need:] == 0xFF).all())
    check_layer(out, so.layer(x.float().cpu().numpy(), ids, w, d1, d2), dt, what)
    again = call(weight, x, to_dev(ids), to_dev(w), ops)
    assert np.array_equal(bits(out), bits(again)), f"{what}: two runs differ"


@pytest.mark.parametrize("weight", ["fp8", "int8"])
def test_layer_missing_foreign_and_repeated_experts(weight):
    rng = np.random.default_rng(8)
    T, E, k, H, I = 9, 5, 4, 256, 256
    ops, (d1, d2) = make(rng, weight, E, H, I)
    x = torch.from_numpy(rng.standard_normal((T, H))).to(torch.bfloat16).cuda()
    ids = choose(rng, T, E, k)
    ids[0] = -1                                            # a token with no expert here
    ids[1] = [E, -3, 2**31 - 1, -2**31]
    ids[2] = [3, 3, 3, 3]                                  # one expert four times
    ids[3] = [0, -1, 0, 1]
    w = rng.uniform(0.1, 1.0, (T, k)).astype(np.float32)
    w[0] = np.nan                                          # weights of experts that do not run are not read
    out = call(weight, x, to_dev(ids), to_dev(w), ops)
    w[0] = 0
    assert bool((out[:2] == 0).all())
    check_layer(out[2:], so.layer(x.float().cpu().numpy(), ids, w, d1, d2)[2:], "bf16", f"{weight} special ids")
    none = call(weight, x, torch.full((T, k), -1, dtype=torch.int32, device="cuda"), to_dev(w), ops)
    assert bool((none == 0).all())


@pytest.mark.parametrize("weight", ["fp8", "int8"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_layer_non_finite_values_stay_in_their_token_and_expert(weight, bad):
    rng = np.random.default_rng(9)
    T, E, k, H, I = 20, 4, 2, 256, 128
    ops, (d1, d2) = make(rng, weight, E, H, I)
    x = torch.from_numpy(rng.standard_normal((T, H))).to(torch.bfloat16).cuda()
    ids = choose(rng, T, E, k)
    ids[4] = -1
    ids[:, 0][ids[:, 0] == 3] = 0
    ids[:, 1][ids[:, 1] == 3] = 1
    ids[19] = [3, 0]
    w = rng.uniform(0.1, 1.0, (T, k)).astype(np.float32)
    ref = so.layer(x.float().cpu().numpy(), ids, w, d1, d2)
    x[7, 100] = bad                                        # a token that runs
    x[4] = bad                                             # one that does not
    if weight == "fp8":
        ops[1][3] = 255                                    # expert 3: NaN scales
    else:
        ops[1][3] = bad
    out = call(weight, x, to_dev(ids), to_dev(w), ops)
    o = out.float().cpu().numpy()
    assert not np.isfinite(o[7]).any() and not np.isfinite(o[19]).any()
    keep = [t for t in range(T) if t not in (7, 19)]
    check_layer(out[keep], ref[keep], "bf16", f"{weight} beside {bad}")


def test_layer_extreme_scale_bytes():
    """E8M0 bytes near both ends: 2^-127 (a subnormal float) against 2^100."""
    rng = np.random.default_rng(10)
    T, E, k, H, I = 3, 2, 1, 128, 128
    ops, _ = make(rng, "fp8", E, H, I)
    x = torch.from_numpy(rng.standard_normal((T, H))).to(torch.bfloat16).cuda()
    ids = np.array([[0], [1], [0]], np.int32)
    w = np.ones((T, k), np.float32)
    ops[1][0] = 127 - 10
    ops[3][0] = 0                                          # 2^-127
    ops[1][1] = 0
    ops[3][1] = 254
    d1 = so.dequantize_fp8(ops[0].view(torch.uint8).cpu().numpy(), ops[1].cpu().numpy())
    d2 = so.dequantize_fp8(ops[2].view(torch.uint8).cpu().numpy(), ops[3].cpu().numpy())
    out = call("fp8", x, to_dev(ids), to_dev(w), ops).float().cpu().numpy()
    ref = so.layer(x.float().cpu().numpy(), ids, w, d1, d2)
    ref[1] = 0.0          # its hidden values, below 2^-230, vanish in fp32; the others are tiny numbers of bf16's range
    assert np.all(np.isfinite(out))
    assert np.all(np.abs(out - ref) <= 2.0 ** -8 * np.abs(ref) * 1.01 + 2.0 ** -12 * np.abs(ref).max(1, keepdims=True) + 2.0 ** -126)


@pytest.mark.parametrize("T,E,k,H,I", [(2, 6, 3, 512, 384), (90, 9, 3, 1152, 1408)])
@pytest.mark.parametrize("offset", [1, 2, 3])
def test_layer_scale_bytes_at_any_alignment(T, E, k, H, I, offset):
    """E8M0 scales are bytes and may start anywhere; the kernels read them in words."""
    rng = np.random.default_rng(T + offset)
    (w1, s1, w2, s2), (d1, d2) = make(rng, "fp8", E, H, I)

    def moved(s):
        flat = torch.full((s.numel() + 8,), 200, dtype=torch.uint8, device="cuda")
        flat[offset:offset + s.numel()] = s.reshape(-1)
        return flat[offset:offset + s.numel()].view(s.shape)

    x = torch.from_numpy(rng.standard_normal((T, H))).to(torch.bfloat16).cuda()
    ids, w = choose(rng, T, E, k), rng.uniform(0.1, 1.0, (T, k)).astype(np.float32)
    out = call("fp8", x, to_dev(ids), to_dev(w), (w1, moved(s1), w2, moved(s2)))
    check_layer(out, so.layer(x.float().cpu().numpy(), ids, w, d1, d2), "bf16", f"scales at {offset}")


def test_layer_on_a_stream_without_a_workspace():
    rng = np.random.default_rng(31)
    T, E, k, H, I = 3, 5, 2, 256, 256
    ops, (d1, d2) = make(rng, "int8", E, H, I)
    x = torch.from_numpy(rng.standard_normal((T, H))).to(torch.bfloat16).cuda()
    ids, w = choose(rng, T, E, k), rng.uniform(0.1, 1.0, (T, k)).astype(np.float32)
    di, dw = to_dev(ids), to_dev(w)
    outs = [torch.zeros_like(x) for _ in range(2)]
    torch.cuda.synchronize()
    ref = so.layer(x.float().cpu().numpy(), ids, w, d1, d2)
    s = torch.cuda.Stream()
    for stream, out in zip((s, s.cuda_stream), outs):     # a Stream, and its handle
        call("int8", x, di, dw, ops, out=out, stream=stream)
        s.synchronize()
        check_layer(out, ref, "bf16", "on a stream")


def test_layer_hidden_values_beyond_half_precision():
    """float16 tokens whose hidden rows pass 65504 and come back into range."""
    rng = np.random.default_rng(12)
    T, E, k, H, I = 4, 2, 2, 256, 256
    ops, (d1, d2) = make(rng, "int8", E, H, I)
    ops[1].mul_(600.0)
    ops[3].mul_(2.0 ** -14)
    x = torch.from_numpy(rng.standard_normal((T, H))).to(torch.float16).cuda()
    ids = choose(rng, T, E, k)
    w = rng.uniform(0.1, 1.0, (T, k)).astype(np.float32)
    ref = so.layer(x.float().cpu().numpy(), ids, w, d1 * np.float32(600.0), d2 * 2.0 ** -14)
    assert np.abs(d1 * 600 @ x.float().cpu().numpy().T).max() ** 2 > 1e5
    check_layer(call("int8", x, to_dev(ids), to_dev(w), ops), ref, "f16", "large hidden values")


def test_layer_and_router_in_a_graph_on_a_stream():
    rng = np.random.default_rng(13)
    T, E, k, H, I = 6, 12, 3, 256, 384
    ops, _ = make(rng, "fp8", E, H, I)
    x = torch.from_numpy(rng.standard_normal((T, H))).to(torch.bfloat16).cuda()
    logits = torch.from_numpy(rng.standard_normal((T, E))).float().cuda()
    ids = torch.zeros(T, k, dtype=torch.int32, device="cuda")
    w = torch.zeros(T, k, device="cuda")
    out = torch.zeros_like(x)
    ws = torch.empty(gfg.moe_layer_workspace_bytes(T, k, H, I), dtype=torch.uint8, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())

    def launches():
        gfg.moe_topk(logits, ids, w, stream=s)
        gfg.moe_fp8_layer(x, ids, w, *ops, out, workspace=ws, stream=s)

    with torch.cuda.stream(s):
        launches()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        launches()
    for r in range(4):
        logits.copy_(torch.from_numpy(rng.standard_normal((T, E))))              # another routing each replay
        out.fill_(3.0)
        ws.fill_(0xFF)
        torch.cuda.synchronize()
        with torch.cuda.stream(s):
            g.replay()
        torch.cuda.synchronize()
        got = out.clone()
        with torch.cuda.stream(s):
            launches()
        torch.cuda.synchronize()
        assert torch.equal(got, out), f"replay {r}"


def test_layer_no_tokens():
    rng = np.random.default_rng(14)
    ops, _ = make(rng, "fp8", 2, 128, 128)
    x = torch.empty(0, 128, dtype=torch.bfloat16, device="cuda")
    out = call("fp8", x, torch.empty(0, 2, dtype=torch.int32, device="cuda"), torch.empty(0, 2, device="cuda"), ops)
    assert out.shape == (0, 128)


# ------------------------------------------------------------------ limits and offsets
@pytest.mark.parametrize("weight,T,E,k,H,I", [("fp8", 2, 3, 2, 32256, 128), ("int8", 2, 3, 2, 32256, 128), ("fp8", 3, 3, 1, 128, 32256),
                                              ("int8", 70, 2, 1, 128, 32256), ("fp8", 70, 2, 2, 16512, 128)])
def test_layer_long_rows(weight, T, E, k, H, I):
    what = f"{weight} long rows T={T} H={H} I={I}"
    print(f"[moe] {what}", flush=True)
    rng = np.random.default_rng(H + I + T)
    ops, (d1, d2) = make(rng, weight, E, H, I)
    x = torch.from_numpy(rng.standard_normal((T, H))).to(torch.bfloat16).cuda()
    ids, w = choose(rng, T, E, k), rng.uniform(0.1, 1.0, (T, k)).astype(np.float32)
    out = call(weight, x, to_dev(ids), to_dev(w), ops)
    check_layer(out, so.layer(x.float().cpu().numpy(), ids, w, d1, d2), "bf16", what)


@pytest.mark.parametrize("T", [2, 70])
def test_layer_largest_experts(T):
    """The longest rows both ways: an expert of 2.08 + 1.04 GB, the second one past 32-bit offsets."""
    E, k, H, I = 2, 1, 32256, 32256
    print(f"[moe] largest experts T={T}", flush=True)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(T)

    def weight(N, K):
        q = torch.randint(-96, 97, (E, N, K), dtype=torch.int8, device="cuda", generator=gen)
        return q, (torch.rand(E, N, device="cuda", generator=gen) + 0.5) / (56 * K ** 0.5)

    def times(v, q, s):                                   # v [R, K] . (q s)^T in float64, a few rows of q at a time
        return torch.cat([v @ (a.double() * b.double()[:, None]).T.contiguous() for a, b in zip(q.split(2016), s.split(2016))], 1)

    (w1, s1), (w2, s2) = weight(2 * I, H), weight(H, I)
    x = torch.randn(T, H, device="cuda", generator=gen).to(torch.bfloat16)
    ids = (torch.arange(T, device="cuda") % E).int().view(T, 1)
    w = torch.rand(T, 1, device="cuda", generator=gen) + 0.1
    out = call("int8", x, ids, w, (w1, s1, w2, s2))
    ref = torch.empty(T, H, dtype=torch.float64, device="cuda")
    for e in range(E):
        rows = ids[:, 0] == e
        gu = times(x[rows].double(), w1[e], s1[e])
        g, u = gu.chunk(2, 1)
        ref[rows] = w[rows].double() * times(g * torch.sigmoid(g) * u, w2[e], s2[e])
    check_layer(out, ref.cpu().numpy(), "bf16", f"largest experts T={T}")


def test_layer_on_two_streams_at_once():
    rng = np.random.default_rng(41)
    E, k, H, I = 24, 4, 1024, 512
    ops, (d1, d2) = make(rng, "fp8", E, H, I)
    work = []
    for T in (40, 3):
        x = torch.from_numpy(rng.standard_normal((T, H))).to(torch.bfloat16).cuda()
        ids, w = choose(rng, T, E, k), rng.uniform(0.1, 1.0, (T, k)).astype(np.float32)
        ws = torch.empty(gfg.moe_layer_workspace_bytes(T, k, H, I), dtype=torch.uint8, device="cuda")
        work.append((x, to_dev(ids), to_dev(w), ws, torch.zeros(8, T, H, dtype=torch.bfloat16, device="cuda"),
                     so.layer(x.float().cpu().numpy(), ids, w, d1, d2), torch.cuda.Stream()))
    torch.cuda.synchronize()
    for i in range(8):
        for x, ids, w, ws, outs, _, s in work:
            call("fp8", x, ids, w, ops, out=outs[i], workspace=ws, stream=s)
    torch.cuda.synchronize()
    for x, _, _, _, outs, ref, _ in work:
        check_layer(outs[0], ref, "bf16", f"two streams T={x.shape[0]}")
        assert all(torch.equal(outs[0], o) for o in outs)


def test_calls_refuse_tensors_that_do_not_fit():
    T, E, k, H, I = 2, 4, 2, 256, 128
    ops, _ = make(np.random.default_rng(5), "fp8", E, H, I)
    x, out = (torch.zeros(T, H, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    ids, w = torch.zeros(T, k, dtype=torch.int32, device="cuda"), torch.zeros(T, k, device="cuda")
    wide = torch.zeros(T, 2 * H, dtype=torch.bfloat16, device="cuda")
    for bad in (dict(x=wide[:, ::2]), dict(x=x.float()), dict(x=x[:1]), dict(ids=ids.long()), dict(ids=ids[:, :1].expand(T, k)),
                dict(w=w.half()), dict(w=w[:, :1]), dict(out=out.half()), dict(out=out.cpu()), dict(w=w.cpu())):
        a = dict(x=x, ids=ids, w=w, out=out) | bad
        with pytest.raises((TypeError, ValueError)):
            gfg.moe_fp8_layer(a["x"], a["ids"], a["w"], *ops, a["out"])
    with pytest.raises(ValueError):
        gfg.moe_fp8_layer(x, ids, w, ops[0], ops[1][:, :1], ops[2], ops[3], out)
    with pytest.raises(TypeError):
        gfg.moe_fp8_layer(x, ids, w, *ops, out, workspace=torch.empty(1 << 20, device="cuda"))
    with pytest.raises(Exception, match="workspace"):
        gfg.moe_fp8_layer(x, ids, w, *ops, out, workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError):
        gfg.moe_topk(torch.zeros(T, E, device="cuda"), ids, w, score="softplus")
    with pytest.raises(ValueError):
        gfg.moe_topk(torch.zeros(E, T, device="cuda").T, ids, w)


def test_topk_many_tokens():
    """More tokens than one launch has workgroups for; the last ones count."""
    T, E, k = (1 << 22) + 5, 8, 2
    gen = torch.Generator(device="cuda")
    gen.manual_seed(8)
    logits = torch.randn(T, E, device="cuda", generator=gen)
    ids = torch.full((T, k), -7, dtype=torch.int32, device="cuda")
    w = torch.full((T, k), -7.0, device="cuda")
    gfg.moe_topk(logits, ids, w)
    top, idx = logits.topk(k, dim=1)
    assert torch.equal(ids, idx.int())
    assert torch.allclose(w, torch.softmax(top, 1), atol=1e-6, rtol=0)
