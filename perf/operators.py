"""The serving operators of a mixture-of-experts block, as cases to measure.

Three operators: the 8-bit integer matrix product with one scale per token and
per output channel (from 16-bit activations, the token quantizer included),
the top-k router, and the whole expert layer for a few tokens.

``run`` computes them in plain torch operations in 32 bits, or, where ``own``
is true, through this package's entry points on the same state.
"""
import math
import random

import torch

own = False

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
TILE = 128      # the contiguous layout pads each expert's rows to a multiple of this


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one decoded token through a linear layer (7168 x 2304, an expert's down projection): latency and 16 MB of weights
        dict(name="linear_one_token", op="linear", M=1, N=7168, K=2304, dt="bf16", bias=False),
        # a small ragged batch, odd output width, K a multiple of 16 only, float16, bias
        dict(name="linear_ragged", op="linear", M=77, N=1003, K=1072, dt="f16", bias=True),
        # prefill through one wide layer (the repository's dense shape)
        dict(name="linear_prefill", op="linear", M=4096, N=4096, K=16384, dt="bf16", bias=False),
        # prefill through 8 experts of 4096 rows, the contiguous layout (the benchmark's default shape)
        dict(name="grouped_contiguous", op="contig", G=8, rows=4096, ragged=False, N=7168, K=2304, dt="bf16"),
        # 8 experts with 0 to 1024 rows each in fixed buffers, the masked layout
        dict(name="grouped_masked", op="masked", G=8, rows=1024, N=2048, K=7168, dt="bf16"),
        # the router of one decoded token: pure latency
        dict(name="route_one_token", op="route", T=1, E=256, k=8, dt="bf16", score="softmax", renorm=True),
        # the router of a prefill batch, 385 experts (an odd count), top 9
        dict(name="route_prefill", op="route", T=4096, E=385, k=9, dt="f32", score="sigmoid", renorm=True),
        # one decoded token through a 385-expert layer at its 4-way tensor-parallel share
        dict(name="layer_fp8_one_token", op="layer", w="fp8", T=1, E=385, ep=1, k=9, H=7168, I=512, dt="bf16"),
        # a decode batch of 32 through the same layer: about half of the experts are hit, one or two rows each
        dict(name="layer_fp8_decode", op="layer", w="fp8", T=32, E=385, ep=1, k=9, H=7168, I=512, dt="bf16"),
        # few large experts and many rows for each of them
        dict(name="layer_fp8_dense_routing", op="layer", w="fp8", T=100, E=8, ep=1, k=2, H=4096, I=1792, dt="bf16"),
        # a handful of tokens, integer weights, float16
        dict(name="layer_int8_few", op="layer", w="int8", T=5, E=64, ep=1, k=6, H=2048, I=1408, dt="f16"),
        # one of 8 expert-parallel ranks: seven eighths of the choices belong to other ranks
        dict(name="layer_int8_parallel", op="layer", w="int8", T=48, E=48, ep=8, k=8, H=4096, I=1024, dt="bf16"),
    ]


def _spread(rng, lo, hi):
    """A whole number spread evenly over the logarithm of [lo, hi]."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    while True:
        case = _draw(rng)
        if 3072 not in case.values():     # no configuration of this repository has it
            return case


def _draw(rng):
    op = rng.choice(["linear", "linear", "contig", "masked", "route", "layer", "layer", "layer"])
    if op == "linear":
        return dict(op=op, M=_spread(rng, 1, 4096), N=_spread(rng, 64, 4096), K=16 * _spread(rng, 8, 1024),
                    dt=rng.choice(["bf16", "f16"]), bias=rng.random() < 0.5)
    if op == "contig":
        return dict(op=op, G=rng.randint(1, 8), rows=_spread(rng, 16, 4096), ragged=True, N=_spread(rng, 128, 7168),
                    K=16 * _spread(rng, 8, 144), dt=rng.choice(["bf16", "f16"]))
    if op == "masked":
        return dict(op=op, G=rng.randint(1, 8), rows=_spread(rng, 16, 1024), N=_spread(rng, 128, 2048),
                    K=16 * _spread(rng, 8, 448), dt=rng.choice(["bf16", "f16"]))
    if op == "route":
        E = _spread(rng, 8, 385)
        return dict(op=op, T=_spread(rng, 1, 4096), E=E, k=rng.randint(1, min(E, 9)), dt=rng.choice(["f32", "bf16", "f16"]),
                    score=rng.choice(["softmax", "sigmoid"]), renorm=rng.random() < 0.7)
    while True:
        E, T, H, I = _spread(rng, 8, 385), _spread(rng, 1, 100), 128 * _spread(rng, 8, 56), 128 * _spread(rng, 1, 16)
        k = rng.randint(1, min(E, 9))
        if T * k * 2 * I * H <= 2_100_000_000 and E * 3 * I * H <= 4_200_000_000:
            return dict(op=op, w=rng.choice(["fp8", "int8"]), T=T, E=E, ep=rng.choice([1, 1, 8]), k=k, H=H, I=I,
                        dt=rng.choice(["bf16", "f16"]))


def _group_rows(case):
    """Rows of each group: part of the case, so the same for every seed."""
    G, rows = case["G"], case["rows"]
    r = random.Random(1000003 * G + 8191 * rows + case["N"])
    if case["op"] == "masked":
        got = [r.randint(0, rows) for _ in range(G)]
        got[r.randrange(G)] = rows
        return got
    return [r.randint(1, rows) for _ in range(G)] if case["ragged"] else [rows] * G


# ------------------------------------------------------------------ inputs
def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(int(seed))
    op = case["op"]
    if op == "route":
        logits = torch.randn(case["T"], case["E"], generator=gen, device=dev) * 1.5
        return dict(case=case, logits=logits.to(DT[case["dt"]]),
                    ids=torch.empty(case["T"], case["k"], dtype=torch.int32, device=dev),
                    weights=torch.empty(case["T"], case["k"], dtype=torch.float32, device=dev))
    if op == "layer":
        return _prepare_layer(case, gen, dev)
    dt, N, K = DT[case["dt"]], case["N"], case["K"]

    def tokens(*shape):   # token vectors of different sizes, as they leave a residual stream
        x = torch.randn(*shape, generator=gen, device=dev)
        return (x * torch.exp2(torch.rand(*shape[:-1], 1, generator=gen, device=dev) * 6 - 3)).to(dt)

    G = case.get("G", 1)
    w = _int8_codes((G, N, K), gen, dev)
    ws = (torch.rand(G, N, generator=gen, device=dev) * 1.5 + 0.5) / (32 * math.sqrt(K))
    s = dict(case=case, w=w, ws=ws)
    if op == "linear":
        s["x"] = tokens(case["M"], K)
        s["bias"] = torch.randn(N, generator=gen, device=dev) if case["bias"] else None
        s["w"], s["ws"] = w[0], ws[0]
        rows = (case["M"],)
        s["workspace"] = _workspace(dev)
    else:
        counts = _group_rows(case)
        if op == "contig":
            parts = [torch.cat([torch.full((m,), g, dtype=torch.int32), torch.full((-m % TILE,), -1, dtype=torch.int32)])
                     for g, m in enumerate(counts)]
            s["layout"] = torch.cat(parts).to(dev)
            starts = [0]
            for m in counts[:-1]:
                starts.append(starts[-1] + m + -m % TILE)
            s["starts"], s["most"] = torch.tensor(starts, device=dev), max(counts)
            rows = (s["layout"].numel(),)
            s["x"] = tokens(*rows, K) * (s["layout"] >= 0)[:, None].to(dt)
        else:
            s["masked_m"] = torch.tensor(counts, dtype=torch.int32, device=dev)
            rows = (G, case["rows"])
            s["x"] = tokens(*rows, K)
        s["q"] = torch.empty(*rows, K, dtype=torch.int8, device=dev)
        s["qs"] = torch.empty(*rows, dtype=torch.float32, device=dev)
    s["d"] = torch.zeros(*rows, N, dtype=dt, device=dev)
    return s


def _workspace(dev):
    """The scratch memory that a program keeps for all of its layers."""
    return torch.empty(128 << 20, dtype=torch.uint8, device=dev)


def _int8_codes(shape, gen, dev):
    x = torch.randn(shape, generator=gen, device=dev, dtype=torch.bfloat16)
    return x.mul_(32).round_().clamp_(-127, 127).to(torch.int8)


def _prepare_layer(case, gen, dev):
    T, E, k, H, I = (case[n] for n in ("T", "E", "k", "H", "I"))
    s = dict(case=case, x=torch.randn(T, H, generator=gen, device=dev).to(DT[case["dt"]]))
    # k different experts a token; those of other expert-parallel ranks are marked -1
    ids = torch.rand(T, E * case["ep"], generator=gen, device=dev).argsort(-1)[:, :k].to(torch.int32)
    s["ids"] = torch.where(ids < E, ids, -1).contiguous()
    p = torch.exp(torch.randn(T, k, generator=gen, device=dev))
    s["weights"] = p / p.sum(-1, keepdim=True)

    def fp8(N, K):
        codes = torch.randn(E, N, K, generator=gen, device=dev, dtype=torch.bfloat16).mul_(96).clamp_(-448, 448)
        t = 127 - round(math.log2(96 * math.sqrt(K)))
        scale = torch.randint(t - 1, t + 2, (E, N // 128, K // 128), generator=gen, device=dev, dtype=torch.uint8)
        return codes.to(torch.float8_e4m3fn), scale

    def int8(N, K):
        return (_int8_codes((E, N, K), gen, dev),
                (torch.rand(E, N, generator=gen, device=dev) * 1.5 + 0.5) / (32 * math.sqrt(K)))

    make = fp8 if case["w"] == "fp8" else int8
    s["w1"], s["s1"] = make(2 * I, H)
    s["w2"], s["s2"] = make(H, I)
    s["workspace"] = _workspace(dev)
    s["out"] = torch.zeros(T, H, dtype=s["x"].dtype, device=dev)
    return s


# ------------------------------------------------------------------ one pass
def run(s):
    op = s["case"]["op"]
    if own:
        import fp8_block_scaled_amd as gfg
        c = s["case"]
        if op == "linear":
            return gfg.int8_linear(s["x"], s["w"], s["ws"], s["d"], bias=s["bias"], workspace=s["workspace"])
        if op == "route":
            gfg.moe_topk(s["logits"], s["ids"], s["weights"], score=c["score"], renormalize=c["renorm"])
            return s["ids"], s["weights"]
        if op == "layer":
            layer = gfg.moe_fp8_layer if c["w"] == "fp8" else gfg.moe_int8_layer
            return layer(s["x"], s["ids"], s["weights"], s["w1"], s["s1"], s["w2"], s["s2"], s["out"],
                         workspace=s["workspace"])
        gfg.int8_quantize_token_device(s["x"], s["q"], s["qs"])
        if op == "contig":
            return gfg.grouped_int8_gemm_contiguous(s["q"], s["qs"], s["w"], s["ws"], s["layout"], s["d"])
        return gfg.grouped_int8_gemm_masked(s["q"], s["qs"], s["w"], s["ws"], s["masked_m"], s["d"])
    return {"linear": _linear, "contig": _contig, "masked": _masked, "route": _route, "layer": _layer}[op](s)


def _quantized(x):
    """Per-token integer codes (as float32) and scales: s = amax / 127, q = rint(x * (127 / amax))."""
    x = x.float()
    amax = x.abs().amax(-1, keepdim=True).clamp_min(2.0 ** -100)
    top = torch.full_like(amax, 127.0)
    return (x * (top / amax)).round(), amax / top


def _linear(s):
    q, qs = _quantized(s["x"])
    d = (q @ s["w"].float().t()) * qs * s["ws"]
    if s["bias"] is not None:
        d = d + s["bias"]
    return d.to(s["x"].dtype)


def _contig(s):
    # every expert's rows side by side, up to the longest run; then back to their places
    q, qs = _quantized(s["x"])
    row = torch.arange(q.shape[0], device=q.device)
    at = (s["starts"][:, None] + row[:s["most"]]).clamp_max(q.shape[0] - 1)
    d = torch.bmm(s["w"].float(), q[at].transpose(1, 2).contiguous()).transpose(1, 2) * s["ws"][:, None, :]
    g = s["layout"].long().clamp_min(0)
    d = d[g, (row - s["starts"][g]).clamp_max(s["most"] - 1)] * qs
    return torch.where((s["layout"] >= 0)[:, None], d, 0.0).to(s["x"].dtype)


def _masked(s):
    q, qs = _quantized(s["x"])
    d = torch.bmm(s["w"].float(), q.transpose(1, 2).contiguous()).transpose(1, 2) * s["ws"][:, None, :] * qs
    rows = torch.arange(d.shape[1], device=d.device)
    return torch.where((rows < s["masked_m"][:, None])[:, :, None], d, 0.0).to(s["x"].dtype)


def _route(s):
    l, k = s["logits"].float(), s["case"]["k"]
    ids = torch.sort(l, dim=-1, descending=True, stable=True)[1][:, :k]
    if s["case"]["score"] == "softmax":
        p = torch.exp(l - l.amax(-1, keepdim=True))
        p = p / p.sum(-1, keepdim=True)
    else:
        p = 1.0 / (1.0 + torch.exp(-l))
    w = p.gather(1, ids)
    if s["case"]["renorm"]:
        w = w / w.sum(-1, keepdim=True)
    return ids.to(torch.int32), w


def _dequantized(w, scale):
    """[n, N, K] float32 of integer codes with a scale per row, or of E4M3 codes with an E8M0 byte per 128 x 128 block."""
    n, N, K = w.shape
    if w.dtype == torch.int8:
        return w.float() * scale[:, :, None]
    w = w.view(torch.float8_e4m3fn).float().view(n, N // 128, 128, K // 128, 128)
    return (w * torch.exp2(scale.float() - 127.0)[:, :, None, :, None]).view(n, N, K)


def _layer(s):
    T, k = s["ids"].shape
    E, x = s["w1"].shape[0], s["x"].float()
    w1, w2 = (w if w.dtype == torch.int8 else w.view(torch.uint8) for w in (s["w1"], s["w2"]))
    if E <= T * k:
        # every expert on every token; those that a token did not choose have weight zero
        chosen = s["ids"][None] == torch.arange(E, device=x.device)[:, None, None]
        c = torch.where(chosen, s["weights"], 0.0).sum(-1)
        h = _swiglu(torch.bmm(_dequantized(w1, s["s1"]), x.t().expand(E, -1, -1).contiguous()))
        y = torch.bmm(_dequantized(w2, s["s2"]), h) * c[:, None, :]
        return y.sum(0).t().to(s["x"].dtype)
    # every chosen pair's own copy of its expert
    here = (s["ids"] >= 0).reshape(-1)
    ids = s["ids"].reshape(-1).long().clamp_min(0)
    h = _swiglu(torch.bmm(_dequantized(w1[ids], s["s1"][ids]), x.repeat_interleave(k, 0)[:, :, None]))
    y = torch.bmm(_dequantized(w2[ids], s["s2"][ids]), h)[:, :, 0]
    y = torch.where(here[:, None], y, 0.0) * s["weights"].reshape(-1, 1)
    return y.view(T, k, -1).sum(1).to(s["x"].dtype)


def _swiglu(gu):
    """[n, 2I, columns]: gate rows, then up rows."""
    g, u = gu.chunk(2, 1)
    return g / (1.0 + torch.exp(-g)) * u


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    op = case["op"]
    if op == "route":
        T, E, k = case["T"], case["E"], case["k"]
        return dict(bytes=T * E * (4 if case["dt"] == "f32" else 2) + 8 * T * k, flops=4 * T * E)
    if op == "layer":
        T, E, k, H, I = (case[n] for n in ("T", "E", "k", "H", "I"))
        total = E * case["ep"]
        hit = E * (1.0 - (1.0 - k / total) ** T)          # experts expected to have a row
        scales = 3 * I * H / 16384 if case["w"] == "fp8" else 4 * (2 * I + H)
        return dict(bytes=hit * (3 * I * H + scales) + 4 * T * H + 8 * T * k, flops=6.0 * T * k / case["ep"] * I * H)
    N, K = case["N"], case["K"]
    if op == "linear":
        M, G, bias = case["M"], 1, 4 * N * case["bias"]
    else:
        counts = _group_rows(case)
        M, G, bias = sum(counts), sum(m > 0 for m in counts), 0
    return dict(bytes=2 * M * K + G * N * (K + 4) + 2 * M * N + bias, flops=2.0 * M * N * K)


# ------------------------------------------------------------------ the definitions in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    return {"linear": _exact_product, "contig": _exact_product, "masked": _exact_product, "route": _exact_route,
            "layer": _exact_layer}[case["op"]](s)


def _exact_product(s):
    w, ws = s["w"], s["ws"].double()
    x = s["x"].reshape(-1, s["x"].shape[-1]).double()
    scale = x.abs().max(dim=1).values.clamp(min=2.0 ** -100) / 127
    q = torch.round(x / scale[:, None])
    out = torch.zeros(x.shape[0], w.shape[-2], dtype=torch.float64, device=x.device)
    for g in range(s["case"].get("G", 1)):
        if "layout" in s:
            rows = (s["layout"] == g).nonzero()[:, 0]
        elif "masked_m" in s:
            rows = torch.arange(int(s["masked_m"][g]), device=x.device) + g * s["case"]["rows"]
        else:
            rows = torch.arange(x.shape[0], device=x.device)
        wg, wsg = (w, ws) if w.dim() == 2 else (w[g], ws[g])
        out[rows] = torch.mm(q[rows], wg.double().t()) * torch.outer(scale[rows], wsg)
    if s.get("bias") is not None:
        out += s["bias"].double()
    return out.view(s["d"].shape)


def _exact_route(s):
    l = s["logits"].double().cpu()
    k, c = s["case"]["k"], s["case"]
    E = l.shape[1]
    # ties to the lowest index: expert i precedes expert j when it has the larger logit, or the same and i < j
    ids = torch.argsort(-l, dim=1, stable=True)[:, :k]
    p = torch.softmax(l, 1) if c["score"] == "softmax" else torch.sigmoid(l)
    w = p[torch.arange(l.shape[0])[:, None], ids]
    if c["renorm"]:
        w = w / w.sum(1)[:, None]
    assert int(ids.max()) < E
    return ids.to(torch.int32), w


def _exact_layer(s):
    c, x = s["case"], s["x"].double()
    T, I = c["T"], c["I"]
    out = torch.zeros(T, c["H"], dtype=torch.float64, device=x.device)

    def matrix(w, sc, e):
        if c["w"] == "int8":
            return w[e].double() * sc[e].double()[:, None]
        t = torch.pow(torch.tensor(2.0, dtype=torch.float64, device=w.device), sc[e].double() - 127)
        return w[e].to(torch.float32).double() * t.repeat_interleave(128, 0).repeat_interleave(128, 1)

    for e in s["ids"].unique().tolist():
        if e < 0:
            continue
        tok, j = (s["ids"] == e).nonzero(as_tuple=True)
        gu = torch.mm(x[tok], matrix(s["w1"], s["s1"], e).t())
        h = gu[:, :I] * torch.sigmoid(gu[:, :I]) * gu[:, I:]
        y = torch.mm(h, matrix(s["w2"], s["s2"], e).t())
        out.index_add_(0, tok, y * s["weights"][tok, j].double()[:, None])
    return out
