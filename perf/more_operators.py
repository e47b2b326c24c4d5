"""The operators of a block on FP8 weights, served and trained, as cases to measure.

The FP8 linear layer with one scale per 128 channels of a token and per
128 x 128 block of the weight (from one token to prefill), its training step
(weights quantized in both orientations, forward, the three gradients), the
norms on both sides of the residual sum with their backward pass, alone and as
the quantizer of the next linear layer, and the router's balance loss with the
gradient of its logits.

``run`` computes them in plain torch operations in 32 bits, or, where ``own``
is true, through this package's entry points on the same state.
"""
import math

import torch

own = False

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
B = 128          # elements of a scale block
EPS = 1e-6       # of the norms


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one decoded token through a linear layer (7168 x 2304, an expert's down projection): latency and 16 MB of weights
        dict(name="linear_one_token", op="linear", M=1, N=7168, K=2304, dt="bf16", bias=False),
        # a small ragged batch, odd output width, a last block of 48 channels, float16, bias
        dict(name="linear_ragged", op="linear", M=77, N=1003, K=1072, dt="f16", bias=True),
        # prefill through one wide layer (the repository's dense shape)
        dict(name="linear_prefill", op="linear", M=4096, N=4096, K=16384, dt="bf16", bias=False),
        # a training step of a small layer on a ragged batch, both widths no multiple of the block
        dict(name="train_ragged", op="train", M=300, N=528, K=1040, dt="f16"),
        # a training step of an expert's down projection on 4096 tokens
        dict(name="train_layer", op="train", M=4096, N=7168, K=2304, dt="bf16"),
        # between two blocks of one decoded token: pure latency
        dict(name="norm_one_token", op="norm", M=1, H=7168, dt="bf16", rdt="bf16", post=True, gate="channel"),
        # between two blocks of a prefill, a 32-bit residual stream
        dict(name="norm_prefill", op="norm", M=4096, H=7168, dt="bf16", rdt="f32", post=True, gate="channel"),
        # backward, an odd width, one gate value a token
        dict(name="norm_backward_odd", op="norm_backward", M=333, H=2049, dt="f16", rdt="f16", post=True, gate="token"),
        # backward of a training batch
        dict(name="norm_backward_batch", op="norm_backward", M=8192, H=4096, dt="bf16", rdt="bf16", post=True, gate="channel"),
        # the end of one block and the first linear layer of the next: the norm hands its rows over in 8 bits
        dict(name="norm_into_linear", op="norm_linear", M=512, H=7168, N=2048, dt="bf16", rdt="bf16"),
        # the router's loss and gradient for a few tokens of one sequence
        dict(name="router_few", op="router", T=77, E=64, k=6, S=1, dt="f32", score="softmax", renorm=True, z=1e-3),
        # a training batch of 8 padded sequences over 385 experts
        dict(name="router_batch", op="router", T=32768, E=385, k=9, S=8, dt="bf16", score="sigmoid", renorm=True, z=0.0),
    ]


def _spread(rng, lo, hi):
    """A whole number spread evenly over the logarithm of [lo, hi]."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["linear", "linear", "train", "norm", "norm_backward", "norm_linear", "router"])
    dt = rng.choice(["bf16", "f16"])
    if op == "linear":
        return dict(op=op, M=_spread(rng, 1, 4096), N=_spread(rng, 64, 4096), K=16 * _spread(rng, 8, 1024), dt=dt,
                    bias=rng.random() < 0.5)
    if op == "train":
        return dict(op=op, M=_spread(rng, 16, 4096), N=16 * _spread(rng, 8, 448), K=16 * _spread(rng, 8, 144), dt=dt)
    if op == "norm_linear":
        return dict(op=op, M=_spread(rng, 1, 1024), H=16 * _spread(rng, 16, 448), N=_spread(rng, 64, 2048), dt=dt,
                    rdt=rng.choice([dt, "f32"]))
    if op == "router":
        E = _spread(rng, 8, 385)
        return dict(op=op, T=_spread(rng, 1, 32768), E=E, k=rng.randint(1, min(E, 9)), S=rng.randint(1, 8),
                    dt=rng.choice(["f32", "bf16", "f16"]), score=rng.choice(["softmax", "sigmoid"]),
                    renorm=rng.random() < 0.7, z=rng.choice([0.0, 1e-3]))
    return dict(op=op, M=_spread(rng, 1, 4096), H=_spread(rng, 64, 8192), dt=dt, rdt=rng.choice([dt, "f32"]),
                post=rng.random() < 0.7, gate=rng.choice(["none", "channel", "token"]))


# ------------------------------------------------------------------ inputs
def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(int(seed))
    s = dict(case=case)
    {"linear": _prepare_linear, "train": _prepare_train, "norm": _prepare_norm, "norm_backward": _prepare_norm_backward,
     "norm_linear": _prepare_norm_linear, "router": _prepare_router}[case["op"]](s, case, gen, dev)
    return s


def _randn(gen, dev, *shape):
    return torch.randn(*shape, generator=gen, device=dev)


def _tokens(gen, dev, dt, *shape):
    """Token vectors of different sizes, as they leave a residual stream."""
    x = _randn(gen, dev, *shape)
    return (x * torch.exp2(torch.rand(*shape[:-1], 1, generator=gen, device=dev) * 6 - 3)).to(DT[dt])


def _blocks(n):
    return (n + B - 1) // B


def _fp8_weight(gen, dev, N, K):
    """E4M3 codes and E8M0 bytes of a weight whose outputs are about as large as its inputs."""
    codes = _randn(gen, dev, N, K).mul_(96).clamp_(-448, 448).to(torch.float8_e4m3fn)
    t = 127 - round(math.log2(96 * math.sqrt(K)))
    scale = torch.randint(t - 1, t + 2, (_blocks(N), _blocks(K)), generator=gen, device=dev, dtype=torch.uint8)
    return codes, scale


def _workspace(dev):
    """The scratch memory that a program keeps for all of its layers."""
    return torch.empty(256 << 20, dtype=torch.uint8, device=dev)


def _prepare_linear(s, c, gen, dev):
    M, N, K, dt = c["M"], c["N"], c["K"], c["dt"]
    s["x"] = _tokens(gen, dev, dt, M, K)
    s["w"], s["ws"] = _fp8_weight(gen, dev, N, K)
    s["bias"] = _randn(gen, dev, N) if c["bias"] else None
    s["d"] = torch.empty(M, N, dtype=DT[dt], device=dev)
    s["workspace"] = _workspace(dev)


def _prepare_train(s, c, gen, dev):
    M, N, K, dt = c["M"], c["N"], c["K"], c["dt"]
    s["x"], s["dy"] = _tokens(gen, dev, dt, M, K), _tokens(gen, dev, dt, M, N)
    s["master"] = _randn(gen, dev, N, K) / math.sqrt(K)
    s["bias"] = _randn(gen, dev, N)
    new = lambda *shape, **kw: torch.empty(*shape, device=dev, **kw)  # noqa: E731
    s["q"], s["qs"] = new(N, K, dtype=torch.float8_e4m3fn), new(_blocks(N), _blocks(K), dtype=torch.uint8)
    s["qt"], s["qts"] = new(K, N, dtype=torch.float8_e4m3fn), new(_blocks(K), _blocks(N), dtype=torch.uint8)
    s["y"], s["dx"], s["dw"] = new(M, N, dtype=DT[dt]), new(M, K, dtype=DT[dt]), new(N, K, dtype=DT[dt])
    s["dbias"] = new(N)
    s["workspace"] = _workspace(dev)


def _prepare_norm(s, c, gen, dev):
    M, H = c["M"], c["H"]
    s["y"] = _tokens(gen, dev, c["dt"], M, H)
    s["residual"] = (4 * _randn(gen, dev, M, H)).to(DT[c["rdt"]])
    s["weight"] = 1 + 0.2 * _randn(gen, dev, H)
    s["post"] = 1 + 0.2 * _randn(gen, dev, H) if c.get("post", True) else None
    gate = c.get("gate", "channel")
    s["gate"] = None if gate == "none" else _randn(gen, dev, H) if gate == "channel" else _randn(gen, dev, M, 1)
    s["alpha"] = 0.8
    s["out"] = torch.empty_like(s["residual"])
    s["normed"] = torch.empty_like(s["y"])
    s["stats"] = torch.empty(2, M, device=dev)


def _prepare_norm_backward(s, c, gen, dev):
    _prepare_norm(s, c, gen, dev)
    M, H = c["M"], c["H"]
    # what the forward pass left: its output as it is stored, and the two rows of statistics
    y = s["y"].float()
    ry = torch.rsqrt(y.square().mean(-1) + EPS)
    u = y * ry[:, None] * s["post"] if s["post"] is not None else y
    out = s["alpha"] * s["residual"].float() + (u if s["gate"] is None else s["gate"] * u)
    s["out"] = out.to(DT[c["rdt"]])
    s["stats"] = torch.stack([ry, torch.rsqrt(out.square().mean(-1) + EPS)])
    s["dout"] = _randn(gen, dev, M, H).to(DT[c["rdt"]])
    s["dnormed"] = _randn(gen, dev, M, H).to(DT[c["dt"]])
    s["dresidual"], s["dy"] = torch.empty_like(s["out"]), torch.empty_like(s["y"])
    s["dweight"] = torch.empty(H, device=dev)
    s["dpost"] = torch.empty(H, device=dev) if s["post"] is not None else None
    s["dgate"] = torch.empty_like(s["gate"]) if s["gate"] is not None else None
    s["workspace"] = _workspace(dev)


def _prepare_norm_linear(s, c, gen, dev):
    _prepare_norm(s, c, gen, dev)
    M, H, N = c["M"], c["H"], c["N"]
    s["w"], s["ws"] = _fp8_weight(gen, dev, N, H)
    s["q"] = torch.empty(M, H, dtype=torch.float8_e4m3fn, device=dev)
    # one row of scale bytes per 128 channels, each padded to a multiple of 4 bytes
    s["qs"] = torch.empty(_blocks(H), (M + 3) // 4 * 4, dtype=torch.uint8, device=dev)[:, :M]
    s["d"] = torch.empty(M, N, dtype=DT[c["dt"]], device=dev)


def _prepare_router(s, c, gen, dev):
    T, E, k, S = c["T"], c["E"], c["k"], c["S"]
    logits = _randn(gen, dev, T, E) * 1.5
    s["logits"] = logits.to(DT[c["dt"]])
    ids = torch.sort(s["logits"].float(), dim=-1, descending=True, stable=True)[1][:, :k].to(torch.int32)
    # sequences of different lengths; the last sixteenth of each is padding, which no expert takes
    cuts = torch.linspace(0, T, S + 1, dtype=torch.float64).square() / max(T, 1)
    offsets = cuts.round().to(torch.int32).to(dev)
    t = torch.arange(T, device=dev)
    seq = torch.searchsorted(offsets[1:].contiguous(), t, right=True).clamp_max(S - 1)
    begin, end = offsets[seq].long(), offsets[seq + 1].long()
    padded = (t - begin) * 16 >= (end - begin) * 15 + 15
    s["ids"] = torch.where(padded[:, None], -1, ids).contiguous()
    s["offsets"] = offsets if S > 1 else None
    s["dweights"] = _randn(gen, dev, T, k)
    s["dloss"] = torch.rand((), generator=gen, device=dev) + 0.5
    s["loss"] = torch.empty((), device=dev)
    s["counts"] = torch.empty(S, E, dtype=torch.int32, device=dev)
    s["factors"] = torch.empty(S, E + 1, device=dev)
    s["dlogits"] = torch.empty_like(s["logits"])
    s["workspace"] = _workspace(dev)


ALPHA, SCALE = 0.01, 2.5      # weight of the balance loss, and the factor of the router's weights


# ------------------------------------------------------------------ one pass
def run(s):
    c = s["case"]
    op = c["op"]
    if own:
        import fp8_block_scaled_amd as gfg
        if op == "linear":
            return gfg.fp8_linear(s["x"], s["w"], s["ws"], s["d"], bias=s["bias"], workspace=s["workspace"])
        if op == "train":
            gfg.fp8_quantize_weight_device(s["master"], s["q"], s["qs"], s["qt"], s["qts"])
            gfg.fp8_linear(s["x"], s["q"], s["qs"], s["y"], bias=s["bias"], workspace=s["workspace"])
            gfg.fp8_linear_backward(s["dy"], s["x"], s["qt"], s["qts"], dx=s["dx"], dw=s["dw"], dbias=s["dbias"],
                                    workspace=s["workspace"])
            return s["y"], s["dx"], s["dw"], s["dbias"]
        if op == "norm":
            gfg.residual_norm(s["y"], s["residual"], s["weight"], post_weight=s["post"], gate=s["gate"], alpha=s["alpha"],
                              eps=EPS, out=s["out"], normed=s["normed"], stats=s["stats"])
            return s["out"], s["normed"], s["stats"]
        if op == "norm_backward":
            gfg.residual_norm_backward(s["dout"], s["dnormed"], s["out"], s["y"], s["stats"], s["weight"],
                                       post_weight=s["post"], gate=s["gate"], alpha=s["alpha"], dresidual=s["dresidual"],
                                       dy=s["dy"], dweight=s["dweight"], dpost_weight=s["dpost"], dgate=s["dgate"],
                                       workspace=s["workspace"])
            return s["dresidual"], s["dy"], s["dweight"], s["dpost"], s["dgate"]
        if op == "norm_linear":
            gfg.residual_norm_fp8(s["y"], s["residual"], s["weight"], post_weight=s["post"], gate=s["gate"],
                                  alpha=s["alpha"], eps=EPS, out=s["out"], q=s["q"], scale=s["qs"], stats=s["stats"])
            gfg.fp8_gemm(s["q"], s["qs"], s["w"], s["ws"], s["d"])
            return s["out"], s["d"]
        gfg.moe_balance_loss(s["logits"], s["ids"], score=c["score"], alpha=ALPHA, z=c["z"], seq_offsets=s["offsets"],
                             loss=s["loss"], counts=s["counts"], factors=s["factors"], workspace=s["workspace"])
        gfg.moe_router_backward(s["logits"], s["ids"], s["dlogits"], dweights=s["dweights"], score=c["score"],
                                renormalize=c["renorm"], scale=SCALE, factors=s["factors"], dloss=s["dloss"],
                                seq_offsets=s["offsets"])
        return s["loss"], s["counts"], s["dlogits"]
    return {"linear": _linear, "train": _train, "norm": _norm, "norm_backward": _norm_backward, "norm_linear": _norm_linear,
            "router": _router}[op](s)


def _exponent(amax):
    """The smallest t with 448 * 2^t >= amax (0 for amax = 0): 448 = 0.875 * 2^9."""
    m, e = torch.frexp(amax)
    return torch.where(amax > 0, torch.where(m <= 0.875, e - 9, e - 8), 0)


def _through_fp8(x):
    """The values that E4M3 codes of x [R, C] stand for, one power-of-two scale per row and 128 columns."""
    R, C = x.shape
    x = torch.nn.functional.pad(x.float(), (0, -C % B)).view(R, -1, B)
    scale = torch.ldexp(torch.ones((), device=x.device), _exponent(x.abs().amax(-1, keepdim=True)))
    return ((x / scale).to(torch.float8_e4m3fn).float() * scale).view(R, -1)[:, :C]


def _weight_through_fp8(w):
    """The same with one scale per block of 128 x 128."""
    N, K = w.shape
    x = torch.nn.functional.pad(w.float(), (0, -K % B, 0, -N % B)).view(_blocks(N), B, _blocks(K), B)
    scale = torch.ldexp(torch.ones((), device=x.device), _exponent(x.abs().amax((1, 3), keepdim=True)))
    return ((x / scale).to(torch.float8_e4m3fn).float() * scale).view(_blocks(N) * B, -1)[:N, :K]


def _dequantized(w, scale):
    N, K = w.shape
    s = torch.exp2(scale.float() - 127.0)
    return w.float() * s.repeat_interleave(B, 0)[:N].repeat_interleave(B, 1)[:, :K]


def _linear(s):
    d = _through_fp8(s["x"]) @ _dequantized(s["w"], s["ws"]).t()
    if s["bias"] is not None:
        d = d + s["bias"]
    return d.to(s["x"].dtype)


def _train(s):
    dt = s["x"].dtype
    w = _weight_through_fp8(s["master"])
    y = _through_fp8(s["x"]) @ w.t() + s["bias"]
    dx = _through_fp8(s["dy"]) @ w
    dw = _through_fp8(s["dy"].t()) @ _through_fp8(s["x"].t()).t()
    return y.to(dt), dx.to(dt), dw.to(dt), s["dy"].float().sum(0)


def _norm_of(s):
    y = s["y"].float()
    ry = torch.rsqrt(y.square().mean(-1, keepdim=True) + EPS)
    u = y * ry * s["post"] if s["post"] is not None else y
    out = s["alpha"] * s["residual"].float() + (u if s["gate"] is None else s["gate"] * u)
    ro = torch.rsqrt(out.square().mean(-1, keepdim=True) + EPS)
    return out, out * ro * s["weight"], torch.stack([ry[:, 0], ro[:, 0]])


def _norm(s):
    out, normed, stats = _norm_of(s)
    if s["post"] is None:
        stats[0] = 1.0
    return out.to(s["residual"].dtype), normed.to(s["y"].dtype), stats


def _norm_backward(s):
    y, out, dz = s["y"].float(), s["out"].float(), s["dnormed"].float()
    ry, ro = s["stats"][0][:, None], s["stats"][1][:, None]
    zhat = out * ro
    h = dz * s["weight"]
    g = s["dout"].float() + ro * (h - zhat * (h * zhat).mean(-1, keepdim=True))
    yhat = y * ry if s["post"] is not None else y
    u = yhat * s["post"] if s["post"] is not None else y
    du = g if s["gate"] is None else g * s["gate"]
    dgate = None
    if s["gate"] is not None:
        dgate = (g * u).sum(0) if s["gate"].dim() == 1 else (g * u).sum(1, keepdim=True)
    dy, dpost = du, None
    if s["post"] is not None:
        dpost = (du * yhat).sum(0)
        h = du * s["post"]
        dy = ry * (h - yhat * (h * yhat).mean(-1, keepdim=True))
    return (s["alpha"] * g).to(s["out"].dtype), dy.to(s["y"].dtype), (dz * zhat).sum(0), dpost, dgate


def _norm_linear(s):
    out, normed, _ = _norm_of(s)
    d = _through_fp8(normed) @ _dequantized(s["w"], s["ws"]).t()
    return out.to(s["residual"].dtype), d.to(s["y"].dtype)


def _router(s):
    c = s["case"]
    T, E, k, S = c["T"], c["E"], c["k"], c["S"]
    l, ids = s["logits"].float(), s["ids"].long()
    dev = l.device
    top = l.amax(-1, keepdim=True)
    e = torch.exp(l - top)
    lse = top[:, 0] + torch.log(e.sum(-1))
    softmax = e / e.sum(-1, keepdim=True)
    score = softmax if c["score"] == "softmax" else 1.0 / (1.0 + torch.exp(-l))
    p = score / score.sum(-1, keepdim=True)
    chosen = (ids >= 0) & (ids < E)
    counted = chosen.any(-1)
    seq = torch.zeros(T, dtype=torch.long, device=dev)
    if s["offsets"] is not None:
        seq = torch.searchsorted(s["offsets"][1:].long(), torch.arange(T, device=dev), right=True).clamp_max(S - 1)
    n = torch.zeros(S, device=dev).index_add(0, seq, counted.float())
    n = n.clamp_min(1.0)
    hit = (chosen[:, :, None] & (ids[:, :, None] == torch.arange(E, device=dev))).sum(1)
    counts = torch.zeros(S, E, dtype=torch.long, device=dev).index_add(0, seq, hit)
    P = torch.zeros(S, E, device=dev).index_add(0, seq, torch.where(counted[:, None], p, 0.0))
    f = counts * (E / k) / n[:, None]
    Z = torch.zeros(S, device=dev).index_add(0, seq, torch.where(counted, lse.square(), 0.0))
    loss = (ALPHA * (f * P).sum(-1) / n + c["z"] * Z / n).sum() / S
    # the gradient of the loss, and of the weights that the chosen experts got
    a = (ALPHA / S * f / n[:, None])[seq]
    inner = a - (a * p).sum(-1, keepdim=True)
    d = softmax * inner if c["score"] == "softmax" else score * (1 - score) / score.sum(-1, keepdim=True) * inner
    d = d + (2 * c["z"] / S) * (lse / n[seq])[:, None] * softmax
    d = torch.where(counted[:, None], d, 0.0) * s["dloss"]
    at = ids.clamp(0, E - 1)
    dw = torch.where(chosen, s["dweights"] * SCALE, 0.0)
    if c["renorm"]:
        sc = torch.where(chosen, score.gather(1, at), 0.0)
        total = sc.sum(-1, keepdim=True)
        w = torch.where(total > 0, sc / total, 0.0)
        dw = torch.where(chosen & (total > 0), (dw - (dw * w).sum(-1, keepdim=True)) / total, 0.0)
    ds = torch.zeros(T, E, device=dev).scatter_add(1, at, dw)
    if c["score"] == "softmax":
        d = d + softmax * (ds - (ds * softmax).sum(-1, keepdim=True))
    else:
        d = d + ds * score * (1 - score)
    return loss, counts.to(torch.int32), d.to(s["logits"].dtype)


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    op = case["op"]
    size = lambda dt: 4 if dt == "f32" else 2  # noqa: E731
    if op == "linear":
        M, N, K = case["M"], case["N"], case["K"]
        return dict(bytes=2 * M * K + N * K + N * K / 16384 + 2 * M * N + 4 * N * case["bias"], flops=2.0 * M * N * K)
    if op == "train":
        M, N, K = case["M"], case["N"], case["K"]
        # in: x, dy, the master weight, the bias; out: y, dx, dw, its bias; the weight's codes in both orientations
        return dict(bytes=2 * M * (2 * K + 2 * N) + N * K * (4 + 2 + 2) + 8 * N, flops=6.0 * M * N * K)
    if op == "router":
        T, E, k, S = (case[n] for n in ("T", "E", "k", "S"))
        return dict(bytes=2 * T * E * size(case["dt"]) + 8 * T * k + 4 * S * E, flops=30.0 * T * E)
    M, H, y, r = case["M"], case["H"], size(case["dt"]), size(case["rdt"])
    if op == "norm":
        return dict(bytes=M * H * (2 * y + 2 * r) + 12 * H, flops=10.0 * M * H)
    if op == "norm_backward":
        return dict(bytes=M * H * (3 * y + 3 * r) + 24 * H, flops=24.0 * M * H)
    N = case["N"]
    return dict(bytes=M * H * (y + 2 * r) + 12 * H + N * H + 2 * M * N, flops=2.0 * M * N * H + 10.0 * M * H)


# ------------------------------------------------------------------ the definitions in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    return {"linear": _exact_linear, "train": _exact_train, "norm": _exact_norm, "norm_backward": _exact_norm_backward,
            "norm_linear": _exact_norm_linear, "router": _exact_router}[case["op"]](s)


def _e4m3(v):
    """The nearest E4M3 values, ties to the even code: steps of 2^(e-3) from 2^e on, of 2^-9 below 2^-6."""
    step = torch.exp2(torch.floor(torch.log2(v.abs().clamp_min(2.0 ** -6))) - 3)
    return torch.round(v / step) * step


def _codes(x, rows):
    """x [R, C] in 64 bits, rounded to E4M3 in blocks of `rows` x 128."""
    R, C = x.shape
    z = torch.zeros(-(-R // rows) * rows, _blocks(C) * B, dtype=torch.float64, device=x.device)
    z[:R, :C] = x
    blocks = z.view(-(-R // rows), rows, _blocks(C), B).transpose(1, 2).reshape(-1, rows * B)
    amax = blocks.abs().max(dim=1, keepdim=True).values
    t = torch.floor(torch.log2(amax.clamp_min(1e-300) / 448.0))
    t = torch.where(448.0 * torch.exp2(t) < amax, t + 1, t)
    t = torch.where(amax > 0, t, torch.zeros_like(t))
    q = _e4m3(blocks / torch.exp2(t)) * torch.exp2(t)
    return q.view(-(-R // rows), _blocks(C), rows, B).transpose(1, 2).reshape(z.shape)[:R, :C]


def _exact_weight(s):
    w, sc = s["w"].float().double(), torch.pow(2.0, s["ws"].double() - 127)
    i, j = (torch.arange(n, device=w.device) // B for n in w.shape)
    return w * sc[i][:, j]


def _exact_linear(s):
    d = torch.mm(_codes(s["x"].double(), 1), _exact_weight(s).t())
    return d if s["bias"] is None else d + s["bias"].double()


def _exact_train(s):
    x, dy, w = s["x"].double(), s["dy"].double(), _codes(s["master"].double(), B)
    y = torch.addmm(s["bias"].double(), _codes(x, 1), w.t())
    dx = torch.mm(_codes(dy, 1), w)
    dw = torch.mm(_codes(dy.t().contiguous(), 1), _codes(x.t().contiguous(), 1).t())
    return y, dx, dw, dy.sum(dim=0)


def _exact_forward(s):
    y, r = s["y"].double(), s["residual"].double()
    ry = 1.0 / torch.sqrt((y * y).mean(dim=1) + EPS)
    u = y
    if s["post"] is not None:
        u = torch.einsum("mh,m,h->mh", y, ry, s["post"].double())
    if s["gate"] is not None:
        u = u * s["gate"].double()
    out = s["alpha"] * r + u
    ro = 1.0 / torch.sqrt((out * out).mean(dim=1) + EPS)
    return out, torch.einsum("mh,m,h->mh", out, ro, s["weight"].double()), ry, ro


def _exact_norm(s):
    out, normed, ry, ro = _exact_forward(s)
    return out, normed, torch.stack([ry if s["post"] is not None else torch.ones_like(ro), ro])


def _exact_norm_linear(s):
    out, normed, _, _ = _exact_forward(s)
    return out, torch.mm(_codes(normed, 1), _exact_weight(s).t())


def _exact_norm_backward(s):
    H = s["case"]["H"]
    y, out, dz = s["y"].double(), s["out"].double(), s["dnormed"].double()
    ry, ro = s["stats"].double()
    # z_h = w_h ro x_h with d(ro)/d(x_j) = -ro^3 x_j / H, so the gradient of x is ro w dz - ro^3 x (w dz . x) / H
    wdz = dz * s["weight"].double()
    g = s["dout"].double() + ro[:, None] * wdz - (ro ** 3 * (wdz * out).sum(dim=1) / H)[:, None] * out
    dweight = torch.mv((dz * out).t(), ro)
    gate = torch.ones((), dtype=torch.float64, device=y.device) if s["gate"] is None else s["gate"].double()
    post = s["post"].double() if s["post"] is not None else None
    u = y if post is None else y * ry[:, None] * post
    dgate = None if s["gate"] is None else (g * u).sum(dim=0 if s["gate"].dim() == 1 else 1).view(s["gate"].shape)
    if post is None:
        return s["alpha"] * g, g * gate, dweight, None, dgate
    dpost = torch.mv((g * gate * y).t(), ry)
    wdu = g * gate * post
    dy = ry[:, None] * wdu - (ry ** 3 * (wdu * y).sum(dim=1) / H)[:, None] * y
    return s["alpha"] * g, dy, dweight, dpost, dgate


def _exact_router(s):
    c = s["case"]
    T, E, k, S = c["T"], c["E"], c["k"], c["S"]
    l = s["logits"].double().cpu().requires_grad_(True)
    ids = s["ids"].cpu().long()
    here = (ids >= 0) & (ids < E)
    score = torch.softmax(l, 1) if c["score"] == "softmax" else torch.sigmoid(l)
    p = score if c["score"] == "softmax" else score / score.sum(1)[:, None]
    lse = torch.logsumexp(l, 1)
    cuts = [0, T] if s["offsets"] is None else s["offsets"].tolist()
    loss, counts = 0.0, torch.zeros(S, E, dtype=torch.int32)
    for q in range(S):
        rows = torch.arange(cuts[q], cuts[q + 1])
        rows = rows[here[rows].any(1)]
        n = rows.numel()
        if n:
            counts[q] = torch.bincount(ids[rows][here[rows]], minlength=E).int()
            f = counts[q].double() * E / (k * n)
            loss = loss + (ALPHA * torch.dot(f, p[rows].mean(0)) + c["z"] * lse[rows].square().mean()) / S
    w = torch.where(here, score.gather(1, ids.clamp(0, E - 1)), 0.0)
    if c["renorm"]:
        w = w / w.sum(1, keepdim=True).clamp_min(1e-300)
    (loss * s["dloss"].double().cpu() + (SCALE * w * s["dweights"].double().cpu()).sum()).backward()
    return loss.detach(), counts, l.grad
