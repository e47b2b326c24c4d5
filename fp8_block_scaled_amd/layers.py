"""The rest of a block on FP8 weights, served and trained: torch-facing calls.

The dense FP8 linear layer (``fp8_linear``, ``fp8_gemm``), its gradients
(``fp8_linear_backward``) and the quantizer of its weights
(``fp8_quantize_weight_device``); the norms around a block with its gate and
residual sum (``residual_norm``, ``residual_norm_fp8`` for the FP8 operand of the
next product, ``residual_norm_backward``); the router's balance loss and gradient
(``moe_balance_loss``, ``moe_router_backward``).  Argument marshalling only, as in
``serving.py``: shapes, types and devices are checked, the work runs in the
library's HIP kernels, asynchronously on ``stream`` (default: the current one),
and nothing falls back.  Outputs are the caller's tensors, or new ones where they
are not given, and are returned.
"""
from __future__ import annotations

import torch

from . import load_library
from .serving import _F8, _F32, _I32, _IN, _OUT, _SCORE, _U8, _call, _device, _dims, _empty, _handle, _ptr, _scratch

_GRAD = {**_OUT, torch.float32: 2}
_GATE_NONE, _GATE_CHANNEL, _GATE_TOKEN = 0, 1, 2


def _blocks(n):
    return (n + 127) // 128


def _opt(t, name, dtypes, shape, device):
    return None if t is None else _ptr(t, name, dtypes, shape, device)


def _scale_rows(t, name, shape, device):
    """Address and row stride of a scale tensor [blocks, rows] whose rows are dense (its blocks may lie further apart)."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != torch.uint8:
        raise TypeError(f"{name} has dtype {t.dtype}, expected one of {_U8}")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    blocks, rows = shape
    ld = t.stride(0) if blocks > 1 else rows
    if (rows > 1 and t.stride(1) != 1) or ld < rows:
        raise ValueError(f"{name} must have dense rows that do not overlap")
    return t.data_ptr(), ld


# ------------------------------------------------------------------ FP8 linear layer
def fp8_quantize_weight_device(w, q=None, scale=None, q_t=None, scale_t=None, transposed=False, stream=None):
    """Blocks of 128 x 128: w [N, K] or [G, N, K] float32, bfloat16 or float16 -> (q, scale), or with ``transposed``
    (or ``q_t`` and ``scale_t``) -> (q, scale, q_t, scale_t).

    q has w's shape, scale [.., ceil(N/128), ceil(K/128)] uint8; q_t [.., K, N] and scale_t [.., ceil(K/128),
    ceil(N/128)] are the same codes and scales transposed (N a multiple of 16).  Tensors that are not given are
    allocated.
    """
    dev = _device(w, "w")
    if w.dim() not in (2, 3):
        raise ValueError("w must have 2 or 3 dimensions")
    lead, (N, K) = tuple(w.shape[:-2]), w.shape[-2:]
    transposed = transposed or q_t is not None or scale_t is not None
    new = lambda t, dtype, *shape: t if t is not None else _empty(lead + shape, dtype, dev, stream)  # noqa: E731
    q, scale = new(q, torch.float8_e4m3fn, N, K), new(scale, torch.uint8, _blocks(N), _blocks(K))
    if transposed:
        q_t, scale_t = new(q_t, torch.float8_e4m3fn, K, N), new(scale_t, torch.uint8, _blocks(K), _blocks(N))
    _call(dev, load_library().fp8_quantize_weight_device,
        _ptr(w, "w", _IN, w.shape, dev), _IN[w.dtype], lead[0] if lead else 1, N, K, _ptr(q, "q", _F8, w.shape, dev),
        _ptr(scale, "scale", _U8, lead + (_blocks(N), _blocks(K)), dev), _opt(q_t, "q_t", _F8, lead + (K, N), dev),
        _opt(scale_t, "scale_t", _U8, lead + (_blocks(K), _blocks(N)), dev), _handle(stream, dev))
    return (q, scale, q_t, scale_t) if transposed else (q, scale)


def fp8_gemm(a, a_scale, b, b_scale, d, bias=None, stream=None):
    """d = a . b^T (+ bias) of E4M3 operands: a [M, K] with a_scale [ceil(K/128), M] (its rows may lie further apart
    than M bytes), b [N, K] with b_scale [ceil(N/128), ceil(K/128)], E8M0 scales, bias [N] float32, d [M, N] bfloat16
    or float16.  K a multiple of 16, any M and N."""
    dev = _device(d, "d")
    M, K = _dims(a, "a", 2)
    N = _dims(b, "b", 2)[0]
    sa, ld = _scale_rows(a_scale, "a_scale", (_blocks(K), M), dev)
    _call(dev, load_library().fp8_gemm,
        _ptr(a, "a", _F8, (M, K), dev), sa, ld, _ptr(b, "b", _F8, (N, K), dev),
        _ptr(b_scale, "b_scale", _U8, (_blocks(N), _blocks(K)), dev), _opt(bias, "bias", _F32, (N,), dev),
        _ptr(d, "d", _OUT, (M, N), dev), M, N, K, _OUT[d.dtype], _handle(stream, dev))
    return d


def fp8_linear_workspace_bytes(M, K):
    """Bytes of workspace that ``fp8_linear`` needs for x [M, K]."""
    return int(load_library().fp8_linear_workspace_bytes(M, K))


def fp8_linear(x, w, w_scale, d, bias=None, workspace=None, stream=None):
    """d = Q(x) . w^T (+ bias), Q the E4M3 quantizer with one scale per token and 128 channels: x [M, K] float32,
    bfloat16 or float16, w, w_scale and d as b, b_scale and d of ``fp8_gemm``.

    ``workspace``: a uint8 tensor of at least ``fp8_linear_workspace_bytes(M, K)`` bytes (allocated if None).  Calls
    on different streams need workspaces of their own.
    """
    dev = _device(d, "d")
    M, K = _dims(x, "x", 2)
    N = _dims(w, "w", 2)[0]
    lib = load_library()
    keep, ws, nbytes = _scratch(workspace, M * K + _blocks(K) * (M + 3), dev, stream)
    _call(dev, lib.fp8_linear,
        _ptr(x, "x", _IN, (M, K), dev), _IN[x.dtype], _ptr(w, "w", _F8, (N, K), dev),
        _ptr(w_scale, "w_scale", _U8, (_blocks(N), _blocks(K)), dev), _opt(bias, "bias", _F32, (N,), dev),
        _ptr(d, "d", _OUT, (M, N), dev), M, N, K, _OUT[d.dtype], ws, nbytes, _handle(stream, dev))
    return d


def fp8_linear_backward_workspace_bytes(M, N, K):
    """Bytes of workspace that ``fp8_linear_backward`` needs for dy [M, N] and x [M, K]."""
    return int(load_library().fp8_linear_backward_workspace_bytes(M, N, K))


def fp8_linear_backward(dy, x, w_t, w_t_scale, dx=None, dw=None, dbias=None, accumulate=False, workspace=None, stream=None):
    """The gradients of ``fp8_linear`` that have a tensor: dx = Q(dy) . w, dw = Q(dy^T) . Q(x^T)^T, dbias = sum of dy.

    dy [M, N] and x [M, K] of one type (x None without dw); w_t [K, N] with w_t_scale [ceil(K/128), ceil(N/128)], the
    transposed weight (both None without dx); dx [M, K] bfloat16 or float16, dw [N, K] one of these or float32,
    dbias [N] float32.  ``accumulate`` adds to dw (float32) and dbias.  N and K multiples of 16.  ``workspace``: at
    least ``fp8_linear_backward_workspace_bytes(M, N, K)`` bytes, as for ``fp8_linear``.  Returns (dx, dw, dbias).
    """
    dev = _device(dy, "dy")
    M, N = _dims(dy, "dy", 2)
    if dw is not None:
        K = _dims(dw, "dw", 2)[1]
    elif dx is not None:
        K = _dims(dx, "dx", 2)[1]
    elif dbias is not None:
        K = 16 if x is None else _dims(x, "x", 2)[1]
    else:
        raise ValueError("dx, dw and dbias are all None")
    if dw is not None and x is None:
        raise ValueError("dw needs x")
    if dx is not None and (w_t is None or w_t_scale is None):
        raise ValueError("dx needs w_t and w_t_scale")
    dy_ptr = _ptr(dy, "dy", _IN, (M, N), dev)
    x_ptr = _opt(x, "x", (dy.dtype,), (M, K), dev)
    wt, ws = _opt(w_t, "w_t", _F8, (K, N), dev), _opt(w_t_scale, "w_t_scale", _U8, (_blocks(K), _blocks(N)), dev)
    dx_ptr, dw_ptr = _opt(dx, "dx", _OUT, (M, K), dev), _opt(dw, "dw", _GRAD, (N, K), dev)
    db_ptr = _opt(dbias, "dbias", _F32, (N,), dev)
    lib = load_library()
    need = 0 if workspace is not None else int(lib.fp8_linear_backward_workspace_bytes(M, N, K))
    keep, work, nbytes = _scratch(workspace, need, dev, stream)
    _call(dev, lib.fp8_linear_backward,
        dy_ptr, x_ptr, _IN[dy.dtype], wt, ws, dx_ptr, dw_ptr, db_ptr, M, N, K, 0 if dx is None else _OUT[dx.dtype],
        0 if dw is None else _GRAD[dw.dtype], bool(accumulate), work, nbytes, _handle(stream, dev))
    return dx, dw, dbias


# ------------------------------------------------------------------ norms around a block
def _gate(gate, M, H, device, name="gate"):
    if gate is None:
        return None, _GATE_NONE
    if isinstance(gate, torch.Tensor) and gate.dim() == 2:
        return _ptr(gate, name, _F32, (M, 1), device), _GATE_TOKEN
    return _ptr(gate, name, _F32, (H,), device), _GATE_CHANNEL


def _norm_inputs(y, residual, weight, post_weight, gate, normed=None):
    dev = _device(residual, "residual")
    M, H = _dims(residual, "residual", 2)
    dtype = residual.dtype if y is None else getattr(y, "dtype", None)
    if y is None and dtype == torch.float32 and getattr(normed, "dtype", None) in _IN:
        dtype = normed.dtype                               # (without y the normed rows alone have this type)
    if dtype not in _IN:
        raise TypeError(f"y has dtype {dtype}, expected one of {tuple(_IN)}")
    if residual.dtype not in (dtype, torch.float32):
        raise TypeError(f"residual has dtype {residual.dtype}, expected {dtype} or torch.float32")
    g, kind = _gate(gate, M, H, dev)
    return dev, M, H, dtype, (
        _opt(y, "y", _IN, (M, H), dev), _ptr(residual, "residual", _IN, (M, H), dev), _opt(weight, "weight", _F32, (H,), dev),
        _opt(post_weight, "post_weight", _F32, (H,), dev), g, kind)


def residual_norm(y, residual, weight, post_weight=None, gate=None, alpha=1.0, eps=1e-6, out=None, normed=None, stats=None,
                  stream=None):
    """out = alpha * residual + gate * u and normed = out * rstd(out) * weight, with u = y * rstd(y) * post_weight, or
    u = y without post_weight, and rstd(v) = 1 / sqrt(mean(v^2) + eps) over a row.

    y [M, H] float32, bfloat16 or float16, or None (u = 0); residual [M, H] of y's type or float32; weight and
    post_weight [H] float32 (weight None: no normed rows); gate float32, [H] (one a channel) or [M, 1] (one a row);
    out like residual (may be residual itself), normed like y (without y of residual's type, or of any of the three beside
    a float32 residual); stats [2, M] float32, rstd(y) and rstd(out), for the backward call.  Returns (out, normed,
    stats); out is allocated where it is not given and there is a y, normed where it is not given and there is a weight,
    stats never.
    """
    dev, M, H, dtype, inputs = _norm_inputs(y, residual, weight, post_weight, gate, normed)
    if out is None and (y is not None or weight is None):
        out = _empty((M, H), residual.dtype, dev, stream)
    if normed is None and weight is not None:
        normed = _empty((M, H), dtype, dev, stream)
    _call(dev, load_library().residual_norm,
        *inputs, alpha, eps, _opt(out, "out", (residual.dtype,), (M, H), dev), _opt(normed, "normed", (dtype,), (M, H), dev),
        _opt(stats, "stats", _F32, (2, M), dev), M, H, _IN[dtype], _IN[residual.dtype], _handle(stream, dev))
    return out, normed, stats


def residual_norm_fp8(y, residual, weight, post_weight=None, gate=None, alpha=1.0, eps=1e-6, out=None, q=None, scale=None,
                      stats=None, stream=None):
    """``residual_norm`` with the normed rows as the FP8 operand of the next product: q [M, H] E4M3 codes and scale
    [ceil(H/128), M] uint8 E8M0 (its rows may lie further apart than M bytes).  H a multiple of 16.

    Returns (out, q, scale, stats); a new scale has rows padded to a multiple of 4 bytes, new codes are float8_e4m3fn.
    """
    dev, M, H, dtype, inputs = _norm_inputs(y, residual, weight, post_weight, gate)
    if out is None and y is not None:
        out = _empty((M, H), residual.dtype, dev, stream)
    if q is None:
        q = _empty((M, H), torch.float8_e4m3fn, dev, stream)
    if scale is None:
        scale = _empty((_blocks(H), (M + 3) // 4 * 4), torch.uint8, dev, stream)[:, :M]
    scale_ptr, ld = _scale_rows(scale, "scale", (_blocks(H), M), dev)
    _call(dev, load_library().residual_norm_fp8,
        *inputs, alpha, eps, _opt(out, "out", (residual.dtype,), (M, H), dev), _ptr(q, "q", _F8, (M, H), dev), scale_ptr, ld,
        _opt(stats, "stats", _F32, (2, M), dev), M, H, _IN[dtype], _IN[residual.dtype], _handle(stream, dev))
    return out, q, scale, stats


def residual_norm_backward_workspace_bytes(M, H):
    """Bytes of workspace that ``residual_norm_backward`` needs for M rows of H."""
    return int(load_library().residual_norm_backward_workspace_bytes(M, H))


def residual_norm_backward(dout, dnormed, out, y, stats, weight, post_weight=None, gate=None, alpha=1.0, dresidual=None,
                           dy=None, dweight=None, dpost_weight=None, dgate=None, accumulate=False, workspace=None, stream=None):
    """The gradients of ``residual_norm`` (and, through the quantizer as through the identity, of ``residual_norm_fp8``)
    that have a tensor, from those of out and normed (either may be None).

    out, y and stats are the forward call's, the other inputs its own.  dresidual is like out, dy like y, dweight and
    dpost_weight [H] float32, dgate like gate.  ``accumulate`` adds to dweight, dpost_weight and a channel gate's
    dgate.  ``workspace``: at least ``residual_norm_backward_workspace_bytes(M, H)`` bytes (allocated if None); calls on
    different streams need workspaces of their own.  Returns (dresidual, dy, dweight, dpost_weight, dgate).
    """
    first = next((t for t in (dout, dnormed) if t is not None), None)
    if first is None:
        raise ValueError("dout and dnormed are both None")
    dev = _device(first, "dout" if dout is not None else "dnormed")
    M, H = _dims(first, "dout" if dout is not None else "dnormed", 2)
    rdtype = next((t.dtype for t in (out, dout, dresidual) if t is not None), None)
    dtype = next((t.dtype for t in (y, dnormed, dy) if t is not None), rdtype)
    rdtype = dtype if rdtype is None else rdtype
    if dtype not in _IN:
        raise TypeError(f"y has dtype {dtype}, expected one of {tuple(_IN)}")
    if rdtype not in (dtype, torch.float32):
        raise TypeError(f"out has dtype {rdtype}, expected {dtype} or torch.float32")
    g, kind = _gate(gate, M, H, dev)
    shape = (M, H)
    rows, wide = lambda t, name: _opt(t, name, (dtype,), shape, dev), lambda t, name: _opt(t, name, (rdtype,), shape, dev)  # noqa: E731
    vector = lambda t, name: _opt(t, name, _F32, (H,), dev)  # noqa: E731
    args = [wide(dout, "dout"), rows(dnormed, "dnormed"), wide(out, "out"), rows(y, "y"), _opt(stats, "stats", _F32, (2, M), dev),
            vector(weight, "weight"), vector(post_weight, "post_weight"), g, kind, alpha, wide(dresidual, "dresidual"),
            rows(dy, "dy"), vector(dweight, "dweight"), vector(dpost_weight, "dpost_weight"),
            _opt(dgate, "dgate", _F32, (M, 1) if kind == _GATE_TOKEN else (H,), dev)]
    lib = load_library()
    need = 0 if workspace is not None else int(lib.residual_norm_backward_workspace_bytes(M, H))
    keep, work, nbytes = _scratch(workspace, need, dev, stream)
    _call(dev, lib.residual_norm_backward, *args, bool(accumulate), M, H, _IN[dtype], _IN[rdtype], work, nbytes, _handle(stream, dev))
    return dresidual, dy, dweight, dpost_weight, dgate


# ------------------------------------------------------------------ training of the router
def moe_balance_workspace_bytes(T, E, S=1):
    """Bytes of workspace that ``moe_balance_loss`` needs for T tokens of S sequences over E experts."""
    return int(load_library().moe_balance_workspace_bytes(T, E, S))


def moe_balance_loss(logits, ids, score="softmax", alpha=1.0, z=0.0, seq_offsets=None, loss=None, counts=None, factors=None,
                     workspace=None, stream=None):
    """How unevenly each sequence's tokens spread over the experts: (loss, counts, factors).

    loss = 1/S sum_s (alpha * sum_e f_e P_e + z * mean logsumexp(logits)^2) over the S sequences (one without
    ``seq_offsets`` [S + 1] int32), f_e = counts[s, e] * E / (k n), P_e the mean over the sequence's n tokens of the
    softmax, or of the sigmoids over their sum.  A token without an id in [0, E) (padding) does not count.

    logits [T, E] float32, bfloat16 or float16; ids [T, k] int32, as ``moe_topk`` gives them; loss [] float32; counts
    [S, E] int32; factors [S, E + 1] float32, for ``moe_router_backward``; all three are allocated where they are not
    given.  ``workspace``: at least ``moe_balance_workspace_bytes(T, E, S)`` bytes (allocated if None); calls on
    different streams need workspaces of their own.
    """
    dev = _device(logits, "logits")
    T, E = _dims(logits, "logits", 2)
    k = _dims(ids, "ids", 2)[1]
    S = 1 if seq_offsets is None else _dims(seq_offsets, "seq_offsets", 1)[0] - 1
    if score not in _SCORE:
        raise ValueError(f"score is {score!r}, expected one of {tuple(_SCORE)}")
    if S < 1:
        raise ValueError("seq_offsets must have at least two entries")
    new = lambda t, dtype, shape: t if t is not None else _empty(shape, dtype, dev, stream)  # noqa: E731
    loss, counts = new(loss, torch.float32, ()), new(counts, torch.int32, (S, E))
    factors = new(factors, torch.float32, (S, E + 1))
    lib = load_library()
    need = 0 if workspace is not None else int(lib.moe_balance_workspace_bytes(T, E, S))
    keep, work, nbytes = _scratch(workspace, need, dev, stream)
    _call(dev, lib.moe_balance_loss,
        _ptr(logits, "logits", _IN, (T, E), dev), _IN[logits.dtype], _ptr(ids, "ids", _I32, (T, k), dev),
        _opt(seq_offsets, "seq_offsets", _I32, (S + 1,), dev), _ptr(loss, "loss", _F32, (), dev),
        _ptr(counts, "counts", _I32, (S, E), dev), _ptr(factors, "factors", _F32, (S, E + 1), dev), T, E, k, S,
        _SCORE[score], alpha, z, work, nbytes, _handle(stream, dev))
    return loss, counts, factors


def moe_router_backward(logits, ids, dlogits, dweights=None, score="softmax", renormalize=True, scale=1.0, factors=None,
                        dloss=None, seq_offsets=None, stream=None):
    """dlogits [T, E] (the logits' type): the gradient of ``dloss * loss + sum(dweights * weights)``.

    ``weights`` are ``moe_topk``'s for these ids, score, renormalize and scale, dweights [T, k] float32 their gradient;
    ``factors`` (with the same ``seq_offsets``) and dloss [] float32 belong to ``moe_balance_loss``.  Either part may
    be left out.
    """
    dev = _device(logits, "logits")
    T, E = _dims(logits, "logits", 2)
    k = _dims(ids, "ids", 2)[1]
    S = 1 if seq_offsets is None else _dims(seq_offsets, "seq_offsets", 1)[0] - 1
    if score not in _SCORE:
        raise ValueError(f"score is {score!r}, expected one of {tuple(_SCORE)}")
    _call(dev, load_library().moe_router_backward,
        _ptr(logits, "logits", _IN, (T, E), dev), _IN[logits.dtype], _ptr(ids, "ids", _I32, (T, k), dev),
        _opt(dweights, "dweights", _F32, (T, k), dev), _opt(factors, "factors", _F32, (S, E + 1), dev),
        _opt(dloss, "dloss", _F32, (), dev), _opt(seq_offsets, "seq_offsets", _I32, (S + 1,), dev),
        _ptr(dlogits, "dlogits", (logits.dtype,), (T, E), dev), T, E, k, S, _SCORE[score], bool(renormalize), scale,
        _handle(stream, dev))
    return dlogits
