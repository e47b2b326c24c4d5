"""Serving a mixture-of-experts block from 8-bit weights: torch-facing calls.

The router (``moe_topk``), the expert layer for a few tokens
(``moe_fp8_layer``, ``moe_int8_layer``) and the 8-bit integer products
(``int8_linear``, ``int8_gemm``, ``grouped_int8_gemm_*``) with their token
quantizer.  As for the other calls, this is argument marshalling only: shapes,
types and devices are checked, the work runs in the library's HIP kernels,
asynchronously on ``stream`` (default: the current one), and nothing falls
back.  Outputs are the caller's tensors and are returned.
"""
from __future__ import annotations

import torch

from . import IN_BF16, IN_F16, IN_F32, OUT_BF16, OUT_F16, _check, _check_stream, _on, load_library

try:
    from ._args import address as _address
except ImportError:                                        # built for another torch or not at all: Python answers
    def _address(t, dtypes, shape, index):
        return None

_IN = {torch.float32: IN_F32, torch.bfloat16: IN_BF16, torch.float16: IN_F16}
_OUT = {torch.bfloat16: OUT_BF16, torch.float16: OUT_F16}
_SCORE = {"softmax": 0, "sigmoid": 1}
_I8, _I32, _F32, _U8 = (torch.int8,), (torch.int32,), (torch.float32,), (torch.uint8,)
_F8 = (torch.float8_e4m3fn, torch.uint8)


def _ptr(t, name, dtypes, shape, device):
    """The address of a dense GPU tensor of one of the types, of that shape."""
    at = _address(t, dtypes, shape, device.index)
    if at is not None:
        return at
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype in dtypes and t.shape == shape and t.device == device and t.is_contiguous():
        return t.data_ptr()
    if t.dtype not in dtypes:
        raise TypeError(f"{name} has dtype {t.dtype}, expected one of {tuple(dtypes)}")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    raise ValueError(f"{name} must be contiguous")


def _device(t, name):
    """The GPU that a call runs on: that of its output, whichever is current."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be on a GPU")
    return t.device


def _dims(t, name, n):
    if not isinstance(t, torch.Tensor) or t.dim() != n:
        raise ValueError(f"{name} must be a torch.Tensor with {n} dimensions")
    return t.shape


# the current stream's handle without a Stream object around it (a quarter of a small call's time), and the current
# device without the check that there is one (its tensors show that)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _handle(stream, device):
    if stream is None:
        if _raw_stream is not None:
            return _raw_stream(device.index)
        return torch.cuda.current_stream(device).cuda_stream
    _check_stream(stream, device)
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _call(device, entry, *args):
    """Call an entry point on ``device``: it is current already, or made current for the call."""
    if _current_device() == device.index:
        _check(entry(*args))
    else:
        _on(device, entry, *args)


def _empty(shape, dtype, device, stream):
    """A new tensor that belongs to the stream that the call runs on (so that its memory is not reused too early)."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    handle = _handle(stream, device)
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(handle, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _scratch(workspace, needed, device, stream):
    """The workspace with its address and size; a new one where the caller keeps none."""
    if workspace is None:
        workspace = _empty(max(needed, 16), torch.uint8, device, stream)
    elif not isinstance(workspace, torch.Tensor) or workspace.dtype != torch.uint8 or not workspace.is_contiguous():
        raise TypeError("workspace must be a contiguous uint8 tensor")
    elif workspace.device != device:
        raise ValueError(f"workspace is on {workspace.device}, expected {device}")
    return workspace, workspace.data_ptr(), workspace.numel()


# ------------------------------------------------------------------ 8-bit integer products
def int8_quantize_token_device(x, q=None, scale=None, stream=None):
    """One scale per row: x [..., K] float32, bfloat16 or float16 -> (q [..., K] int8, scale [...] float32).

    ``scale = amax / 127`` and ``q = rint(x * (127 / amax))`` with ``amax = max(max|x|, 2**-100)``; a row with a
    NaN or an infinity gets scale NaN.  ``q`` and ``scale`` are allocated where they are not given.
    """
    dev = _device(x, "x")
    if x.dim() < 1:
        raise ValueError("x must have at least one dimension")
    if q is None:
        q = _empty(x.shape, torch.int8, dev, stream)
    if scale is None:
        scale = _empty(x.shape[:-1], torch.float32, dev, stream)
    K = x.shape[-1]
    M = x.numel() // K if K else 0
    _call(dev, load_library().int8_quantize_token_device,
        _ptr(x, "x", _IN, x.shape, dev), _IN[x.dtype], M, K, _ptr(q, "q", _I8, x.shape, dev),
        _ptr(scale, "scale", _F32, x.shape[:-1], dev), _handle(stream, dev))
    return q, scale


def int8_gemm(a, a_scale, b, b_scale, d, bias=None, stream=None):
    """d = (a . b^T) * a_scale[:, None] * b_scale (+ bias): a [M, K] and b [N, K] int8, a_scale [M], b_scale [N]
    and bias [N] float32, d [M, N] bfloat16 or float16.  K a multiple of 16."""
    dev = _device(d, "d")
    M, K = _dims(a, "a", 2)
    N = _dims(b, "b", 2)[0]
    _call(dev, load_library().int8_gemm,
        _ptr(a, "a", _I8, (M, K), dev), _ptr(a_scale, "a_scale", _F32, (M,), dev), _ptr(b, "b", _I8, (N, K), dev),
        _ptr(b_scale, "b_scale", _F32, (N,), dev), None if bias is None else _ptr(bias, "bias", _F32, (N,), dev),
        _ptr(d, "d", _OUT, (M, N), dev), M, N, K, _OUT[d.dtype], _handle(stream, dev))
    return d


def int8_linear_workspace_bytes(M, K):
    """Bytes of workspace that ``int8_linear`` needs for x [M, K]."""
    return int(load_library().int8_linear_workspace_bytes(M, K))


def int8_linear(x, b, b_scale, d, bias=None, workspace=None, stream=None):
    """The token quantizer and ``int8_gemm`` in one call: x [M, K] float32, bfloat16 or float16.

    ``workspace``: a uint8 tensor of at least ``int8_linear_workspace_bytes(M, K)`` bytes (allocated if None).
    Calls on different streams need workspaces of their own.
    """
    dev = _device(d, "d")
    M, K = _dims(x, "x", 2)
    N = _dims(b, "b", 2)[0]
    lib = load_library()
    keep, ws, nbytes = _scratch(workspace, M * (K + 4), dev, stream)
    _call(dev, lib.int8_linear,
        _ptr(x, "x", _IN, (M, K), dev), _IN[x.dtype], _ptr(b, "b", _I8, (N, K), dev),
        _ptr(b_scale, "b_scale", _F32, (N,), dev), None if bias is None else _ptr(bias, "bias", _F32, (N,), dev),
        _ptr(d, "d", _OUT, (M, N), dev), M, N, K, _OUT[d.dtype], ws, nbytes, _handle(stream, dev))
    return d


def grouped_int8_gemm_contiguous(a, a_scale, b, b_scale, grouped_layout, d, stream=None):
    """d[rows of expert g] = a[rows] . b[g]^T with both scales: a [M, K], b [G, N, K] int8, a_scale [M], b_scale
    [G, N] float32, grouped_layout [M] int32 (as in ``grouped_fp8_gemm_contiguous``), d [M, N]."""
    dev = _device(d, "d")
    M, K = _dims(a, "a", 2)
    G, N = _dims(b, "b", 3)[:2]
    _call(dev, load_library().grouped_int8_gemm_contiguous,
        _ptr(a, "a", _I8, (M, K), dev), _ptr(a_scale, "a_scale", _F32, (M,), dev), _ptr(b, "b", _I8, (G, N, K), dev),
        _ptr(b_scale, "b_scale", _F32, (G, N), dev), _ptr(grouped_layout, "grouped_layout", _I32, (M,), dev),
        _ptr(d, "d", _OUT, (M, N), dev), M, N, K, G, _OUT[d.dtype], _handle(stream, dev))
    return d


def grouped_int8_gemm_masked(a, a_scale, b, b_scale, masked_m, d, stream=None):
    """d[g, m < masked_m[g]] = a[g, m] . b[g]^T with both scales: a [G, M_max, K], b [G, N, K] int8, a_scale
    [G, M_max], b_scale [G, N] float32, masked_m [G] int32 (device), d [G, M_max, N]."""
    dev = _device(d, "d")
    G, Mmax, K = _dims(a, "a", 3)
    N = _dims(b, "b", 3)[1]
    _call(dev, load_library().grouped_int8_gemm_masked,
        _ptr(a, "a", _I8, (G, Mmax, K), dev), _ptr(a_scale, "a_scale", _F32, (G, Mmax), dev),
        _ptr(b, "b", _I8, (G, N, K), dev), _ptr(b_scale, "b_scale", _F32, (G, N), dev),
        _ptr(masked_m, "masked_m", _I32, (G,), dev), _ptr(d, "d", _OUT, (G, Mmax, N), dev), G, Mmax, N, K,
        _OUT[d.dtype], _handle(stream, dev))
    return d


# ------------------------------------------------------------------ mixture of experts
def moe_topk(logits, ids, weights, score="softmax", bias=None, renormalize=True, scale=1.0, stream=None):
    """The k = ids.shape[1] experts of each token's largest logits and their weights.

    logits [T, E] float32, bfloat16 or float16; ids [T, k] int32; weights [T, k] float32; ``score`` "softmax" or
    "sigmoid"; bias [E] float32 chooses by score + bias.  Experts with logit -inf or NaN are never chosen; missing
    choices get id -1 and weight 0.  Returns (ids, weights).
    """
    dev = _device(ids, "ids")
    T, E = _dims(logits, "logits", 2)
    k = _dims(ids, "ids", 2)[1]
    if score not in _SCORE:
        raise ValueError(f"score is {score!r}, expected one of {tuple(_SCORE)}")
    _call(dev, load_library().moe_topk,
        _ptr(logits, "logits", _IN, (T, E), dev), _IN[logits.dtype],
        None if bias is None else _ptr(bias, "bias", _F32, (E,), dev), _ptr(ids, "ids", _I32, (T, k), dev),
        _ptr(weights, "weights", _F32, (T, k), dev), T, E, k, _SCORE[score], bool(renormalize), scale,
        _handle(stream, dev))
    return ids, weights


def moe_layer_workspace_bytes(T, k, H, I):
    """Bytes of workspace that the layers need for T tokens of k experts each."""
    return int(load_library().moe_layer_workspace_bytes(T, k, H, I))


def _layer(entry, x, topk_ids, topk_weights, w1, w1_scale, w2, w2_scale, out, workspace, stream, wtypes, stype, block):
    dev = _device(out, "out")
    T, H = _dims(x, "x", 2)
    k = _dims(topk_ids, "topk_ids", 2)[1]
    E, _, I = _dims(w2, "w2", 3)
    s1, s2 = ((E, 2 * I // block, H // block), (E, H // block, I // block)) if block else ((E, 2 * I), (E, H))
    keep, ws, nbytes = _scratch(workspace, T * k * (H + I) * 4, dev, stream)
    _call(dev, entry,
        _ptr(x, "x", _OUT, (T, H), dev), _OUT[x.dtype], _ptr(topk_ids, "topk_ids", _I32, (T, k), dev),
        _ptr(topk_weights, "topk_weights", _F32, (T, k), dev), _ptr(w1, "w1", wtypes, (E, 2 * I, H), dev),
        _ptr(w1_scale, "w1_scale", stype, s1, dev), _ptr(w2, "w2", wtypes, (E, H, I), dev),
        _ptr(w2_scale, "w2_scale", stype, s2, dev), _ptr(out, "out", (x.dtype,), (T, H), dev), T, k, E, H, I, ws, nbytes,
        _handle(stream, dev))
    return out


def moe_fp8_layer(x, topk_ids, topk_weights, w1, w1_scale, w2, w2_scale, out, workspace=None, stream=None):
    """out[t] = sum_j topk_weights[t, j] * W2[e] (silu(g) * u), g | u = W1[e] x[t], e = topk_ids[t, j].

    x and out [T, H] bfloat16 or float16; topk_ids [T, k] int32 (outside [0, E): no contribution); w1 [E, 2I, H]
    and w2 [E, H, I] e4m3 with E8M0 scales [E, 2I/128, H/128] and [E, H/128, I/128], as in the grouped FP8 GEMMs.
    At most 1024 pairs T * k.  ``workspace``: a uint8 tensor of ``moe_layer_workspace_bytes(T, k, H, I)`` bytes
    (allocated if None); calls on different streams need workspaces of their own.
    """
    return _layer(load_library().moe_fp8_layer, x, topk_ids, topk_weights, w1, w1_scale, w2, w2_scale, out, workspace,
                  stream, _F8, _U8, 128)


def moe_int8_layer(x, topk_ids, topk_weights, w1, w1_scale, w2, w2_scale, out, workspace=None, stream=None):
    """The same layer on int8 weights with one float32 scale per output channel: w1_scale [E, 2I], w2_scale [E, H],
    as in the grouped int8 products."""
    return _layer(load_library().moe_int8_layer, x, topk_ids, topk_weights, w1, w1_scale, w2, w2_scale, out, workspace,
                  stream, _I8, _F32, 0)
