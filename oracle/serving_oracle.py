"""Plain float64 definitions of the serving operators (test infrastructure only).

    quantizer   s = max(max|x|, 2^-100) / 127, q = rint(x * (127 / max(..))), each a single float32 rounding
    product     d[m, n] = (sum_k a[m, k] b[n, k]) * a_scale[m] * b_scale[n] (+ bias[n])
    router      the k largest logits (or scores plus bias), ties to the lowest index, and their scores
    layer       out[t] = sum_j w[t, j] * W2[e] (silu(g) * u),  g | u = W1[e] x[t],  e = ids[t, j]
"""
from __future__ import annotations

import numpy as np

from .fp8_oracle import decode_e4m3, e8m0_value


def quantize_token(x: np.ndarray):
    """x [..., K] (float32 values) -> (q int8, scale float32), bit for bit as defined."""
    x = np.asarray(x, np.float32)
    q = np.zeros(x.shape, np.int8)
    scale = np.full(x.shape[:-1], np.nan, np.float32)
    for i in np.ndindex(x.shape[:-1]):
        row = x[i]
        if not np.all(np.isfinite(row)):
            continue
        amax = np.maximum(np.max(np.abs(row), initial=np.float32(0)), np.float32(2.0 ** -100))
        scale[i] = amax / np.float32(127)
        q[i] = np.rint(row * (np.float32(127) / amax)).astype(np.int8)
    return q, scale


def int8_product(a, a_scale, b, b_scale, bias=None):
    """a [M, K], b [N, K] int8 -> float64 [M, N]."""
    acc = np.asarray(a, np.float64) @ np.asarray(b, np.float64).T      # exact: |sums| < 2^31
    d = acc * np.asarray(a_scale, np.float64)[:, None] * np.asarray(b_scale, np.float64)[None, :]
    return d if bias is None else d + np.asarray(bias, np.float64)[None, :]


def topk(logits, k, score="softmax", bias=None, renormalize=True, scale=1.0):
    """(ids [T, k], weights [T, k] float64); see the entry point for masked experts."""
    l = np.asarray(logits, np.float64).copy()
    l[np.isnan(l)] = -np.inf
    T, E = l.shape
    ids = np.full((T, k), -1, np.int32)
    w = np.zeros((T, k))
    for t in range(T):
        row = l[t]
        if score == "softmax":
            m = row.max()
            e = np.array([0.0 if v == -np.inf else 1.0 if v == m else np.exp(v - m) for v in row])
            p = e / e.sum() if e.sum() > 0 else e
        else:
            with np.errstate(over="ignore"):
                p = 1.0 / (1.0 + np.exp(-row))
        s = row if bias is None else np.where(row > -np.inf, p + np.asarray(bias, np.float64), -np.inf)
        order = [e for e in sorted(range(E), key=lambda e: (-s[e], e)) if s[e] > -np.inf][:k]
        ids[t, :len(order)] = order
        w[t, :len(order)] = p[order]
        if renormalize and w[t].sum() > 0:
            w[t] /= w[t].sum()
    return ids, w * scale


def dequantize_fp8(q, scale):
    """q [E, N, K] e4m3 codes, scale [E, N/128, K/128] E8M0 bytes -> float64."""
    s = e8m0_value(np.asarray(scale)).astype(np.float64)
    return decode_e4m3(np.asarray(q)).astype(np.float64) * s.repeat(128, 1).repeat(128, 2)


def dequantize_int8(q, scale):
    return np.asarray(q, np.float64) * np.asarray(scale, np.float64)[..., None]


def layer(x, ids, weights, w1, w2):
    """x [T, H], w1 [E, 2I, H], w2 [E, H, I] (dequantized, float64) -> [T, H]."""
    x = np.asarray(x, np.float64)
    T, k = np.shape(ids)
    E, H, I = w2.shape
    out = np.zeros((T, H))
    for t in range(T):
        for j in range(k):
            e = int(ids[t][j])
            if not 0 <= e < E:
                continue
            gu = w1[e] @ x[t]
            g, u = gu[:I], gu[I:]
            with np.errstate(over="ignore"):
                out[t] += float(weights[t][j]) * (w2[e] @ (g / (1.0 + np.exp(-g)) * u))
    return out
