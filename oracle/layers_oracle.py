"""Plain float64 definitions of the operators around a block's products (test infrastructure only).

    linear      y = Q(x) W^T + b;  dx = Q(dy) W,  dW = Q(dy^T) Q(x^T)^T,  db = sum dy, Q in blocks of 1 x 128
    norms       u = y rstd(y) wp,  out = alpha r + g u,  normed = out rstd(out) w, and the gradients
    router      loss = 1/S sum_s (alpha sum_e f_e P_e + z mean lse^2), and the gradient of the logits from it and
                from the weights
"""
from __future__ import annotations

import numpy as np

from .fp8_oracle import dequantize_act, quantize_act_1x128


def through_fp8(x):
    """The values that x [R, C] has in E4M3 with one scale per row and 128 columns."""
    return dequantize_act(*quantize_act_1x128(np.ascontiguousarray(x)))


def linear(x, w, bias=None):
    """x [M, K] (float32 values), w [N, K] (dequantized)."""
    y = through_fp8(x) @ np.asarray(w, np.float64).T
    return y if bias is None else y + np.asarray(bias, np.float64)


def linear_backward(dy, x, w):
    dw = through_fp8(np.asarray(dy).T) @ through_fp8(np.asarray(x).T).T
    return through_fp8(dy) @ np.asarray(w, np.float64), dw, np.asarray(dy, np.float64).sum(0)


def rstd(v, eps):
    return 1.0 / np.sqrt((v * v).mean(1, keepdims=True) + eps)


def residual_norm(y, residual, weight, post=None, gate=None, alpha=1.0, eps=1e-6):
    """(out, normed, rstd(y) or 1, rstd(out)); gate [H] or [M, 1]."""
    out, ry = alpha * np.asarray(residual, np.float64), np.ones((len(residual), 1))
    if y is not None:
        u = np.asarray(y, np.float64)
        if post is not None:
            ry = rstd(u, eps)
            u = u * ry * post
        out = out + (u if gate is None else gate * u)
    ro = rstd(out, eps)
    return out, None if weight is None else out * ro * weight, ry, ro


def residual_norm_backward(dout, dnormed, out, y, ry, ro, weight, post=None, gate=None, alpha=1.0):
    """(dresidual, dy, dweight, dpost, dgate), those without an operand None."""
    f = lambda v: None if v is None else np.asarray(v, np.float64)  # noqa: E731
    dout, dnormed, out, y, post, gate = (f(v) for v in (dout, dnormed, out, y, post, gate))
    G = 0.0 if dout is None else dout
    dweight = None
    if dnormed is not None and weight is not None:
        zh, h = out * ro, dnormed * weight
        G = G + ro * (h - zh * (h * zh).mean(1, keepdims=True))
        dweight = (dnormed * zh).sum(0)
    if y is None:
        return alpha * G, None, dweight, None, None
    yh = y if post is None else y * ry
    u = yh if post is None else yh * post
    du = G if gate is None else G * gate
    dgate = None if gate is None else (G * u).sum(0) if gate.ndim == 1 else (G * u).sum(1, keepdims=True)
    if post is None:
        return alpha * G, du * np.ones_like(y), dweight, None, dgate
    h = post * du
    return alpha * G, ry * (h - yh * (h * yh).mean(1, keepdims=True)), dweight, (du * yh).sum(0), dgate


def _scores(logits, score):
    """(the router's scores, their normalized form p, the softmax, logsumexp), masked experts 0."""
    l = np.asarray(logits, np.float64).copy()
    l[np.isnan(l)] = -np.inf
    top = l.max(1, keepdims=True)
    safe = np.where(np.isfinite(top), top, 0.0)
    e = np.exp(l - safe)
    total = e.sum(1, keepdims=True)
    softmax = e / np.where(total > 0, total, 1.0)
    lse = np.where(total > 0, safe + np.log(np.where(total > 0, total, 1.0)), 0.0)[:, 0]
    if score == "softmax":
        return softmax, softmax, softmax, lse
    s = np.where(l >= 0, 1 / (1 + np.exp(-np.abs(l))), np.exp(-np.abs(l)) / (1 + np.exp(-np.abs(l))))
    z = s.sum(1, keepdims=True)
    return s, s / np.where(z > 0, z, 1.0), softmax, lse


def _sequences(T, offsets):
    return [(0, T)] if offsets is None else [(int(a), int(b)) for a, b in zip(offsets[:-1], offsets[1:])]


def balance(logits, ids, score="softmax", alpha=1.0, z=0.0, offsets=None):
    """(loss, counts [S, E], factors [S, E + 1])."""
    T, E = np.shape(logits)
    ids = np.asarray(ids)
    k, here = ids.shape[1], (ids >= 0) & (ids < E)
    _, p, _, lse = _scores(logits, score)
    spans = _sequences(T, offsets)
    S, loss = len(spans), 0.0
    counts, factors = np.zeros((S, E), np.int64), np.zeros((S, E + 1))
    for s, (a, b) in enumerate(spans):
        rows = [t for t in range(a, b) if here[t].any()]
        n = len(rows)
        if not n:
            continue
        for t in rows:
            np.add.at(counts[s], ids[t][here[t]], 1)
        f = counts[s] * E / (k * n)
        loss += (alpha * (f * p[rows].mean(0)).sum() + z * (lse[rows] ** 2).mean()) / S
        factors[s, :E], factors[s, E] = alpha * f / (S * n), 2 * z / (S * n)
    return loss, counts, factors


def topk_weights(logits, ids, score, renormalize, scale):
    sc = _scores(logits, score)[0]
    here = (ids >= 0) & (ids < sc.shape[1])
    w = np.where(here, np.take_along_axis(sc, np.clip(ids, 0, sc.shape[1] - 1), 1), 0.0)
    if renormalize:
        total = w.sum(1, keepdims=True)
        w = np.where(total > 0, w / np.where(total > 0, total, 1.0), 0.0)
    return w * scale


def router_backward(logits, ids, dweights=None, score="softmax", renormalize=True, scale=1.0, factors=None, dloss=0.0,
                    offsets=None):
    T, E = np.shape(logits)
    ids = np.asarray(ids)
    here = (ids >= 0) & (ids < E)
    sc, p, softmax, lse = _scores(logits, score)
    total = sc.sum(1)
    d = np.zeros((T, E))
    if factors is not None:
        for s, (a, b) in enumerate(_sequences(T, offsets)):
            for t in range(a, b):
                if not here[t].any():
                    continue
                inner = factors[s, :E] - (factors[s, :E] * p[t]).sum()
                d[t] += dloss * (p[t] * inner if score == "softmax" else sc[t] * (1 - sc[t]) / total[t] * inner)
                d[t] += dloss * factors[s, E] * lse[t] * softmax[t]
    if dweights is not None:
        for t in range(T):
            g = np.zeros(E)
            at, dw = ids[t][here[t]], scale * np.asarray(dweights, np.float64)[t][here[t]]
            if renormalize:
                chosen = sc[t, at]
                if chosen.sum() <= 0:
                    continue
                dw = (dw - (dw * chosen).sum() / chosen.sum()) / chosen.sum()
            np.add.at(g, at, dw)
            d[t] += softmax[t] * (g - (g * softmax[t]).sum()) if score == "softmax" else g * sc[t] * (1 - sc[t])
    return d
