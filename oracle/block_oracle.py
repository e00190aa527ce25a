"""NumPy oracle of the operators around the W4A16 linears in a decoder block (test infrastructure).

Written from the formulas in 64 bits, without the library's code: the row quantizer and product in
8-bit integers, the residual update with its norms, and the mixture-of-experts layer.
"""
from __future__ import annotations

import numpy as np

f16, f32, f64 = np.float16, np.float32, np.float64


def scaled_rows(v, s=None, divide=True):
    """fp16(v / s) or fp16(v * s) through fp32, as the equivalent transform defines it."""
    v = np.asarray(v, f16)
    if s is None:
        return v
    with np.errstate(over="ignore", invalid="ignore", divide="ignore"):
        return (v.astype(f32) / s if divide else v.astype(f32) * s).astype(f16)


def quantize_rows(v):
    """(codes int8, step fp32): step = max|v| / 127 per row, code = rint(RN32(v / step))."""
    a = np.abs(np.asarray(v, f16).astype(f32))
    amax = a.max(axis=1)                                   # NaN propagates
    with np.errstate(invalid="ignore", divide="ignore"):
        step = (amax / f32(127)).astype(f32)
        q = np.rint((np.asarray(v, f16).astype(f32) / step[:, None]).astype(f32))
    live = (amax > 0) & np.isfinite(amax)
    return np.where(live[:, None], q, 0).astype(np.int8), step


def w8a8(xq, sx, wq, sw):
    """The product in exact integers, scaled in 64 bits."""
    acc = np.asarray(xq, f64) @ np.asarray(wq, f64).T      # exact: |acc| < 2^31
    return acc * np.asarray(sx, f64)[:, None] * np.asarray(sw, f64)[None, :]


def residual_norm(y, residual, weight, post_weight=None, gate=None, alpha=1.0, eps=1e-6, s=None):
    """(h, x, t) in 64 bits; t = alpha * gate * post-norm(y), the part that is added to the residual."""
    t = np.asarray(y, f64)
    M = t.shape[0]
    if post_weight is not None:
        t = t / np.sqrt((t * t).mean(1, keepdims=True) + eps) * np.asarray(post_weight, f64)
    if gate is not None:
        t = t * np.repeat(np.asarray(gate, f64), M // gate.shape[0], axis=0)
    t = alpha * t
    h = t + (0.0 if residual is None else np.asarray(residual, f64))
    x = h / np.sqrt((h * h).mean(1, keepdims=True) + eps) * np.asarray(weight, f64)
    return h, x if s is None else x / np.asarray(s, f64), t


def silu(v):
    with np.errstate(over="ignore"):
        return v / (1.0 + np.exp(-v))


def route(x, router, top, renormalize):
    """(ids [T, top], p [T, top]) by the logits in 64 bits, ties to the lowest index; and the smallest
    distance between a chosen logit and one that is not (infinite if all are chosen)."""
    logits = np.asarray(x, f64) @ np.asarray(router, f64).T
    order = np.argsort(-logits, axis=1, kind="stable")
    ids = order[:, :top]
    e = np.exp(logits - logits.max(1, keepdims=True))
    p = np.take_along_axis(e, ids, 1)
    p = p / (p if renormalize else e).sum(1, keepdims=True)
    gap = np.inf
    if top < logits.shape[1]:
        l = np.take_along_axis(logits, order, 1)
        gap = (l[:, top - 1] - l[:, top]).min()
    return ids, p, gap


def moe(x, router, gate_up, down, top, renormalize, h_scale=None):
    """(y, bound) of the layer with dequantized experts gate_up [E, 2I, K], down [E, K, I].

    bound: the error that the definition's roundings allow. Sums of products in fp32 on tensor cores are
    taken as off by at most 2^-18 of the sum of magnitudes, p, SiLU and the division by h_scale as off by
    2^-16; h as off by 2^-20 of its largest value; y is rounded to fp16 at the end."""
    x = np.asarray(x, f64)
    I = down.shape[2]
    ids, p, gap = route(x, router, top, renormalize)
    y, err = np.zeros_like(x), np.zeros_like(x)
    for t in range(x.shape[0]):
        for e, w in zip(ids[t], p[t]):
            gu, mag = gate_up[e] @ x[t], np.abs(gate_up[e]) @ np.abs(x[t])
            g, u = gu[:I], gu[I:]
            s = 1.0 if h_scale is None else np.asarray(h_scale[e], f64)
            h = w * silu(g) * u / s
            sig = 1.0 / (1.0 + np.exp(-np.clip(g, -700, 700)))
            slope = np.abs(sig * (1.0 + g * (1.0 - sig)))
            dh = w / s * 2.0 ** -18 * (slope * np.abs(u) * mag[:I] + np.abs(silu(g)) * mag[I:])
            dh = dh + np.abs(h) * 2.0 ** -16 + np.abs(h).max() * 2.0 ** -20
            a = np.abs(down[e])
            y[t] += down[e] @ h
            err[t] += a @ dh + 2.0 ** -18 * (a @ np.abs(h))
    return y, err + 2.0 ** -11 * (np.abs(y) + err) + 2.0 ** -25, gap
