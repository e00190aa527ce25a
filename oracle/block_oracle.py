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
