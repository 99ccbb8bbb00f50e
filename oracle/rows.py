"""fp64 oracle of the row operators, the 8-bit product and log probabilities (plain numpy).

Test infrastructure only, like the rest of this package: written from the definitions in
``include/nvfp4.h``, sharing no code with the HIP path.
"""
from __future__ import annotations

import numpy as np


def bf16(x):
    """Nearest bf16 of float64 values, ties to even, as float64."""
    x = np.asarray(x, np.float64)
    with np.errstate(all="ignore"):
        _, e = np.frexp(x)
        ulp = np.ldexp(1.0, np.maximum(e, -125) - 8)
        y = np.where(np.isfinite(x), np.rint(x / ulp) * ulp, x)
        return np.where(np.abs(y) >= 2.0 ** 128, np.copysign(np.inf, y), y)


def to_type(x, name):
    """Values of type "bf16" or "f32" nearest to float64 ones."""
    with np.errstate(over="ignore", invalid="ignore"):
        return bf16(x) if name == "bf16" else np.asarray(x, np.float64).astype(np.float32).astype(np.float64)


def rms_norm(x, weight, eps, offset=0.0, residual=None, residual_type=None):
    """(y, h): the norm before its rounding, and the stream as it is stored."""
    h = np.asarray(x, np.float64)
    if residual is not None:
        h = to_type(h + residual, residual_type)
    with np.errstate(all="ignore"):
        r = 1.0 / np.sqrt(np.mean(h * h, axis=1, keepdims=True) + float(np.float32(eps)))
        return h * r * (np.asarray(weight, np.float64) + float(np.float32(offset))), h


def swiglu(x):
    """silu(gate) * up of rows [gate | up], not rounded."""
    g, u = np.split(np.asarray(x, np.float64), 2, axis=1)
    with np.errstate(all="ignore"):
        return g * u / (1.0 + np.exp(-g))


def codes(y):
    """(codes int8, scale float32) of rows."""
    y = np.asarray(y, np.float64)
    with np.errstate(all="ignore"):
        most = np.where(np.isnan(y).any(axis=1), np.nan, np.nanmax(np.where(np.isnan(y), 0, np.abs(y)), axis=1))
        scale = (most / 127.0).astype(np.float32)
        q = np.rint(y / scale.astype(np.float64)[:, None])
    none = ~((scale > 0) & np.isfinite(scale))
    q = np.where(none[:, None], 0.0, q)
    return np.clip(q, -127, 127).astype(np.int8), scale


def int8_gemm(a, a_scale, w, w_scale, bias=None):
    """(y, s): the product, and the sum of magnitudes that its last steps round (w and bias apart)."""
    acc = a.astype(np.float64) @ w.astype(np.float64).T  # whole numbers below 2^53
    y = acc * a_scale.astype(np.float64)[:, None] * w_scale.astype(np.float64)
    s = np.abs(y)
    return (y, s) if bias is None else (y + bias.astype(np.float64), s)


def logprobs(x, tokens, k, scale):
    """(logprob, entropy, top tokens, top log probabilities, lp, E, E2): lp all log probabilities; E and
    E2 the means of |z - max z| and its square under p, for error bounds."""
    x = np.asarray(x, np.float64)
    rows, V = x.shape
    z = x * float(np.float32(scale))
    m = z.max(axis=1, keepdims=True)
    m = np.where(np.isneginf(m), 0.0, m)
    with np.errstate(invalid="ignore"):
        d = z - m
    e = np.exp(d)
    s = e.sum(axis=1, keepdims=True)
    with np.errstate(divide="ignore", invalid="ignore"):
        lp = np.where(s == 0, -np.inf, d - np.log(s))
        fine = np.where(np.isneginf(d), 0.0, d)
        E, E2 = ((e * np.abs(fine) ** i).sum(axis=1) / np.where(s == 0, 1, s)[:, 0] for i in (1, 2))
        entropy = np.where(s[:, 0] == 0, 0.0, np.log(s[:, 0]) + E)
    t = np.asarray(tokens).reshape(rows, -1)
    out = np.where((t >= 0) & (t < V), np.take_along_axis(lp, np.clip(t, 0, V - 1), axis=1), -np.inf)
    order = np.stack([np.lexsort((np.arange(V), -(r + 0.0))) for r in x])[:, :k] if rows else np.zeros((0, k), int)
    return out, entropy, order, np.take_along_axis(lp, order, axis=1), lp, E, E2
