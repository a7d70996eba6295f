"""Float64 oracle of the operators around the block: norm + modulation, gated
residual, and the dual GEMM's epilogue.  Plain NumPy on float64 values, with no
rounding; the caller rounds or bounds."""
from __future__ import annotations

import numpy as np


def norm(x, kind="layer", weight=None, bias=None, eps=1e-6):
    """Row norm of x [M][K]: (x - mean) / sqrt(var + eps) w + b ("layer"), or
    x / sqrt(mean x^2 + eps) w + b ("rms")."""
    x = np.asarray(x, np.float64)
    mean = x.mean(axis=1, keepdims=True) if kind == "layer" else 0.0
    d = x - mean
    n = d / np.sqrt((d * d).mean(axis=1, keepdims=True) + eps)
    if weight is not None:
        n = n * np.asarray(weight, np.float64)
    if bias is not None:
        n = n + np.asarray(bias, np.float64)
    return n


def rows_of(M, rows, index=None, group=None):
    """Modulation row of each of M tokens, -1 for a padding token."""
    if index is None:
        return np.arange(M) // (group if group is not None else max(M, 1))
    index = np.asarray(index, np.int64)
    return np.where((index >= 0) & (index < rows), index, -1)


def modulate(n, i, scale=None, shift=None):
    """n (1 + scale_i) + shift_i, 0 on padding tokens (i < 0)."""
    h = np.array(n, np.float64)
    k = np.maximum(i, 0)
    if scale is not None:
        h = h * (1.0 + np.asarray(scale, np.float64)[k])
    if shift is not None:
        h = h + np.asarray(shift, np.float64)[k]
    h[np.asarray(i) < 0] = 0.0
    return h


def gated(x, y, i, gate=None):
    """x + gate_i y, x itself on padding tokens."""
    x = np.asarray(x, np.float64)
    y = np.array(y, np.float64)
    if gate is not None:
        y = np.asarray(gate, np.float64)[np.maximum(i, 0)] * y
    y[np.asarray(i) < 0] = 0.0
    return x + y


def activation(v, act="none"):
    v = np.asarray(v, np.float64)
    if act == "gelu":
        return 0.5 * v * (1.0 + np.tanh(np.sqrt(2.0 / np.pi) * (v + 0.044715 * v ** 3)))
    if act == "silu":
        return v / (1.0 + np.exp(-v))
    return v


def epilogue(v, i, bias=None, act="none", gate=None, residual=None):
    """residual + gate_i act(v + bias); padding tokens: the residual (or 0)."""
    v = np.asarray(v, np.float64)
    if bias is not None:
        v = v + np.asarray(bias, np.float64)
    r = np.zeros_like(v) if residual is None else residual
    return gated(r, activation(v, act), i, gate)
