"""Rotary positions and head norms in 64 bits, written from the formulas (test helper)."""
import math

import numpy as np


def frequencies(n, base, scaling=0, factor=1.0, original=0):
    """Radians per position of the n pairs of an axis, and the gain on cosines and sines."""
    i = np.arange(n, dtype=np.float64)
    if scaling == 2:
        base = base * factor ** (n / (n - 1))
    f = base ** (-i / n)
    if scaling == 1:
        f = f / factor
    gain = 1.0
    if scaling == 3:
        w = np.clip((original * f / (2 * math.pi) - 1) / 31, 0, 1)
        f = f * (w + (1 - w) / factor)
        gain = 0.1 * math.log(factor) + 1
    return f, gain


def pair_columns(rot, axes, layout):
    """(first, second) value of every rotated pair, the pairs axis by axis."""
    n = rot // 2 // axes
    first = [ax * 2 * n + (i if layout == 0 else 2 * i) for ax in range(axes) for i in range(n)]
    second = [c + (n if layout == 0 else 1) for c in first]
    return np.array(first), np.array(second)


def rotate(x, pos, rot, axes, layout, base, scaling=0, factor=1.0, original=0):
    """x [rows, heads, D] float64, pos [axes, rows] -> rotated x, and |a| + |b| of each value's pair."""
    n = rot // 2 // axes
    f, gain = frequencies(n, base, scaling, factor, original)
    t = np.concatenate([pos[a].astype(np.float64)[:, None] * f for a in range(axes)], axis=1)[:, None, :]
    c, s = gain * np.cos(t), gain * np.sin(t)
    i, j = pair_columns(rot, axes, layout)
    y, size = x.copy(), np.abs(x)
    y[..., i] = x[..., i] * c - x[..., j] * s
    y[..., j] = x[..., j] * c + x[..., i] * s
    size[..., i] = size[..., j] = gain * (np.abs(x[..., i]) + np.abs(x[..., j]))
    return y, size


def head_norm(x, gamma, norm, eps):
    if norm == 1:
        x = x - x.mean(-1, keepdims=True)
    return x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * gamma
