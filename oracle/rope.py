"""Plain CPU form of the rotary positions with several axes (numpy, fp64)."""
from __future__ import annotations

import numpy as np


def frequencies(dims, theta=10000.0):
    """(axis, angular frequency) of every pair: axis a of width d has theta^(-2 i / d), i = 0 .. d / 2 - 1."""
    axis = np.array([a for a, d in enumerate(dims) for _ in range(d // 2)], np.int64)
    freq = np.array([theta ** (-2.0 * i / d) for d in dims for i in range(d // 2)], np.float64)
    return axis, freq


def rms_norm(x, w, eps):
    x = np.asarray(x, np.float64)
    return x / np.sqrt((x * x).mean(axis=-1, keepdims=True) + eps) * np.asarray(w, np.float64)


def rotate(x, pos, axis, freq, pairing="interleaved", inverse=False):
    """x [T, H, D], pos [T, axes] -> the rotated heads (values past the pairs as they are)."""
    y = np.array(x, np.float64)
    P = len(freq)
    if P == 0:
        return y
    angle = np.asarray(pos, np.float64)[:, axis] * freq
    c, s = np.cos(angle)[:, None, :], np.sin(-angle if inverse else angle)[:, None, :]
    first, second = (slice(0, 2 * P, 2), slice(1, 2 * P, 2)) if pairing == "interleaved" else (slice(0, P), slice(P, 2 * P))
    a, b = y[..., first].copy(), y[..., second].copy()
    y[..., first], y[..., second] = a * c - b * s, a * s + b * c
    return y
