"""Plain CPU form of the 8-bit layers (numpy, fp64): E4M3 with one fp32 scale
per block of 128.

Per block: amax over its finite values, s = max(fp32(amax / 448), 2^-120),
code = e4m3(clamp(fp32(v * fp32(1 / s)), -448, 448)), nearest, ties to even.
Activations [M, K]: a block is 128 channels of a row, scales [ceil(K/128), M].
Weights, given as [K, N] and stored as [N, K]: a block is 128 x 128, scales
[ceil(N/128), ceil(K/128)]. Codes are handled as the values they stand for.
"""
from __future__ import annotations

import numpy as np

BLOCK = 128
E4M3_MAX = 448.0
SCALE_MIN = 2.0 ** -120


def e4m3_round(t: np.ndarray) -> np.ndarray:
    """Nearest E4M3 value (ties to even mantissa) of fp64 values in [-448,
    448]: the grid around t has the step 2^(e - 3), e = floor(log2 |t|), and
    2^-9 below 2^-6."""
    t = np.asarray(t, np.float64)
    _, e = np.frexp(np.where(np.isfinite(t), t, 0.0))
    step = np.ldexp(1.0, np.maximum(e - 1, -6) - 3)
    return np.rint(t / step) * step


def _scale(amax):
    s = (np.asarray(amax, np.float64) / E4M3_MAX).astype(np.float32)
    return np.maximum(s, np.float32(SCALE_MIN))


def _codes(v, s):
    """v fp64, s fp32 (broadcast): the definition's fp32 roundings in turn."""
    r = (1.0 / s.astype(np.float64)).astype(np.float32)
    with np.errstate(over="ignore", invalid="ignore"):
        t = (v * r.astype(np.float64)).astype(np.float32).astype(np.float64)
    return e4m3_round(np.clip(t, -E4M3_MAX, E4M3_MAX))


def _finite_abs(v):
    return np.where(np.isfinite(v), np.abs(v), 0.0)


def quantize_act(x: np.ndarray):
    """x [M, K] (values of bf16 activations) -> (code values fp64 [M, K], scales fp32 [ceil(K/128), M])."""
    x = np.asarray(x, np.float64)
    M, K = x.shape
    kb = -(-K // BLOCK)
    q, s = np.empty((M, K)), np.empty((kb, M), np.float32)
    for b in range(kb):
        v = x[:, b * BLOCK:(b + 1) * BLOCK]
        s[b] = _scale(_finite_abs(v).max(axis=1))
        q[:, b * BLOCK:(b + 1) * BLOCK] = _codes(v, s[b][:, None])
    return q, s


def quantize_weight(w: np.ndarray):
    """w [K, N] -> (code values fp64 [N, K], scales fp32 [ceil(N/128), ceil(K/128)])."""
    v = np.asarray(w, np.float64).T
    N, K = v.shape
    q, s = np.empty((N, K)), np.empty((-(-N // BLOCK), -(-K // BLOCK)), np.float32)
    for i in range(s.shape[0]):
        for b in range(s.shape[1]):
            at = (slice(i * BLOCK, (i + 1) * BLOCK), slice(b * BLOCK, (b + 1) * BLOCK))
            s[i, b] = _scale(_finite_abs(v[at]).max())
            q[at] = _codes(v[at], s[i, b])
    return q, s


def linear(qx, sx, qw, sw, bias=None):
    """(y, mag, peak): the fp64 product before the activation; the sum of the
    magnitudes of its terms (the scale of fp32 rounding errors); and the sum
    over each 8 consecutive channels of the largest term's magnitude (the
    scale of what a matrix pipe loses that aligns 8 products to the largest)."""
    qx, qw = np.asarray(qx, np.float64), np.asarray(qw, np.float64)
    y, mag, peak = (np.zeros((qx.shape[0], qw.shape[0])) for _ in range(3))
    rows = np.arange(qw.shape[0]) // BLOCK
    for b in range(sx.shape[0]):
        a, c = qx[:, b * BLOCK:(b + 1) * BLOCK], qw[:, b * BLOCK:(b + 1) * BLOCK]
        s = np.asarray(sx[b], np.float64)[:, None] * np.asarray(sw, np.float64)[rows, b][None, :]
        y += (a @ c.T) * s
        mag += (np.abs(a) @ np.abs(c).T) * np.abs(s)
        for k in range(0, a.shape[1], 8):
            top = np.zeros_like(y)
            for i in range(k, min(k + 8, a.shape[1])):
                np.maximum(top, np.abs(a[:, i])[:, None] * np.abs(c[:, i])[None, :], out=top)
            peak += top * np.abs(s)
    if bias is not None:
        y, mag = y + bias, mag + np.abs(bias)
    return y, mag, peak


def rising(offsets, M):
    """Group bounds as the kernels read them: values clamped into [0, M], one
    that falls counting as the largest before it."""
    return np.maximum.accumulate(np.clip(np.asarray(offsets, np.int64), 0, M)).tolist()


def grouped_linear(qx, sx, offsets, qw, sw, bias=None):
    """linear() with group g's weight for the rows offsets[g] .. offsets[g + 1]; other rows are NaN."""
    y = np.full((qx.shape[0], qw.shape[1]), np.nan)
    mag, peak = np.zeros_like(y), np.zeros_like(y)
    for g in range(len(offsets) - 1):
        r = slice(offsets[g], offsets[g + 1])
        y[r], mag[r], peak[r] = linear(qx[r], sx[:, r], qw[g], sw[g], None if bias is None else bias[g])
    return y, mag, peak
