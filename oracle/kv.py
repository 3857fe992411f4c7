"""Plain CPU form of the paged 8-bit cache of keys and values and of attention
over it (numpy, fp64).

Codes are handled as the values they stand for, by token: [pages, page, heads,
64 C] with an exponent per block of 16 tokens, [pages, page / 16, heads].
pack() and unpack() translate to and from the library's bytes.
"""
from __future__ import annotations

import numpy as np

from .fp8 import E4M3_MAX, e4m3_round

EXP_MIN = -120


def e4m3_values() -> np.ndarray:
    """The 256 codes' values: sign, 4 exponent bits (bias 7), 3 of mantissa; 0x7f and 0xff are NaN."""
    c = np.arange(256)
    e, m = (c >> 3) & 15, c & 7
    v = np.where(e == 0, np.ldexp(m / 8.0, -6), np.ldexp(1.0 + m / 8.0, e - 7))
    v = np.where((c & 127) == 127, np.nan, v)
    return np.where(c & 128, -v, v)


_VALUES = e4m3_values()
_ORDER = np.argsort(_VALUES[:127], kind="stable")


def encode(v: np.ndarray) -> np.ndarray:
    """E4M3 bytes of values that are on the grid (zeros without sign; NaN 0x7f)."""
    v = np.asarray(v, np.float64)
    a = np.where(np.isnan(v), 0.0, np.abs(v))
    i = np.searchsorted(_VALUES[:127], a)
    assert (_VALUES[:127][i] == a).all(), "a value off the grid"
    c = i.astype(np.uint8) | np.where(np.signbit(v) & (a > 0), 128, 0).astype(np.uint8)
    return np.where(np.isnan(v), 127, c).astype(np.uint8)


def layout(C: int):
    """(token of the block, channel) of every byte of a block's C runs, keys and values."""
    j, c = np.arange(1024)[None, :], np.arange(C)[:, None]
    keys = (np.broadcast_to(j // 16 % 16, (C, 1024)), 64 * c + 16 * (j // 256) + j % 16)
    values = (np.broadcast_to(4 * (j // 256) + j % 4, (C, 1024)), 64 * c + 16 * (j // 4 % 4) + j // 16 % 16)
    return keys, values


def pack(k, v, ke, ve):
    """Values on the grid (before their exponents) [pages, page, H, 64 C] and exponents -> data, scales bytes."""
    pages, page, H, W = k.shape
    C = W // 64
    data = np.empty((pages, H, page // 64, 2, 4, C, 1024), np.uint8)
    scales = np.empty((pages, H, page // 64, 2, 4), np.uint8)
    for side, (x, e) in enumerate(((k, ke), (v, ve))):
        t, d = layout(C)[side]
        b = encode(x).reshape(pages, page // 64, 4, 16, H, W).transpose(0, 4, 1, 2, 3, 5)
        data[:, :, :, side] = b[:, :, :, :, t, d]
        scales[:, :, :, side] = (e.reshape(pages, page // 64, 4, H).transpose(0, 3, 1, 2) + 127).astype(np.uint8)
    return data, scales


def unpack(data, scales):
    """The library's bytes -> (k, v, ke, ve) as pack() takes them."""
    pages, H, tiles, _, _, C, _ = data.shape
    out = []
    for side in range(2):
        t, d = layout(C)[side]
        x = np.empty((pages, H, tiles, 4, 16, 64 * C))
        x[:, :, :, :, t, d] = _VALUES[data[:, :, :, side]]
        out.append(x.transpose(0, 2, 3, 4, 1, 5).reshape(pages, tiles * 64, H, 64 * C))
    for side in range(2):
        out.append(scales[:, :, :, side].astype(np.int64).transpose(0, 2, 3, 1).reshape(pages, tiles * 4, H) - 127)
    return tuple(out)


def exponent(amax):
    """Least e with amax <= 448 * 2^e, at least EXP_MIN."""
    m, x = np.frexp(np.asarray(amax, np.float64))
    e = np.where(m <= 0.875, x - 9, x - 8)
    return np.where(np.asarray(amax) > 0, np.maximum(e, EXP_MIN), EXP_MIN)


def rising(offsets, T):
    return np.maximum.accumulate(np.clip(np.asarray(offsets, np.int64), 0, T))


def append(state, k, v, table, lengths, offsets):
    """state (k, v, ke, ve) of unpack(), written in place: the call's keys
    (already normed and rotated) and values [T, H, D]. Returns {(page, block):
    (first slot of the call, one past its last)}."""
    touched = {}
    pages, page, H, W = state[0].shape
    off = rising(offsets, k.shape[0])
    for b in range(table.shape[0]):
        n, length = int(off[b + 1] - off[b]), max(0, int(lengths[b]))
        start = length - n
        for blk in range(max(start, 0) // 16, -(-length // 16)):
            if n == 0 or blk * 16 >= table.shape[1] * page:
                continue
            p = int(table[b, blk * 16 // page])
            if not 0 <= p < pages:
                continue
            s0, s1 = max(max(start, 0) - blk * 16, 0), min(length - blk * 16, 16)
            if s1 <= s0:
                continue
            at = blk * 16 % page
            touched[(p, at // 16)] = (s0, s1)
            rows = slice(int(off[b]) + blk * 16 + s0 - start, int(off[b]) + blk * 16 + s1 - start)
            for side, x in enumerate((k, v)):
                x = np.asarray(x[rows], np.float64)                         # [s1 - s0, H, D]
                e = exponent(np.where(np.isfinite(x), np.abs(x), 0.0).max(axis=(0, 2)))
                old = state[2 + side][p, at // 16]
                e = np.maximum(e, old) if s0 > 0 else e
                block = state[side][p, at:at + 16]
                block[:s0] = e4m3_round(np.ldexp(block[:s0], (old - e)[None, :, None]))
                block[s0:] = 0.0
                block[s0:s1, :, :x.shape[2]] = e4m3_round(np.clip(np.ldexp(x, -e[None, :, None]), -E4M3_MAX, E4M3_MAX))
                state[2 + side][p, at // 16] = e
    return touched


def read(state, table, n):
    """(keys, values, present) of the first n tokens of a sequence with pages `table`: [n, H, 64 C] each."""
    pages, page, H, W = state[0].shape
    t = np.arange(min(n, len(table) * page))
    p = np.asarray(table, np.int64)[t // page] if len(t) else np.zeros(0, np.int64)
    there = (p >= 0) & (p < pages)
    p = np.where(there, p, 0)
    return (*(np.ldexp(state[i][p, t % page], state[2 + i][p, t % page // 16][..., None]) for i in range(2)), there)


def attend(state, q, table, lengths, offsets, causal=True, window=0, scale=None):
    """(y, mag, rss, peak): the outputs, NaN for tokens of no sequence; sum_j w_j
    |v_j|; sqrt(sum_j (w_j v_j)^2); and per (token, head) the largest over the
    keys seen of the sum over each 8 consecutive channels of the largest
    |scale q_d k_d| (the scale of what a matrix pipe loses that aligns 8
    products to the largest)."""
    q = np.asarray(q, np.float64)
    T, hq, D = q.shape
    H = state[0].shape[2]
    scale = 1.0 / np.sqrt(D) if scale is None else scale
    y = np.full(q.shape, np.nan)
    mag, rss, peak = np.zeros(q.shape), np.zeros(q.shape), np.zeros((T, hq))
    off = rising(offsets, T)
    for b in range(table.shape[0]):
        n, length = int(off[b + 1] - off[b]), max(0, int(lengths[b]))
        k, v, there = read(state, table[b], length)
        at = np.arange(k.shape[0])
        for i in range(n):
            t, pos = int(off[b]) + i, length - n + i
            seen = there & (at < (pos + 1 if causal else length))
            if window:
                seen = seen & (at > pos - window)
            for h in range(hq):
                kh, vh = k[seen, h // (hq // H), :D], v[seen, h // (hq // H), :D]
                if not len(kh):
                    y[t, h] = 0.0
                    continue
                prod = scale * q[t, h] * kh
                s = prod.sum(axis=1)
                w = np.exp(s - s.max())
                w /= w.sum()
                y[t, h] = w @ vh
                mag[t, h] = w @ np.abs(vh)
                rss[t, h] = np.sqrt((w * w) @ (vh * vh))
                pad = np.zeros((len(kh), -(-D // 8) * 8))
                pad[:, :D] = np.abs(prod)
                peak[t, h] = pad.reshape(len(kh), -1, 8).max(axis=2).sum(axis=1).max()
    return y, mag, rss, peak
