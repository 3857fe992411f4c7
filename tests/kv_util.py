"""Caches, batches and bounds for the tests of the paged 8-bit cache."""
import numpy as np
import torch

from oracle import kv as okv


def bf16(rng, shape, scale=1.0):
    """(bf16 tensor on the CPU, its values)"""
    t = torch.from_numpy(rng.standard_normal(shape) * scale).to(torch.bfloat16)
    return t, t.double().numpy()


def random_state(rng, pages, page, H, D, loud=4.0):
    """A full cache: keys with a few loud channels."""
    W = -(-D // 64) * 64
    out = []
    for side in range(2):
        x = rng.standard_normal((pages, page, H, W))
        if side == 0:
            x *= np.where(rng.random((H, W)) < 0.05, loud, 1.0)
        x[..., D:] = 0.0
        e = okv.exponent(np.abs(x).reshape(pages, page // 16, 16, H, W).max(axis=(2, 4)))
        out.append((okv.e4m3_round(np.ldexp(x, -np.repeat(e, 16, axis=1)[..., None])), e))
    return [out[0][0], out[1][0], out[0][1], out[1][1]]


def paged(rng, lengths, page, spare=1, width=None):
    """(pages, table): every sequence's pages in any order, -1 past its length."""
    need = [-(-max(0, n) // page) for n in lengths]
    pages = sum(need) + spare
    order = rng.permutation(pages)
    table = np.full((len(lengths), max(need + [0]) if width is None else width), -1, np.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    return pages, table


def cum(counts):
    return np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)


def attend_bound(y, mag, rss, peak):
    """How far an output may be from the definition's.

    A score: the two E4M3 instructions drop what falls 13 bits below the largest
    of 8 products, at most 7 x 2^-13 of it for the queries' first parts and a
    sixteenth of that for what those leave: ds <= 7 x 2^-13 x 17/16 x peak; what
    the second part rounds is below 2^-18 of a query's largest channel, and
    peak x 2^-16 covers it where that channel counts (2^-12 added). A weight is
    then off by the factor e^(2 ds), its exponential by 2^-20. Rounded to
    bf16 it is off by half a step, 2^-8 of itself; those errors are independent
    and bounded, so their sum passes 8 x 2^-8 x sqrt(sum (w v)^2) once in 10^13
    (Hoeffding), and never 2^-8 x sum w |v|. The output rounds by 2^-8 of itself."""
    ds = 2.0 ** -13 * 7 * 17 / 16 * peak[..., None] + 2.0 ** -12
    e = np.expm1(2 * ds) * mag + 2.0 ** -18 * mag + np.minimum(2.0 ** -8 * mag, 8 * 2.0 ** -8 * rss)
    return e * (1 + 2.0 ** -8) + 2.0 ** -8 * np.abs(y) + 1e-30
