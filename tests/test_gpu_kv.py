"""GPU parity of the paged 8-bit cache: appending against the fp64 oracle
(codes and exponents exact where the inputs are), attention over it at the
sizes, masks and layouts where it can go wrong."""
import numpy as np
import pytest
import torch

from gpu_util import note
from kv_util import attend_bound, bf16, cum, paged, random_state

pytestmark = pytest.mark.gpu

import bit_quantized_diffusion_svdq_amd as svdq
from oracle import kv as okv, rope as orope


def dev(a, dt=None):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda() if dt is None else torch.from_numpy(np.ascontiguousarray(a)).to(dt).cuda()


def cache_of(state, H, D, page):
    data, scales = okv.pack(*state)
    return svdq.KVCache(data.shape[0], H, D, page_size=page, data=dev(data), scales=dev(scales))


def state_of(cache):
    return list(okv.unpack(cache.data.cpu().numpy(), cache.scales.cpu().numpy()))


# ---------------------------------------------------------------- attention

# counts, tokens before, heads, key heads, D, page, causal, window
ATTEND = [
    ([1], [0], 1, 1, 8, 64, True, 0),
    ([1], [0], 3, 1, 128, 64, False, 0),
    ([1], [76], 24, 24, 128, 64, True, 0),
    ([1, 1, 1], [63, 64, 500], 8, 2, 128, 64, True, 0),
    ([1] * 5, [0, 15, 16, 1000, 333], 12, 1, 64, 128, True, 0),
    ([1, 1], [700, 90], 6, 2, 72, 64, True, 100),
    ([1, 1], [700, 90], 16, 1, 256, 192, False, 0),
    ([1, 1], [700, 90], 3, 3, 136, 64, True, 1),
    ([2, 2], [61, 640], 48, 2, 96, 64, True, 0),
    ([3], [2000], 8, 2, 128, 64, True, 65),
    ([5, 1, 30], [10, 130, 77], 6, 2, 40, 64, True, 0),
    ([5, 1, 30], [10, 130, 77], 6, 2, 200, 64, False, 50),
    ([130, 7], [0, 300], 2, 1, 128, 64, True, 0),
    ([257], [64], 4, 4, 64, 64, True, 0),
    ([100, 300], [1000, 5], 3, 1, 128, 128, True, 130),
    ([130], [1200], 1, 1, 128, 64, False, 0),
    ([140, 70], [10, 333], 2, 2, 256, 64, True, 0),
    ([140, 70], [10, 333], 2, 2, 176, 64, False, 0),
]


def run_attend(cache, state, q, qv, table, lengths, offsets, causal, window, scale=None, uniform=False, **kw):
    got = cache.attend(q, dev(table), dev(np.asarray(lengths, np.int32)), None if uniform else dev(offsets), causal=causal,
                       window=window, scale=scale, **kw)
    torch.cuda.synchronize()
    y, mag, rss, peak = okv.attend(state, qv, table, lengths, offsets, causal, window, scale)
    g = got.double().cpu().numpy()
    there = ~np.isnan(y)
    err, bound = np.abs(g - y)[there], attend_bound(y, mag, rss, peak)[there]
    assert (err <= bound).all(), f"{(~(err <= bound)).sum()} of {err.size} outside the bound, worst {np.nanmax(err / bound):.3g}"
    return got


@pytest.mark.parametrize("case", range(len(ATTEND)))
def test_attend(case):
    counts, before, hq, H, D, page, causal, window = ATTEND[case]
    note(f"kv attend {ATTEND[case]}")
    rng = np.random.default_rng(case)
    lengths = [a + b for a, b in zip(counts, before)]
    pages, table = paged(rng, lengths, page)
    state = random_state(rng, pages, page, H, D)
    q, qv = bf16(rng, (sum(counts), hq, D), 2.0)
    run_attend(cache_of(state, H, D, page), state, q.cuda(), qv, table, lengths, cum(counts), causal, window,
               uniform=len(set(counts)) == 1 and case % 2 == 0)


# ---------------------------------------------------------------- appending

# counts, tokens before, heads, key heads, D, axes, pairing, norm, page, queries
APPEND = [
    ([1], [0], 1, 1, 8, (8,), "interleaved", False, 64, True),
    ([1], [76], 24, 24, 128, (16, 56, 56), "interleaved", True, 64, True),
    ([1, 1, 1], [15, 16, 200], 8, 2, 128, (128,), "half", True, 64, True),
    ([5, 1, 40], [3, 0, 30], 6, 3, 64, (16, 24, 24), "half", False, 64, True),
    ([5, 0, 40], [3, 0, 30], 6, 3, 72, (24, 24, 24), "interleaved", True, 128, False),
    ([17, 64], [15, 64], 6, 2, 96, (32, 32), "half", True, 192, True),
    ([33, 2], [1, 63], 5, 5, 256, (64, 96, 96), "interleaved", True, 64, True),
    ([33, 2], [1, 63], 5, 5, 200, (40, 40), "half", True, 64, True),
    ([20, 3], [7, 9], 4, 1, 128, None, None, False, 64, True),
    ([20, 3], [7, 9], 4, 4, 136, None, None, True, 64, True),
    ([700], [100], 9, 9, 64, (64,), "interleaved", True, 64, True),
    ([1300, 900], [100, 1], 3, 3, 128, (44, 42, 42), "half", False, 128, True),
]


def near(a, b, rel):
    return okv.exponent(a * (1 - rel)), okv.exponent(b * (1 + rel))


def turned(x, pos, dims, pairing, w, eps):
    """(values, what they may be off by): test_gpu_rope's bound, 2^-19 of the pair's magnitudes."""
    v = x if w is None else orope.rms_norm(x, w, eps)
    if dims is None:
        return v, 2.0 ** -21 * np.abs(v) if w is not None else np.zeros_like(v)
    axis, freq = orope.frequencies(dims)
    P = len(freq)
    mag = np.abs(v)
    s = (slice(0, 2 * P, 2), slice(1, 2 * P, 2)) if pairing == "interleaved" else (slice(0, P), slice(P, 2 * P))
    both = mag[..., s[0]] + mag[..., s[1]]
    mag[..., s[0]] = both
    mag[..., s[1]] = both
    return orope.rotate(v, pos, axis, freq, pairing), 2.0 ** -19 * mag


def check_append(cache, was, k, kerr, v, table, lengths, offsets):
    """The cache after a call against the oracle from the state before it.
    Values: bit for bit. Keys: the exponent that the block's largest value
    gives, give or take its error; the code within half a step of the key,
    besides its error (a step is 2^-3 of the value's power of two, 2^-9 at
    the least). What the call does not touch stays."""
    got = state_of(cache)
    ref = [a.copy() for a in was]
    touched = okv.append(ref, k, v, table, lengths, offsets)
    np.testing.assert_array_equal(got[1], ref[1])
    np.testing.assert_array_equal(got[3], ref[3])
    off = okv.rising(offsets, k.shape[0])
    page = was[0].shape[1]
    mask = np.ones(was[0].shape[:2], bool)
    blocks = np.ones(was[2].shape[:2], bool)
    for b in range(table.shape[0]):
        n = int(off[b + 1] - off[b])
        start = int(lengths[b]) - n
        for blk in range(max(start, 0) // 16, -(-int(lengths[b]) // 16)):
            p, at = int(table[b, blk * 16 // page]) if blk * 16 // page < table.shape[1] else -1, blk * 16 % page
            if (p, at // 16) not in touched:
                continue
            s0, s1 = touched[(p, at // 16)]
            mask[p, at:at + 16] = blocks[p, at // 16] = False
            rows = slice(int(off[b]) + blk * 16 + s0 - start, int(off[b]) + blk * 16 + s1 - start)
            x, xe = k[rows], kerr[rows]
            e = got[2][p, at // 16]
            lo = okv.exponent(np.maximum(np.abs(x) - xe, 0).max(axis=(0, 2)))
            hi = okv.exponent((np.abs(x) + xe).max(axis=(0, 2)))
            if s0:
                lo, hi = np.maximum(lo, was[2][p, at // 16]), np.maximum(hi, was[2][p, at // 16])
            assert ((e >= lo) & (e <= hi)).all(), f"page {p} block {at // 16}: exponents {e} outside [{lo}, {hi}]"
            c = got[0][p, at:at + 16]
            want = np.clip(np.ldexp(x, -e[None, :, None]), -448, 448)
            step = np.ldexp(1.0, np.maximum(np.frexp(np.maximum(np.abs(want), 2.0 ** -6))[1] - 1, -6) - 3)
            d = np.abs(c[s0:s1, :, :x.shape[2]] - want)
            assert (d <= step / 2 + np.ldexp(xe, -e[None, :, None]) * 1.01).all(), f"keys off by up to {(d / step).max():.3g} steps"
            assert (c[s1:] == 0).all() and (c[:, :, x.shape[2]:] == 0).all()
            same = e == was[2][p, at // 16]
            np.testing.assert_array_equal(c[:s0], okv.e4m3_round(np.ldexp(was[0][p, at:at + s0], (was[2][p, at // 16] - e)[None, :, None])))
            assert s0 == 0 or (c[:s0, same] == was[0][p, at:at + s0][:, same]).all()
    np.testing.assert_array_equal(got[0][mask], was[0][mask])
    np.testing.assert_array_equal(got[2][blocks], was[2][blocks])


@pytest.mark.parametrize("case", range(len(APPEND)))
def test_append(case):
    counts, before, hq, H, D, dims, pairing, norm, page, queries = APPEND[case]
    note(f"kv append {APPEND[case]}")
    rng = np.random.default_rng(100 + case)
    T, lengths = sum(counts), [a + b for a, b in zip(counts, before)]
    pages, table = paged(rng, lengths, page)
    was = random_state(rng, pages, page, H, D)
    cache = cache_of(was, H, D, page)
    flat, fv = bf16(rng, (T, hq + 2 * H, D), 1.0)
    loud = torch.from_numpy(np.where(rng.random((T, 1, 1)) < 0.2, 6.0, 1.0))     # some blocks grow, some do not
    flat = (flat.double() * loud).to(torch.bfloat16)
    fv = flat.double().numpy()
    q, k, v = flat.cuda().split((hq, H, H), dim=1)
    qv, kv, vv = fv[:, :hq], fv[:, hq:hq + H], fv[:, hq + H:]
    w = [torch.from_numpy(1 + 0.2 * rng.standard_normal(D)).to(torch.bfloat16) if norm else None for _ in range(2)]
    wn = [None if x is None else x.double().numpy() for x in w]
    pos = rng.integers(-500, 4096, (T, 1 if dims is None else len(dims))).astype(np.int32)
    plan = None if dims is None else svdq.RopePlan(dims, head_dim=D, pairing=pairing)
    out = cache.append(k, v, dev(table), dev(np.asarray(lengths, np.int32)), dev(cum(counts)),
                       pos=None if plan is None else dev(pos), plan=plan, k_norm=None if w[1] is None else w[1].cuda(),
                       q=q if queries else None, q_norm=w[0].cuda() if queries and norm else None)
    torch.cuda.synchronize()
    assert queries or out is None
    kr, kerr = turned(kv, pos, dims, pairing, wn[1], 1e-6)
    check_append(cache, was, kr, kerr, vv, table, lengths, cum(counts))
    if queries:
        qr, qerr = turned(qv, pos, dims, pairing, wn[0], 1e-6)
        d = np.abs(out.double().cpu().numpy() - qr)
        assert (d <= qerr * (1 + 2.0 ** -8) + 2.0 ** -8 * np.abs(qr) + 1e-37).all()


def set_code(cache, page, h, token, d, side, code):
    """The byte of one channel of one token."""
    t, ch = okv.layout(cache.data.shape[5])[side]
    at = np.argwhere((t == token % 16) & (ch == d))[0]
    cache.data[page, h, token // 64, side, token % 64 // 16, int(at[0]), int(at[1])] = code


@pytest.mark.parametrize("T,before", [(1, 200), (3, 200), (20, 200), (150, 100)])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_values_that_are_not_finite(T, before, D):
    """A NaN among the keys or values reaches the queries that see it (keys:
    whole outputs, values: their channel) and no others, wherever the order, the
    window or the sequence's end hides it; what lies past the end may be
    anything."""
    note(f"kv attend NaN {T} {before} {D}")
    rng = np.random.default_rng(T + D)
    H, hq, page, window = 2, 4, 128, 150
    n = T + before
    pages, table = paged(rng, [n], page, spare=0)
    state = random_state(rng, pages, page, H, D)
    q, _ = bf16(rng, (T, hq, D))
    q = q.cuda()
    lengths = dev(np.asarray([n], np.int32))
    for causal, win in ((True, 0), (True, window), (False, 0)):
        cache = cache_of(state, H, D, page)
        clean = cache.attend(q, dev(table), lengths, causal=causal, window=win)
        # past the end: every byte a NaN
        for t in range(n, -(-n // page) * page):
            p = int(table[0, t // page])
            for d in range(0, D, 7):
                set_code(cache, p, 0, t % page, d, 0, 0x7F)
                set_code(cache, p, 1, t % page, d, 1, 0xFF)
        assert torch.equal(cache.attend(q, dev(table), lengths, causal=causal, window=win), clean)
        # a NaN value and a NaN key among the tokens
        vt, kt = n - 1 - T // 2, n - 1 - T // 3
        set_code(cache, int(table[0, vt // page]), 0, vt % page, 5, 1, 0x7F)
        set_code(cache, int(table[0, kt // page]), 1, kt % page, 3, 0, 0xFF)
        got = cache.attend(q, dev(table), lengths, causal=causal, window=win)
        want = clean.clone()
        for i in range(T):
            pos = before + i
            sees = lambda t: (not causal or t <= pos) and (not win or t > pos - win)
            if sees(vt):
                want[i, :2, 5] = float("nan")
            if sees(kt):
                want[i, 2:] = float("nan")
        assert torch.equal(got.isnan(), want.isnan())
        assert torch.equal(got.nan_to_num(nan=7.0), want.nan_to_num(nan=7.0))
    # a query that is not finite gives NaN, alone
    bad = q.clone()
    bad[T // 2, 1, 3], bad[0, 3, 0] = float("inf"), float("nan")
    cache = cache_of(state, H, D, page)
    clean, got = (cache.attend(x, dev(table), lengths) for x in (q, bad))
    assert got[T // 2, 1].isnan().all() and got[0, 3].isnan().all()
    got[T // 2, 1], got[0, 3] = clean[T // 2, 1], clean[0, 3]
    assert torch.equal(got, clean)
