"""Attention over the paged 8-bit cache at the ends of fp32's range: scales that
are huge, scores far below zero, in both kernels, whole and in pieces. The
oracle has all of them in 64 bits."""
import numpy as np
import pytest
import torch

from gpu_util import note
from kv_util import attend_bound, bf16, cum, paged, random_state
from test_gpu_kv import cache_of, dev, run_attend, state_of

pytestmark = pytest.mark.gpu

import bit_quantized_diffusion_svdq_amd as svdq
from oracle import kv as okv

# counts, tokens before, heads, key heads, causal, window: few rows, with pieces; more, with and without splits
SHAPES = [
    ([2], [127], 2, 1, True, 0),
    ([1, 1, 1], [0, 700, 64], 4, 2, True, 90),
    ([3], [2600], 2, 1, True, 0),
    ([40, 2], [100, 5], 2, 2, False, 30),
    ([130], [0], 1, 1, True, 0),
    ([150, 7], [30, 900], 2, 1, True, 70),
    ([140], [1900], 2, 1, True, 0),
]


def case(i, D, hidden=False):
    """A cache, its batch and queries; hidden: some queries see nothing (a missing page, tokens before
    position 0)."""
    counts, before, hq, H, causal, window = SHAPES[i]
    rng = np.random.default_rng(1000 + i)
    lengths = [a + b for a, b in zip(counts, before)]
    pages, table = paged(rng, lengths, 64)
    state = random_state(rng, pages, 64, H, D)
    if hidden:
        table[-1, :1] = -1
        lengths[0] -= min(counts[0], before[0] + 1, 9)       # (fewer tokens than the call has of it, or none before)
    q, qv = bf16(rng, (sum(counts), hq, D))
    return state, table, lengths, cum(counts), q, qv, H, causal, window


@pytest.mark.parametrize("i", range(len(SHAPES)))
@pytest.mark.parametrize("D", [64, 200])
@pytest.mark.parametrize("up", [27, 28, 60, 105])
def test_large_scales(i, D, up):
    """scale = 2^up over queries as much smaller: the scaled scores are the usual ones, and a query that
    sees nothing gives zeros. (q 2^-105 keeps all bits: a row's exponent is at least -120, its second
    parts' step 2^-129.) The largest scale of all, over queries of zeros, gives the mean."""
    note(f"kv scale 2^{up} {SHAPES[i]} {D}")
    state, table, lengths, offs, q, qv, H, causal, window = case(i, D, hidden=True)
    f = 2.0 ** -up
    run_attend(cache_of(state, H, D, 64), state, (q.double() * f).bfloat16().cuda(), qv * f, table, lengths, offs, causal, window,
               scale=2.0 ** up / 8)
    run_attend(cache_of(state, H, D, 64), state, torch.zeros_like(q).cuda(), 0 * qv, table, lengths, offs, causal, window,
               scale=2.0 ** 127 / 1.5)


@pytest.mark.parametrize("i", range(len(SHAPES)))
@pytest.mark.parametrize("D", [64, 200])
@pytest.mark.parametrize("scale", [2.0 ** -149, 2.0 ** -126, 1e-30])
def test_least_scales(i, D, scale):
    """Weights are all alike, and what is hidden has none."""
    note(f"kv scale {scale} {SHAPES[i]} {D}")
    state, table, lengths, offs, q, qv, H, causal, window = case(i, D, hidden=True)
    run_attend(cache_of(state, H, D, 64), state, q.cuda(), qv, table, lengths, offs, causal, window, scale=scale)


@pytest.mark.parametrize("i", range(len(SHAPES)))
@pytest.mark.parametrize("up", [20, 45])
def test_scores_far_below_zero(i, up):
    """Every score finite and below -1e30 (keys below zero, queries above), the scale as small: a mean of
    values as any other. With scaled scores in the thousands, over values that are all the same, it is that
    value: the weights' sum is the weighted values' divided by it, whatever the weights are."""
    note(f"kv scores below -1e30, 2^{up} {SHAPES[i]}")
    state, table, lengths, offs, q, qv, H, causal, window = case(i, 64)
    state[0] = -np.abs(state[0])
    state[2] = state[2] + 65
    q = (q.double().abs() + 1) * 2.0 ** up
    q = q.bfloat16()
    qv = q.double().numpy()
    there = [p for row in table for p in row if p >= 0]
    keys = np.ldexp(state[0], np.repeat(state[2], 16, axis=1)[..., None])[there].sum(axis=3)
    assert (keys.max() * 2.0 ** up < -1e30) == (up == 45)      # (20: the same work where nothing is extreme)
    run_attend(cache_of(state, H, 64, 64), state, q.cuda(), qv, table, lengths, offs, causal, window, scale=2.0 ** (-65 - up) / 8)
    state[1][:] = state[1][:1, :1]
    state[3][:] = 0
    want = torch.from_numpy(state[1][0, 0]).cuda().bfloat16().repeat_interleave(q.shape[1] // H, 0)
    got = cache_of(state, H, 64, 64).attend(q.cuda(), dev(table), dev(np.asarray(lengths, np.int32)), dev(offs), causal=causal,
                                            window=window, scale=2.0 ** (-57 - up))
    assert torch.equal(got, want.expand_as(got))


@pytest.mark.parametrize("i", range(len(SHAPES)))
def test_values_near_the_largest(i):
    """bf16's largest values go into the cache as 2^128. Queries that do not see them do not change; those
    that do have them by their weight."""
    note(f"kv largest values {SHAPES[i]}")
    counts, before, hq, H, causal, window = SHAPES[i]
    state, table, lengths, offs, q, qv, *_ = case(i, 64)
    rng = np.random.default_rng(i)
    caches = [cache_of(state, H, 64, 64) for _ in range(2)]
    kv = [bf16(rng, (sum(lengths), H, 64))[0].cuda() for _ in range(2)]
    big = kv[1].clone()
    at = []
    for b, n in enumerate(lengths):                       # (the last ones: early queries do not see them)
        first = int(cum(lengths)[b])
        for t in (n - 1, n - counts[b] // 2 - 1):
            big[first + t, 0, 5], big[first + t, 0, 6] = 3.38e38, -3.38e38
            at.append((b, t))
    for cache, v in zip(caches, (kv[1], big)):
        cache.append(kv[0], v, dev(table), dev(np.asarray(lengths, np.int32)), dev(cum(lengths)))
    args = (dev(table), dev(np.asarray(lengths, np.int32)), dev(offs))
    q, qv = (0.1 * q).bfloat16(), (0.1 * q).bfloat16().double().numpy()
    clean, got = (c.attend(q.cuda(), *args, causal=causal, window=window) for c in caches)
    y = okv.attend(state_of(caches[1]), qv, table, lengths, offs, causal, window)[0]
    fits = np.abs(y) < 2.0 ** 126                         # (a row of a few keys: past bf16)
    assert torch.equal(got.isfinite() | ~torch.from_numpy(fits).cuda(), torch.ones_like(got, dtype=torch.bool))
    g, bound = got.double().cpu().numpy(), attend_bound(*okv.attend(state_of(caches[1]), qv, table, lengths, offs, causal, window))
    assert (np.abs(g - y)[fits] <= bound[fits]).all()
    # what sees none of them, and the channels beside them but for their block's coarser steps, is as it was
    other = torch.ones(hq, dtype=torch.bool)
    other[:hq // H] = False
    assert torch.equal(got[:, other], clean[:, other])
    hidden = 0
    for b in range(len(counts)):
        for r in range(counts[b]):
            pos = lengths[b] - counts[b] + r
            sees = [t for bb, t in at if bb == b and (t <= pos if causal else True) and not (window and t <= pos - window)]
            same = not sees and not [t for bb, t in at if bb == b and t // 16 <= pos // 16]   # (nor their blocks' steps)
            hidden += same
            if same:
                assert torch.equal(got[int(offs[b]) + r], clean[int(offs[b]) + r])
    assert hidden or max(counts) < 32 or not causal


@pytest.mark.parametrize("i", range(len(SHAPES)))
@pytest.mark.parametrize("D", [64, 200])
def test_large_values_under_large_weights(i, D):
    """Weights are taken from a reference up to 2^8 below the largest, and values of 2^120 are read under them."""
    note(f"kv large values {SHAPES[i]} {D}")
    state, table, lengths, offs, q, qv, H, causal, window = case(i, D)
    state[3] = state[3] + 121
    run_attend(cache_of(state, H, D, 64), state, q.cuda(), qv, table, lengths, offs, causal, window)
    # the least exponents: bf16's own step is 2^-133, that of a 64th of the values
    state[3] = np.maximum(state[3] - 121 - 113, okv.EXP_MIN)
    y, mag, rss, peak = okv.attend(state, qv, table, lengths, offs, causal, window)
    got = cache_of(state, H, D, 64).attend(q.cuda(), dev(table), dev(np.asarray(lengths, np.int32)), dev(offs), causal=causal,
                                            window=window).double().cpu().numpy()
    assert (np.abs(got - y) <= attend_bound(y, mag, rss, peak) - 1e-30 + 2.0 ** -127).all()


@pytest.mark.parametrize("T,hq", [(2, 2), (40, 2)])
def test_exponents_that_no_append_writes(T, hq):
    """A values' byte above 247 counts as 247, under attention and where a block is gone on with."""
    note(f"kv exponents {T} {hq}")
    rng = np.random.default_rng(T)
    n, D = 150, 64
    pages, table = paged(rng, [n], 64)
    state = random_state(rng, pages, 64, 1, D)
    state[1] = np.where(state[1] >= 0, 2.0 ** -6, -2.0 ** -6)
    state[3][:] = 120
    caches = [cache_of(state, 1, D, 64) for _ in range(2)]
    caches[1].scales[:, :, :, 1, ::2] = 255
    caches[1].scales[:, :, :, 1, 1::2] = 248
    q, qv = bf16(rng, (T, hq, D))
    args = (dev(table), dev(np.asarray([n], np.int32)))
    a, b = (c.attend(q.cuda(), *args) for c in caches)
    assert torch.equal(a, b) and a.isfinite().all()
    run_attend(caches[0], state, q.cuda(), qv, table, [n], cum([T]), True, 0)
    k, v = (bf16(rng, (7, 1, D), 2.0 ** 118)[0].cuda() for _ in range(2))
    for c, byte in zip(caches, (247, 255)):
        c.scales[:] = byte
        c.append(k, v, *args)
    p, at = int(table[0, (n - 7) // 64]), (n - 7) % 64
    assert torch.equal(caches[0].data, caches[1].data)
    for c in caches:
        assert (c.scales[p, 0, 0, :, at // 16] == 247).all()


@pytest.mark.parametrize("D", [8, 40, 72, 136, 200])
@pytest.mark.parametrize("turns", [False, True])
def test_channels_past_the_head(D, turns):
    """They stay zeros where a key's norm is a NaN as well (a NaN or, with eps 0, a key of zeros)."""
    note(f"kv channels past {D}")
    T, H = 40, 2
    cache = svdq.KVCache(1, H, D)
    k = torch.randn(T, H, D, generator=torch.Generator().manual_seed(D)).bfloat16()
    k[3, 0, 1], k[20, 1, D - 1], k[7, 1], k[33] = float("nan"), float("inf"), 0.0, float("nan")
    k = k.cuda()
    more = dict(pos=torch.ones(T, 1, dtype=torch.int32, device="cuda"), plan=svdq.RopePlan((8,), head_dim=D)) if turns else {}
    for eps in (1e-6, 0.0):
        cache.data.zero_()
        cache.append(k, k, dev(np.zeros((1, 1), np.int32)), dev(np.asarray([T], np.int32)), eps=eps,
                     k_norm=torch.ones(D, dtype=torch.bfloat16, device="cuda"), **more)
        keys, values, *_ = state_of(cache)
        assert (keys[..., D:] == 0).all() and (values[..., D:] == 0).all() and (keys[0, T:] == 0).all()
        assert np.isnan(keys[0, 3, 0, :D]).all() and np.isnan(keys[0, 7, 1, :D]).all() == (eps == 0.0)
        assert np.isnan(keys[0, 20, 1, D - 1]) and np.isnan(values[0, 33, 0, :D]).all()
