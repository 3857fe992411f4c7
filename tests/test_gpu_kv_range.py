"""Attention over the paged 8-bit cache at the ends of fp32's range: scales that
are huge, scores far below zero, in both kernels, whole and in pieces. The
oracle has all of them in 64 bits."""
import numpy as np
import pytest
import torch

from gpu_util import note
from kv_util import bf16, cum, paged, random_state
from test_gpu_kv import cache_of, dev, run_attend

pytestmark = pytest.mark.gpu

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
@pytest.mark.parametrize("up", [27, 28, 60, 105])
def test_large_scales(i, up):
    """scale = 2^up over queries as much smaller: the scaled scores are the usual ones, and a query that
    sees nothing gives zeros. (q 2^-105 keeps all bits: a row's exponent is at least -120, its second
    parts' step 2^-129.) The largest scale of all, over queries of zeros, gives the mean."""
    note(f"kv scale 2^{up} {SHAPES[i]}")
    state, table, lengths, offs, q, qv, H, causal, window = case(i, 64, hidden=True)
    f = 2.0 ** -up
    run_attend(cache_of(state, H, 64, 64), state, (q.double() * f).bfloat16().cuda(), qv * f, table, lengths, offs, causal, window,
               scale=2.0 ** up / 8)
    run_attend(cache_of(state, H, 64, 64), state, torch.zeros_like(q).cuda(), 0 * qv, table, lengths, offs, causal, window,
               scale=2.0 ** 127 / 1.5)


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
