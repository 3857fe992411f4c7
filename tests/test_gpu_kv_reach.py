"""What the attention kernels reach, beside the bounds that no output may pass
(kv_util): their rms error, one key that takes all, a loud query channel; and
batches whose kernel or plan goes by something else than their sequences: single
tokens and a prompt in one call, tables far wider than what is stored."""
import numpy as np
import pytest
import torch

from gpu_util import note
from kv_util import attend_bound, bf16, cum, paged, random_state
from test_gpu_kv import cache_of, dev, run_attend

pytestmark = pytest.mark.gpu

import bit_quantized_diffusion_svdq_amd as svdq
from oracle import kv as okv


def batch(seed, counts, before, hq, H, D, loud=4.0, q_scale=1.0, page=64, width=None):
    rng = np.random.default_rng(seed)
    lengths = [a + b for a, b in zip(counts, before)]
    pages, table = paged(rng, lengths, page, width=width)
    state = random_state(rng, pages, page, H, D, loud=loud)
    q, qv = bf16(rng, (sum(counts), hq, D), q_scale)
    return state, table, lengths, cum(counts), q, qv


@pytest.mark.parametrize("counts,before,hq,H,D", [
    ([1] * 12, [700, 90, 333, 800, 20, 64, 500, 410, 77, 128, 900, 256], 16, 4, 128), ([30], [400], 4, 4, 64), ([150], [300], 2, 2, 128),
    ([100, 60], [40, 500], 3, 1, 256), ([140], [100], 2, 1, 72), ([2], [4000], 24, 2, 128)])
def test_rms(counts, before, hq, H, D):
    """Errors that are independent from key to key add up by their squares. bf16 weights: half a step is 2^-8
    of a weight at the most, evenly spread errors have rms 2^-8 / sqrt(3) of it, and rss = sqrt(sum (w v)^2)
    takes them; a score: of each 8 products 7 may lose up to 2^-13 of the largest, of either sign: rms
    sqrt(7 / 3) 2^-13 17/16 sqrt(sum over the eights) <= the same of `peak`, and as much of a weight; the
    output's own rounding, 2^-8 / sqrt(3) of it. A weight's error is all channels' of its row, so as many
    errors are independent as there are (token, head) rows: 1.5 leaves six deviations of the mean over 150."""
    note(f"kv rms {counts[:3]} {D}")
    state, table, lengths, offs, q, qv = batch(D + len(counts), counts, before, hq, H, D)
    y, mag, rss, peak = okv.attend(state, qv, table, lengths, offs, True, 0)
    got = cache_of(state, H, D, 64).attend(q.cuda(), dev(table), dev(np.asarray(lengths, np.int32)), dev(offs))
    err = got.double().cpu().numpy() - y
    weight = 2.0 ** -16 / 3 + 7 / 3 * (2.0 ** -13 * 17 / 16 * peak[..., None]) ** 2
    want = np.sqrt((weight * rss ** 2 + 2.0 ** -16 / 3 * y ** 2).mean())
    rms = np.sqrt((err ** 2).mean())
    print(f"rms error {rms:.3g}, {rms / np.sqrt((y ** 2).mean()):.3g} of the outputs', expected at most {want:.3g}")
    assert rms <= 1.5 * want


@pytest.mark.parametrize("counts,before,hq,H,D,scale,loud", [
    ([1], [300], 5, 1, 128, 30.0, 40.0), ([37], [100], 5, 1, 128, 30.0, 40.0), ([150], [300], 2, 2, 64, 8.0, 60.0), ([2], [5000], 4, 2, 64, 20.0, 30.0)])
def test_one_key_takes_all(counts, before, hq, H, D, scale, loud):
    """Where the largest score leads by more than twice what scores are off by and 60 (a factor of e^60), the
    output is that key's value, bit for bit: it has four significant bits."""
    note(f"kv one key {counts} {D}")
    state, table, lengths, offs, q, qv = batch(D + len(counts), counts, before, hq, H, D, loud=loud)
    got = cache_of(state, H, D, 64).attend(q.cuda(), dev(table), dev(np.asarray(lengths, np.int32)), scale=scale).double().cpu().numpy()
    keys, values, _ = okv.read(state, table[0], lengths[0])
    took = 0
    for t in range(counts[0]):
        pos = lengths[0] - counts[0] + t
        for h in range(hq):
            prod = scale * qv[t, h] * keys[:pos + 1, h // (hq // H), :D]
            s = prod.sum(axis=1)
            off = 7 * 2.0 ** -13 * 17 / 16 * np.abs(prod).reshape(len(s), -1, 8).max(axis=2).sum(axis=1).max()
            off += scale * np.abs(qv[t, h]).max() * 2.0 ** -10 / 224 * np.abs(keys[:pos + 1, h // (hq // H), :D]).sum(axis=1).max()
            first, second = np.sort(s)[-1:-3:-1]
            if first - second > 2 * off + 60:
                took += 1
                assert (got[t, h] == values[s.argmax(), h // (hq // H), :D]).all(), f"token {t} head {h}"
    assert took >= counts[0] * hq // 2, f"{took} rows"


@pytest.mark.parametrize("loud", [2.0 ** 6, 2.0 ** 8])
@pytest.mark.parametrize("T,D", [(1, 64), (3, 128), (150, 128), (150, 200)])
def test_loud_query_channel(T, D, loud):
    """A query channel that dwarfs the rest, over keys that are zeros there. A query is two E4M3 numbers over
    its row's power of two, the second's least step 2^-9, so a channel is off by up to 2^-10 of 1 / 224 of the
    row's largest (exact where bf16's last bit is no finer than that step: from 1 / 896 of the largest on)."""
    note(f"kv loud query {T} {D} {loud}")
    state, table, lengths, offs, q, qv = batch(T + D, [T], [200], 4, 2, D)
    state[0][..., 3] = 0.0
    q[..., 3] = loud
    qv = q.double().numpy()
    got = cache_of(state, 2, D, 64).attend(q.cuda(), dev(table), dev(np.asarray(lengths, np.int32))).double().cpu().numpy()
    y, mag, rss, peak = okv.attend(state, qv, table, lengths, offs)
    keys = np.ldexp(state[0], np.repeat(state[2], 16, axis=1)[..., None])
    most = np.abs(keys).sum(axis=3).max()
    extra = loud * 2.0 ** -10 / 224 * most / np.sqrt(D)
    bound = attend_bound(y, mag, rss, peak + extra / (2.0 ** -13 * 7 * 17 / 16))
    assert (np.abs(got - y) <= bound).all()
    # all other channels a 512th of it and more: as exact as without it
    q = torch.where(q == loud, q, torch.copysign(q.abs().clamp(min=loud / 512), q))
    qv = q.double().numpy()
    run_attend(cache_of(state, 2, D, 64), state, q.cuda(), qv, table, lengths, offs, True, 0)


@pytest.mark.parametrize("singles,prompt,hq,H,window", [
    (20, 300, 2, 1, 0),                                   # 32 rows a sequence on the average: the few-rows kernel, with a prompt
    (21, 600, 1, 1, 70), (70, 1000, 4, 2, 0),
    (3, 300, 2, 1, 0), (9, 500, 3, 1, 70), (70, 1200, 4, 2, 0)])     # more: single tokens in row tiles of 128
def test_single_tokens_and_a_prompt(singles, prompt, hq, H, window):
    note(f"kv mixed {singles} {prompt} {hq}")
    rng = np.random.default_rng(singles)
    at = singles // 2
    counts = [1] * at + [prompt] + [1] * (singles - at)
    before = rng.integers(0, 400, singles + 1).tolist()
    state, table, lengths, offs, q, qv = batch(singles, counts, before, hq, H, 64)
    run_attend(cache_of(state, H, 64, 64), state, q.cuda(), qv, table, lengths, offs, True, window)


@pytest.mark.parametrize("T,hq,H,width,splits", [(1, 4, 2, 4096, 0), (300, 4, 2, 4096, 10), (140, 2, 2, 2048, 10), (512, 4, 4, 2048, 3)])
@pytest.mark.parametrize("before", [0, 700])
def test_tables_far_wider(T, hq, H, width, splits, before):
    """Room for 131072 tokens and more, a few hundred there: most pieces and splits of the plan, which knows
    the table's width only, are empty."""
    note(f"kv wide table {T} {width} {before}")
    D = 64
    state, table, lengths, offs, q, qv = batch(T, [T], [before], hq, H, D, width=width)
    cache = cache_of(state, H, D, 64)
    if splits:
        groups = -(-T * (hq // H) // 128) * H
        need = svdq.svdq_kv_attend_workspace_size(svdq.KvCacheDesc(None, None, state[0].shape[0], H, D, 64),
                                                  svdq.KvBatchDesc(None, None, None, T, 1, width), hq)
        assert need >= groups * 128 * splits * (D + 2) * 4
    wide = run_attend(cache, state, q.cuda(), qv, table, lengths, offs, True, 0, uniform=True)
    again = cache.attend(q.cuda(), dev(table), dev(np.asarray(lengths, np.int32)))
    assert torch.equal(wide, again)
