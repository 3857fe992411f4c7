"""The queries that KVCache.append turns beside the keys that it stores: the
tokens that belong to a sequence are the same ones for both, whatever the
offsets say, and positions may be fp32."""
import numpy as np
import pytest
import torch

from gpu_util import note
from kv_util import bf16, cum, paged, random_state
from test_gpu_kv import cache_of, check_append, dev, run_attend, state_of, turned

pytestmark = pytest.mark.gpu

import bit_quantized_diffusion_svdq_amd as svdq
from oracle import kv as okv
from oracle.fp8 import e4m3_round


def both(rng, counts_or_offsets, lengths, hq, H, D, dims, pairing, norm, pos, T):
    """One call over given offsets: keys, values and queries against the oracle, rows of no sequence as
    they were, and what attention makes of it, in place."""
    offsets = np.asarray(counts_or_offsets, np.int32)
    pages, table = paged(rng, lengths, 64)
    was = random_state(rng, pages, 64, H, D)
    cache = cache_of(was, H, D, 64)
    flat, fv = bf16(rng, (T, hq + 2 * H, D))
    w = (1 + 0.2 * torch.randn(D, generator=torch.Generator().manual_seed(1))).bfloat16() if norm else None
    wn = None if w is None else w.double().numpy()
    gpu = flat.cuda()
    q, k, v = gpu.split((hq, H, H), dim=1)
    out = torch.full((T, hq, D), 7.0, dtype=torch.bfloat16, device="cuda")
    plan = svdq.RopePlan(dims, head_dim=D, pairing=pairing)
    args = (dev(table), dev(np.asarray(lengths, np.int32)), dev(offsets))
    kw = dict(pos=dev(pos), plan=plan, k_norm=None if w is None else w.cuda(), q_norm=None if w is None else w.cuda())
    assert cache.append(k, v, *args, q=q, q_out=out, **kw) is out
    torch.cuda.synchronize()
    kr, kerr = turned(fv[:, hq:hq + H], pos, dims, pairing, wn, 1e-6)
    check_append(cache, was, kr, kerr, fv[:, hq + H:], table, np.clip(lengths, 0, None), offsets)
    qr, qerr = turned(fv[:, :hq], pos, dims, pairing, wn, 1e-6)
    off = okv.rising(offsets, T)
    owned = np.zeros(T, bool)
    owned[off[0]:off[-1]] = True
    d = np.abs(out.double().cpu().numpy() - qr)
    assert (d <= qerr * (1 + 2.0 ** -8) + 2.0 ** -8 * np.abs(qr) + 1e-37)[owned].all()
    assert (out.cpu()[torch.from_numpy(~owned)] == 7.0).all()
    turned_out = out.clone()
    again = cache_of(was, H, D, 64)
    assert again.append(k, v, *args, q=q, q_out=q, **kw) is q         # in place: the rest of the buffer stays
    want = flat.clone()
    want[torch.from_numpy(owned), :hq] = out.cpu()[torch.from_numpy(owned)]
    assert torch.equal(gpu.cpu(), want)
    run_attend(cache, state_of(cache), turned_out, turned_out.double().cpu().numpy(), table, lengths, offsets, True, 0, out=out)
    return owned


@pytest.mark.parametrize("hq", [2, 24])
@pytest.mark.parametrize("offsets", [[0, 9, 3], [0, 9, 9], [2, 11, -4], [0, 12, 5], [-3, 99, 1], [3, 3, 2], [8, 2, 10], [5, 1, 0], [40, 3, 7]])
def test_offsets_that_fall(offsets, hq):
    note(f"kv queries, offsets {offsets} {hq}")
    rng = np.random.default_rng(5)
    T = 12
    pos = rng.integers(0, 500, (T, 2)).astype(np.int32)
    both(rng, offsets, [70, 40], hq, 2, 72, (32, 40), "interleaved", True, pos, T)


@pytest.mark.parametrize("peak", [0, 1, 63, 64, 65, 128, 129])
def test_many_offsets_that_fall(peak):
    """The largest offset anywhere in more of them than a wave has lanes."""
    note(f"kv queries, largest offset {peak}")
    rng = np.random.default_rng(peak)
    T, B = 40, 129
    offsets = np.minimum(np.arange(B + 1) // 8, 12).astype(np.int32)
    offsets[peak] = 33
    pos = rng.integers(0, 500, (T, 1)).astype(np.int32)
    owned = both(rng, offsets, [35] * B, 2, 1, 64, (64,), "half", False, pos, T)
    assert owned.sum() == (0 if peak == 0 else 33)


@pytest.mark.parametrize("counts,before,dims,pairing,norm,D", [
    ([1], [76], (16, 56, 56), "interleaved", True, 128),
    ([5, 1, 40], [3, 0, 30], (16, 24, 24), "half", False, 64),
    ([17, 64], [15, 64], (32, 32), "half", True, 96),
    ([33, 600], [1, 63], (40, 40), "interleaved", True, 200),
    ([33, 2], [1, 63], (64, 96, 96), "half", True, 256),
])
def test_positions_in_fp32(counts, before, dims, pairing, norm, D):
    """Positions between whole ones, far ones and ones below zero, of keys as of queries."""
    note(f"kv fp32 positions {counts} {D}")
    rng = np.random.default_rng(D)
    T = sum(counts)
    pos = (rng.standard_normal((T, len(dims))) * np.where(rng.random((T, 1)) < 0.3, 3e5, 40.0)).astype(np.float32)
    both(rng, cum(counts), [a + b for a, b in zip(counts, before)], 4, 2, D, dims, pairing, norm, pos, T)


@pytest.mark.parametrize("pairing,norm", [("interleaved", True), ("half", False)])
def test_keys_are_rounded_once(pairing, norm):
    """14 million codes against the 64-bit keys'. Angles are 2^-29 off at the most and the root 2^-28, so a
    key is off by some 2^-28 of itself; a power of two has 8 borders between codes, so a code in 2^24 / 2 may be
    another: about one of 14 million. (Rounded to 32 bits first, a key within 2^-24 of a border comes to lie on it: 7.)"""
    note(f"kv codes {pairing} {norm}")
    rng = np.random.default_rng(77)
    T, H, D, dims = 4608, 24, 128, (16, 56, 56)
    cache = svdq.KVCache(T // 64, H, D)
    k, kv = bf16(rng, (T, H, D))
    w = torch.from_numpy(1 + 0.2 * rng.standard_normal(D)).bfloat16()
    pos = rng.integers(0, 4096, (T, 3)).astype(np.int32)
    cache.append(k.cuda(), k.cuda(), dev(np.arange(T // 64, dtype=np.int32)[None]), dev(np.asarray([T], np.int32)), pos=dev(pos),
                 plan=svdq.RopePlan(dims, head_dim=D, pairing=pairing), k_norm=w.cuda() if norm else None)
    keys, _, exps, _ = state_of(cache)
    x = turned(kv, pos, dims, pairing, w.double().numpy() if norm else None, 1e-6)[0].reshape(T // 64, 64, H, D)
    e = okv.exponent(np.abs(x).reshape(T // 64, 4, 16, H, D).max(axis=(2, 4)))
    np.testing.assert_array_equal(exps, e)
    other = int((keys != e4m3_round(np.ldexp(x, -np.repeat(e, 16, axis=1)[..., None]))).sum())
    print(f"{other} codes of {keys.size} are others")
    assert other <= 3


@pytest.mark.parametrize("D", [64, 72, 256])
def test_ties_go_to_even(D):
    """Keys that lie on a border between codes, with no norm and a rotation by no angle, and beside one."""
    note(f"kv ties {D}")
    T, H = 64, 2
    rng = np.random.default_rng(D)
    k = torch.from_numpy(np.ldexp(rng.integers(-31, 32, (T, H, D)).astype(np.float64), rng.integers(-12, 3, (T, 1, D)))).bfloat16()
    k[::16, :, 0] = 448.0                                 # (exponent 0: borders at odd numbers of 2^-4 of a power of two)
    cache = svdq.KVCache(1, H, D)
    for more in ({}, dict(pos=torch.zeros(T, 1, dtype=torch.int32, device="cuda"), plan=svdq.RopePlan((D,), head_dim=D))):
        cache.append(k.cuda(), k.cuda(), dev(np.zeros((1, 1), np.int32)), dev(np.asarray([T], np.int32)), **more)
        keys, values, ke, ve = state_of(cache)
        assert (ke == 0).all() and (ve == 0).all()
        want = e4m3_round(k.double().numpy())
        np.testing.assert_array_equal(keys[0, :, :, :D], want)
        np.testing.assert_array_equal(values[0, :, :, :D], want)


@pytest.mark.parametrize("D", [64, 200])
def test_squares_past_fp32(D):
    """A head whose squares add up past fp32 becomes zeros, of keys as of queries; one just below is normed."""
    note(f"kv squares past fp32 {D}")
    T, H = 20, 2
    x = torch.ones(T, H, D)
    x[3] = 5e18                                           # (their mean does not pass it)
    x[7, 1], x[11, 0] = 1e30, 3e38
    x[5] = (3e38 / D) ** 0.5
    x = x.bfloat16().cuda()
    cache = svdq.KVCache(1, H, D)
    w = torch.ones(D, dtype=torch.bfloat16, device="cuda")
    q = cache.append(x, x, dev(np.zeros((1, 1), np.int32)), dev(np.asarray([T], np.int32)), k_norm=w, q=x, q_norm=w)
    keys, _, e, _ = state_of(cache)
    keys = np.ldexp(keys[0, :T, :, :D], np.repeat(e[0], 16, axis=0)[:T, :, None])
    want = np.ones((T, H, D))
    want[3] = want[7, 1] = want[11, 0] = 0.0
    np.testing.assert_array_equal(q.double().cpu().numpy(), want)
    np.testing.assert_array_equal(keys, want)
