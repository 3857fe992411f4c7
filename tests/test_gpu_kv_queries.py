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
