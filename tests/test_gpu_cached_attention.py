"""The cache, its attention and the 8-bit layers' residual together, as a
decoder's block runs them: a ragged chunk, then single tokens, eager and as a
captured graph, against the oracles stage by stage."""
import numpy as np
import pytest
import torch

from gpu_util import note
from kv_util import cum, paged, random_state
from test_gpu_fp8 import acts, biases, check_product, np64, weights
from test_gpu_fp8_residual import check as check_residual, stream
from test_gpu_kv import cache_of, check_append, dev, run_attend, state_of, turned

pytestmark = pytest.mark.gpu

import bit_quantized_diffusion_svdq_amd as svdq
from oracle import fp8 as ofp8

H, HK, D, K, PAGE, DIMS = 6, 2, 72, 160, 64, (24, 24, 24)
N = (H + 2 * HK) * D


def parts(norms=True, window=0):
    qkv = svdq.Fp8Linear.from_quantized(svdq.quantize_fp8(weights(K, N, 1), biases(N, 2)))
    out = svdq.Fp8Linear.from_quantized(svdq.quantize_fp8(weights(H * D, K, 3), biases(K, 4)))
    w = [(1 + 0.1 * biases(D, i)) if norms else None for i in (5, 6)]
    plan = svdq.RopePlan(DIMS, head_dim=D)
    return svdq.FusedQKV(qkv, plan, H, HK, *w), out


def positions(lengths, counts):
    t = np.concatenate([np.arange(n - c, n) for n, c in zip(lengths, counts)])
    return np.stack([t // 16, t // 4 % 4, t % 4], axis=1).astype(np.int32)


@pytest.mark.parametrize("norms,window", [(True, 0), (False, 40)])
def test_block_by_stages(norms, window):
    note(f"CachedAttention {norms} {window}")
    rng = np.random.default_rng(1)
    qkv, out = parts(norms, window)
    pages, table = paged(rng, [200, 90], PAGE)
    state = random_state(rng, pages, PAGE, HK, D)
    cache = cache_of(state, HK, D, PAGE)
    block = svdq.CachedAttention(qkv, out, cache, window=window)
    gate = biases(K, 7)
    lengths = np.zeros(2, np.int32)
    for step, counts in enumerate(([130, 3], [1, 1], [1, 1], [20, 60])):
        lengths += np.asarray(counts, np.int32)
        T, off, pos = sum(counts), cum(counts), positions(lengths, counts)
        x = acts(T, K, 10 + step)
        res = stream(T, K, torch.bfloat16, step)
        args = (dev(pos), dev(table), dev(lengths), dev(off))
        before = [a.copy() for a in state_of(cache)]
        y = block(x, *args, residual=res, gate=gate)
        # the same by hand, each stage against its oracle on what the one before gave
        flat = qkv.layer(x)
        check_product(flat, ofp8.linear(*ofp8.quantize_act(np64(x)), np64(qkv.layer.qw), qkv.layer.sw.cpu().numpy(),
                                        np64(qkv.layer.bias)), K)
        q, k, v = flat.unflatten(1, (H + 2 * HK, D)).split((H, HK, HK), dim=1)
        wn = [None if w is None else np64(w) for w in (qkv.q_norm, qkv.k_norm)]
        kr, kerr = turned(np64(k), pos, DIMS, "interleaved", wn[1], 1e-6)
        check_append(cache, before, kr, kerr, np64(v), table, lengths, off)
        qr, qerr = turned(np64(q), pos, DIMS, "interleaved", wn[0], 1e-6)
        again = cache_of(before, HK, D, PAGE)
        q = again.append(k, v, *args[1:], pos=args[0], plan=qkv.plan, k_norm=qkv.k_norm, q=q, q_norm=qkv.q_norm)
        assert torch.equal(again.data, cache.data) and torch.equal(again.scales, cache.scales)
        assert (np.abs(np64(q) - qr) <= qerr * (1 + 2.0 ** -8) + 2.0 ** -8 * np.abs(qr) + 1e-37).all()
        o = run_attend(cache, state_of(cache), q, np64(q), table, lengths, off, True, window).flatten(1)
        plain = out(o)
        check_product(plain, ofp8.linear(*ofp8.quantize_act(np64(o)), np64(out.qw), out.sw.cpu().numpy(), np64(out.bias)), H * D)
        check_residual(y, plain, res, gate)
        assert torch.equal(y, out(o, residual=res, gate=gate))
        # in place in the residual stream
        cache.data.copy_(cache_of(before, HK, D, PAGE).data)
        cache.scales.copy_(cache_of(before, HK, D, PAGE).scales)
        assert torch.equal(block(x, *args, residual=res, gate=gate, y=res), y) and torch.equal(res, y)


def test_block_captured():
    """Single tokens of three sequences in one graph, the step's state advanced on the GPU between
    replays; every replay against the eager block on a cache of its own."""
    note("CachedAttention captured")
    qkv, out = parts()
    B, width = 3, 2
    table = torch.arange(B * width, dtype=torch.int32, device="cuda").reshape(B, width)
    caches = [svdq.KVCache(B * width, HK, D) for _ in range(2)]
    blocks = [svdq.CachedAttention(qkv, out, c) for c in caches]
    x = torch.zeros(B, K, dtype=torch.bfloat16, device="cuda")
    y = torch.zeros(B, K, dtype=torch.bfloat16, device="cuda")
    pos = torch.zeros(B, 3, dtype=torch.int32, device="cuda")
    lengths = torch.zeros(B, dtype=torch.int32, device="cuda")
    start = torch.tensor([0, 14, 60], dtype=torch.int32, device="cuda")

    def step():
        blocks[1](x, pos, table, lengths, residual=x, y=y)

    graph = svdq.CapturedSequence(step)
    caches[1].data.zero_(), caches[1].scales.fill_(7)
    lengths.copy_(start)
    for i in range(8):
        x.copy_(acts(B, K, i))
        lengths.add_(1)
        pos.copy_(torch.stack([lengths - 1, lengths % 7, lengths % 5], dim=1))
        want = blocks[0](x, pos, table, lengths, residual=x)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want)
        assert torch.equal(caches[0].data, caches[1].data) and torch.equal(caches[0].scales, caches[1].scales)


def test_block_over_four_bits():
    """A W4A4 projection on either side (no residual there)."""
    note("CachedAttention over SvdqLinear")
    Kw, h, hk, d = 256, 4, 1, 64
    g = torch.Generator().manual_seed(0)
    w = (torch.randn((Kw, (h + 2 * hk) * d), generator=g) * 0.05).bfloat16().cuda()
    wo = (torch.randn((h * d, Kw), generator=g) * 0.05).bfloat16().cuda()
    x = acts(40, Kw, 1)
    qkv = svdq.SvdqLinear.from_quantized(svdq.quantize_layer(w, acts(128, Kw, 2), rank=16))
    out = svdq.SvdqLinear.from_quantized(svdq.quantize_layer(wo, acts(128, h * d, 3), rank=16))
    fused = svdq.FusedQKV(qkv, svdq.RopePlan((64,)), h, hk)
    table = torch.tensor([[1], [0]], dtype=torch.int32, device="cuda")
    lengths = torch.tensor([20, 33], dtype=torch.int32, device="cuda")
    pos = torch.arange(40, dtype=torch.int32, device="cuda").reshape(40, 1)
    caches = [svdq.KVCache(2, hk, d) for _ in range(2)]
    y = svdq.CachedAttention(fused, out, caches[0])(x, pos, table, lengths)
    q, k, v = (t.contiguous() for t in qkv(x).unflatten(1, (h + 2 * hk, d)).split((h, hk, hk), dim=1))
    q = caches[1].append(k, v, table, lengths, pos=pos, plan=fused.plan, q=q)
    assert torch.equal(y, out(caches[1].attend(q, table, lengths).flatten(1)))
    with pytest.raises(ValueError):
        svdq.CachedAttention(fused, out, caches[0])(x, pos, table, lengths, residual=x)


def test_block_refuses_before_it_writes():
    note("CachedAttention refuses")
    qkv, out = parts()
    cache = svdq.KVCache(2, HK, D)
    block = svdq.CachedAttention(qkv, out, cache)
    x, pos = acts(4, K, 0), torch.zeros(4, 3, dtype=torch.int32, device="cuda")
    table, lengths = torch.zeros(1, 1, dtype=torch.int32, device="cuda"), torch.full((1,), 4, dtype=torch.int32, device="cuda")
    bad = torch.zeros(4, K + 1, dtype=torch.bfloat16, device="cuda")
    for kw in (dict(residual=bad), dict(gate=biases(K, 0)), dict(residual=x.float()), dict(y=bad), dict(residual=x, gate=biases(K + 1, 0)),
               dict(residual=x.cpu())):
        with pytest.raises(ValueError):
            block(x, pos, table, lengths, **kw)
    for a in ((x, pos[:3], table, lengths), (x, pos, table, lengths.long()), (x, pos, table.cpu(), lengths), (x[:, :8], pos, table, lengths)):
        with pytest.raises(ValueError):
            block(*a)
    torch.cuda.synchronize()
    assert (cache.data == 0).all() and (cache.scales == 7).all()
