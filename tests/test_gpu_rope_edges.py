"""Rotary positions where a call can go wrong: values that are not finite
beside channels that do not turn, tokens of no group, many tokens of every
type and pairing."""
import numpy as np
import pytest
import torch

from gpu_util import note

pytestmark = pytest.mark.gpu

import bit_quantized_diffusion_svdq_amd as svdq
from oracle import rope as orope
from test_gpu_rope import check, heads, np64, positions


@pytest.mark.parametrize("T", [9, 600])
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("pairing", ["interleaved", "half"])
@pytest.mark.parametrize("dims", [(16, 8), (0,)])
def test_values_past_the_pairs_stand_alone(T, dt, pairing, dims):
    """Channels past the pairs do not turn, so an infinity or a NaN in one of
    them stays in it: each such channel is its value (times its weight), with
    or without pairs in the head."""
    note(f"rope_axes past the pairs {T} {dt} {pairing} {dims}")
    D, P2 = 64, sum(dims)
    q = heads(T, 3, D, 1, dt)
    clean = q.clone()
    q[4, 1, 40], q[5, 0, 47], q[6, 2, 56] = float("inf"), float("nan"), float("-inf")
    pos, plan = positions(T, len(dims), 2), svdq.RopePlan(dims, head_dim=D, pairing=pairing)
    got, want = svdq.rope_axes(q, None, pos, plan), svdq.rope_axes(clean, None, pos, plan)
    keep = torch.isfinite(q)
    assert torch.equal(got[keep], want[keep]) and torch.equal(want[..., P2:], clean[..., P2:])
    assert got[4, 1, 40] == float("inf") and got[5, 0, 47].isnan() and got[6, 2, 56] == float("-inf")
    # with a norm: a weight that is not finite spoils its own channel only
    w = (1 + 0.1 * heads(1, 1, D, 7, torch.float32)).flatten().to(dt)
    want = svdq.rope_axes(clean, None, pos, plan, q_norm=w)
    w[41], w[50] = float("inf"), float("nan")
    got = svdq.rope_axes(clean, None, pos, plan, q_norm=w)
    keep = torch.isfinite(w)
    assert torch.equal(got[..., keep], want[..., keep])
    assert torch.isinf(got[..., 41]).all() and got[..., 50].isnan().all()


@pytest.mark.parametrize("T,offs", [(7, [0, 7]), (30, [2, 10, 10, 20]), (30, [30, 30]), (1, [0, 0]), (700, [3, 500, 690])])
def test_tokens_of_no_group_stay(T, offs):
    note(f"rope_axes groups {T} {offs}")
    H, HK, D = 3, 1, 64
    q, k, pos, plan = heads(T, H, D, 1), heads(T, HK, D, 2), positions(T, 2, 3), svdq.RopePlan((32, 32))
    w = (1 + 0.1 * heads(1, 1, D, 7)).flatten()
    want_q, want_k = svdq.rope_axes(q, k, pos, plan, q_norm=w, k_norm=w)
    o = torch.tensor(offs, dtype=torch.int32, device="cuda")
    inside = torch.zeros(T, dtype=torch.bool, device="cuda")
    inside[offs[0]:offs[-1]] = True
    for in_place in (False, True):
        qo, ko = (q.clone(), k.clone()) if in_place else (torch.full_like(q, -3.0), torch.full_like(k, -3.0))
        before = qo.clone(), ko.clone()
        src = (qo, ko) if in_place else (q, k)
        svdq.rope_axes(*src, pos, plan, q_norm=w, k_norm=w, q_out=qo, k_out=ko, offsets=o)
        for got, want, old in ((qo, want_q, before[0]), (ko, want_k, before[1])):
            assert torch.equal(got[inside], want[inside]) and torch.equal(got[~inside], old[~inside])


def test_qkv_block_leaves_rows_of_no_group():
    """FusedQKV over a grouped layer into a given buffer: the rows that the
    projection leaves as they are are not turned either; a graph of it, its
    offsets moving between replays, does the same."""
    note("FusedQKV over Fp8GroupedLinear, rows of no group")
    from test_gpu_fp8 import acts, weights
    T, K, H, D = 50, 144, 2, 32
    N = 3 * H * D
    layer = svdq.Fp8GroupedLinear.from_quantized(svdq.quantize_fp8(weights(K, N, 1, groups=2)))
    plan = svdq.RopePlan((16, 16))
    block = svdq.FusedQKV(layer, plan, H)
    x, pos = acts(T, K, 2), positions(T, 2, 3)
    y, o = torch.empty((T, N), dtype=torch.bfloat16, device="cuda"), torch.zeros(3, dtype=torch.int32, device="cuda")
    graph = svdq.CapturedSequence(lambda: block(x, pos, o, y=y))
    for offs in ([4, 20, 41], [0, 0, 50], [7, 7, 7], [0, 30, 33]):
        o.copy_(torch.tensor(offs, dtype=torch.int32))
        full = layer(x, o)
        wq, wk, wv = full.unflatten(1, (3 * H, D)).split(H, dim=1)
        rq, rk = svdq.rope_axes(wq, wk, pos, plan)
        for replay in (False, True):
            y.fill_(-3.0)
            q, k, v = y.unflatten(1, (3 * H, D)).split(H, dim=1)
            if replay:
                graph.replay()
            else:
                block(x, pos, o, y=y)
            torch.cuda.synchronize()
            r = slice(offs[0], offs[-1])
            assert torch.equal(q[r], rq[r]) and torch.equal(k[r], rk[r]) and torch.equal(v[r], wv[r])
            assert (y[:offs[0]] == -3.0).all() and (y[offs[-1]:] == -3.0).all()


# More than two tokens a CU run other instances (four loads in flight) than fewer do, and up to
# about 3000 of them several waves share a token: 1024 tokens of 24 + 24 heads of 128 are 6 + 6
# loads in three shares, of which the second holds the last queries and the first keys.
MANY = [
    # T, Hq, Hk, D, dims, pairing, norm, dtype
    (600, 3, 1, 64, (16, 24, 24), "interleaved", False, torch.float32),
    (600, 3, 1, 64, (16, 24, 24), "half", True, torch.float32),
    (700, 5, 2, 72, (24, 16, 24), "interleaved", True, torch.float32),
    (700, 5, 2, 72, (24, 16, 24), "half", True, torch.bfloat16),
    (530, 24, 24, 128, (32, 32), "half", True, torch.float32),
    (530, 24, 24, 128, (32, 32), "interleaved", True, torch.float32),
    (600, 4, 3, 128, (32, 32), "half", False, torch.bfloat16),
    (600, 4, 3, 128, (32, 32), "interleaved", True, torch.bfloat16),
    (1024, 24, 24, 128, (16, 56, 56), "interleaved", True, torch.bfloat16),
    (1024, 24, 24, 128, (16, 56, 56), "half", True, torch.bfloat16),
    (1024, 24, 8, 128, (16, 56, 56), "half", True, torch.float32),
    (1024, 21, 27, 128, (16, 56, 56), "interleaved", False, torch.float32),
    (3100, 7, 7, 128, (16, 56, 56), "half", True, torch.bfloat16),
    (3100, 6, 2, 256, (64, 96, 96), "interleaved", True, torch.float32),
    (520, 2, 1, 512, (128, 128, 128, 128), "half", True, torch.float32),
    (2000, 40, 1, 8, (8,), "interleaved", True, torch.bfloat16),
]


@pytest.mark.parametrize("T,hq,hk,D,dims,pairing,norm,dt", MANY)
def test_many_tokens(T, hq, hk, D, dims, pairing, norm, dt):
    note(f"rope_axes {T} x {hq}+{hk} x {D} {dims} {pairing} norm={norm} {dt}")
    q, k, pos = heads(T, hq, D, 1, dt), heads(T, hk, D, 2, dt), positions(T, len(dims), 3)
    qn = (1 + 0.3 * heads(1, 1, D, 4, torch.float32)).flatten().to(dt) if norm else None
    kn = (1 + 0.3 * heads(1, 1, D, 5, torch.float32)).flatten().to(dt) if norm else None
    plan = svdq.RopePlan(dims, head_dim=D, pairing=pairing)
    qo, ko = svdq.rope_axes(q, k, pos, plan, q_norm=qn, k_norm=kn)
    check(qo, q, pos, dims, pairing, qn)
    check(ko, k, pos, dims, pairing, kn)
    qi, ki = q.clone(), k.clone()
    svdq.rope_axes(qi, ki, pos, plan, q_norm=qn, k_norm=kn, q_out=qi, k_out=ki)
    assert torch.equal(qi, qo) and torch.equal(ki, ko)
    back = svdq.rope_axes(q, None, pos, plan, q_norm=qn, inverse=True)
    check(back, q, pos, dims, pairing, qn, inverse=True)
