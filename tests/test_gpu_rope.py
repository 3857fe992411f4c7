"""GPU parity of the rotary positions with several axes against the fp64
oracle, over head widths, pairings, layouts, types and far positions."""
import numpy as np
import pytest
import torch

from gpu_util import note

pytestmark = pytest.mark.gpu

import bit_quantized_diffusion_svdq_amd as svdq
from oracle import rope as orope


def np64(t):
    return t.detach().double().cpu().numpy()


def heads(T, H, D, seed, dt=torch.bfloat16):
    return torch.randn((T, H, D), generator=torch.Generator().manual_seed(seed)).to(dt).cuda()


def positions(T, axes, seed, dt=torch.int32, top=4096):
    g = torch.Generator().manual_seed(seed)
    p = torch.randint(-top // 8, top, (T, axes), generator=g)
    return (p.to(dt) if dt == torch.int32 else p.float() + torch.rand((T, axes), generator=g)).cuda()


def check(got, x, pos, dims, pairing, w=None, eps=1e-6, inverse=False, theta=10000.0):
    """Per pair: sine and cosine are off by at most 2^-21 (the part of a turn
    rounded to 32 bits, 2^-26 turns = 2^-23 rad, and the functions' 2 ulp),
    the two products and their sum by 3 x 2^-24, the norm's factor by less
    than 2^-21 (sums over at most 512 squares in lanes and a tree, a root, a
    division and two products): 2^-19 (|a| + |b|) covers them. bf16 adds half
    a step, 2^-8 of the value."""
    v = np64(x) if w is None else orope.rms_norm(np64(x), np64(w), eps)
    axis, freq = orope.frequencies(dims, theta)
    ref = orope.rotate(v, np64(pos), axis, freq, pairing, inverse)
    P = len(freq)
    mag = np.abs(v)
    s = (slice(0, 2 * P, 2), slice(1, 2 * P, 2)) if pairing == "interleaved" else (slice(0, P), slice(P, 2 * P))
    both = mag[..., s[0]] + mag[..., s[1]]
    mag[..., s[0]] = both
    mag[..., s[1]] = both
    bound = 2.0 ** -19 * mag + 1e-37
    if got.dtype == torch.bfloat16:
        bound = bound * (1 + 2.0 ** -8) + 2.0 ** -8 * np.abs(ref)
    err = np.abs(np64(got) - ref)
    assert (err <= bound).all(), f"{(err > bound).sum()} outside the bound, worst ratio {(err / bound).max():.3g}"


CASES = [
    # T, Hq, Hk, D, dims, pairing, norm, dtype, positions
    (1, 1, 1, 8, (8,), "interleaved", False, torch.bfloat16, torch.int32),
    (1, 24, 24, 128, (16, 56, 56), "interleaved", True, torch.bfloat16, torch.int32),
    (3, 5, 1, 64, (16, 24, 24), "half", True, torch.bfloat16, torch.int32),
    (17, 3, 3, 72, (24, 24, 24), "interleaved", True, torch.bfloat16, torch.float32),
    (17, 3, 2, 72, (24, 24, 24), "half", True, torch.float32, torch.int32),
    (9, 2, 1, 96, (32, 32, 32), "half", False, torch.float32, torch.float32),
    (33, 4, 2, 128, (32, 32), "half", True, torch.bfloat16, torch.int32),
    (33, 4, 2, 128, (32, 32), "interleaved", True, torch.bfloat16, torch.int32),
    (5, 7, 3, 256, (64, 96, 96), "interleaved", True, torch.float32, torch.int32),
    (4, 2, 1, 512, (128, 128, 128, 128), "half", True, torch.bfloat16, torch.int32),
    (6, 3, 1, 40, (6, 6, 4, 8), "interleaved", True, torch.bfloat16, torch.float32),
    (6, 3, 1, 40, (6, 6, 4, 8), "half", False, torch.float32, torch.int32),
    (2, 3, 3, 64, (), "half", True, torch.bfloat16, torch.int32),
    (2200, 3, 1, 128, (44, 42, 42), "half", False, torch.bfloat16, torch.int32),
    (2300, 9, 9, 64, (64,), "interleaved", True, torch.bfloat16, torch.int32),
]


@pytest.mark.parametrize("T,hq,hk,D,dims,pairing,norm,dt,pt", CASES)
def test_rope(T, hq, hk, D, dims, pairing, norm, dt, pt):
    note(f"rope_axes {T} x {hq}+{hk} x {D} {dims} {pairing} norm={norm} {dt} {pt}")
    if not dims:
        dims = (0,)                                # no pair turns: the norm alone
    q, k = heads(T, hq, D, 1, dt), heads(T, hk, D, 2, dt)
    pos = positions(T, len(dims), 3, pt)
    qn = (1 + 0.3 * heads(1, 1, D, 4, torch.float32)).flatten().to(dt) if norm else None
    kn = (1 + 0.3 * heads(1, 1, D, 5, torch.float32)).flatten().to(dt) if norm else None
    plan = svdq.RopePlan(dims, head_dim=D, pairing=pairing)
    qo, ko = svdq.rope_axes(q, k, pos, plan, q_norm=qn, k_norm=kn)
    check(qo, q, pos, dims, pairing, qn)
    check(ko, k, pos, dims, pairing, kn)
    only = svdq.rope_axes(q, None, pos, plan, q_norm=qn)
    assert torch.equal(only, qo)
    qo, ko = svdq.rope_axes(q, k, pos, plan, k_norm=kn)          # one side normed
    check(qo, q, pos, dims, pairing)
    check(ko, k, pos, dims, pairing, kn)


def test_far_positions_and_theta():
    """Positions up to 2^31 and fractions of a step keep their angle."""
    note("rope_axes far positions")
    T, D, dims = 64, 64, (32, 32)
    q = heads(T, 2, D, 1, torch.float32)
    plan = svdq.RopePlan(dims, theta=(10000.0, 256.0))
    pos = torch.randint(2 ** 30, 2 ** 31 - 1, (T, 2), generator=torch.Generator().manual_seed(2)).to(torch.int32).cuda()
    axis, f0 = orope.frequencies(dims)
    freq = np.where(axis == 0, f0, 256.0 ** (np.log(f0) / np.log(10000.0)))
    v = np64(q)
    for inverse in (False, True):
        got = np64(svdq.rope_axes(q, None, pos, plan, inverse=inverse))
        # fp64 leaves 2^31 / 2 pi turns x 2^-52 in the kernel and the same again in the reference
        ref = orope.rotate(v, np64(pos), axis, freq, "interleaved", inverse)
        mag = np.abs(v[..., 0::2]) + np.abs(v[..., 1::2])
        bound = np.repeat((2.0 ** -19 + 2.0 ** -18) * mag, 2, axis=2)
        assert (np.abs(got - ref) <= bound).all()


def test_views_layouts_and_in_place():
    """Views of a fused [Q | K | V] output, head-major outputs, in place;
    the value columns and everything around the outputs stay."""
    note("rope_axes layouts")
    T, H, HK, D, dims = 130, 6, 2, 64, (16, 24, 24)
    flat = heads(T, 1, (H + 2 * HK) * D + 16, 1)[:, 0]
    y = flat[:, 8:8 + (H + 2 * HK) * D]
    h = y.unflatten(1, (H + 2 * HK, D))
    q, k, v = h.split((H, HK, HK), dim=1)
    pos = positions(T, 3, 2)
    plan = svdq.RopePlan(dims)
    want_q, want_k = svdq.rope_axes(q, k, pos, plan)
    check(want_q, q, pos, dims, "interleaved")
    qh, kh = torch.empty((H, T, D), dtype=q.dtype, device="cuda"), torch.empty((HK, T, D), dtype=q.dtype, device="cuda")
    svdq.rope_axes(q, k, pos, plan, q_out=qh.transpose(0, 1), k_out=kh.transpose(0, 1))
    assert torch.equal(qh.transpose(0, 1), want_q) and torch.equal(kh.transpose(0, 1), want_k)
    back_q, back_k = svdq.rope_axes(qh.transpose(0, 1), kh.transpose(0, 1), pos, plan, inverse=True)
    # there and back: two bf16 roundings of a pair's members, each 2^-8 of the pair's length at most
    pair = np.sqrt(np64(q)[..., 0::2] ** 2 + np64(q)[..., 1::2] ** 2)
    assert (np.abs(np64(back_q) - np64(q)) <= np.repeat(2.5 * 2.0 ** -8 * pair, 2, axis=2)).all()
    before = flat.clone()
    svdq.rope_axes(q, k, pos, plan, q_out=q, k_out=k)
    assert torch.equal(q, want_q) and torch.equal(k, want_k)
    lo, hi = 8 + (H + HK) * D, 8
    assert torch.equal(flat[:, lo:], before[:, lo:]) and torch.equal(flat[:, :hi], before[:, :hi])


def test_gradient_is_the_inverse():
    """<g, R x> has the gradient R^T g = the inverse rotation of g: against
    differences along random directions, in fp32 with the fp64 oracle's R."""
    note("rope_axes gradient")
    T, H, D, dims = 5, 2, 32, (16, 16)
    x, g, d = (heads(T, H, D, s, torch.float32) for s in (1, 2, 3))
    pos = positions(T, 2, 4)
    for pairing in ("interleaved", "half"):
        plan = svdq.RopePlan(dims, pairing=pairing)
        grad = np64(svdq.rope_axes(g, None, pos, plan, inverse=True))
        axis, freq = orope.frequencies(dims)
        f = lambda z: (np64(g) * orope.rotate(z, np64(pos), axis, freq, pairing)).sum()
        h = 2.0 ** -10
        slope = (f(np64(x) + h * np64(d)) - f(np64(x) - h * np64(d))) / (2 * h)
        # R is linear, so the difference is exact up to fp64; grad is within 2^-18 of each element's pair
        assert abs((grad * np64(d)).sum() - slope) <= 2.0 ** -18 * np.abs(np64(g)).sum() * np.abs(np64(d)).max()


def test_streams_graphs_and_non_finite():
    note("rope_axes stream and graph")
    T, H, D = 40, 3, 64
    q, k = heads(T, H, D, 1), heads(T, 1, D, 2)
    pos, plan = positions(T, 3, 3), svdq.RopePlan((16, 24, 24))
    w = (1 + 0.1 * heads(1, 1, D, 7)).flatten()
    want = svdq.rope_axes(q, k, pos, plan, q_norm=w)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = svdq.rope_axes(q, k, pos, plan, q_norm=w, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    qo, ko = torch.empty_like(q), torch.empty_like(k)
    graph = svdq.CapturedSequence(lambda: svdq.rope_axes(q, k, pos, plan, q_norm=w, q_out=qo, k_out=ko))
    for i in range(4):
        q.copy_(heads(T, H, D, 10 + i))
        graph.replay()
        torch.cuda.synchronize()
        want = svdq.rope_axes(q, k, pos, plan, q_norm=w)
        assert torch.equal(qo, want[0]) and torch.equal(ko, want[1])
        qo.zero_()
    # a NaN stays in its pair, with the norm in its head
    q[3, 1, 10] = float("nan")
    bad = svdq.rope_axes(q, None, pos, plan).isnan()
    assert bad[3, 1, 10:12].all() and bad.sum() == 2
    bad = svdq.rope_axes(q, None, pos, plan, q_norm=w).isnan()
    assert bad[3, 1].all() and bad.sum() == D


def test_offsets_past_32_bits():
    """Heads past 2^31 values, in place: the last tokens are those of a short
    sequence, and tokens of zeros stay zero."""
    note("rope_axes past 2^31 values")
    T, H, D = 530_003, 32, 128
    assert T * H * D > 2 ** 31
    plan = svdq.RopePlan((16, 56, 56))
    q = torch.zeros((T, H, D), dtype=torch.bfloat16, device="cuda")
    tail, pos = heads(40, H, D, 1), positions(T, 3, 2)
    q[-40:] = tail
    assert svdq.rope_axes(q, None, pos, plan, q_out=q) is q
    want = svdq.rope_axes(tail, None, pos[-40:].contiguous(), plan)
    assert torch.equal(q[-40:], want) and (q[0] == 0).all() and (q[-41] == 0).all()


@pytest.mark.parametrize("T", [1, 9])
def test_no_pairs_no_positions(T):
    """The C entry without pairs takes no positions and no plan: the norm
    alone, or a copy."""
    note(f"svdq_rope_axes without positions {T}")
    H, D = 3, 40
    q = heads(T, H, D, 1)
    w = (1 + 0.1 * heads(1, 1, D, 7)).flatten()
    plan = svdq.RopePlan((0,), head_dim=D)
    for norm in (None, w):
        y = torch.zeros_like(q)
        side = svdq._lib.RopeHeads(q.data_ptr(), H * D, D, H, None if norm is None else norm.data_ptr(), y.data_ptr(), H * D, D)
        svdq.svdq_rope_axes(side, None, T, D, 0, None, 0, 1, None, None, 0, 0, 0, 1e-6)
        assert torch.equal(y, svdq.rope_axes(q, None, positions(T, 1, 2), plan, q_norm=norm))
        assert norm is not None or torch.equal(y, q)


def test_qkv_block_over_a_four_bit_layer():
    """FusedQKV over a W4A4 layer is the layer's call and then the rotation."""
    note("FusedQKV over SvdqLinear")
    T, K, H, D = 50, 256, 4, 64
    g = torch.Generator().manual_seed(1)
    w = (torch.randn((K, 3 * H * D), generator=g) * 0.05).to(torch.bfloat16).cuda()
    x = torch.randn((T, K), generator=g).to(torch.bfloat16).cuda()
    layer = svdq.SvdqLinear.from_quantized(svdq.quantize_layer(w, x, rank=16))
    plan = svdq.RopePlan((16, 24, 24))
    pos = positions(T, 3, 2)
    y = layer(x)
    wq, wk, wv = y.unflatten(1, (3 * H, D)).split(H, dim=1)
    rq, rk = svdq.rope_axes(wq, wk, pos, plan)
    q, k, v = svdq.FusedQKV(layer, plan, H)(x, pos)
    assert torch.equal(q, rq) and torch.equal(k, rk) and torch.equal(v, wv)
