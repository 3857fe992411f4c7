"""Rotary positions where a call can go wrong: values that are not finite
beside channels that do not turn."""
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
