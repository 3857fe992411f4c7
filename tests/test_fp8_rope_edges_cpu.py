"""Host-side checks of the 8-bit layers and the rotary positions at the calls
that could go wrong, without a GPU."""
import numpy as np
import pytest
import torch

import bit_quantized_diffusion_svdq_amd as svdq
from oracle import fp8 as ofp8


# ---------------------------------------------------------------- offsets that fall

@pytest.mark.parametrize("offs", [[0, 9, 0, 9, 0], [9, 7, 5, 3, 1], [-5, 3, 1 << 30, 2, 4], [0, 4, 4, 9], [3, 3, 2, 8, 8, 1, 9]])
def test_rising_bounds_share_no_row(offs):
    M = 9
    b = ofp8.rising(offs, M)
    owners = np.zeros(M, int)
    for lo, hi in zip(b, b[1:]):
        assert 0 <= lo <= hi <= M
        owners[lo:hi] += 1
    assert owners.max() <= 1
    if all(x <= y for x, y in zip(offs, offs[1:])):
        assert b == offs


# ---------------------------------------------------------------- gradients

def _rope_args():
    return dict(q=torch.zeros((4, 3, 32), dtype=torch.bfloat16), k=torch.zeros((4, 1, 32), dtype=torch.bfloat16),
                pos=torch.zeros((4, 2), dtype=torch.int32), plan=svdq.RopePlan((16, 16), device="cpu"))


@pytest.mark.parametrize("name", ["q", "k"])
def test_rope_axes_refuses_to_lose_a_gradient(name):
    a = _rope_args()
    a[name].requires_grad_()
    with pytest.raises(ValueError, match="requires a gradient"):
        svdq.rope_axes(**a)
    with torch.no_grad(), pytest.raises(ValueError, match="GPU device"):     # the next check: the call itself is fine
        svdq.rope_axes(**a)
    a[name] = a[name].detach()
    with pytest.raises(ValueError, match="GPU device"):
        svdq.rope_axes(**a, q_norm=torch.zeros(32, dtype=torch.bfloat16, requires_grad=True))
