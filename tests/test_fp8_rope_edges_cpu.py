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
