"""Every kernel that a product of the 8-bit layers can run, at a size that
takes it: (kernel, output type, dense or grouped). test_fp8_rope_edges_cpu.py
holds that the list is whole and that each size still takes its kernel."""
import numpy as np
import pytest
import torch

from gpu_util import note

pytestmark = pytest.mark.gpu

import bit_quantized_diffusion_svdq_amd as svdq
from test_gpu_fp8 import acts, biases, check_all_and_some, weights

# (kernel's index, fp32 outputs, groups) -> M, K, N
VARIANTS = {
    (0, 0, 0): (2405, 400, 6152), (1, 0, 0): (4700, 144, 2603), (2, 0, 0): (2405, 1168, 4104), (3, 0, 0): (6007, 400, 1288),
    (4, 0, 0): (4111, 1168, 1001), (5, 0, 0): (700, 144, 3000), (6, 0, 0): (3600, 400, 520), (7, 0, 0): (130, 400, 6152),
    (8, 0, 0): (65, 256, 136), (9, 0, 0): (16, 2064, 100), (10, 0, 0): (23, 1040, 1289), (11, 0, 0): (61, 1936, 2049),
    (5, 1, 0): (4111, 400, 520), (8, 1, 0): (129, 144, 1001), (9, 1, 0): (7, 2064, 300), (10, 1, 0): (23, 1040, 1289),
    (11, 1, 0): (257, 1152, 520),
    (0, 0, 3): (2000, 400, 6152), (1, 0, 3): (4700, 144, 2603), (2, 0, 3): (1030, 1168, 9001), (3, 0, 3): (6007, 400, 1288),
    (4, 0, 3): (4111, 1168, 1001), (5, 0, 3): (300, 400, 6152), (6, 0, 3): (1500, 400, 1288), (7, 0, 3): (257, 400, 3000),
    (8, 0, 3): (70, 144, 136), (9, 0, 2): (300, 2064, 72), (10, 0, 5): (23, 1040, 257), (11, 0, 3): (90, 1168, 1288),
    (5, 1, 5): (701, 400, 6152), (8, 1, 3): (70, 144, 136), (9, 1, 3): (300, 528, 128), (10, 1, 5): (23, 1040, 257),
    (11, 1, 5): (61, 1936, 1289),
}


@pytest.mark.parametrize("key", VARIANTS, ids=str)
def test_every_kernel(key):
    """Every output and, in groups, a group of one row, an empty one, a last
    tile with few or no rows for half of its waves, and rows of no group."""
    (index, f32, groups), (M, K, N) = key, VARIANTS[key]
    note(f"fp8 product, kernel {index}, fp32 outputs {f32}, {groups} groups: {M} x {K} x {N}")
    cus = torch.cuda.get_device_properties(0).multi_processor_count
    assert svdq.svdq_gemm_fp8_variant(M, K, N, groups, f32, cus) == index
    dt = torch.float32 if f32 else torch.bfloat16
    qx, sx = svdq.quantize_act_fp8(acts(M, K, M))
    if not groups:
        d = svdq.quantize_fp8(weights(K, N, N), biases(N, K))
        y = svdq.fp8_linear(qx, sx, d["qw"], d["sw"], d["bias"], out_dtype=dt)
        check_all_and_some(y, qx, sx, d["qw"], d["sw"], d["bias"], sorted({0, 1, M // 3, M // 2, M - 1}), K)
        return
    d = svdq.quantize_fp8(weights(K, N, N, groups=groups), biases((groups, N), K))
    cut = max(M * 3 // 5 // 32 * 32 + 5, 2)               # a tile's first rows at the end of the first group
    offs = [1, cut, cut + 1, cut + 1, M - 2, M - 2][:groups] + [M - 2]
    y = torch.full((M, N), -3.0, dtype=dt, device="cuda")
    svdq.fp8_grouped_linear(qx, sx, torch.tensor(offs, dtype=torch.int32, device="cuda"), d["qw"], d["sw"], d["bias"], y=y)
    assert (y[:1] == -3.0).all() and (y[M - 2:] == -3.0).all()
    for g in range(groups):
        n = offs[g + 1] - offs[g]
        if n:
            r = slice(offs[g], offs[g + 1])
            check_all_and_some(y[r], qx[r], sx[:, r].contiguous(), d["qw"][g], d["sw"][g], d["bias"][g], sorted({0, n // 2, n - 1}), K)
