"""The 8-bit layers where a call can go wrong: offsets that fall, rows at
addresses that the kernels cannot read, biases that are views."""
import numpy as np
import pytest
import torch

from gpu_util import note

pytestmark = pytest.mark.gpu

import bit_quantized_diffusion_svdq_amd as svdq
from oracle import fp8 as ofp8
from test_gpu_fp8 import acts, biases, check_product, np64, weights


def falling(kind, M):
    """Offsets of `kind`: rising runs with values that fall among them."""
    if kind == "swap":
        return [0, M, 0, M, 0]
    if kind == "down":
        return [M, M - 2, M - 4, 1]
    if kind == "mixed":
        return [1, 3, 2, M - 3, 4, 4, M - 1, -7, M + 9, 2]
    # over runs of 64 groups: falls inside one, at its end and at the next one's start
    offs = np.sort(np.random.default_rng(5).integers(0, M + 1, 140)).tolist()
    for i in (20, 63, 64, 65, 100, 128):
        offs[i] = offs[i] // 3
    return offs


@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("kind", ["swap", "down", "mixed", "long"])
@pytest.mark.parametrize("M,N,layer", [(12, 72, True), (12, 72, False), (40, 136, True), (700, 1288, False)])
def test_offsets_that_fall(M, N, layer, kind, out):
    """An offset that falls counts as the largest before it: every row has one
    owner at the most, and rows without one stay."""
    offs = falling(kind, M)
    note(f"grouped 8-bit layer, falling offsets {kind} {M} x {N} {out} layer={layer}")
    K, E = 272, len(offs) - 1
    lay = svdq.Fp8GroupedLinear.from_quantized(svdq.quantize_fp8(weights(K, N, 1, groups=E), biases((E, N), 2)))
    x = acts(M, K, 3)
    o = torch.tensor(offs, dtype=torch.int32, device="cuda")
    y = torch.full((M, N), -3.0, dtype=out, device="cuda")
    qx, sx = svdq.quantize_act_fp8(x)
    if layer:
        lay(x, o, y=y)
    else:
        svdq.fp8_grouped_linear(qx, sx, o, lay.qw, lay.sw, lay.bias, y=y)
    ref = ofp8.grouped_linear(np64(qx), sx.cpu().numpy(), ofp8.rising(offs, M), np64(lay.qw), lay.sw.cpu().numpy(), np64(lay.bias))
    inside = ~np.isnan(ref[0][:, 0])
    assert (np64(y)[~inside] == -3.0).all()
    if inside.any():
        check_product(y[torch.from_numpy(inside).cuda()], [r[inside] for r in ref], K)


@pytest.mark.parametrize("M,K", [(1, 400), (5, 400), (16, 4096), (40, 272), (300, 144)])
def test_rows_at_any_address(M, K):
    """Activations at any address of a bf16 value, dense or strided, are those
    of an aligned copy: the activation pass, a dense and a grouped layer."""
    note(f"8-bit layers on unaligned rows {M} x {K}")
    N = 136
    x = acts(M, K, 1)
    lay = svdq.Fp8Linear.from_quantized(svdq.quantize_fp8(weights(K, N, 2), biases(N, 3)))
    grp = svdq.Fp8GroupedLinear(torch.stack([lay.qw.view(torch.uint8)] * 2).view(lay.qw.dtype), torch.stack([lay.sw] * 2))
    offs = torch.tensor([0, M // 2, M], dtype=torch.int32, device="cuda")
    want_q, want_s = svdq.quantize_act_fp8(x)
    want, want_g = lay(x), grp(x, offs)
    buf = torch.zeros(M * (K + 48) + 64, dtype=torch.bfloat16, device="cuda")
    for off in (1, 4, 7):
        for ld in (K, K + 40, K + 3):
            v = buf[off:off + M * ld].view(M, ld)[:, :K]
            v.copy_(x)
            q, s = svdq.quantize_act_fp8(v)
            assert torch.equal(q.view(torch.uint8), want_q.view(torch.uint8)) and torch.equal(s, want_s)
            assert torch.equal(lay(v), want) and torch.equal(grp(v, offs), want_g)


def test_quantised_layers_take_any_bias_view():
    """A bias that is a view of something wider makes a layer that runs."""
    note("quantize_fp8 with a strided bias")
    K, N = 144, 72
    w, b = weights(K, N, 1, groups=2), biases((2, 2 * N), 2)
    x, offs = acts(9, K, 3), torch.tensor([0, 4, 9], dtype=torch.int32, device="cuda")
    grp = svdq.Fp8GroupedLinear.from_quantized(svdq.quantize_fp8(w, b[:, ::2]))
    want = svdq.Fp8GroupedLinear.from_quantized(svdq.quantize_fp8(w, b[:, ::2].contiguous()))(x, offs)
    assert torch.equal(grp(x, offs), want)
    lay = svdq.Fp8Linear.from_quantized(svdq.quantize_fp8(w[1], b[1, 1::2]))
    assert torch.equal(lay(x), svdq.Fp8Linear(lay.qw, lay.sw, b[1, 1::2].contiguous())(x))
