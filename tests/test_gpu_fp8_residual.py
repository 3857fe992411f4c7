"""The 8-bit layers that join a residual stream, on every kernel that a product
can run, against the product without it (which test_gpu_fp8*.py hold against
the oracle)."""
import pytest
import torch

from gpu_util import note

pytestmark = pytest.mark.gpu

import bit_quantized_diffusion_svdq_amd as svdq
from test_gpu_fp8 import acts, biases, weights
from test_gpu_fp8_variants import VARIANTS

BF16, F32 = torch.bfloat16, torch.float32


def check(y, plain, res, gate):
    """y = round(res + gate * a), a the product before rounding. fp32 outputs:
    `plain` is a itself, and one fused step rounds by 2^-24 of the result (2^-50 for
    the reference in 64 bits). bf16: a is within half a step, 2^-8 of |a|, of
    `plain`, so within 2^-8 (1 + 2^-7) |plain|; the result rounds by 2^-8 of itself."""
    g = torch.ones_like(plain, dtype=torch.float64) if gate is None else gate.double().expand(plain.shape)
    want = res.double() + g * plain.double()
    if y.dtype == F32:
        bound = 2.0 ** -24 * (1 + 1e-6) * want.abs() + 2.0 ** -149
    else:
        e = 2.0 ** -8 * (1 + 2.0 ** -7) * (g * plain.double()).abs() + 2.0 ** -22 * (res.double().abs() + (g * plain.double()).abs())
        bound = e * (1 + 2.0 ** -8) + 2.0 ** -8 * want.abs() + 1e-38
    d = (y.double() - want).abs()
    assert bool((d <= bound).all()), f"{int((d > bound).sum())} outside the bound, worst {float((d / bound).max()):.3g}"


def stream(M, N, dt, seed, ld=None, off=0):
    g = torch.Generator().manual_seed(seed)
    ld = N if ld is None else ld
    flat = (torch.randn(M * ld + off + 8, generator=g) * 2).to(dt).cuda()
    return flat[off:off + M * ld].view(M, ld)[:, :N]


@pytest.mark.parametrize("key", VARIANTS, ids=str)
def test_every_kernel(key):
    (index, f32, groups), (M, K, N) = key, VARIANTS[key]
    note(f"fp8 residual, kernel {index}, fp32 outputs {f32}, {groups} groups: {M} x {K} x {N}")
    dt = F32 if f32 else BF16
    qx, sx = svdq.quantize_act_fp8(acts(M, K, M))
    ld = N if index % 2 else N + 4 - N % 4 + 4
    res = stream(M, N, dt, index, ld)
    act = "gelu_tanh" if index % 3 == 1 else "none"
    if not groups:
        d = svdq.quantize_fp8(weights(K, N, N), biases(N, K))
        gate = biases(N, 7) if index % 4 else None
        plain = svdq.fp8_linear(qx, sx, d["qw"], d["sw"], d["bias"], act=act, out_dtype=dt)
        y = svdq.fp8_linear(qx, sx, d["qw"], d["sw"], d["bias"], act=act, out_dtype=dt, residual=res, gate=gate)
        check(y, plain, res, gate)
        same = res.clone()
        svdq.fp8_linear(qx, sx, d["qw"], d["sw"], d["bias"], act=act, residual=same, gate=gate, y=same)
        assert torch.equal(same, y)
        return
    d = svdq.quantize_fp8(weights(K, N, N, groups=groups), biases((groups, N), K))
    gate = biases((groups, N), 7) if index % 4 else None
    cut = max(M * 3 // 5 // 32 * 32 + 5, 2)
    offs = [1, cut, cut + 1, cut + 1, M - 2, M - 2][:groups] + [M - 2]
    o = torch.tensor(offs, dtype=torch.int32, device="cuda")
    plain = svdq.fp8_grouped_linear(qx, sx, o, d["qw"], d["sw"], d["bias"], act=act, out_dtype=dt)
    y = torch.full((M, N), -3.0, dtype=dt, device="cuda")
    svdq.fp8_grouped_linear(qx, sx, o, d["qw"], d["sw"], d["bias"], act=act, y=y, residual=res, gate=gate)
    assert (y[:1] == -3.0).all() and (y[M - 2:] == -3.0).all()
    for g in range(groups):
        r = slice(offs[g], offs[g + 1])
        check(y[r], plain[r], res[r], None if gate is None else gate[g])
    same = res.clone()
    svdq.fp8_grouped_linear(qx, sx, o, d["qw"], d["sw"], d["bias"], act=act, residual=same, gate=gate, y=same)
    assert torch.equal(same[1:M - 2], y[1:M - 2]) and torch.equal(same[:1], res[:1]) and torch.equal(same[M - 2:], res[M - 2:])


@pytest.mark.parametrize("M,K,N", [(1, 16, 1), (1, 4096, 300), (3, 2064, 33), (16, 1536, 100), (17, 272, 129), (300, 528, 264)])
@pytest.mark.parametrize("dt", [BF16, F32])
@pytest.mark.parametrize("groups", [0, 2])
def test_layers(M, K, N, dt, groups):
    """From activations: one launch for few rows, two for more; strided, odd and
    unaligned residuals; in place."""
    note(f"fp8 residual layer {M} x {K} x {N} {dt} {groups}")
    x = acts(M, K, M)
    more = {}
    if groups:
        lin = svdq.Fp8GroupedLinear.from_quantized(svdq.quantize_fp8(weights(K, N, N, groups=groups), biases((groups, N), K)))
        more["offsets"] = torch.tensor([0, M // 2, M], dtype=torch.int32, device="cuda")
        gate = biases((groups, N), 3)
        rows = torch.tensor([0] * (M // 2) + [1] * (M - M // 2), device="cuda")
        per_row = gate[rows]
    else:
        lin = svdq.Fp8Linear.from_quantized(svdq.quantize_fp8(weights(K, N, N), biases(N, K)))
        gate = biases(N, 3)
        per_row = gate
    plain = lin(x, out_dtype=dt, **more)
    for ld, off in ((N, 0), (N + 3, 1), (N + 8, 8)):
        res = stream(M, N, dt, ld, ld, off)
        y = lin(x, out_dtype=dt, residual=res, gate=gate, **more)
        check(y, plain, res, per_row)
        same = torch.empty_strided((M, N), (ld, 1), dtype=dt, device="cuda").copy_(res)
        assert lin(x, y=same, residual=same, gate=gate, **more) is same
        assert torch.equal(same, y)
    y = lin(x, out_dtype=dt, residual=plain, **more)
    check(y, plain, plain, None)


def test_values_that_are_not_finite():
    """A NaN or an infinity of the stream stays in its place; a gate of zero takes nothing of a finite product."""
    M, K, N = 40, 272, 136
    lin = svdq.Fp8Linear.from_quantized(svdq.quantize_fp8(weights(K, N, N), biases(N, K)))
    x, res = acts(M, K, M), stream(M, N, BF16, 5)
    clean = lin(x, residual=res)
    dirty = res.clone()
    dirty[3, 7], dirty[30, 100] = float("nan"), float("-inf")
    y = lin(x, residual=dirty)
    assert y[3, 7].isnan() and y[30, 100] == float("-inf")
    y[3, 7], y[30, 100] = clean[3, 7], clean[30, 100]
    assert torch.equal(y, clean)
    assert torch.equal(lin(x, residual=res, gate=torch.zeros(N, dtype=BF16, device="cuda")), res)
