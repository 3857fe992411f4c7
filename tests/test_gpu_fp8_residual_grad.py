"""Gradients and the 8-bit layers' residual: refused where they would be lost."""
import pytest
import torch

from gpu_util import note

pytestmark = pytest.mark.gpu

import bit_quantized_diffusion_svdq_amd as svdq
from test_gpu_fp8 import acts, biases, weights


@pytest.mark.parametrize("M", [3, 40])                    # one launch, two
@pytest.mark.parametrize("groups", [0, 2])
def test_refused_while_recording(M, groups):
    note(f"fp8 residual, gradients, {M} rows, {groups} groups")
    K, N = 272, 136
    x, res = acts(M, K, 1), acts(M, N, 2)
    if groups:
        lin = svdq.Fp8GroupedLinear.from_quantized(svdq.quantize_fp8(weights(K, N, N, groups=groups), biases((groups, N), K)))
        more, gate = dict(offsets=torch.tensor([0, M // 2, M], dtype=torch.int32, device="cuda")), biases((groups, N), 3)
        product = svdq.fp8_grouped_linear
    else:
        lin = svdq.Fp8Linear.from_quantized(svdq.quantize_fp8(weights(K, N, N), biases(N, K)))
        more, gate, product = {}, biases(N, 3), svdq.fp8_linear
    want = lin(x, residual=res, gate=gate, **more)
    qx, sx = svdq.quantize_act_fp8(x)
    a = {"qx": qx, "sx": sx, "qw": lin.qw, "sw": lin.sw, "bias": lin.bias, **more}
    for name in ("residual", "gate"):
        kw = dict(residual=res, gate=gate)
        kw[name] = kw[name].clone().requires_grad_()
        before = kw["residual"].detach().clone()
        with pytest.raises(ValueError, match="gradient"):
            lin(x, **kw, **more)
        with pytest.raises(ValueError, match="gradient"):
            lin(x, y=kw["residual"], **kw, **more)
        with pytest.raises(ValueError, match="gradient"):
            product(**a, **kw)
        assert torch.equal(kw["residual"], before)
        with torch.no_grad():
            assert torch.equal(lin(x, **kw, **more), want)
    # added outside, it is recorded
    r = res.clone().requires_grad_()
    (r + lin(x, **more)).sum().backward()
    assert (r.grad == 1).all()
