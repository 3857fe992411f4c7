"""What the residual of the 8-bit layers and the block around the cache refuse,
on tensors of the CPU: before anything would run."""
import pytest
import torch

import bit_quantized_diffusion_svdq_amd as svdq
from bit_quantized_diffusion_svdq_amd.fp8 import _residual


def t(*shape, dtype=torch.bfloat16):
    return torch.zeros(*shape, dtype=dtype)


def block(**kw):
    """4 query heads over 2 of 64, K = 32 (an 8-bit output projection)."""
    class Layer:
        K, N = 32, 8 * 64

        def __call__(self, x):
            raise AssertionError("the projection ran")

    out = svdq.Fp8Linear(t(32, 256, dtype=torch.float8_e4m3fn), t(1, 2, dtype=torch.float32))
    qkv = svdq.FusedQKV(Layer(), svdq.RopePlan((64,), device="cpu"), 4, 2)
    return svdq.CachedAttention(qkv, out, svdq.KVCache(2, 2, 64, device="cpu"), **kw)


GOOD = dict(x=t(3, 32), pos=t(3, 1, dtype=torch.int32), table=t(1, 1, dtype=torch.int32), lengths=t(1, dtype=torch.int32),
            residual=t(3, 32), gate=t(32))


@pytest.mark.parametrize("name", ["residual", "gate"])
def test_residual_refuses_a_gradient(name):
    a = dict(residual=t(3, 8), gate=t(8))
    a[name] = a[name].requires_grad_()
    cpu = torch.device("cpu")
    with pytest.raises(ValueError, match="gradient"):
        _residual(a["residual"], a["gate"], 3, 8, torch.bfloat16, (), cpu)
    with torch.no_grad():
        assert _residual(a["residual"], a["gate"], 3, 8, torch.bfloat16, (), cpu).ld == 8
    assert _residual(a["residual"].detach(), a["gate"].detach(), 3, 8, torch.bfloat16, (), cpu).ld == 8


@pytest.mark.parametrize("name", ["x", "residual", "gate"])
def test_block_refuses_a_gradient(name):
    a = dict(GOOD)
    a[name] = a[name].clone().requires_grad_()
    with pytest.raises(ValueError, match="gradient"):
        block()(**a)


@pytest.mark.parametrize("kw", [dict(scale=0.0), dict(scale=-1.0), dict(scale=float("nan")), dict(scale=float("inf")),
                                dict(scale=3e38), dict(window=-1), dict(window=1 << 31)], ids=str)
def test_block_refuses_what_attention_would(kw):
    """At once, not after a call has written its keys and values."""
    with pytest.raises(ValueError, match="scale|window"):
        block(**kw)
    assert block(scale=2.0 ** 126, window=(1 << 31) - 1).scale == 2.0 ** 126
