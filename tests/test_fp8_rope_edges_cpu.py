"""Host-side checks of the 8-bit layers and the rotary positions at the calls
that could go wrong, without a GPU."""
import ctypes

import numpy as np
import pytest
import torch

import bit_quantized_diffusion_svdq_amd as svdq
from oracle import fp8 as ofp8
from test_fp8_rope_cpu import (A, ALIGN, B, C, D, E, F, NULL, OK, SHAPE, _act, _few, _few_grouped, _gemm, _heads, _weight, lib,
                               valid)


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


# ---------------------------------------------------------------- tokens in groups

def _rope(lib, q=None, k=None, offs=E + 64, groups=2, T=5):
    q = _heads() if q is None else q
    return lib.svdq_rope_axes_grouped(ctypes.addressof(q), ctypes.addressof(k) if k else None, T, 64, 0, C, 0, 3, D, E, 32, 0, 0,
                                      1e-6, offs, groups, None)


def test_rope_axes_grouped_rejects(lib):
    assert _rope(lib, groups=0) == SHAPE and _rope(lib, groups=-1) == SHAPE and _rope(lib, groups=65537) == SHAPE
    assert _rope(lib, offs=None) == NULL and _rope(lib, offs=E + 2) == ALIGN
    assert _rope(lib, T=0, offs=None) == OK
    valid(_rope(lib))
    valid(_rope(lib, k=_heads(heads=0), groups=65536))


@pytest.mark.parametrize("offs", [torch.zeros(3, dtype=torch.int64), torch.zeros(1, dtype=torch.int32),
                                  torch.zeros((2, 2), dtype=torch.int32), torch.zeros(6, dtype=torch.int32)[::2]])
def test_rope_axes_refuses_offsets(offs, monkeypatch):
    class Gpu(torch.Tensor):
        """A host tensor that says it is on a GPU: the checks before the call."""
        device = torch.device("cuda", 0)

    a = {n: t.as_subclass(Gpu) if isinstance(t, torch.Tensor) else t for n, t in _rope_args().items()}
    a["plan"].turns = a["plan"].turns.as_subclass(Gpu)
    with pytest.raises(ValueError, match="offsets must be"):
        svdq.rope_axes(**a, offsets=offs)


# ---------------------------------------------------------------- a block's refusals come first

class NotCalled:
    """A layer that must not run: its call would overwrite y."""
    N, K = 192, 144

    def __call__(self, *a, **kw):
        raise AssertionError("the projection ran")


def _y(M=3, ld=192, off=0, dt=torch.bfloat16):
    return torch.zeros(M * ld + off + 8, dtype=dt)[off:off + M * ld].view(M, ld)[:, :192]


@pytest.mark.parametrize("kw,text", [
    (dict(y=_y(dt=torch.float32)), "y must be"), (dict(y=_y(ld=196)), "y must be"), (dict(y=_y(off=4)), "y must be"),
    (dict(y=_y(M=4)), "y must be"), (dict(y=torch.zeros((192, 3), dtype=torch.bfloat16).t()), "y must be"),
    (dict(y=_y(M=1).expand(3, 192)), "y must be"), (dict(pos=torch.zeros((3, 3), dtype=torch.int32)), "pos must be"),
    (dict(pos=torch.zeros((3, 2), dtype=torch.int64)), "pos must be"), (dict(x=torch.zeros(144, dtype=torch.bfloat16)), "x must be"),
    (dict(pos=torch.zeros((3, 2), device="meta")), "pos is on"), (dict(y=torch.zeros((3, 192), dtype=torch.bfloat16, device="meta")), "y is on"),
])
def test_qkv_block_refuses_before_it_writes(kw, text):
    block = svdq.FusedQKV(NotCalled(), svdq.RopePlan((16, 16), device="cpu"), 2)
    a = dict(x=torch.zeros((3, 144), dtype=torch.bfloat16), pos=torch.zeros((3, 2), dtype=torch.int32)) | kw
    with pytest.raises(ValueError, match=text):
        block(**a)
    for good in (None, _y(), _y(ld=200), _y(off=8)):
        with pytest.raises(AssertionError, match="ran"):
            block(torch.zeros((3, 144), dtype=torch.bfloat16), torch.zeros((3, 2), dtype=torch.int32), y=good)


def test_qkv_block_refuses_norms_elsewhere():
    norm = torch.ones(32, dtype=torch.bfloat16, device="meta")
    block = svdq.FusedQKV(NotCalled(), svdq.RopePlan((16, 16), device="cpu"), 2, k_norm=norm)
    with pytest.raises(ValueError, match="k_norm is on"):
        block(torch.zeros((3, 144), dtype=torch.bfloat16), torch.zeros((3, 2), dtype=torch.int32))
    with pytest.raises(ValueError, match="q_norm"):
        svdq.FusedQKV(NotCalled(), svdq.RopePlan((16, 16), device="cpu"), 2, q_norm=torch.ones(64, dtype=torch.bfloat16)[::2])


# ---------------------------------------------------------------- outputs over other tensors

@pytest.mark.parametrize("q,k", [
    (dict(x=A, y=C), dict(x=C, y=A)),                       # the outputs swapped
    (dict(x=A, y=B), dict(x=C, y=B)), (dict(x=A, y=C), dict(x=C, y=B)), (dict(x=A, y=B), dict(x=C, y=A)),
    (dict(x=A, y=A, yts=512), dict(x=C, y=C)), (dict(x=A, y=A, yts=64, yhs=320), dict(x=C, y=C)),
    (dict(x=A, y=A), dict(x=C, y=C, ts=0)), (dict(x=A, y=A), dict(x=C, y=C, hs=0)),
])
def test_rope_axes_rejects_outputs_over_other_tensors(lib, q, k):
    assert _rope(lib, q=_heads(**q), k=_heads(**k)) == SHAPE and b"" != lib.svdq_last_error()


def test_rope_axes_accepts_in_place(lib):
    valid(_rope(lib, q=_heads(x=A, y=A), k=_heads(x=C, y=C)))
    valid(_rope(lib, q=_heads(x=A, y=B), k=_heads(x=A, y=F)))                            # one input for both
    valid(_rope(lib, q=_heads(x=A, y=A, ts=0, hs=0, heads=1), T=1))                      # strides of one element
    valid(_rope(lib, q=_heads(x=A, y=B), k=_heads(x=A, y=B, heads=0)))


# ---------------------------------------------------------------- streams

def test_a_stream_of_another_gpu_is_refused():
    """Its kernels would run on the GPU that the tensors are not on."""
    from types import SimpleNamespace
    from bit_quantized_diffusion_svdq_amd.fp8 import _on
    t = SimpleNamespace(is_cuda=True, device=torch.device("cuda", 1))
    with pytest.raises(ValueError, match="stream is on cuda:0"):
        _on(t, SimpleNamespace(device=torch.device("cuda", 0)))


# ---------------------------------------------------------------- which kernel a product runs

def _geometric(lo, hi, n):
    return sorted({int(round(lo * (hi / lo) ** (i / (n - 1)))) for i in range(n)})


def test_every_kernel_that_a_product_can_run_has_a_gpu_test():
    """Over sizes of one row to tens of thousands: no kernel outside the GPU
    tests' list, and every size of the list still takes its kernel."""
    from test_gpu_fp8_variants import VARIANTS
    for (index, f32, groups), (M, K, N) in VARIANTS.items():
        assert svdq.svdq_gemm_fp8_variant(M, K, N, groups, f32, 256) == index
    seen = {(svdq.svdq_gemm_fp8_variant(M, max(16, K // 16 * 16), N, E, f32, 256), f32, E > 0)
            for M in _geometric(1, 70000, 25) for K in _geometric(16, 24576, 14) for N in _geometric(1, 32768, 16)
            for E in (0, 1, 3, 8, 33, 256) for f32 in (0, 1)}
    assert seen == {(index, f32, groups > 0) for index, f32, groups in VARIANTS}


@pytest.mark.parametrize("a", [(0, 16, 1, 0, 0, 256), (1, 24, 1, 0, 0, 256), (1, 16, 0, 0, 0, 256), (1, 16, 1, -1, 0, 256),
                               (1, 16, 1, 65537, 0, 256), (1, 16, 1, 0, 2, 256), (1, 16, 1, 0, 0, 0), (1 << 31, 16, 1, 0, 0, 256),
                               (1 << 30, 16, 1 << 20, 0, 0, 256)])
def test_variant_refuses(lib, a):
    with pytest.raises(svdq.SvdqError):
        svdq.svdq_gemm_fp8_variant(*a)
    assert lib.svdq_gemm_fp8_variant(1, 16, 1, 0, 0, 256, None) == NULL


# ---------------------------------------------------------------- outputs that start at another array

def test_outputs_over_inputs_are_rejected(lib):
    ws = dict(M=17, ws=B, wsb=17 * 2048 + 17 * 64)
    for status in (_act(lib, qx=A), _act(lib, sx=A), _act(lib, sx=B), _weight(lib, qw=A), _weight(lib, sw=A), _weight(lib, sw=B),
                   _gemm(lib, False, y=A), _gemm(lib, True, y=C), _few(lib, y=A), _few(lib, y=C), _few_grouped(lib, y=A),
                   _few(lib, **ws, y=B), _few(lib, **{**ws, "ws": A}), _few_grouped(lib, **ws, y=C)):
        assert status == SHAPE and b"overlap" in lib.svdq_last_error()
    valid(_few(lib, **ws, y=A))                              # with a workspace x is read before y is written
