"""8-bit layers: E4M3 weights and activations with an fp32 scale per block of
128 (weights 128 x 128, activations 128 channels of a row), dense and grouped.

For the projections that 4 bits hurt: the donmalab.com page (section on the
two schemes) keeps precision-sensitive projections out of the 4-bit path, and
the remio.ai page (section on the loading path) names a scheme per module.
``Fp8Linear`` stands beside ``SvdqLinear``; ``Fp8GroupedLinear`` holds several
weights of one shape, and the rows of a batch, sorted by group, each meet
their group's (the experts of a mixture, or the text and image streams of a
joint block in one launch).

Marshalling only: the arithmetic is the library's. Tensors may live on any
GPU; a call runs on that GPU's current stream, or on ``stream``, and
allocates what it needs there.
"""
from __future__ import annotations

import contextlib
import ctypes
from dataclasses import dataclass

import torch

from . import _lib
from ._lib import _check, _check_rows, _check_same_device, _require, load_library

BLOCK = 128
E4M3 = torch.float8_e4m3fn


def blocks(n: int) -> int:
    """Blocks of 128 that cover n channels."""
    return (n + BLOCK - 1) // BLOCK


def _on(t: torch.Tensor, stream=None):
    """The tensor's GPU made current, if it is not, and the given stream (a
    torch stream or a raw handle), so that what a call allocates belongs to the
    stream that uses it. (Host tensors: the checks that follow refuse them.)"""
    if not t.is_cuda:
        return _HERE
    if stream is None:
        return _HERE if t.device.index == torch.cuda.current_device() else torch.cuda.device(t.device)
    if isinstance(stream, int):
        stream = torch.cuda.ExternalStream(stream, device=t.device) if stream else torch.cuda.default_stream(t.device)
    elif stream.device != t.device:
        raise ValueError(f"stream is on {stream.device}, the tensors are on {t.device}")
    return torch.cuda.stream(stream)


def _stream_now() -> int:
    """The current stream's handle (small calls are bound by Python: these
    entry points marshal by hand what _lib's functions take apart)."""
    return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())


def _address(t):
    return None if t is None else t.data_ptr()


_HERE = contextlib.nullcontext()
_F32, _BF16 = torch.float32, torch.bfloat16


def _aligned_copy(x):
    """Dense rows at an address that the kernels can read, for rows at one they
    cannot (16 bytes at a time: a broadcast or unaligned stride or address).
    (contiguous() would keep a dense view where it is.)"""
    return x.clone(memory_format=torch.contiguous_format)


def quantize_act_fp8(x: torch.Tensor, stream=None):
    """x: bf16 [M, K] on the GPU (K a multiple of 16; rows may be strided; where
    the row stride is not a multiple of 8 or the address not one of 16 bytes a
    copy is read) -> (qx E4M3 [M, K], sx fp32 [ceil(K/128), M]):
    per row and 128 channels s = max(amax / 448, 2^-120), code = e4m3(x / s)
    (include/svdq.h gives every rounding)."""
    if not (x.is_cuda and x.dtype is _BF16 and x.dim() == 2 and x.is_contiguous()):
        _check_rows(x, "x", _BF16)              # the slow way: says what is wrong, if anything is
        _require(x.shape[1] >= 16 and x.shape[1] % 16 == 0, f"x must have K a positive multiple of 16, got {x.shape[1]}")
        _check_same_device(x)
    M, K = x.shape
    if K < 16 or K % 16:
        raise ValueError(f"x must have K a positive multiple of 16, got {K}")
    ldx = x.stride(0) if M > 1 else K
    with _on(x, stream):
        if ldx < K or ldx % 8 or x.data_ptr() % 16:
            x, ldx = _aligned_copy(x), K
        # (x.new_empty costs half a us less than torch.empty)
        qx, sx = x.new_empty(M, K, dtype=E4M3), x.new_empty(blocks(K), M, dtype=_F32)
        _check(load_library().svdq_quantize_act_fp8(x.data_ptr(), M, K, ldx, qx.data_ptr(), sx.data_ptr(), _stream_now()),
               "svdq_quantize_act_fp8")
    return qx, sx


def _check_product(qx, sx, qw, sw, bias, act, out_dtype, y, groups):
    """Argument checks of the dense (groups 0) and the grouped product. The
    first condition is the usual call and costs the least; what it does not
    pass is looked at one by one and refused with a reason."""
    lead = (groups,) if groups else ()
    dev = qx.device
    if (y is None and qx.dtype is E4M3 and qw.dtype is E4M3 and sx.dtype is _F32 and sw.dtype is _F32
            and dev.type == "cuda" and qw.device == dev and sx.device == dev and sw.device == dev
            and qx.dim() == 2 and qw.dim() == 2 + len(lead) and qx.is_contiguous() and qw.is_contiguous()
            and sx.is_contiguous() and sw.is_contiguous() and act in _lib.ACT
            and (out_dtype is _BF16 or out_dtype is _F32)):
        M, K = qx.shape
        N = qw.shape[-2]
        kb = blocks(K)
        if (K >= 16 and K % 16 == 0 and N >= 1 and qw.shape == (*lead, N, K) and sx.shape == (kb, M)
                and sw.shape == (*lead, blocks(N), kb)
                and (bias is None or (bias.dtype is _BF16 and bias.shape == (*lead, N) and bias.is_contiguous()
                                      and bias.device == dev))):
            return M, K, N, out_dtype
    _check_rows(qx, "qx", E4M3)
    _require(qx.is_contiguous(), "qx must be contiguous [M, K]")
    M, K = qx.shape
    _require(K >= 16 and K % 16 == 0, f"qx must have K a positive multiple of 16, got {K}")
    _require(qw.dim() == 2 + len(lead) and qw.dtype == E4M3 and qw.is_contiguous() and qw.shape[-1] == K
             and qw.shape[:-2] == lead, f"qw must be contiguous E4M3 {[*lead, 'N', K]}, got {tuple(qw.shape)} {qw.dtype}")
    N = qw.shape[-2]
    _require(N >= 1, "qw must have at least one output row")
    _require(tuple(sx.shape) == (blocks(K), M) and sx.dtype == _F32
             and (sx.is_contiguous() or sx.numel() <= 1),
             f"sx must be contiguous fp32 [{blocks(K)}, {M}], got {tuple(sx.shape)} {sx.dtype}")
    want = (*lead, blocks(N), blocks(K))
    _require(tuple(sw.shape) == want and sw.dtype == _F32 and sw.is_contiguous(),
             f"sw must be contiguous fp32 {list(want)}, got {tuple(sw.shape)} {sw.dtype}")
    if bias is not None:
        _require(tuple(bias.shape) == (*lead, N) and bias.dtype == _BF16 and bias.is_contiguous(),
                 f"bias must be contiguous bf16 {[*lead, N]}, got {tuple(bias.shape)} {bias.dtype}")
    _require(act in _lib.ACT, f"act must be one of {sorted(_lib.ACT)}, got {act!r}")
    if y is not None:
        out_dtype = y.dtype
        _require(y.dim() == 2 and tuple(y.shape) == (M, N) and (y.stride(1) == 1 or N == 1)
                 and (y.stride(0) >= N or M <= 1),
                 f"y must be [{M}, {N}] with contiguous columns and rows that do not overlap")
    _require(out_dtype in (_BF16, _F32), f"y must be bf16 or fp32, got {out_dtype}")
    _check_same_device(qx, sx=sx, qw=qw, sw=sw, bias=bias, y=y)
    return M, K, N, out_dtype


def _output(y, M, N, out_dtype, like):
    """(y, its row stride)"""
    if y is None:
        return like.new_empty(M, N, dtype=out_dtype), N
    return y, y.stride(0) if M > 1 else N


def _residual(residual, gate, M, N, dtype, lead, dev):
    """What the outputs join, or None: checked (``dtype``: the outputs')."""
    if torch.is_grad_enabled() and ((residual is not None and residual.requires_grad)
                                    or (gate is not None and gate.requires_grad)):
        raise ValueError("residual or gate requires a gradient, which this call does not record: call it under torch.no_grad() "
                         "or on detached tensors, or add the layer's outputs outside")
    if residual is None:
        if gate is not None:
            raise ValueError("gate needs a residual")
        return None
    if not (residual.shape == (M, N) and residual.dtype is dtype and (residual.stride(1) == 1 or N == 1)
            and (residual.stride(0) >= N or M <= 1)):
        raise ValueError(f"residual must be {dtype} [{M}, {N}] with contiguous columns and rows that do not overlap, got "
                         f"{tuple(residual.shape)} {residual.dtype}, strides {residual.stride()}")
    if gate is not None and not (gate.dtype is _BF16 and gate.shape == (*lead, N) and gate.is_contiguous()):
        raise ValueError(f"gate must be contiguous bf16 {[*lead, N]}, got {tuple(gate.shape)} {gate.dtype}")
    if residual.device != dev or (gate is not None and gate.device != dev):
        raise ValueError(f"residual or gate is not on {dev}")
    return _lib.Fp8Residual(residual.data_ptr(), residual.stride(0) if M > 1 else N, _address(gate))


def fp8_linear(qx, sx, qw, sw, bias=None, act: str = "none", out_dtype=torch.bfloat16, y=None, stream=None,
               residual=None, gate=None):
    """act(sum_b sx sw P_b + bias) for already quantised activations: qx E4M3
    [M, K], sx fp32 [ceil(K/128), M] (quantize_act_fp8), qw E4M3 [N, K], sw
    fp32 [ceil(N/128), ceil(K/128)], bias bf16 [N] or None -> y [M, N] (bf16
    or fp32; rows of a given y may be strided; y must not overlap the inputs).
    residual [M, N] of the outputs' type (rows may be strided; y itself: in
    place): the outputs are residual + gate * act(...), gate bf16 [N] or None
    (ones), joined in fp32 before the one rounding. Nothing is recorded for
    autograd: a residual or gate that requires a gradient is refused while it is on.

    The output type also chooses the sums. bf16: the E4M3 matrix instructions,
    which drop what falls 13 bits below the largest of each 8 products, 1.4e-5
    to 3.1e-5 of the outputs' rms (a fiftieth of their rounding; outputs that
    cancel to a twentieth of the others lose as much as to the rounding).
    fp32: every product and sum in fp32, at half the matrix rate; round its
    result where bf16 outputs of such sums are wanted."""
    M, K, N, out_dtype = _check_product(qx, sx, qw, sw, bias, act, out_dtype, y, 0)
    res = _residual(residual, gate, M, N, out_dtype, (), qx.device)
    with _on(qx, stream):
        y, ldy = _output(y, M, N, out_dtype, qx)
        if res is not None:
            _check(load_library().svdq_gemm_fp8_residual(
                qx.data_ptr(), sx.data_ptr(), M, K, qw.data_ptr(), sw.data_ptr(), N, None, 0, _address(bias), _lib.ACT[act],
                ctypes.addressof(res), y.data_ptr(), out_dtype is _F32, ldy, _stream_now()), "svdq_gemm_fp8_residual")
            return y
        _check(load_library().svdq_gemm_fp8(qx.data_ptr(), sx.data_ptr(), M, K, qw.data_ptr(), sw.data_ptr(), N,
                                            _address(bias), _lib.ACT[act], y.data_ptr(), out_dtype is _F32, ldy,
                                            _stream_now()), "svdq_gemm_fp8")
    return y


def _groups(offsets) -> int:
    if not (offsets.dtype is torch.int32 and offsets.dim() == 1 and offsets.numel() >= 2 and offsets.is_contiguous()):
        raise ValueError(f"offsets must be a contiguous int32 vector of groups + 1 values, got {tuple(offsets.shape)} "
                         f"{offsets.dtype}")
    return offsets.numel() - 1


def fp8_grouped_linear(qx, sx, offsets, qw, sw, bias=None, act: str = "none", out_dtype=torch.bfloat16, y=None,
                       stream=None, residual=None, gate=None):
    """fp8_linear with a weight per group: rows offsets[g] .. offsets[g + 1] - 1
    of qx meet qw[g] [N, K], sw[g], bias[g]. offsets: int32 [groups + 1] on
    the GPU, rising, within [0, M] (read there: no synchronisation, so bad
    values are not reported: they are clamped, and one that falls counts as
    the largest before it). Rows of
    no group (before offsets[0], from offsets[-1] on) are left as they are in
    a given y and are unspecified in a new one. The sums are fp8_linear's, and
    so is residual; gate is bf16 [groups, N]."""
    groups = _groups(offsets)
    M, K, N, out_dtype = _check_product(qx, sx, qw, sw, bias, act, out_dtype, y, groups)
    if offsets.device != qx.device:
        raise ValueError(f"offsets is on {offsets.device}, expected {qx.device}")
    res = _residual(residual, gate, M, N, out_dtype, (groups,), qx.device)
    with _on(qx, stream):
        y, ldy = _output(y, M, N, out_dtype, qx)
        if res is not None:
            _check(load_library().svdq_gemm_fp8_residual(
                qx.data_ptr(), sx.data_ptr(), M, K, qw.data_ptr(), sw.data_ptr(), N, offsets.data_ptr(), groups,
                _address(bias), _lib.ACT[act], ctypes.addressof(res), y.data_ptr(), out_dtype is _F32, ldy, _stream_now()),
                "svdq_gemm_fp8_residual")
            return y
        _check(load_library().svdq_gemm_fp8_grouped(qx.data_ptr(), sx.data_ptr(), M, K, qw.data_ptr(), sw.data_ptr(), N,
                                                    offsets.data_ptr(), groups, _address(bias), _lib.ACT[act],
                                                    y.data_ptr(), out_dtype is _F32, ldy, _stream_now()),
               "svdq_gemm_fp8_grouped")
    return y


def _workspace_bytes(M, K) -> int:
    """svdq_linear_fp8_workspace_size, without the call."""
    kb = blocks(K)
    return 0 if M <= 16 and M * kb <= 256 else M * K + 4 * kb * M


def _layer(x, qw, sw, bias, act, out_dtype, y, offsets=None, residual=None, gate=None):
    """The layer in one call, or None for a call that is not the usual one
    (the two passes then do it, or say what is wrong)."""
    M, K = x.shape
    kb = blocks(K)
    dev = x.device
    lead = () if offsets is None else (offsets.numel() - 1,)
    if not (M > 0 and x.is_cuda and x.dtype is _BF16 and K >= 16 and K % 16 == 0
            and x.stride(1) == 1 and qw.dtype is E4M3 and sw.dtype is _F32 and qw.device == dev and sw.device == dev
            and qw.dim() == 2 + len(lead) and qw.is_contiguous() and sw.is_contiguous() and act in _lib.ACT):
        return None
    N = qw.shape[-2]
    if not (1 <= N < 1 << 22 and qw.shape == (*lead, N, K) and sw.shape == (*lead, blocks(N), kb)
            and (bias is None or (bias.dtype is _BF16 and bias.shape == (*lead, N) and bias.is_contiguous()
                                  and bias.device == dev))
            and (offsets is None or offsets.device == dev)):
        return None
    need = _workspace_bytes(M, K)
    ldx = x.stride(0) if M > 1 else K
    if y is None:
        if not (out_dtype is _BF16 or out_dtype is _F32):
            return None
        y, ldy = x.new_empty(M, N, dtype=out_dtype), N
    else:
        ldy = y.stride(0) if y.dim() == 2 and M > 1 else N
        if not (y.shape == (M, N) and (y.dtype is _BF16 or y.dtype is _F32) and y.device == dev
                and (y.stride(1) == 1 or N == 1) and ldy >= N):
            return None
        if not need and y.untyped_storage().data_ptr() == x.untyped_storage().data_ptr():
            x, ldx = _aligned_copy(x), K         # in place: y is written while x is read
    if ldx < K or ldx % 8 or x.data_ptr() % 16:
        x, ldx = _aligned_copy(x), K
    f32 = y.dtype is _F32
    res = None
    if residual is not None or gate is not None:
        res = _residual(residual, gate, M, N, y.dtype, lead, dev)
    ws = x.new_empty(need, dtype=torch.uint8) if need else None
    if res is not None:
        _check(load_library().svdq_linear_fp8_residual(
            x.data_ptr(), M, K, ldx, qw.data_ptr(), sw.data_ptr(), N, _address(offsets), lead[0] if lead else 0, _address(bias),
            _lib.ACT[act], ctypes.addressof(res), y.data_ptr(), f32, ldy, _address(ws), need, _stream_now()),
            "svdq_linear_fp8_residual")
        return y
    if offsets is None:
        _check(load_library().svdq_linear_fp8(x.data_ptr(), M, K, ldx, qw.data_ptr(), sw.data_ptr(), N, _address(bias),
                                              _lib.ACT[act], y.data_ptr(), f32, ldy, _address(ws), need, _stream_now()),
               "svdq_linear_fp8")
    else:
        _check(load_library().svdq_linear_fp8_grouped(x.data_ptr(), M, K, ldx, qw.data_ptr(), sw.data_ptr(), N,
                                                      offsets.data_ptr(), lead[0], _address(bias), _lib.ACT[act],
                                                      y.data_ptr(), f32, ldy, _address(ws), need, _stream_now()),
               "svdq_linear_fp8_grouped")
    return y


@dataclass
class Fp8Linear:
    """One 8-bit layer's device arrays."""
    qw: torch.Tensor                # E4M3 [N, K]
    sw: torch.Tensor                # fp32 [ceil(N/128), ceil(K/128)]
    bias: torch.Tensor | None = None  # bf16 [N]

    @property
    def K(self) -> int:
        return self.qw.shape[-1]

    @property
    def N(self) -> int:
        return self.qw.shape[-2]

    @classmethod
    def from_quantized(cls, d: dict) -> "Fp8Linear":
        """From the dict quantize_fp8() returns."""
        return cls(d["qw"], d["sw"], d.get("bias"))

    def __call__(self, x: torch.Tensor, act: str = "none", out_dtype=torch.bfloat16, y=None,
                 stream=None, residual=None, gate=None) -> torch.Tensor:
        """Y [M, N] for bf16 activations x [M, K]: the activation pass, then
        the product, in one call on one stream; in one launch for few rows (M
        <= 16 and M * ceil(K / 128) <= 256: single tokens, pooled
        conditioning). bf16 outputs are summed by the E4M3 matrix
        instructions, fp32 outputs in fp32 (fp8_linear gives the difference).
        residual, gate: Y = residual + gate * act(...), as fp8_linear's."""
        if x.dim() != 2 or x.shape[1] != self.K:
            raise ValueError(f"x must be [M, {self.K}], got {tuple(x.shape)}")
        with _on(x, stream):                     # (the codes are freed on the stream that reads them)
            out = _layer(x, self.qw, self.sw, self.bias, act, out_dtype, y, None, residual, gate)
            if out is not None:
                return out
            qx, sx = quantize_act_fp8(x)
            return fp8_linear(qx, sx, self.qw, self.sw, self.bias, act, out_dtype, y, residual=residual, gate=gate)


@dataclass
class Fp8GroupedLinear:
    """Weights of one shape for several groups of rows."""
    qw: torch.Tensor                # E4M3 [groups, N, K]
    sw: torch.Tensor                # fp32 [groups, ceil(N/128), ceil(K/128)]
    bias: torch.Tensor | None = None  # bf16 [groups, N]

    @property
    def groups(self) -> int:
        return self.qw.shape[0]

    @property
    def K(self) -> int:
        return self.qw.shape[-1]

    @property
    def N(self) -> int:
        return self.qw.shape[-2]

    @classmethod
    def from_quantized(cls, d: dict) -> "Fp8GroupedLinear":
        """From the dict quantize_fp8() returns for a weight [groups, K, N]."""
        return cls(d["qw"], d["sw"], d.get("bias"))

    def __call__(self, x: torch.Tensor, offsets: torch.Tensor, act: str = "none", out_dtype=torch.bfloat16, y=None,
                 stream=None, residual=None, gate=None) -> torch.Tensor:
        """Y [M, N] for bf16 activations x [M, K] sorted by group
        (fp8_grouped_linear's offsets); one call, one launch for few rows,
        the sums and the residual, as Fp8Linear (gate [groups, N])."""
        if x.dim() != 2 or x.shape[1] != self.K:
            raise ValueError(f"x must be [M, {self.K}], got {tuple(x.shape)}")
        if _groups(offsets) != self.groups:
            raise ValueError(f"offsets must hold {self.groups + 1} values, got {offsets.numel()}")
        with _on(x, stream):
            out = _layer(x, self.qw, self.sw, self.bias, act, out_dtype, y, offsets, residual, gate)
            if out is not None:
                return out
            qx, sx = quantize_act_fp8(x)
            return fp8_grouped_linear(qx, sx, offsets, self.qw, self.sw, self.bias, act, out_dtype, y, residual=residual,
                                      gate=gate)
