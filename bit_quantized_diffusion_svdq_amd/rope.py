"""Rotary positions with several axes (time, height, width of images and
video) on the query and key heads of an attention block.

A diffusion transformer's attention reads the fused [Q | K | V] projection
(fused.py) through an optional RMS norm of each head and a rotation whose
angles come from positions on several axes: every axis owns a run of a head's
pairs, with frequencies theta^(-2 i / d) over its d channels. One launch
norms and rotates queries and keys, in place or into buffers of any layout.

Marshalling only: the arithmetic is the library's.
"""
from __future__ import annotations

import math
from typing import Sequence

import torch

from . import _lib
from ._lib import RopeHeads, _check_same_device, _require
from .fp8 import _on

PAIRING = {"interleaved": 0, "half": 1}


class RopePlan:
    """How the pairs of a head belong to the axes of a position: axis a owns
    ``dims[a]`` channels (even; their sum a multiple of 8, at most
    ``head_dim``; channels past it do not turn), pair i of it turning by
    position * theta^(-2 i / dims[a]). ``theta`` is one number or one per
    axis; ``freqs`` gives every pair's angular frequency instead. ``pairing``
    "interleaved": pair i of a head is channels (2i, 2i + 1); "half": (i, i +
    pairs)."""

    def __init__(self, dims: Sequence[int], head_dim: int | None = None, theta=10000.0,
                 pairing: str = "interleaved", freqs: Sequence[float] | None = None, device="cuda"):
        dims = [int(d) for d in dims]
        _require(1 <= len(dims) <= 8, f"dims must name 1 to 8 axes, got {len(dims)}")
        _require(all(d >= 0 and d % 2 == 0 for d in dims), f"every axis needs an even number of channels, got {dims}")
        turned = sum(dims)
        self.head_dim = turned if head_dim is None else int(head_dim)
        _require(self.head_dim % 8 == 0 and 8 <= self.head_dim <= 512,
                 f"head_dim must be a multiple of 8 in [8, 512], got {self.head_dim}")
        _require(turned % 8 == 0 and turned <= self.head_dim,
                 f"the axes' channels ({turned}) must add up to a multiple of 8, at most head_dim {self.head_dim}")
        _require(pairing in PAIRING, f"pairing must be one of {sorted(PAIRING)}, got {pairing!r}")
        self.dims, self.axes, self.pairs, self.pairing = tuple(dims), len(dims), turned // 2, pairing
        thetas = [float(t) for t in theta] if isinstance(theta, (list, tuple)) else [float(theta)] * len(dims)
        _require(len(thetas) == len(dims) and all(t > 0 for t in thetas), "theta must be one positive number or one per axis")
        if freqs is None:
            freqs = [th ** (-2.0 * i / d) for d, th in zip(dims, thetas) for i in range(d // 2)]
        freqs = [float(f) for f in freqs]
        _require(len(freqs) == self.pairs, f"freqs must hold {self.pairs} values, got {len(freqs)}")
        # an empty array still needs an address
        self.turns = torch.tensor([f / (2.0 * math.pi) for f in freqs] or [0.0], dtype=torch.float64, device=device)
        self.axis = torch.tensor([a for a, d in enumerate(dims) for _ in range(d // 2)] or [0], dtype=torch.int32,
                                 device=device)


def _heads(x, name, D):
    _require(x.dim() == 3 and x.shape[2] == D, f"{name} must be [T, heads, {D}], got {tuple(x.shape)}")
    _require(x.stride(2) == 1, f"{name} must have contiguous heads (stride(2) == 1)")


def _strides(x):
    """Token and head stride; an axis of one element has none of its own."""
    T, H, D = x.shape
    hs = x.stride(1) if H > 1 else D
    return (x.stride(0) if T > 1 else max(H * hs, D)), hs


def _side(x, y, norm):
    ts, hs = _strides(x)
    yts, yhs = _strides(y)
    return RopeHeads(x.data_ptr(), ts, hs, x.shape[1], None if norm is None else norm.data_ptr(), y.data_ptr(), yts, yhs)


def rope_axes(q, k, pos, plan: RopePlan, q_norm=None, k_norm=None, eps: float = 1e-6, inverse: bool = False,
              q_out=None, k_out=None, stream=None):
    """q [T, Hq, D] and k [T, Hk, D] (or None), bf16 or fp32, strided views
    allowed (token and head strides multiples of 8), rotated by pos [T, axes]
    (int32 or fp32) after an RMS norm of each head where q_norm / k_norm [D]
    is given: (q', k'), or q' alone if k is None. q_out / k_out may be q / k
    themselves (in place) or buffers of any such layout. inverse undoes the
    rotation; without a norm it is also its gradient."""
    D = plan.head_dim
    _heads(q, "q", D)
    T = q.shape[0]
    _require(q.dtype in (torch.bfloat16, torch.float32), f"q must be bf16 or fp32, got {q.dtype}")
    _require(q.shape[1] >= 1, "q must have at least one head")
    sides = [("q", q, q_norm, q_out)]
    if k is not None:
        _heads(k, "k", D)
        _require(k.shape[0] == T and k.dtype == q.dtype, f"k must have {T} tokens of {q.dtype}, got {tuple(k.shape)} {k.dtype}")
        sides.append(("k", k, k_norm, k_out))
    else:
        _require(k_norm is None and k_out is None, "k_norm and k_out need k")
    for name, x, norm, out in sides:
        if norm is not None:
            _require(tuple(norm.shape) == (D,) and norm.dtype == q.dtype and norm.is_contiguous(),
                     f"{name}_norm must be a contiguous {q.dtype} vector of {D} values")
        if out is not None:
            _heads(out, f"{name}_out", D)
            _require(out.shape == x.shape and out.dtype == q.dtype, f"{name}_out must be {tuple(x.shape)} {q.dtype}")
    _require(tuple(pos.shape) == (T, plan.axes) and pos.dtype in (torch.int32, torch.float32) and pos.is_contiguous(),
             f"pos must be contiguous int32 or fp32 [{T}, {plan.axes}], got {tuple(pos.shape)} {pos.dtype}")
    _check_same_device(q, k=k, pos=pos, q_norm=q_norm, k_norm=k_norm, q_out=q_out, k_out=k_out, plan=plan.turns)
    with _on(q):
        outs = [torch.empty((T, x.shape[1], D), dtype=q.dtype, device=q.device) if out is None else out
                for _, x, _, out in sides]
        structs = [_side(x, o, norm) for (_, x, norm, _), o in zip(sides, outs)]
        _lib.svdq_rope_axes(structs[0], structs[1] if k is not None else None, T, D, int(q.dtype == torch.float32),
                            pos, int(pos.dtype == torch.float32), plan.axes, plan.turns, plan.axis, plan.pairs,
                            PAIRING[plan.pairing], int(inverse), eps, stream)
    return (outs[0], outs[1]) if k is not None else outs[0]
