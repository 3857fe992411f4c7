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

import ctypes
import math
from typing import Sequence

import torch

from ._lib import RopeHeads, _check, _require, load_library
from .fp8 import _groups, _on, _stream_now

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
    if x.dim() != 3 or x.shape[2] != D:
        raise ValueError(f"{name} must be [T, heads, {D}], got {tuple(x.shape)}")
    if x.stride(2) != 1:
        raise ValueError(f"{name} must have contiguous heads (stride(2) == 1)")


def _check_side(name, x, norm, out, D, dt, dev):
    if norm is not None and not (norm.dtype is dt and norm.shape == (D,) and norm.is_contiguous()):
        raise ValueError(f"{name}_norm must be a contiguous {dt} vector of {D} values")
    if out is not None:
        _heads(out, f"{name}_out", D)
        if out.shape != x.shape or out.dtype is not dt:
            raise ValueError(f"{name}_out must be {tuple(x.shape)} {dt}")
    if dev.type == "cuda":
        for t in (norm, out):
            if t is not None and t.device != dev:
                raise ValueError(f"{name}_norm or {name}_out is on {t.device}, expected {dev}")


def _strides(x, T, H, D):
    """Token and head stride; an axis of one element has none of its own."""
    ts, hs, _ = x.stride()
    if H == 1:
        hs = D
    return (ts if T > 1 else H * hs), hs


def _side(x, y, norm, T, H, D):
    ts, hs = _strides(x, T, H, D)
    yts, yhs = (H * D, D) if y is None else _strides(y, T, H, D)
    if y is None:
        y = x.new_empty(T, H, D)
    return y, RopeHeads(x.data_ptr(), ts, hs, H, None if norm is None else norm.data_ptr(), y.data_ptr(), yts, yhs)


def rope_axes(q, k, pos, plan: RopePlan, q_norm=None, k_norm=None, eps: float = 1e-6, inverse: bool = False,
              q_out=None, k_out=None, stream=None, offsets=None):
    """q [T, Hq, D] and k [T, Hk, D] (or None), bf16 or fp32, strided views
    allowed (token and head strides multiples of 8), rotated by pos [T, axes]
    (int32 or fp32) after an RMS norm of each head where q_norm / k_norm [D]
    is given: (q', k'), or q' alone if k is None. q_out / k_out may be q / k
    themselves (in place) or buffers of any such layout; addresses are
    multiples of 16 bytes. inverse undoes the rotation; without a norm that is
    also how a gradient goes back through it. Nothing is recorded for
    autograd: q and k that require a gradient are refused while it is on, the
    norms' weights are taken as constants. offsets (int32 [groups + 1] on the
    GPU, as a grouped layer takes them): tokens of no group are left as they
    are in a given output and are unspecified in a new one."""
    D, dt, dev = plan.head_dim, q.dtype, q.device
    _heads(q, "q", D)
    T, hq, _ = q.shape
    if dt is not torch.bfloat16 and dt is not torch.float32:
        raise ValueError(f"q must be bf16 or fp32, got {dt}")
    if hq < 1:
        raise ValueError("q must have at least one head")
    if (q.requires_grad or (k is not None and k.requires_grad)) and torch.is_grad_enabled():
        raise ValueError("q or k requires a gradient, which this call does not record: call it under torch.no_grad() or "
                         "on detached tensors (inverse=True turns a gradient back)")
    hk = 0
    if k is not None:
        _heads(k, "k", D)
        hk = k.shape[1]
        if k.shape[0] != T or k.dtype is not dt:
            raise ValueError(f"k must have {T} tokens of {dt}, got {tuple(k.shape)} {k.dtype}")
    elif k_norm is not None or k_out is not None:
        raise ValueError("k_norm and k_out need k")
    if q_norm is not None or q_out is not None:
        _check_side("q", q, q_norm, q_out, D, dt, dev)
    if k_norm is not None or k_out is not None:
        _check_side("k", k, k_norm, k_out, D, dt, dev)
    f32_pos = pos.dtype is torch.float32
    if not ((f32_pos or pos.dtype is torch.int32) and pos.shape == (T, plan.axes) and pos.is_contiguous()):
        raise ValueError(f"pos must be contiguous int32 or fp32 [{T}, {plan.axes}], got {tuple(pos.shape)} {pos.dtype}")
    if dev.type != "cuda":
        raise ValueError(f"tensors must be on a GPU device, got {dev}")
    if pos.device != dev or plan.turns.device != dev or (k is not None and k.device != dev):
        raise ValueError(f"k, pos or the plan is not on {dev}")
    groups = 0
    if offsets is not None:
        groups = _groups(offsets)
        if offsets.device != dev:
            raise ValueError(f"offsets is on {offsets.device}, expected {dev}")
    with _on(q, stream):
        q_out, qs = _side(q, q_out, q_norm, T, hq, D)
        ks = None
        if k is not None:
            k_out, ks = _side(k, k_out, k_norm, T, hk, D)
        q_at, k_at = ctypes.addressof(qs), None if ks is None else ctypes.addressof(ks)
        if not groups:
            _check(load_library().svdq_rope_axes(q_at, k_at, T, D, dt is torch.float32, pos.data_ptr(), f32_pos,
                                                 plan.axes, plan.turns.data_ptr(), plan.axis.data_ptr(), plan.pairs,
                                                 PAIRING[plan.pairing], bool(inverse), eps, _stream_now()),
                   "svdq_rope_axes")
        else:
            _check(load_library().svdq_rope_axes_grouped(q_at, k_at, T, D, dt is torch.float32, pos.data_ptr(), f32_pos,
                                                         plan.axes, plan.turns.data_ptr(), plan.axis.data_ptr(),
                                                         plan.pairs, PAIRING[plan.pairing], bool(inverse), eps,
                                                         offsets.data_ptr(), groups, _stream_now()),
                   "svdq_rope_axes_grouped")
    return q_out if k is None else (q_out, k_out)
