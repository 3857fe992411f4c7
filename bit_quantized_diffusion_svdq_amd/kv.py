"""A paged cache of keys and values in 8 bits, and attention over it, for
blocks whose tokens come in steps or chunks (autoregressive video, text).

A fused projection's keys go into the cache through their norm and rotation
(``KVCache.append``, which turns the queries in the same launch), and the
queries read it (``KVCache.attend``). The cache holds E4M3 codes with one power
of two per 16 tokens, head and side, on pages that the caller deals out;
everything that changes from step to step (page tables, lengths, offsets) is
read on the GPU, so a captured graph follows it.

Marshalling only: the arithmetic is the library's.
"""
from __future__ import annotations

import ctypes
import math

import torch

from . import _lib
from ._lib import KvBatchDesc, KvCacheDesc, RopeHeads, _check, _require, load_library
from .fp8 import _on, _stream_now
from .rope import PAIRING, RopePlan

_BF16, _I32 = torch.bfloat16, torch.int32
_NO_TURN = (None, 0, 1, None, None, 0, 0)


def _heads_of(x, name, T, D):
    """(heads, token stride, head stride) of a source or an output [T, heads, D]; an axis of one
    element has no stride of its own."""
    shape = x.shape
    if len(shape) != 3 or shape[0] != T or shape[2] != D or x.dtype is not _BF16:
        raise ValueError(f"{name} must be bf16 [{T}, heads, {D}], got {tuple(shape)} {x.dtype}")
    ts, hs, es = x.stride()
    if es != 1:
        raise ValueError(f"{name} must have contiguous heads (stride(2) == 1)")
    H = shape[1]
    if H == 1:
        hs = D
    return H, (ts if T > 1 else H * hs), hs


def _norm_at(name, w, D, gpu):
    if not (w.dtype is _BF16 and w.shape == (D,) and w.is_contiguous()):
        raise ValueError(f"{name} must be a contiguous bf16 vector of {D} values")
    if w.get_device() != gpu:
        raise ValueError(f"{name} is on {w.device}, the cache on cuda:{gpu}")
    return w.data_ptr()


class KVCache:
    """``pages`` pages of ``page_size`` tokens (a multiple of 64) of
    ``kv_heads`` key and value heads of ``head_dim`` channels (a multiple of 8,
    at most 256; kept as the next multiple of 64). ``data`` uint8 [pages,
    kv_heads, page_size / 64, 2, 4, ceil(head_dim / 64), 1024] and ``scales`` uint8
    [pages, kv_heads, page_size / 64, 2, 4] may be given (include/svdq.h has
    their layout); else they are allocated. Pages need no clearing between
    users.

    A batch of B sequences: ``table`` int32 [B, width], row b the pages of
    sequence b in order (a number outside [0, pages): no page; its tokens are
    neither stored nor seen); ``lengths`` int32 [B], tokens of each sequence in
    the cache once the call's are in; ``offsets`` int32 [B + 1] where the call's
    T tokens, sorted by sequence, begin and end (None: T / B each). All on the
    GPU and read there: bad values are not reported, and nothing outside the
    arrays is touched."""

    def __init__(self, pages: int, kv_heads: int, head_dim: int, page_size: int = 64, device="cuda", data=None,
                 scales=None):
        _require(pages >= 1 and kv_heads >= 1, f"pages and kv_heads must be positive, got {pages} and {kv_heads}")
        _require(head_dim % 8 == 0 and 8 <= head_dim <= 256, f"head_dim must be a multiple of 8 in [8, 256], got {head_dim}")
        _require(page_size % 64 == 0 and 64 <= page_size <= 65536,
                 f"page_size must be a multiple of 64 in [64, 65536], got {page_size}")
        self.pages, self.kv_heads, self.head_dim, self.page_size = int(pages), int(kv_heads), int(head_dim), int(page_size)
        lead = (self.pages, self.kv_heads, self.page_size // 64, 2, 4)
        shape = (*lead, -(-self.head_dim // 64), 1024)
        for name, t, want in (("data", data, shape), ("scales", scales, lead)):
            _require(t is None or (tuple(t.shape) == want and t.dtype is torch.uint8 and t.is_contiguous()),
                     f"{name} must be contiguous uint8 {list(want)}")
        _require(data is None or scales is None or data.device == scales.device, "data and scales must be on one device")
        device = device if data is None and scales is None else (data if data is not None else scales).device
        self._data = torch.zeros(shape, dtype=torch.uint8, device=device) if data is None else data
        self._scales = torch.full(lead, 7, dtype=torch.uint8, device=device) if scales is None else scales
        _require(self._data.data_ptr() % 16 == 0 and self._scales.data_ptr() % 8 == 0,
                 "data needs an address of 16 bytes, scales of 8")
        self._desc = KvCacheDesc(self._data.data_ptr(), self._scales.data_ptr(), self.pages, self.kv_heads, self.head_dim,
                                 self.page_size)
        self._at = ctypes.addressof(self._desc)
        self._gpu = self._data.get_device()          # (numbers compare in half the time of devices)

    @property
    def data(self) -> torch.Tensor:                  # (not to be bound anew: the calls have its address)
        return self._data

    @property
    def scales(self) -> torch.Tensor:
        return self._scales

    def _batch(self, T, table, lengths, offsets):
        if not (table.dtype is _I32 and table.dim() == 2 and table.shape[0] >= 1 and table.is_contiguous()):
            raise ValueError(f"table must be contiguous int32 [sequences, width], got {tuple(table.shape)} {table.dtype}")
        B, width = table.shape
        if not (lengths.dtype is _I32 and lengths.shape == (B,) and lengths.is_contiguous()):
            raise ValueError(f"lengths must be a contiguous int32 vector of {B} values, got {tuple(lengths.shape)} {lengths.dtype}")
        if offsets is None:
            if T % B:
                raise ValueError(f"{T} tokens are not a multiple of {B} sequences: offsets are needed")
        elif not (offsets.dtype is _I32 and offsets.shape == (B + 1,) and offsets.is_contiguous()):
            raise ValueError(f"offsets must be a contiguous int32 vector of {B + 1} values, got {tuple(offsets.shape)} {offsets.dtype}")
        gpu = self._gpu
        if gpu < 0:
            raise ValueError(f"the cache must be on a GPU device, got {self.data.device}")
        if table.get_device() != gpu or lengths.get_device() != gpu or (offsets is not None and offsets.get_device() != gpu):
            raise ValueError(f"table, lengths or offsets is not on cuda:{gpu}")
        return KvBatchDesc(table.data_ptr(), lengths.data_ptr(), None if offsets is None else offsets.data_ptr(), T, B, width)

    def append(self, k, v, table, lengths, offsets=None, pos=None, plan: RopePlan | None = None, k_norm=None, q=None,
               q_norm=None, q_out=None, eps: float = 1e-6, stream=None):
        """k and v bf16 [T, kv_heads, head_dim] (strided views allowed, token
        and head strides multiples of 8, addresses of 16 bytes) into the cache:
        keys through an RMS norm of each head (k_norm [head_dim]) and the
        rotation of ``plan`` at pos [T, axes] (int32 or fp32) where given, then
        both as E4M3 codes (the keys' norm and rotation in 64 bits, rounded once).
        q [T, heads, head_dim]: its norm and rotation (as rope_axes') in the same launch, into q_out (q itself, a buffer of any such layout, or a
        new one), which is returned. Tokens of no sequence are neither stored nor
        turned. Nothing is recorded for autograd: k, v and q that require a
        gradient are refused while it is on."""
        D, gpu = self.head_dim, self._gpu
        if k.dim() != 3:
            raise ValueError(f"k must be [T, {self.kv_heads}, {D}], got {tuple(k.shape)}")
        T = k.shape[0]
        if (k.requires_grad or v.requires_grad or (q is not None and q.requires_grad)) and torch.is_grad_enabled():
            raise ValueError("k, v or q requires a gradient, which this call does not record: call it under torch.no_grad() "
                             "or on detached tensors")
        kh, kts, khs = _heads_of(k, "k", T, D)
        vh, vts, vhs = _heads_of(v, "v", T, D)
        if kh != self.kv_heads or vh != kh:
            raise ValueError(f"k has {kh} heads and v {vh}, the cache {self.kv_heads}")
        if plan is None:
            if pos is not None:
                raise ValueError("pos and plan belong together")
            turn = _NO_TURN
        else:
            if pos is None:
                raise ValueError("pos and plan belong together")
            if plan.head_dim != D:
                raise ValueError(f"the plan turns heads of {plan.head_dim}, the cache holds {D}")
            f32_pos = pos.dtype is torch.float32
            if not ((f32_pos or pos.dtype is _I32) and pos.shape == (T, plan.axes) and pos.is_contiguous()):
                raise ValueError(f"pos must be contiguous int32 or fp32 [{T}, {plan.axes}], got {tuple(pos.shape)} {pos.dtype}")
            if pos.get_device() != gpu or plan.turns.get_device() != gpu:
                raise ValueError(f"pos is on {pos.device}, the plan on {plan.turns.device}, the cache on {self.data.device}")
            turn = (pos.data_ptr(), f32_pos, plan.axes, plan.turns.data_ptr(), plan.axis.data_ptr(), plan.pairs,
                    PAIRING[plan.pairing])
        batch = self._batch(T, table, lengths, offsets)
        if k.get_device() != gpu or v.get_device() != gpu:
            raise ValueError(f"k is on {k.device}, v on {v.device}, the cache on cuda:{gpu}")
        k_norm = None if k_norm is None else _norm_at("k_norm", k_norm, D, gpu)
        qs = q_at = None
        if q is not None:
            qh, qts, qhs = _heads_of(q, "q", T, D)
            if qh < 1:
                raise ValueError("q must have at least one head")
            yts, yhs = qh * D, D
            if q_out is not None:
                yh, yts, yhs = _heads_of(q_out, "q_out", T, D)
                if yh != qh:
                    raise ValueError(f"q_out must have {qh} heads, got {yh}")
            if q.get_device() != gpu or (q_out is not None and q_out.get_device() != gpu):
                raise ValueError(f"q or q_out is not on cuda:{gpu}")
            q_norm = None if q_norm is None else _norm_at("q_norm", q_norm, D, gpu)
        elif q_norm is not None or q_out is not None:
            raise ValueError("q_norm and q_out need q")
        with _on(k, stream):
            if q is not None:
                if q_out is None:
                    q_out = q.new_empty(T, qh, D)
                qs = RopeHeads(q.data_ptr(), qts, qhs, qh, q_norm, q_out.data_ptr(), yts, yhs)
                q_at = ctypes.addressof(qs)
            ks = RopeHeads(k.data_ptr(), kts, khs, kh, k_norm)
            vs = RopeHeads(v.data_ptr(), vts, vhs, vh)
            _check(load_library().svdq_kv_append(self._at, ctypes.addressof(batch), q_at, ctypes.addressof(ks),
                                                 ctypes.addressof(vs), *turn, eps, _stream_now()), "svdq_kv_append")
        return q_out

    def attend(self, q, table, lengths, offsets=None, causal: bool = True, window: int = 0, scale: float | None = None,
               out=None, stream=None):
        """softmax(scale q k^T) v over each sequence's cached tokens, for its
        last tokens' queries q bf16 [T, heads, head_dim] (heads a multiple of
        kv_heads; query head i reads key head i // (heads // kv_heads); strides
        as append's) -> [T, heads, head_dim]. The query at position p sees the
        keys of [max(0, p - window + 1), p + 1) if causal, else up to the
        sequence's length; window 0: from 0. One that sees none gives zeros.
        scale: 1 / sqrt(head_dim) by default. out: q itself or a buffer of any
        such layout; rows of no sequence are left as they are in it and are
        unspecified in a new one. Nothing is recorded for autograd.

        Scores are summed by the E4M3 matrix instructions, which drop what falls
        13 bits below the largest of each 8 products (at most 9e-4 of a score's
        larger terms); query channels below 1/896 of the largest are off by up to
        2^-17.8 of it; weights are rounded to bf16 before they meet the values,
        statistics and sums are fp32. Outputs are some 2.1e-3 of their size from
        the definition's (rms; their own rounding to bf16 is 1.7e-3 of that).

        The sequences of a call run in one kernel, which the mean of their tokens
        chooses: single tokens and prompts take less time in a call each. Work and
        workspace are planned for sequences as long as ``table`` is wide: 512
        queries of 24 heads over 1000 keys take 34 us with a table for 1024
        tokens, 66 us and 102 MB with one for 131072."""
        D, gpu = self.head_dim, self._gpu
        if q.dim() != 3:
            raise ValueError(f"q must be [T, heads, {D}], got {tuple(q.shape)}")
        if q.requires_grad and torch.is_grad_enabled():
            raise ValueError("q requires a gradient, which this call does not record: call it under torch.no_grad() or on "
                             "a detached tensor")
        T = q.shape[0]
        H, ts, hs = _heads_of(q, "q", T, D)
        if H < 1 or H % self.kv_heads:
            raise ValueError(f"q must have a multiple of {self.kv_heads} heads, got {H}")
        if scale is None:
            scale = 1.0 / math.sqrt(D)
        if not (0.0 < scale < math.inf):
            raise ValueError(f"scale must be positive and finite, got {scale}")
        if not 0 <= window < 1 << 31:
            raise ValueError(f"window must be in [0, 2^31), got {window}")
        batch = self._batch(T, table, lengths, offsets)
        yts, yhs = H * D, D
        if out is not None:
            yh, yts, yhs = _heads_of(out, "out", T, D)
            if yh != H:
                raise ValueError(f"out must have {H} heads, got {yh}")
        if q.get_device() != gpu or (out is not None and out.get_device() != gpu):
            raise ValueError(f"q or out is not on cuda:{gpu}")
        lib, at = load_library(), ctypes.addressof(batch)
        with _on(q, stream):
            if out is None:
                out = q.new_empty(T, H, D)
            need = ctypes.c_int64(0)
            _check(lib.svdq_kv_attend_workspace_size(self._at, at, H, ctypes.addressof(need)), "svdq_kv_attend_workspace_size")
            ws = q.new_empty(need.value, dtype=torch.uint8) if need.value else None
            qs = RopeHeads(q.data_ptr(), ts, hs, H, None, out.data_ptr(), yts, yhs)
            _check(lib.svdq_kv_attend(self._at, at, ctypes.addressof(qs), scale, bool(causal), window,
                                      None if ws is None else ws.data_ptr(), need.value, _stream_now()), "svdq_kv_attend")
        return out
