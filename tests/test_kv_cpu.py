"""Host-side checks of the paged 8-bit cache, its attention and the 8-bit
layers' residual that need no GPU: statuses of the C entry points, refusals of
the Python ones, and the oracle's own rules."""
import ctypes

import numpy as np
import pytest
import torch

import bit_quantized_diffusion_svdq_amd as svdq
from bit_quantized_diffusion_svdq_amd import _lib
from kv_util import cum, paged, random_state
from oracle import kv as okv
from oracle.fp8 import e4m3_round

OK, NULL, SHAPE, ALIGN, UNSUP, DEVICE = 0, 1, 2, 3, 4, 5
A = 0x7F0000000000
B, C, D, E, F, G, H, I = (A + i * 0x1000000 for i in range(1, 9))


@pytest.fixture(scope="module")
def lib():
    return svdq.load_library()


def valid(status):
    """A well-formed call: the capability check without a GPU."""
    if torch.cuda.is_available():
        pytest.skip("a GPU is present: well-formed calls on these placeholder pointers would launch")
    assert status == DEVICE


# ---------------------------------------------------------------- C ABI

CACHE = dict(data=A, scales=B, pages=9, heads=4, D=72, page=128)
BATCH = dict(table=C, lengths=D, offsets=E, T=20, sequences=3, width=5)


def heads(**kw):
    h = dict(x=F, ts=12 * 72, hs=72, heads=8, norm=None, y=G, yts=8 * 72, yhs=72)
    h.update(kw)
    return _lib.RopeHeads(h["x"], h["ts"], h["hs"], h["heads"], h["norm"], h["y"], h["yts"], h["yhs"])


def structs(kw):
    cache = _lib.KvCacheDesc(*(kw.get(k, v) for k, v in CACHE.items()))
    batch = _lib.KvBatchDesc(*(kw.get(k, v) for k, v in BATCH.items()))
    return cache, batch


def _append(lib, kw):
    cache, batch = structs(kw)
    q = heads(**kw.get("q", {})) if kw.get("q", 0) is not None else None
    k = heads(**{**dict(x=H, heads=4, y=None), **(kw.get("k") or {})})
    v = heads(**{**dict(x=I, heads=4, y=None), **(kw.get("v") or {})})
    a = dict(pos=B + 0x100000, pdt=0, axes=3, turns=C + 0x100000, axis=D + 0x100000, pairs=36, pairing=0, eps=1e-6)
    a.update({n: kw[n] for n in a if n in kw})
    at = _lib._at
    return lib.svdq_kv_append(None if kw.get("cache", 0) is None else at(cache), None if kw.get("batch", 0) is None else at(batch),
                              at(q), None if kw.get("k", 0) is None else at(k), None if kw.get("v", 0) is None else at(v), a["pos"],
                              a["pdt"], a["axes"], a["turns"], a["axis"], a["pairs"], a["pairing"], a["eps"], None)


def _attend(lib, kw):
    cache, batch = structs(kw)
    q = heads(**kw.get("q", {}))
    need = ctypes.c_int64(-1)
    if lib.svdq_kv_attend_workspace_size(_lib._at(cache), _lib._at(batch), q.heads, ctypes.addressof(need)) != OK:
        need.value = 1 << 40
    a = dict(scale=0.1, causal=1, window=0, ws=I, bytes=need.value)
    a.update({n: kw[n] for n in a if n in kw})
    return lib.svdq_kv_attend(None if kw.get("cache", 0) is None else _lib._at(cache),
                              None if kw.get("batch", 0) is None else _lib._at(batch), _lib._at(q), a["scale"], a["causal"],
                              a["window"], a["ws"], a["bytes"], None)


BOTH = [
    (dict(pages=0), SHAPE), (dict(pages=1 << 31), SHAPE), (dict(heads=0), SHAPE), (dict(heads=65537), SHAPE), (dict(D=0), SHAPE),
    (dict(D=12), SHAPE), (dict(D=264), SHAPE), (dict(page=32), SHAPE), (dict(page=96), SHAPE), (dict(page=65600), SHAPE),
    (dict(T=-1), SHAPE), (dict(T=1 << 24), SHAPE), (dict(sequences=0), SHAPE), (dict(sequences=65537), SHAPE),
    (dict(width=-1), SHAPE), (dict(width=1 << 24), SHAPE), (dict(offsets=None), SHAPE), (dict(cache=None), NULL),
    (dict(batch=None), NULL), (dict(data=None), NULL), (dict(scales=None), NULL), (dict(table=None), NULL),
    (dict(lengths=None), NULL), (dict(data=A + 8), ALIGN), (dict(scales=B + 4), ALIGN), (dict(table=C + 2), ALIGN),
    (dict(lengths=D + 1), ALIGN), (dict(offsets=E + 2), ALIGN), (dict(q=dict(ts=12 * 72 + 4)), ALIGN),
    (dict(q=dict(x=F + 8)), ALIGN), (dict(q=dict(y=G + 2)), ALIGN), (dict(q=dict(y=None)), NULL), (dict(q=dict(x=None)), NULL),
    (dict(q=dict(yts=64, yhs=72)), SHAPE), (dict(q=dict(hs=-72)), SHAPE), (dict(q=dict(y=F)), SHAPE), (dict(q=dict(y=A)), SHAPE),
    (dict(T=0, data=None, table=None), OK),
]


@pytest.mark.parametrize("kw,status", BOTH + [
    (dict(k=dict(heads=3)), SHAPE), (dict(v=dict(heads=5)), SHAPE), (dict(k=None), NULL), (dict(v=None), NULL),
    (dict(k=dict(x=None)), NULL), (dict(v=dict(x=I + 2)), ALIGN), (dict(k=dict(ts=100)), ALIGN), (dict(v=dict(hs=-8)), SHAPE),
    (dict(v=dict(norm=A)), UNSUP), (dict(k=dict(norm=A + 2)), ALIGN), (dict(pairs=40), SHAPE), (dict(pairs=6), SHAPE),
    (dict(axes=0), SHAPE), (dict(axes=9), SHAPE), (dict(pdt=2), UNSUP), (dict(pairing=2), UNSUP), (dict(eps=-1.0), UNSUP),
    (dict(eps=float("nan")), UNSUP), (dict(pos=None), NULL), (dict(turns=None), NULL), (dict(axis=None), NULL),
    (dict(turns=C + 4), ALIGN), (dict(q=dict(heads=0)), SHAPE), (dict(q=dict(y=H)), SHAPE), (dict(q=dict(y=I)), SHAPE),
    (dict(data=H), SHAPE), (dict(scales=A), SHAPE), (dict(T=(1 << 24) - 1, q=dict(heads=512, yts=512 * 72)), SHAPE),
], ids=str)
def test_append_rejects(lib, kw, status):
    assert _append(lib, kw) == status
    assert status == OK or lib.svdq_last_error()


@pytest.mark.parametrize("kw,status", BOTH + [
    (dict(q=dict(heads=6, yts=6 * 72)), SHAPE), (dict(q=dict(norm=A)), UNSUP), (dict(scale=0.0), UNSUP), (dict(scale=-1.0), UNSUP),
    (dict(scale=float("inf")), UNSUP), (dict(scale=3e38), UNSUP), (dict(scale=float("nan")), UNSUP), (dict(causal=2), UNSUP), (dict(window=-1), SHAPE),
    (dict(bytes=0), SHAPE), (dict(ws=None), NULL), (dict(ws=I + 8), ALIGN), (dict(ws=F), SHAPE), (dict(ws=G), SHAPE),
    (dict(ws=A), SHAPE), (dict(T=(1 << 24) - 1, q=dict(heads=64, yts=64 * 72)), SHAPE),
    (dict(sequences=65536, T=65536, width=1 << 23, offsets=None, page=128), SHAPE),
], ids=str)
def test_attend_rejects(lib, kw, status):
    assert _attend(lib, kw) == status
    assert status == OK or lib.svdq_last_error()


def test_valid_calls(lib):
    valid(_append(lib, {}))
    valid(_append(lib, dict(q=None)))
    valid(_append(lib, dict(pairs=0, pos=None, turns=None, axis=None)))
    valid(_append(lib, dict(q=dict(y=F, yts=12 * 72))))
    valid(_append(lib, dict(width=0, table=None)))
    valid(_attend(lib, {}))
    valid(_attend(lib, dict(q=dict(y=F, yts=12 * 72))))
    valid(_attend(lib, dict(T=21, offsets=None)))
    valid(_attend(lib, dict(width=0, table=None)))


def test_sizes(lib):
    cache = _lib.KvCacheDesc(None, None, 9, 4, 72, 128)
    assert svdq.svdq_kv_cache_sizes(cache) == (9 * 4 * 128 * 128 * 2, 9 * 4 * 2 * 8)
    assert lib.svdq_kv_cache_sizes(_lib._at(cache), None, None) == NULL
    cache.page = 100
    assert lib.svdq_kv_cache_sizes(_lib._at(cache), None, None) == SHAPE
    cache = _lib.KvCacheDesc(None, None, 9, 8, 128, 64)
    small = _lib.KvBatchDesc(None, None, None, 1, 1, 4)
    assert svdq.svdq_kv_attend_workspace_size(cache, small, 8) == 0          # four tiles: one piece
    assert svdq.svdq_kv_attend_workspace_size(cache, _lib.KvBatchDesc(None, None, None, 1, 1, 5), 8) > 0
    assert lib.svdq_kv_attend_workspace_size(_lib._at(cache), _lib._at(small), 8, None) == NULL


RES = dict(qx=A, sx=B, M=33, K=144, qw=C, sw=D, N=77, offs=E, groups=3, bias=None, act=0, x=F, ld=77, gate=G, y=H, ydt=0, ldy=77)


def _residual(lib, layer, kw):
    a = {**RES, **kw}
    r = _lib.Fp8Residual(a["x"], a["ld"], a["gate"])
    at = None if a.get("res", 0) is None else _lib._at(r)
    if layer:
        need = svdq.svdq_linear_fp8_workspace_size(max(a["M"], 0), a["K"])
        return lib.svdq_linear_fp8_residual(a["qx"], a["M"], a["K"], a["K"], a["qw"], a["sw"], a["N"], a["offs"], a["groups"],
                                            a["bias"], a["act"], at, a["y"], a["ydt"], a["ldy"], I, need, None)
    return lib.svdq_gemm_fp8_residual(a["qx"], a["sx"], a["M"], a["K"], a["qw"], a["sw"], a["N"], a["offs"], a["groups"],
                                      a["bias"], a["act"], at, a["y"], a["ydt"], a["ldy"], None)


@pytest.mark.parametrize("layer", [False, True])
@pytest.mark.parametrize("kw,status", [
    (dict(res=None), NULL), (dict(x=None), NULL), (dict(ld=76), SHAPE), (dict(ld=1 << 31), SHAPE), (dict(x=F + 1), ALIGN),
    (dict(x=F + 2, ydt=1), ALIGN), (dict(gate=G + 1), ALIGN), (dict(x=H, ld=80), SHAPE), (dict(groups=-1), SHAPE),
    (dict(M=-1), SHAPE), (dict(act=2), UNSUP), (dict(groups=3, offs=None), NULL), (dict(M=0, x=None), OK),
], ids=str)
def test_residual_rejects(lib, layer, kw, status):
    assert _residual(lib, layer, kw) == status
    assert status == OK or lib.svdq_last_error()


@pytest.mark.parametrize("layer", [False, True])
def test_residual_valid(lib, layer):
    valid(_residual(lib, layer, {}))
    valid(_residual(lib, layer, dict(groups=0, gate=None)))
    valid(_residual(lib, layer, dict(x=H)))
    valid(_residual(lib, layer, dict(M=1, x=H, ld=80)))


# ---------------------------------------------------------------- Python

def t(*shape, dtype=torch.bfloat16):
    return torch.zeros(*shape, dtype=dtype)


def test_cache_refuses():
    for kw in (dict(pages=0), dict(kv_heads=0), dict(head_dim=12), dict(head_dim=264), dict(page_size=32), dict(page_size=100),
               dict(data=t(2, 3, 1, 2, 4, 1, 1024, dtype=torch.uint8)), dict(scales=t(2, 3, 1, 2, 4))):
        with pytest.raises(ValueError):
            svdq.KVCache(**{**dict(pages=3, kv_heads=3, head_dim=64, page_size=64, device="cpu"), **kw})
    with pytest.raises(ValueError):                       # data off its alignment
        svdq.KVCache(1, 1, 64, data=t(8193, dtype=torch.uint8)[1:].view(1, 1, 1, 2, 4, 1, 1024))
    c = svdq.KVCache(3, 2, 136, page_size=128, device="cpu")
    with pytest.raises(AttributeError):                   # the calls have the arrays' addresses
        c.data = c.data.clone()
    with pytest.raises(AttributeError):
        c.scales = c.scales.clone()
    assert tuple(c.data.shape) == (3, 2, 2, 2, 4, 3, 1024) and tuple(c.scales.shape) == (3, 2, 2, 2, 4)


GOOD = dict(k=t(4, 2, 64), v=t(4, 2, 64), table=t(2, 3, dtype=torch.int32), lengths=t(2, dtype=torch.int32), q=t(4, 6, 64))


@pytest.mark.parametrize("kw,word", [
    (dict(k=t(4, 128)), "k must"), (dict(k=t(4, 3, 64)), "heads"), (dict(v=t(3, 2, 64)), "v must"),
    (dict(v=t(4, 2, 64, dtype=torch.float32)), "v must"), (dict(k=t(4, 64, 2).transpose(1, 2)), "contiguous heads"),
    (dict(table=t(6, dtype=torch.int32)), "table"), (dict(table=t(2, 3, dtype=torch.int64)), "table"),
    (dict(lengths=t(3, dtype=torch.int32)), "lengths"), (dict(lengths=t(2, dtype=torch.int64)), "lengths"),
    (dict(offsets=t(2, dtype=torch.int32)), "offsets"), (dict(offsets=t(3, dtype=torch.int64)), "offsets"),
    (dict(table=t(3, 3, dtype=torch.int32), lengths=t(3, dtype=torch.int32)), "offsets are needed"),
    (dict(pos=t(4, 1, dtype=torch.int32)), "belong together"), (dict(plan=svdq.RopePlan((64,), device="cpu")), "belong together"),
    (dict(plan=svdq.RopePlan((32,), device="cpu"), pos=t(4, 1, dtype=torch.int32)), "turns heads"),
    (dict(plan=svdq.RopePlan((64,), device="cpu"), pos=t(4, 2, dtype=torch.int32)), "pos must"),
    (dict(plan=svdq.RopePlan((64,), device="cpu"), pos=t(4, 1, dtype=torch.int64)), "pos must"),
    (dict(k=t(4, 2, 64).requires_grad_()), "gradient"), ({}, "GPU device"),
])
def test_append_refuses(kw, word):
    c = svdq.KVCache(3, 2, 64, device="cpu")
    a = {**GOOD, **kw}
    with pytest.raises(ValueError, match=word):
        c.append(a.pop("k"), a.pop("v"), a.pop("table"), a.pop("lengths"), **a)


@pytest.mark.parametrize("kw,word", [
    (dict(q=t(4, 384)), "q must"), (dict(q=t(4, 5, 64)), "multiple of 2"), (dict(q=t(4, 6, 64, dtype=torch.float16)), "q must"),
    (dict(q=t(4, 6, 64).requires_grad_()), "gradient"), (dict(scale=0.0), "scale"), (dict(scale=float("nan")), "scale"),
    (dict(window=-1), "window"), (dict(window=1 << 31), "window"), (dict(lengths=t(1, dtype=torch.int32)), "lengths"), ({}, "GPU device"),
])
def test_attend_refuses(kw, word):
    c = svdq.KVCache(3, 2, 64, device="cpu")
    a = {**{n: GOOD[n] for n in ("q", "table", "lengths")}, **kw}
    with pytest.raises(ValueError, match=word):
        c.attend(a.pop("q"), a.pop("table"), a.pop("lengths"), **a)


def test_residual_refuses():
    from bit_quantized_diffusion_svdq_amd.fp8 import _residual as r
    cpu = torch.device("cpu")
    assert r(None, None, 3, 8, torch.bfloat16, (), cpu) is None
    for res, gate, lead in ((None, t(8), ()), (t(3, 9), None, ()), (t(3, 8, dtype=torch.float32), None, ()),
                            (t(8, 3).t(), None, ()), (t(1, 8).expand(3, 8), None, ()), (t(3, 8), t(9), ()),
                            (t(3, 8), t(8, dtype=torch.float32), ()), (t(3, 8), t(8), (2,))):
        with pytest.raises(ValueError):
            r(res, gate, 3, 8, torch.bfloat16, lead, cpu)
    assert r(t(3, 12)[:, :8], t(2, 8), 3, 8, torch.bfloat16, (2,), cpu).ld == 12


# ---------------------------------------------------------------- the oracle

def test_oracle_codes():
    v = okv.e4m3_values()
    want = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(np.nan_to_num(v, nan=1e9), np.nan_to_num(want, nan=1e9))
    codes = np.array([c for c in range(256) if c & 127 != 127 and c != 128], np.uint8)
    assert np.array_equal(okv.encode(v[codes]), codes)


@pytest.mark.parametrize("amax,e", [(0.0, -120), (448.0, 0), (448.0001, 1), (224.0, -1), (1.0, -8), (1.75, -8), (1.7500001, -7),
                                    (2.0 ** -140, -120), (3e38, 120)])
def test_oracle_exponent(amax, e):
    assert okv.exponent(amax) == e
    assert e == -120 or 448 * 2.0 ** (e - 1) < amax <= 448 * 2.0 ** e


@pytest.mark.parametrize("H,D,page", [(1, 8, 64), (3, 72, 128), (2, 256, 192)])
def test_oracle_layout(H, D, page):
    """Every byte belongs to one channel of one token, and packing undoes unpacking."""
    rng = np.random.default_rng(D)
    C = -(-D // 64)
    for tok, ch in okv.layout(C):
        assert len(set(zip(tok.ravel().tolist(), ch.ravel().tolist()))) == 16 * 64 * C
    st = random_state(rng, 3, page, H, D)
    data, scales = okv.pack(*st)
    for a, b in zip(okv.unpack(data, scales), st):
        assert np.array_equal(a, b)


def test_oracle_append_step_by_step():
    """Token by token gives what all at once gives, but for what becomes subnormal on the way."""
    rng = np.random.default_rng(0)
    H, D, n = 2, 64, 40
    k, v = rng.standard_normal((2, n, H, D)) * np.exp(rng.standard_normal((2, n, 1, 1)))
    pages, table = paged(rng, [n], 64)
    once = random_state(rng, pages, 64, H, D)
    steps = [a.copy() for a in once]
    okv.append(once, k, v, table, [n], [0, n])
    for i in range(n):
        okv.append(steps, k[i:i + 1], v[i:i + 1], table, [i + 1], [0, 1])
    assert np.array_equal(once[2], steps[2]) and np.array_equal(once[3], steps[3])
    for side in range(2):
        d = np.abs(once[side] - steps[side])
        assert (d[np.abs(once[side]) >= 2.0 ** -5] == 0).all() and d.max() <= 2.0 ** -9
    assert (once[0][table[0, 0], n:48] == 0).all()


def test_oracle_attend():
    """Against a softmax written out, with a window, a missing page and a row that sees nothing."""
    rng = np.random.default_rng(1)
    H, D, page = 1, 8, 64
    pages, table = paged(rng, [130, 3], page)
    st = random_state(rng, pages, page, H, D)
    table[0, 1] = -1
    q = rng.standard_normal((3, 2, D))
    y, mag, rss, peak = okv.attend(st, q, table, [130, 0], [0, 2, 3], causal=True, window=70)
    assert (y[2] == 0).all() and (mag >= np.abs(y) - 1e-12).all() and (rss <= mag + 1e-12).all()
    k, v, there = okv.read(st, table[0], 130)
    seen = [i for i in range(130) if there[i] and 129 - 70 < i]
    s = k[seen, 0, :D] @ q[1, 1] / np.sqrt(D)
    w = np.exp(s) / np.exp(s).sum()
    assert np.allclose(w @ v[seen, 0, :D], y[1, 1]) and len(seen) == 70 - 64


def test_offsets_that_fall():
    assert okv.rising([0, 5, 3, 9, 99], 7).tolist() == [0, 5, 5, 7, 7]
    assert cum([2, 0, 3]).tolist() == [0, 2, 2, 5]
    assert e4m3_round(np.array([0.3])) == 0.3125


def test_block_refuses():
    class Layer:
        def __init__(self, K, N):
            self.K, self.N = K, N

    plan = svdq.RopePlan((64,), device="cpu")
    cache = svdq.KVCache(2, 2, 64, device="cpu")
    qkv = svdq.FusedQKV(Layer(32, 8 * 64), plan, 4, 2)
    svdq.CachedAttention(qkv, Layer(4 * 64, 32), cache)
    grouped = svdq.Fp8GroupedLinear(t(2, 8, 256, dtype=torch.float8_e4m3fn), t(2, 1, 2, dtype=torch.float32))
    for args in ((qkv, Layer(5 * 64, 32), cache), (qkv, Layer(4 * 64, 32), svdq.KVCache(2, 4, 64, device="cpu")),
                 (qkv, Layer(4 * 64, 32), svdq.KVCache(2, 2, 32, device="cpu")), (qkv, grouped, cache),
                 (svdq.FusedQKV(Layer(32, 7 * 64), plan, 3, 2), Layer(3 * 64, 32), cache)):
        with pytest.raises(ValueError):
            svdq.CachedAttention(*args)
