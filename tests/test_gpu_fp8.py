"""GPU parity of the 8-bit layers (E4M3, one fp32 scale per block of 128)
against the fp64 oracle: quantisers bit-exact, products within bounds on fp32
accumulation and one output rounding, at the sizes where tiles, blocks and
vectors end."""
import math

import numpy as np
import pytest
import torch

from gpu_util import note

pytestmark = pytest.mark.gpu

import bit_quantized_diffusion_svdq_amd as svdq
from oracle import fp8 as ofp8, svdq as osv

E4M3 = torch.float8_e4m3fn


def np64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def acts(M, K, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((M, K), generator=g) * scale
    x[:, torch.rand(K, generator=g) < 0.02] *= 20.0
    return x.to(torch.bfloat16).cuda()


def weights(K, N, seed, groups=0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn((*((groups,) if groups else ()), K, N), generator=g) * 0.05).to(torch.bfloat16).cuda()


def biases(shape, seed):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).to(torch.bfloat16).cuda()


def check_product(y, ref64, K, act="none"):
    """ref64 = (y, mag, peak) of the oracle. fp32 part: a block's 128 products
    and the KB block sums each add at most one rounding of the running sum,
    which the sum of magnitudes bounds; a factor 2 covers a matrix pipe that
    truncates: 2 (128 + KB + 4) 2^-24 mag. A bf16 output comes from the E4M3
    matrix instructions, which shift each 8 products to the exponent of the
    largest and drop what is more than 13 bits below it: of the 8, the 7
    others lose less than 2^-13 of the largest each, 7 x 2^-13 peak. GELU passes
    all that on with a slope of at most 1.13 and adds 2^-18 of its value and,
    in the negative tail, 2^-22 of the input. bf16 outputs add half a step,
    2^-8 of the value."""
    y64, mag, peak = ref64
    kb = -(-K // 128)
    bound = 2.0 * (128 + kb + 4) * 2.0 ** -24 * mag + 1e-30
    if y.dtype == torch.bfloat16:
        bound = bound + 7 * 2.0 ** -13 * peak
    ref = y64
    if act == "gelu_tanh":
        ref = osv.gelu_tanh(y64)
        bound = 1.13 * bound + 2.0 ** -18 * np.abs(ref) + 2.0 ** -22 * np.abs(y64)
    if y.dtype == torch.bfloat16:
        bound = bound * (1 + 2.0 ** -8) + 2.0 ** -8 * np.abs(ref)
    got = np64(y)
    bad = ~(np.abs(got - ref) <= bound)
    assert not bad.any(), (f"{bad.sum()} of {bad.size} outputs outside the bound, first at {np.argwhere(bad)[0]}; "
                           f"worst ratio {np.nanmax(np.abs(got - ref) / bound):.3g}")


# ---------------------------------------------------------------- quantisers

@pytest.mark.parametrize("M,K", [(1, 16), (1, 4096), (3, 128), (5, 112), (16, 144), (17, 640), (33, 2064), (130, 272),
                                 (4099, 528), (8200, 512)])
def test_quantize_act(M, K):
    note(f"quantize_act_fp8 {M} x {K}")
    x = acts(M, K, M * 7 + K)
    if M > 2:
        x[1] = 0.0                                   # a row of zeros
        x[2, K // 2:] *= 1e-30
    q, s = svdq.quantize_act_fp8(x)
    assert q.dtype == E4M3 and tuple(q.shape) == (M, K) and tuple(s.shape) == (-(-K // 128), M)
    qo, so = ofp8.quantize_act(np64(x))
    assert np.array_equal(s.cpu().numpy(), so)
    assert np.array_equal(np64(q), qo)


def test_quantize_act_strided_rows_and_guard():
    note("quantize_act_fp8 strided rows")
    big = acts(40, 1024, 3)
    x = big[3:37, 64:64 + 400]
    q, s = svdq.quantize_act_fp8(x)
    qo, so = ofp8.quantize_act(np64(x))
    assert np.array_equal(np64(q), qo) and np.array_equal(s.cpu().numpy(), so)
    # outputs end where they should
    M, K = x.shape
    qb = torch.full((M * K + 64,), 0x55, dtype=torch.uint8, device="cuda")
    sb = torch.full((4 * M + 16,), -7.0, device="cuda")
    svdq.svdq_quantize_act_fp8(x, M, K, x.stride(0), qb, sb)
    assert torch.equal(qb[:M * K].view(E4M3).view(M, K).view(torch.uint8), q.view(torch.uint8))
    assert (qb[M * K:] == 0x55).all() and torch.equal(sb[:4 * M].view(4, M), s) and (sb[4 * M:] == -7.0).all()


def test_quantize_act_values_that_are_not_finite():
    note("quantize_act_fp8 non-finite values")
    x = acts(4, 384, 5)
    x[0, 3], x[0, 130], x[1, 200] = float("inf"), float("-inf"), float("nan")
    x[2, :128] = float("inf")
    x[3] = torch.finfo(torch.bfloat16).max
    q, s = svdq.quantize_act_fp8(x)
    q, s = np64(q), s.cpu().numpy()
    qo, so = ofp8.quantize_act(np64(x))
    assert np.array_equal(s, so) and np.isfinite(s).all()
    assert np.isnan(q[1, 200]) and np.isnan(q).sum() == 1
    assert q[0, 3] == 448 and q[0, 130] == -448 and (q[2, :128] == 448).all() and s[0, 2] == np.float32(2.0 ** -120)
    assert np.array_equal(np.nan_to_num(q, nan=1e9), np.nan_to_num(qo, nan=1e9))


def test_quantize_act_every_code():
    """Every multiple of a half step around each E4M3 value, ties among them."""
    note("quantize_act_fp8 ties")
    codes = torch.arange(0x7F, dtype=torch.uint8).view(E4M3).double()
    mids = (codes[1:] + codes[:-1]) / 2
    v = torch.cat([codes, mids, -codes, -mids]).to(torch.bfloat16)       # exact: 5 bits of mantissa at most
    x = torch.zeros((v.numel(), 128), dtype=torch.bfloat16)
    x[:, 5], x[:, 90] = v, 448.0                                         # the block's scale is 1
    q, s = svdq.quantize_act_fp8(x.cuda())
    assert (s == 1.0).all()
    assert np.array_equal(np64(q)[:, 5], ofp8.e4m3_round(v.double().numpy()))


@pytest.mark.parametrize("K,N", [(16, 1), (128, 128), (144, 8), (272, 129), (2064, 37), (384, 300)])
def test_quantize_weight(K, N):
    note(f"quantize_fp8 {K} x {N}")
    w = weights(K, N, K + N)
    d = svdq.quantize_fp8(w)
    qo, so = ofp8.quantize_weight(np64(w))
    assert np.array_equal(d["sw"].cpu().numpy(), so)
    assert np.array_equal(np64(d["qw"]), qo)


def test_quantize_weight_views_and_groups():
    note("quantize_fp8 views")
    big = weights(160, 512, 1)
    w = big[:, 40:40 + 200]
    assert np.array_equal(np64(svdq.quantize_fp8(w)["qw"]), ofp8.quantize_weight(np64(w))[0])
    w = big[:, 3:3 + 77]                                                # an address the kernel cannot read
    assert np.array_equal(np64(svdq.quantize_fp8(w)["qw"]), ofp8.quantize_weight(np64(w))[0])
    w3 = weights(144, 72, 9, groups=3)
    d = svdq.quantize_fp8(w3)
    for g in range(3):
        q, s = ofp8.quantize_weight(np64(w3[g]))
        assert np.array_equal(np64(d["qw"][g]), q) and np.array_equal(d["sw"][g].cpu().numpy(), s)


# ---------------------------------------------------------------- the product

SIZES = [(1, 16, 1), (1, 128, 16), (1, 4096, 300), (2, 144, 7), (7, 272, 129), (16, 2064, 100), (17, 112, 33),
         (31, 640, 1000), (64, 1040, 257), (65, 256, 136), (100, 384, 128), (128, 128, 128), (129, 400, 1001),
         (200, 2064, 72), (257, 1152, 520), (300, 16, 384), (513, 528, 264), (1030, 272, 130)]


@pytest.mark.parametrize("M,K,N", SIZES)
@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
def test_linear(M, K, N, out):
    note(f"fp8_linear {M} x {K} x {N} {out}")
    x, w, b = acts(M, K, M + K), weights(K, N, K + N), biases(N, N)
    d = svdq.quantize_fp8(w, b)
    qx, sx = svdq.quantize_act_fp8(x)
    act = "gelu_tanh" if (M + N) % 2 else "none"
    y = svdq.fp8_linear(qx, sx, d["qw"], d["sw"], b if M % 3 else None, act=act, out_dtype=out)
    ref = ofp8.linear(np64(qx), sx.cpu().numpy(), np64(d["qw"]), d["sw"].cpu().numpy(), np64(b) if M % 3 else None)
    assert y.dtype == out
    check_product(y, ref, K, act)


@pytest.mark.parametrize("M", [3, 50, 150, 700])
def test_linear_rows_stand_alone(M):
    """A row or a weight column of NaN touches its own outputs only, also
    where the last block of K ends inside a tile's loads; and one row's
    result does not depend on the others."""
    note(f"fp8_linear NaN neighbours {M}")
    K, N = 272, 140
    x, w = acts(M, K, 1), weights(K, N, 2)
    d = svdq.quantize_fp8(w)
    qx, sx = svdq.quantize_act_fp8(x)
    clean = svdq.fp8_linear(qx, sx, d["qw"], d["sw"], out_dtype=torch.float32)
    qn, wn = qx.clone(), d["qw"].clone()
    qn.view(torch.uint8)[M // 2] = 0x7F
    wn.view(torch.uint8)[N // 2] = 0xFF
    y = svdq.fp8_linear(qn, sx, wn, d["sw"], out_dtype=torch.float32)
    keep_m, keep_n = torch.arange(M, device="cuda") != M // 2, torch.arange(N, device="cuda") != N // 2
    assert torch.equal(y[keep_m][:, keep_n], clean[keep_m][:, keep_n])
    assert y[M // 2].isnan().all() and y[:, N // 2].isnan().all()


@pytest.mark.parametrize("M", [5, 90, 400])
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("N,ld,off", [(200, 200, 0), (200, 208, 8), (200, 203, 1), (121, 121, 0), (121, 128, 0),
                                      (6, 12, 4), (200, 204, 4)])
def test_linear_into_views(M, dt, N, ld, off):
    """Outputs into strided, odd and unaligned buffers; nothing else of the
    buffer changes, and the values are those of a plain call."""
    note(f"fp8_linear into a view {M} {dt} {N} {ld} {off}")
    K = 400
    d = svdq.quantize_fp8(weights(K, N, N))
    qx, sx = svdq.quantize_act_fp8(acts(M, K, 4))
    want = svdq.fp8_linear(qx, sx, d["qw"], d["sw"], out_dtype=dt)
    buf = torch.full((M * ld + 64,), -3.0, dtype=dt, device="cuda")
    y = buf[off:off + M * ld].view(M, ld)[:, :N]
    assert svdq.fp8_linear(qx, sx, d["qw"], d["sw"], y=y) is y
    assert torch.equal(y, want)
    rest = torch.ones_like(buf, dtype=torch.bool)
    rest[off:off + M * ld].view(M, ld)[:, :N] = False
    assert (buf[rest] == -3.0).all()


def test_linear_is_deterministic_and_empty_batch():
    note("fp8_linear repeat")
    d = svdq.quantize_fp8(weights(1040, 264, 1))
    for M in (0, 4, 300):
        qx, sx = svdq.quantize_act_fp8(acts(M, 1040, 2))
        a = svdq.fp8_linear(qx, sx, d["qw"], d["sw"])
        b = svdq.fp8_linear(qx, sx, d["qw"], d["sw"])
        assert tuple(a.shape) == (M, 264) and torch.equal(a, b)


def test_large_magnitudes_and_zero_blocks():
    """Scales far from one (2^-60 .. 2^60) and blocks of zeros."""
    note("fp8_linear scales")
    M, K, N = 70, 512, 136
    x, w = acts(M, K, 1).float(), weights(K, N, 2).float()
    x[:, :128] *= 2.0 ** 40
    x[:, 128:256] *= 2.0 ** -60
    x[:, 256:384] = 0
    w[:128] *= 2.0 ** -50
    w[128:256] *= 2.0 ** 60
    d = svdq.quantize_fp8(w.to(torch.bfloat16))
    qx, sx = svdq.quantize_act_fp8(x.to(torch.bfloat16))
    for m in (M, 3):
        y = svdq.fp8_linear(qx[:m].contiguous(), sx[:, :m].contiguous(), d["qw"], d["sw"], out_dtype=torch.float32)
        ref = ofp8.linear(np64(qx[:m]), sx[:, :m].cpu().numpy(), np64(d["qw"]), d["sw"].cpu().numpy())
        check_product(y, ref, K)


# ---------------------------------------------------------------- grouped

GROUPS = [([0, 5], 5, 272, 40), ([0, 0, 3, 3, 4], 4, 128, 129), ([0, 1, 2, 3, 4, 5, 6, 7, 8], 8, 400, 56),
          ([2, 20, 20, 60], 70, 144, 136), ([0, 130, 131, 131, 400], 400, 272, 200),
          ([0, 128, 256, 300], 300, 528, 128), ([10, 700, 1000], 1024, 256, 260), ([0, 0, 0], 6, 128, 24),
          ([0, 300, 300], 300, 2064, 72)]


@pytest.mark.parametrize("offs,M,K,N", GROUPS)
@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
def test_grouped(offs, M, K, N, out):
    note(f"fp8_grouped_linear {offs} of {M} x {K} x {N} {out}")
    E = len(offs) - 1
    x, w, b = acts(M, K, M), weights(K, N, N, groups=E), biases((E, N), K)
    d = svdq.quantize_fp8(w, b)
    qx, sx = svdq.quantize_act_fp8(x)
    o = torch.tensor(offs, dtype=torch.int32, device="cuda")
    y = torch.full((M, N), -3.0, dtype=out, device="cuda")
    act = "gelu_tanh" if E % 2 else "none"
    svdq.fp8_grouped_linear(qx, sx, o, d["qw"], d["sw"], b, act=act, y=y)
    ref = ofp8.grouped_linear(np64(qx), sx.cpu().numpy(), offs, np64(d["qw"]), d["sw"].cpu().numpy(), np64(b))
    inside = ~np.isnan(ref[0][:, 0])
    assert (np64(y)[~inside] == -3.0).all()
    if inside.any():
        check_product(y[torch.from_numpy(inside).cuda()], [r[inside] for r in ref], K, act)


@pytest.mark.parametrize("E,M", [(64, 200), (65, 90), (130, 1500), (200, 64)])
def test_grouped_many_groups(E, M):
    """More groups than a wave has lanes, most of them small or empty."""
    note(f"fp8_grouped_linear {E} groups of {M}")
    K, N = 144, 40
    cut = np.sort(np.random.default_rng(E).integers(0, M + 1, E - 1))
    offs = [0, *cut.tolist(), M]
    d = svdq.quantize_fp8(weights(K, N, 3, groups=E))
    qx, sx = svdq.quantize_act_fp8(acts(M, K, 5))
    y = svdq.fp8_grouped_linear(qx, sx, torch.tensor(offs, dtype=torch.int32, device="cuda"), d["qw"], d["sw"],
                                out_dtype=torch.float32)
    ref = ofp8.grouped_linear(np64(qx), sx.cpu().numpy(), offs, np64(d["qw"]), d["sw"].cpu().numpy())
    check_product(y, ref, K)


# ---------------------------------------------------------------- every tile size

def check_all_and_some(y, qx, sx, qw, sw, bias, rows, K):
    """Every output against an fp32 product of the codes' values on the GPU, a
    few rows against the oracle. The loose bound of the first: the E4M3
    instructions lose at most 7 x 2^-13 of the sum of the largest terms, which
    the sum of all magnitudes bounds; the fp32 sums of either side at most
    2 (K + 8) 2^-24 of it; bf16 outputs half a step, 2^-8 of the value."""
    kb = sx.shape[0]
    xv = qx.float() * sx.t().repeat_interleave(128, 1)[:, :K]
    wv = qw.float() * sw.repeat_interleave(128, 0)[:qw.shape[0]].repeat_interleave(128, 1)[:, :K]
    full, mag = xv @ wv.t(), xv.abs() @ wv.abs().t()
    if bias is not None:
        full, mag = full + bias.float(), mag + bias.float().abs()
    bf = y.dtype == torch.bfloat16
    bound = ((7 * 2.0 ** -13 if bf else 0.0) + 4 * (K + kb + 8) * 2.0 ** -24) * mag
    if bf:
        bound = bound * (1 + 2.0 ** -8) + 2.0 ** -8 * full.abs()
    bad = ~((y.float() - full).abs() <= bound)
    assert not bad.any(), f"{int(bad.sum())} outputs outside the bound, first at {bad.nonzero()[0].tolist()}"
    ref = ofp8.linear(np64(qx[rows]), sx[:, rows].cpu().numpy(), np64(qw), sw.cpu().numpy(),
                      None if bias is None else np64(bias))
    check_product(y[rows], ref, K)


# sizes that between them take every tile size
TILES = [(2405, 400, 6152), (4700, 144, 2603), (2405, 1168, 4104), (6007, 400, 1288), (4111, 1168, 1001), (700, 144, 3000),
         (6007, 400, 6152), (3600, 400, 520), (700, 1168, 3000), (130, 400, 6152), (6007, 1168, 129), (257, 1168, 1001),
         # more than 64 blocks of K: the weight's scales come in two runs
         (2405, 8336, 6152), (4700, 8336, 2603), (2405, 8336, 4104), (6007, 8336, 1288), (4111, 8336, 1001), (700, 8336, 3000),
         (3600, 8336, 520), (130, 8336, 6152), (257, 16400, 1001)]


@pytest.mark.parametrize("M,K,N", TILES)
def test_every_tile_size(M, K, N):
    note(f"fp8_linear tiles {M} x {K} x {N}")
    d = svdq.quantize_fp8(weights(K, N, N), biases(N, K) if M % 2 else None)
    qx, sx = svdq.quantize_act_fp8(acts(M, K, M))
    y = svdq.fp8_linear(qx, sx, d["qw"], d["sw"], d["bias"])
    check_all_and_some(y, qx, sx, d["qw"], d["sw"], d["bias"], [0, 1, M // 3, M // 2 + 5, M - 2, M - 1], K)


@pytest.mark.parametrize("M,K,N", [(4111, 400, 520), (2405, 144, 1001), (300, 1168, 520), (4111, 8336, 520), (257, 16400, 520)])
def test_every_tile_size_fp32(M, K, N):
    note(f"fp8_linear tiles, fp32 outputs {M} x {K} x {N}")
    d = svdq.quantize_fp8(weights(K, N, N), biases(N, K))
    qx, sx = svdq.quantize_act_fp8(acts(M, K, M))
    y = svdq.fp8_linear(qx, sx, d["qw"], d["sw"], d["bias"], out_dtype=torch.float32)
    check_all_and_some(y, qx, sx, d["qw"], d["sw"], d["bias"], [0, 17, M // 2, M - 1], K)


@pytest.mark.parametrize("M,K,N", [(2000, 400, 6152), (4700, 144, 2603), (1030, 1168, 9001), (6007, 400, 1288), (4111, 1168, 1001),
                                   (300, 400, 6152), (1500, 400, 1288), (257, 400, 3000), (90, 1168, 1288)])
def test_every_tile_size_grouped(M, K, N):
    """Three groups, one of a single row, the last tiles of the others with few
    or no rows for half of their waves; rows of no group stay."""
    note(f"fp8_grouped_linear tiles {M} x {K} x {N}")
    d = svdq.quantize_fp8(weights(K, N, N, groups=3), biases((3, N), K))
    qx, sx = svdq.quantize_act_fp8(acts(M, K, M))
    cut = M * 3 // 5 // 32 * 32 + 5                       # a tile's first rows at the end of the first group
    offs = [0, cut, cut + 1, M - 2]
    y = torch.full((M, N), -3.0, dtype=torch.bfloat16, device="cuda")
    svdq.fp8_grouped_linear(qx, sx, torch.tensor(offs, dtype=torch.int32, device="cuda"), d["qw"], d["sw"], d["bias"], y=y)
    assert (y[M - 2:] == -3.0).all()
    for g in range(3):
        r = slice(offs[g], offs[g + 1])
        n = offs[g + 1] - offs[g]
        check_all_and_some(y[r], qx[r], sx[:, r].contiguous(), d["qw"][g], d["sw"][g], d["bias"][g], sorted({0, n // 2, n - 1}), K)


def test_offsets_past_32_bits():
    """A batch whose values, codes and outputs each pass 2^31: the last rows
    are those of a small batch."""
    note("fp8 batch past 2^31 values")
    M, K, N = 264_007, 8208, 8200
    assert M * K > 2 ** 31 and M * N > 2 ** 31
    d = svdq.quantize_fp8(weights(K, N, 1), biases(N, 2))
    tail = acts(300, K, 3)
    x = torch.zeros((M, K), dtype=torch.bfloat16, device="cuda")
    x[-300:] = tail
    qx, sx = svdq.quantize_act_fp8(x)
    qt, st = svdq.quantize_act_fp8(tail)
    assert torch.equal(qx[-300:].view(torch.uint8), qt.view(torch.uint8)) and torch.equal(sx[:, -300:], st)
    assert (qx[:-300].view(torch.uint8) == 0).all()
    del x
    y = svdq.fp8_linear(qx, sx, d["qw"], d["sw"], d["bias"])
    assert torch.equal(y[:1], d["bias"][None]) and torch.equal(y[M - 302:M - 300], d["bias"].expand(2, N))
    check_all_and_some(y[-300:], qt, st, d["qw"], d["sw"], d["bias"], [0, 150, 299], K)
    # the same rows as the second of two groups that share one weight
    two = svdq.fp8_grouped_linear(qx, sx, torch.tensor([0, M - 300, M], dtype=torch.int32, device="cuda"),
                                  d["qw"].expand(2, N, K).contiguous(), d["sw"].expand(2, -1, -1).contiguous(), y=y)
    assert (two[:1] == 0).all() and (two[M - 301] == 0).all()
    check_all_and_some(two[-300:], qt, st, d["qw"], d["sw"], None, [0, 150, 299], K)


@pytest.mark.parametrize("M", [7, 700])
def test_weights_past_32_bits(M):
    """Groups' weights past 2^31 bytes: all rows in the last one."""
    note(f"fp8_grouped_linear weights past 2^31 bytes, {M} rows")
    E, K, N = 33, 8208, 8200
    assert (E - 1) * N * K > 2 ** 31
    qw = torch.zeros((E, N, K), dtype=torch.uint8, device="cuda")
    qw[-1] = torch.randint(0, 0x7F, (N, K), dtype=torch.uint8, generator=torch.Generator().manual_seed(M)).cuda()
    qw = qw.view(E4M3)
    sw = torch.rand((E, -(-N // 128), -(-K // 128)), generator=torch.Generator().manual_seed(1)).cuda()
    qx, sx = svdq.quantize_act_fp8(acts(M, K, 3))
    y = svdq.fp8_grouped_linear(qx, sx, torch.tensor([0] * E + [M], dtype=torch.int32, device="cuda"), qw, sw)
    check_all_and_some(y, qx, sx, qw[-1], sw[-1], None, [0, M - 1], K)


# ---------------------------------------------------------------- how a program has them

def test_layers_on_streams_and_in_a_graph():
    """A dense and a grouped layer called eagerly, on a side stream, and
    replayed from two captured graphs with eager work in between."""
    note("Fp8Linear / Fp8GroupedLinear streams and graphs")
    K, N, M = 272, 264, 150
    dense = svdq.Fp8Linear.from_quantized(svdq.quantize_fp8(weights(K, N, 1), biases(N, 2)))
    grouped = svdq.Fp8GroupedLinear.from_quantized(svdq.quantize_fp8(weights(K, N, 3, groups=2), biases((2, N), 4)))
    offs = torch.tensor([0, 40, M], dtype=torch.int32, device="cuda")
    x = acts(M, K, 5)
    want = dense(x, act="gelu_tanh"), grouped(x, offs)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    on_side = dense(x, act="gelu_tanh", stream=side), grouped(x, offs, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    assert torch.equal(on_side[0], want[0]) and torch.equal(on_side[1], want[1])
    y = [torch.empty_like(w) for w in want]
    graphs = [svdq.CapturedSequence(lambda: dense(x, act="gelu_tanh", y=y[0])),
              svdq.CapturedSequence(lambda: grouped(x, offs, y=y[1]))]
    for i in range(4):
        x.copy_(acts(M, K, 6 + i))
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        assert torch.equal(y[0], dense(x, act="gelu_tanh")) and torch.equal(y[1], grouped(x, offs))
        for t in y:
            t.zero_()


FEW = [(1, 16, 1), (1, 4096, 300), (2, 144, 7), (3, 10240, 24), (7, 272, 129), (16, 2048, 100), (5, 112, 8201),
       (16, 2048, 4200), (9, 1040, 4104), (1, 24576, 40), (1, 32768, 33), (16, 2064, 20), (17, 128, 20)]


@pytest.mark.parametrize("M,K,N", FEW)
@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
def test_layer_of_few_rows(M, K, N, out):
    """A layer on bf16 rows, up to and past what one launch takes, against the
    oracle's codes and products."""
    note(f"Fp8Linear {M} x {K} x {N} {out}")
    x, b = acts(M, K, M + N), biases(N, K)
    lay = svdq.Fp8Linear.from_quantized(svdq.quantize_fp8(weights(K, N, K + N), b if M % 3 else None))
    act = "gelu_tanh" if (M + N) % 2 else "none"
    y = lay(x, act=act, out_dtype=out)
    qx, sx = ofp8.quantize_act(np64(x))
    ref = ofp8.linear(qx, sx, np64(lay.qw), lay.sw.cpu().numpy(), np64(b) if M % 3 else None)
    assert y.dtype == out and tuple(y.shape) == (M, N)
    check_product(y, ref, K, act)


@pytest.mark.parametrize("M,K,N", [(6, 400, 136), (6, 400, 4200)])
def test_layer_of_few_rows_values_that_are_not_finite(M, K, N):
    """Infinities saturate and leave the scale alone, NaN spoils its own row
    only, rows of zeros give the bias: as in the two passes."""
    note(f"Fp8Linear non-finite {M} x {K} x {N}")
    x, b = acts(M, K, 8), biases(N, 9)
    lay = svdq.Fp8Linear.from_quantized(svdq.quantize_fp8(weights(K, N, 10), b))
    clean = lay(x, out_dtype=torch.float32)
    x[1] = 0.0
    x[2, 5], x[2, 300] = float("inf"), float("-inf")
    x[4, 399] = float("nan")
    y = lay(x, out_dtype=torch.float32)
    rest = [0, 3, 5]
    assert torch.equal(y[rest], clean[rest]) and torch.equal(y[1], b.float()) and y[4].isnan().all()
    qx, sx = ofp8.quantize_act(np64(x[2:3]))
    check_product(y[2:3], ofp8.linear(qx, sx, np64(lay.qw), lay.sw.cpu().numpy(), np64(b)), K)


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("N,ld,off", [(200, 200, 0), (200, 203, 1), (121, 128, 0), (4200, 4204, 4)])
def test_layer_of_few_rows_views(dt, N, ld, off):
    """Strided inputs, outputs into strided, odd and unaligned buffers whose
    other values stay, and an output over its own input."""
    note(f"Fp8Linear views {dt} {N} {ld} {off}")
    M, K = 5, 400
    lay = svdq.Fp8Linear.from_quantized(svdq.quantize_fp8(weights(K, N, N)))
    x = acts(40, 1024, 3)[3:3 + M, 64:64 + K]
    want = lay(x.contiguous(), out_dtype=dt)
    assert torch.equal(lay(x, out_dtype=dt), want)
    assert torch.equal(lay(x[:1].expand(M, K), out_dtype=dt), want[:1].expand(M, N))
    buf = torch.full((M * ld + 64,), -3.0, dtype=dt, device="cuda")
    y = buf[off:off + M * ld].view(M, ld)[:, :N]
    assert lay(x, y=y) is y and torch.equal(y, want)
    rest = torch.ones_like(buf, dtype=torch.bool)
    rest[off:off + M * ld].view(M, ld)[:, :N] = False
    assert (buf[rest] == -3.0).all()


@pytest.mark.parametrize("offs,M,K,N", [([0, 1], 1, 144, 40), ([0, 0, 2, 2, 3], 4, 2048, 264), ([0, 16], 16, 2048, 100),
                                        ([1, 4, 4, 15], 16, 400, 4200), ([0] * 70 + [3, 3, 7], 9, 1040, 72),
                                        ([2, 3, 5, 8], 8, 4096, 129), ([0, 0, 0], 5, 128, 24), ([0, 9, 17], 17, 128, 40)])
@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
def test_grouped_layer_of_few_rows(offs, M, K, N, out):
    """Grouped layers on a few bf16 rows: rows of no group stay."""
    note(f"Fp8GroupedLinear {offs[-5:]} of {M} x {K} x {N} {out}")
    E = len(offs) - 1
    lay = svdq.Fp8GroupedLinear.from_quantized(svdq.quantize_fp8(weights(K, N, N, groups=E), biases((E, N), K)))
    x = acts(M + 3, K + 24, M)[2:2 + M, 8:8 + K]
    o = torch.tensor(offs, dtype=torch.int32, device="cuda")
    y = torch.full((M, N), -3.0, dtype=out, device="cuda")
    act = "gelu_tanh" if E % 2 else "none"
    assert lay(x, o, act=act, y=y) is y
    qx, sx = ofp8.quantize_act(np64(x))
    ref = ofp8.grouped_linear(qx, sx, offs, np64(lay.qw), lay.sw.cpu().numpy(), np64(lay.bias))
    inside = ~np.isnan(ref[0][:, 0])
    assert (np64(y)[~inside] == -3.0).all()
    if inside.any():
        check_product(y[torch.from_numpy(inside).cuda()], [r[inside] for r in ref], K, act)
        keep = torch.from_numpy(inside).cuda()
        assert torch.equal(lay(x, o, act=act, out_dtype=out)[keep], y[keep])


@pytest.mark.parametrize("M", [6, 40])
def test_grouped_offsets_that_are_wrong_stay_inside(M):
    """Offsets outside [0, M] or falling are clamped: nothing outside y is
    written (the rows themselves are then unspecified)."""
    note(f"Fp8GroupedLinear with wrong offsets {M}")
    K, N = 272, 72
    lay = svdq.Fp8GroupedLinear.from_quantized(svdq.quantize_fp8(weights(K, N, 1, groups=4)))
    x = acts(M, K, 2)
    for offs in ([-5, 3, 1 << 30, 2, 4], [9, 7, 5, 3, 1], [0, M, 0, M, 0], [-(1 << 31)] * 4 + [(1 << 31) - 1]):
        buf = torch.full((M + 80, N), -3.0, dtype=torch.bfloat16, device="cuda")
        lay(x, torch.tensor(offs, dtype=torch.int32, device="cuda"), y=buf[40:40 + M])
        assert (buf[:40] == -3.0).all() and (buf[40 + M:] == -3.0).all()


@pytest.mark.parametrize("M", [1, 8, 16])
def test_layer_of_few_rows_over_its_input(M):
    note(f"Fp8Linear in place {M}")
    K = N = 1024
    lay = svdq.Fp8Linear.from_quantized(svdq.quantize_fp8(weights(K, N, 1)))
    x = acts(M, K, 2)
    want = lay(x)
    for _ in range(5):
        z = x.clone()
        assert lay(z, y=z) is z and torch.equal(z, want)


def test_layer_of_few_rows_on_streams_and_in_a_graph():
    note("Fp8Linear few rows: streams and graphs")
    K, N, M = 1040, 520, 4
    lay = svdq.Fp8Linear.from_quantized(svdq.quantize_fp8(weights(K, N, 1), biases(N, 2)))
    x = acts(M, K, 5)
    want = lay(x)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = [lay(x, stream=side), lay(x, stream=side.cuda_stream)]
    torch.cuda.synchronize()
    assert all(torch.equal(g, want) for g in got)
    y = torch.empty_like(want)
    graph = svdq.CapturedSequence(lambda: lay(x, y=y))
    for i in range(4):
        x.copy_(acts(M, K, 6 + i))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, lay(x))
        y.zero_()
    assert tuple(lay(x[:0]).shape) == (0, N)


def test_buffers_of_a_call_belong_to_its_stream():
    """Calls on a side stream while the current one allocates and overwrites
    memory of the same sizes: the codes between a layer's two kernels are the
    side stream's, also for a raw handle."""
    note("Fp8Linear on a busy side stream")
    M, K, N = 300, 1024, 512
    lay = svdq.Fp8Linear.from_quantized(svdq.quantize_fp8(weights(K, N, 1)))
    x = acts(M, K, 2)
    want = lay(x)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for s in (side, side.cuda_stream):
        got = []
        for _ in range(20):
            got.append(lay(x, stream=s))
            for shape in ((M, K), (8, M * 4)):
                torch.empty(shape, dtype=torch.uint8, device="cuda").fill_(0x7F)
        torch.cuda.synchronize()
        assert all(torch.equal(g, want) for g in got)


def test_package_round_trip(tmp_path):
    note("save_fp8_layer / load_fp8_layer")
    x = acts(9, 144, 1)
    lay = svdq.Fp8Linear.from_quantized(svdq.quantize_fp8(weights(144, 72, 1), biases(72, 2)))
    svdq.save_fp8_layer(str(tmp_path / "a.safetensors"), lay)
    assert torch.equal(svdq.load_fp8_layer(str(tmp_path / "a.safetensors"))(x), lay(x))
    grp = svdq.Fp8GroupedLinear.from_quantized(svdq.quantize_fp8(weights(144, 72, 3, groups=2)))
    svdq.save_fp8_layer(str(tmp_path / "g.safetensors"), grp)
    offs = torch.tensor([0, 4, 9], dtype=torch.int32, device="cuda")
    assert torch.equal(svdq.load_fp8_layer(str(tmp_path / "g.safetensors"))(x, offs), grp(x, offs))


def test_joint_block_input_in_eight_bits():
    """The operators together, as a joint block uses them: text and image
    rows through weights of their own, head norms and rotary positions in
    place in the fused output, against the oracles' chain."""
    note("FusedQKV over Fp8GroupedLinear")
    from oracle import rope as orope
    T, K, H, HK, D = 77, 400, 4, 2, 64
    N = (H + 2 * HK) * D
    x, b = acts(T, K, 1), biases((2, N), 2)
    layer = svdq.Fp8GroupedLinear.from_quantized(svdq.quantize_fp8(weights(K, N, 3, groups=2), b))
    offs = [0, 20, T]
    pos = torch.randint(0, 64, (T, 3), generator=torch.Generator().manual_seed(4), dtype=torch.int32).cuda()
    qn, kn = (1 + 0.1 * biases(D, 5)), (1 + 0.1 * biases(D, 6))
    block = svdq.FusedQKV(layer, svdq.RopePlan([16, 24, 24]), H, HK, qn, kn)
    q, k, v = block(x, pos, torch.tensor(offs, dtype=torch.int32, device="cuda"))
    assert tuple(q.shape) == (T, H, D) and tuple(k.shape) == tuple(v.shape) == (T, HK, D)
    qx, sx = ofp8.quantize_act(np64(x))
    ref = ofp8.grouped_linear(qx, sx, offs, np64(layer.qw), layer.sw.cpu().numpy(), np64(b))
    # The projection's rounding to bf16 (2^-8 of each value; its fp32 sums are far below)
    # moves a head h by d, |d|_2 <= rel |h|_2, so its direction by at most 2 rel; the norm
    # scales directions by sqrt(D) and at most max |w|, the rotation keeps lengths, and the
    # output rounds once more.
    axis, freq = orope.frequencies([16, 24, 24])
    y64 = ref[0].reshape(T, H + 2 * HK, D)
    for got, lo, hi, w in ((q, 0, H, qn), (k, H, H + HK, kn)):
        want = orope.rotate(orope.rms_norm(y64[:, lo:hi], np64(w), 1e-6), pos.cpu().numpy(), axis, freq)
        err = np.linalg.norm(np64(got) - want, axis=2)
        rel_in = 2.0 ** -8 + 2.0 ** -11          # with the E4M3 sums, 7 x 2^-13 of peaks
        bound = 2 * rel_in * np.abs(np64(w)).max() * math.sqrt(D) + (2.0 ** -8 + 2.0 ** -15) * np.linalg.norm(want, axis=2)
        assert (err <= bound).all(), f"worst ratio {(err / bound).max():.3g}"
    check_product(v.reshape(T, -1), [r[:, (H + HK) * D:] for r in ref], K)


def test_quantize_act_every_maximum():
    """Every finite bf16 magnitude as a block's maximum: the scale's division
    and its reciprocal are rounded correctly, and the codes follow."""
    note("quantize_act_fp8 every maximum")
    amax = torch.arange(0x7F80, dtype=torch.int32).to(torch.int16).view(torch.bfloat16)
    x = torch.zeros((amax.numel(), 128), dtype=torch.bfloat16)
    part = torch.tensor([1.0, -0.7, 0.33, -0.051, 0.0077, 1e-3, 1e-5], dtype=torch.float64)
    x[:, 3:10] = (amax.double()[:, None] * part).to(torch.bfloat16)
    q, s = svdq.quantize_act_fp8(x.cuda())
    qo, so = ofp8.quantize_act(x.double().numpy())
    assert np.array_equal(s.cpu().numpy(), so) and np.array_equal(np64(q), qo)
