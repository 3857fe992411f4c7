"""Host-side checks of the 8-bit layers and the rotary positions that need no
GPU: the C entry points' statuses, the Python entry points' refusals, plans
and packaged files."""
import ctypes

import pytest
import torch

import bit_quantized_diffusion_svdq_amd as svdq
from bit_quantized_diffusion_svdq_amd import _lib

OK, NULL, SHAPE, ALIGN, UNSUP, DEVICE = 0, 1, 2, 3, 4, 5
A = 0x7F0000000000
B, C, D, E, F = (A + i * 0x100000 for i in range(1, 6))
E4M3 = torch.float8_e4m3fn


@pytest.fixture(scope="module")
def lib():
    return svdq.load_library()


def valid(status):
    """A well-formed call: the capability check without a GPU."""
    if torch.cuda.is_available():
        pytest.skip("a GPU is present: well-formed calls on these placeholder pointers would launch")
    assert status == DEVICE


# ---------------------------------------------------------------- C ABI

def _act(lib, **kw):
    a = dict(x=A, M=7, K=144, ldx=144, qx=B, sx=C)
    a.update(kw)
    return lib.svdq_quantize_act_fp8(a["x"], a["M"], a["K"], a["ldx"], a["qx"], a["sx"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(M=-1), SHAPE), (dict(K=0), SHAPE), (dict(K=24), SHAPE), (dict(K=1 << 22), SHAPE), (dict(ldx=128), SHAPE),
    (dict(ldx=148), ALIGN), (dict(x=None), NULL), (dict(qx=None), NULL), (dict(sx=None), NULL), (dict(x=A + 8), ALIGN),
    (dict(qx=B + 8), ALIGN), (dict(sx=C + 2), ALIGN), (dict(M=1 << 40), SHAPE), (dict(M=0, x=None), OK),
])
def test_act_rejects(lib, kw, status):
    assert _act(lib, **kw) == status
    assert status == OK or lib.svdq_last_error()


def _weight(lib, **kw):
    a = dict(w=A, K=144, N=77, ldw=80, qw=B, sw=C)
    a.update(kw)
    return lib.svdq_quantize_weight_fp8(a["w"], a["K"], a["N"], a["ldw"], a["qw"], a["sw"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(K=8), SHAPE), (dict(N=0), SHAPE), (dict(N=1 << 24, ldw=1 << 24), SHAPE), (dict(ldw=72), SHAPE),
    (dict(ldw=77), ALIGN), (dict(w=None), NULL), (dict(qw=None), NULL), (dict(sw=None), NULL), (dict(w=A + 2), ALIGN),
])
def test_weight_rejects(lib, kw, status):
    assert _weight(lib, **kw) == status


def _gemm(lib, grouped, **kw):
    a = dict(qx=A, sx=B, M=33, K=144, qw=C, sw=D, N=77, offs=E, groups=3, bias=None, act=0, y=F, ydt=0, ldy=77)
    a.update(kw)
    if grouped:
        return lib.svdq_gemm_fp8_grouped(a["qx"], a["sx"], a["M"], a["K"], a["qw"], a["sw"], a["N"], a["offs"],
                                         a["groups"], a["bias"], a["act"], a["y"], a["ydt"], a["ldy"], None)
    return lib.svdq_gemm_fp8(a["qx"], a["sx"], a["M"], a["K"], a["qw"], a["sw"], a["N"], a["bias"], a["act"], a["y"],
                             a["ydt"], a["ldy"], None)


@pytest.mark.parametrize("grouped", [False, True])
@pytest.mark.parametrize("kw,status", [
    (dict(M=-1), SHAPE), (dict(M=1 << 31), SHAPE), (dict(K=40), SHAPE), (dict(K=0), SHAPE), (dict(K=1 << 22), SHAPE),
    (dict(N=0), SHAPE), (dict(N=1 << 30, ldy=1 << 30), SHAPE), (dict(ldy=76), SHAPE), (dict(ldy=1 << 31), SHAPE),
    (dict(act=2), UNSUP), (dict(ydt=2), UNSUP), (dict(qx=None), NULL), (dict(sx=None), NULL), (dict(qw=None), NULL),
    (dict(sw=None), NULL), (dict(y=None), NULL), (dict(qx=A + 8), ALIGN), (dict(qw=C + 4), ALIGN),
    (dict(sx=B + 2), ALIGN), (dict(bias=E + 1), ALIGN), (dict(y=F + 1), ALIGN), (dict(y=F + 2, ydt=1), ALIGN),
    (dict(M=1 << 30, N=1 << 20, ldy=1 << 20), SHAPE), (dict(M=0, qx=None), OK),
])
def test_gemm_rejects(lib, grouped, kw, status):
    assert _gemm(lib, grouped, **kw) == status
    assert status == OK or lib.svdq_last_error()


@pytest.mark.parametrize("kw,status", [(dict(groups=0), SHAPE), (dict(groups=-2), SHAPE), (dict(groups=65537), SHAPE),
                                       (dict(offs=None), NULL), (dict(offs=E + 2), ALIGN)])
def test_grouped_rejects(lib, kw, status):
    assert _gemm(lib, True, **kw) == status


def test_well_formed_calls_reach_the_device_check(lib):
    valid(_act(lib))
    valid(_weight(lib))
    valid(_gemm(lib, False))
    valid(_gemm(lib, True, y=F + 2, bias=E))


def _few(lib, **kw):
    a = dict(x=A, M=16, K=2048, ldx=2048, qw=C, sw=D, N=77, bias=None, act=0, y=F, ydt=0, ldy=77, ws=None, wsb=0)
    a.update(kw)
    return lib.svdq_linear_fp8(a["x"], a["M"], a["K"], a["ldx"], a["qw"], a["sw"], a["N"], a["bias"], a["act"], a["y"],
                               a["ydt"], a["ldy"], a["ws"], a["wsb"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(M=-1), SHAPE), (dict(M=17, K=128), SHAPE), (dict(K=2064, ldx=2064), SHAPE), (dict(M=1, K=32784, ldx=32784), SHAPE),
    (dict(M=17, wsb=17 * 2048 + 17 * 64 - 1, ws=B), SHAPE), (dict(M=17, wsb=17 * 2048 + 17 * 64), NULL),
    (dict(M=17, wsb=1 << 20, ws=B + 8), ALIGN), (dict(M=1 << 31), SHAPE), (dict(M=1 << 30, K=1 << 16, ldx=1 << 16), SHAPE),
    (dict(K=40), SHAPE), (dict(K=0), SHAPE), (dict(K=1 << 22), SHAPE), (dict(N=0), SHAPE),
    (dict(N=1 << 23, ldy=1 << 23), SHAPE), (dict(ldx=2032), SHAPE), (dict(ldx=2052), ALIGN), (dict(ldy=76), SHAPE),
    (dict(ldy=1 << 31), SHAPE), (dict(act=2), UNSUP), (dict(ydt=2), UNSUP), (dict(x=None), NULL), (dict(qw=None), NULL),
    (dict(sw=None), NULL), (dict(y=None), NULL), (dict(x=A + 8), ALIGN), (dict(qw=C + 4), ALIGN), (dict(sw=D + 2), ALIGN),
    (dict(bias=E + 1), ALIGN), (dict(y=F + 1), ALIGN), (dict(y=F + 2, ydt=1), ALIGN), (dict(M=0, x=None), OK),
])
def test_layer_of_few_rows_rejects(lib, kw, status):
    assert _few(lib, **kw) == status
    assert status == OK or lib.svdq_last_error()


def _few_grouped(lib, **kw):
    a = dict(x=A, M=16, K=2048, ldx=2048, qw=C, sw=D, N=77, offs=E, groups=5, bias=None, act=0, y=F, ydt=0, ldy=77, ws=None,
             wsb=0)
    a.update(kw)
    return lib.svdq_linear_fp8_grouped(a["x"], a["M"], a["K"], a["ldx"], a["qw"], a["sw"], a["N"], a["offs"], a["groups"],
                                       a["bias"], a["act"], a["y"], a["ydt"], a["ldy"], a["ws"], a["wsb"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(M=17, K=128), SHAPE), (dict(N=(1 << 23) - 8, ldy=1 << 23), SHAPE), (dict(M=17, wsb=1 << 20), NULL), (dict(K=2064, ldx=2064), SHAPE), (dict(groups=0), SHAPE), (dict(groups=-1), SHAPE),
    (dict(groups=65537), SHAPE), (dict(N=1 << 23, ldy=1 << 23), SHAPE), (dict(offs=None), NULL), (dict(offs=E + 2), ALIGN),
    (dict(x=None), NULL), (dict(ldx=2052), ALIGN), (dict(y=F + 1), ALIGN), (dict(act=2), UNSUP), (dict(M=0, offs=None), OK),
])
def test_grouped_layer_of_few_rows_rejects(lib, kw, status):
    assert _few_grouped(lib, **kw) == status
    assert status == OK or lib.svdq_last_error()


def test_layer_of_few_rows_limits(lib):
    valid(_few_grouped(lib))
    valid(_few(lib))
    valid(_few(lib, M=1, K=32768, ldx=1 << 40, bias=E, N=(1 << 23) - 1, ldy=1 << 23))
    valid(_few(lib, M=17, ws=B, wsb=17 * 2048 + 17 * 64))
    valid(_few_grouped(lib, M=4000, ws=B, wsb=4000 * 2048 + 4000 * 64))


def test_layer_workspace(lib):
    from bit_quantized_diffusion_svdq_amd.fp8 import _workspace_bytes
    for M, K in ((0, 16), (1, 16), (1, 32768), (1, 32784), (16, 2048), (16, 2064), (17, 16), (4608, 12288)):
        assert svdq.svdq_linear_fp8_workspace_size(M, K) == _workspace_bytes(M, K)
    assert _workspace_bytes(16, 2048) == 0 and _workspace_bytes(17, 144) == 17 * 144 + 17 * 8
    for M, K in ((-1, 16), (1, 24), (1 << 31, 16)):
        with pytest.raises(svdq.SvdqError):
            svdq.svdq_linear_fp8_workspace_size(M, K)
    assert lib.svdq_linear_fp8_workspace_size(1, 16, None) == NULL


def _heads(**kw):
    a = dict(x=A, ts=256, hs=64, heads=4, norm=None, y=B, yts=256, yhs=64)
    a.update(kw)
    return _lib.RopeHeads(a["x"], a["ts"], a["hs"], a["heads"], a["norm"], a["y"], a["yts"], a["yhs"])


def _rope(lib, q=None, k=None, **kw):
    a = dict(T=5, D=64, dt=0, pos=C, pdt=0, axes=3, turns=D, axis=E, pairs=32, pairing=0, inverse=0, eps=1e-6)
    a.update(kw)
    q = _heads() if q is None else q
    return lib.svdq_rope_axes(ctypes.addressof(q) if q else None, ctypes.addressof(k) if k else None, a["T"], a["D"],
                              a["dt"], a["pos"], a["pdt"], a["axes"], a["turns"], a["axis"], a["pairs"], a["pairing"],
                              a["inverse"], a["eps"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), SHAPE), (dict(D=60), SHAPE), (dict(D=0), SHAPE), (dict(D=520), SHAPE), (dict(pairs=30), SHAPE),
    (dict(pairs=36), SHAPE), (dict(pairs=-4), SHAPE), (dict(axes=0), SHAPE), (dict(axes=9), SHAPE), (dict(dt=2), UNSUP),
    (dict(pdt=2), UNSUP), (dict(pairing=2), UNSUP), (dict(inverse=2), UNSUP), (dict(eps=-1.0), UNSUP),
    (dict(eps=float("nan")), UNSUP), (dict(pos=None), NULL), (dict(turns=None), NULL), (dict(axis=None), NULL),
    (dict(turns=D + 4), ALIGN), (dict(pos=C + 2), ALIGN), (dict(T=0, pos=None), OK),
])
def test_rope_rejects(lib, kw, status):
    assert _rope(lib, **kw) == status
    assert status == OK or lib.svdq_last_error()


@pytest.mark.parametrize("kw,status", [
    (dict(heads=70000), SHAPE), (dict(ts=-8), SHAPE), (dict(hs=60), ALIGN), (dict(yts=252), ALIGN),
    (dict(x=None), NULL), (dict(y=None), NULL), (dict(x=A + 8), ALIGN), (dict(norm=E + 8), ALIGN),
    (dict(yhs=0), SHAPE), (dict(yts=0), SHAPE), (dict(yhs=32), SHAPE), (dict(yts=128), SHAPE),
])
def test_rope_heads_rejects(lib, kw, status):
    assert _rope(lib, q=_heads(**kw)) == status
    assert _rope(lib, k=_heads(**kw)) == status


def test_rope_accepts(lib):
    assert lib.svdq_rope_axes(None, None, 1, 64, 0, C, 0, 1, D, E, 32, 0, 0, 1e-6, None) == NULL
    assert _rope(lib, q=_heads(heads=0)) == SHAPE
    valid(_rope(lib, k=_heads(heads=0)))
    valid(_rope(lib, q=_heads(ts=0, hs=0)))                 # a broadcast input may be read
    valid(_rope(lib, q=_heads(yts=64, yhs=320)))            # head-major output of 5 tokens
    valid(_rope(lib, pairs=0, pos=None))


# ---------------------------------------------------------------- Python entry points

def test_plan():
    p = svdq.RopePlan((16, 56, 56), device="cpu")
    assert (p.head_dim, p.pairs, p.axes) == (128, 64, 3) and p.turns.dtype == torch.float64
    assert p.axis.tolist() == [0] * 8 + [1] * 28 + [2] * 28
    assert float(p.turns[0]) * 2 * 3.141592653589793 == pytest.approx(1.0, rel=1e-15)
    p = svdq.RopePlan((4, 4), head_dim=16, theta=(100.0, 4.0), pairing="half", device="cpu")
    assert (p.turns * 2 * 3.141592653589793).tolist() == pytest.approx([1.0, 0.1, 1.0, 0.5])
    p = svdq.RopePlan((8,), freqs=[1, 2, 3, 4], device="cpu")
    assert (p.turns * 2 * 3.141592653589793).tolist() == pytest.approx([1, 2, 3, 4])
    assert svdq.RopePlan((0,), head_dim=8, device="cpu").pairs == 0


@pytest.mark.parametrize("args,kw", [
    (((),), {}), (((4,) * 9,), {}), (((3, 5),), {}), (((4, 2),), {}), (((16,),), dict(head_dim=8)),
    (((16,),), dict(head_dim=20)), (((520,),), {}), (((16,),), dict(pairing="split")), (((16,),), dict(theta=0.0)),
    (((8, 8),), dict(theta=(1.0,))), (((8,),), dict(freqs=[1.0])), (((-8, 16),), {}),
])
def test_plan_refuses(args, kw):
    with pytest.raises(ValueError):
        svdq.RopePlan(*args, device="cpu", **kw)


def _rope_args(**kw):
    a = dict(q=torch.zeros((4, 3, 32), dtype=torch.bfloat16), k=torch.zeros((4, 1, 32), dtype=torch.bfloat16),
             pos=torch.zeros((4, 2), dtype=torch.int32), plan=svdq.RopePlan((16, 16), device="cpu"))
    a.update(kw)
    return a


bf, f32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("kw,text", [
    (dict(q=torch.zeros((4, 96), dtype=bf)), "q must be"), (dict(q=torch.zeros((4, 3, 64), dtype=bf)), "q must be"),
    (dict(q=torch.zeros((4, 3, 32), dtype=torch.float16)), "bf16 or fp32"),
    (dict(q=torch.zeros((4, 32, 3), dtype=bf).transpose(1, 2)), "contiguous heads"),
    (dict(q=torch.zeros((4, 0, 32), dtype=bf)), "at least one head"),
    (dict(k=torch.zeros((5, 1, 32), dtype=bf)), "k must have"), (dict(k=torch.zeros((4, 1, 32))), "k must have"),
    (dict(k=None, k_norm=torch.zeros(32, dtype=bf)), "need k"), (dict(q_norm=torch.zeros(32)), "q_norm"),
    (dict(k_norm=torch.zeros(16, dtype=bf)), "k_norm"), (dict(q_out=torch.zeros((4, 3, 32))), "q_out"),
    (dict(k_out=torch.zeros((4, 2, 32), dtype=bf)), "k_out"),
    (dict(pos=torch.zeros((4, 3), dtype=torch.int32)), "pos must be"),
    (dict(pos=torch.zeros((4, 2), dtype=torch.int64)), "pos must be"),
    (dict(pos=torch.zeros((2, 4), dtype=torch.int32).t()), "pos must be"),
    (dict(), "GPU device"),
])
def test_rope_axes_refuses(kw, text):
    a = _rope_args(**kw)
    with pytest.raises(ValueError, match=text):
        svdq.rope_axes(a.pop("q"), a.pop("k"), a.pop("pos"), a.pop("plan"), **a)


def _prod(groups=0, **kw):
    lead = (groups,) if groups else ()
    a = dict(qx=torch.zeros((5, 144), dtype=torch.uint8).view(E4M3), sx=torch.ones((2, 5)),
             qw=torch.zeros((*lead, 130, 144), dtype=torch.uint8).view(E4M3), sw=torch.ones((*lead, 2, 2)))
    a.update(kw)
    return a


@pytest.mark.parametrize("kw,text", [
    (dict(qx=torch.zeros((5, 144), dtype=torch.uint8)), "qx must be"),
    (dict(qx=torch.zeros((5, 152), dtype=torch.uint8).view(E4M3)[:, :144]), "contiguous"),
    (dict(qx=torch.zeros((5, 40), dtype=torch.uint8).view(E4M3)), "multiple of 16"),
    (dict(sx=torch.ones((5, 2))), "sx must be"), (dict(sx=torch.ones((2, 5), dtype=torch.float64)), "sx must be"),
    (dict(sx=torch.ones((5, 2)).t()), "sx must be"),
    (dict(qw=torch.zeros((130, 128), dtype=torch.uint8).view(E4M3)), "qw must be"),
    (dict(qw=torch.zeros((130, 144))), "qw must be"), (dict(sw=torch.ones((1, 2))), "sw must be"),
    (dict(bias=torch.zeros(130)), "bias must be"), (dict(bias=torch.zeros(144, dtype=bf)), "bias must be"),
    (dict(act="relu"), "act must be"), (dict(out_dtype=torch.float16), "bf16 or fp32"),
    (dict(y=torch.zeros((5, 131), dtype=bf)), "y must be"), (dict(y=torch.zeros((130, 5), dtype=bf).t()), "y must be"),
    (dict(y=torch.zeros((1, 130), dtype=bf).expand(5, 130)), "y must be"), (dict(), "GPU device"),
])
def test_fp8_linear_refuses(kw, text):
    a = _prod(**kw)
    with pytest.raises(ValueError, match=text):
        svdq.fp8_linear(a.pop("qx"), a.pop("sx"), a.pop("qw"), a.pop("sw"), **a)


@pytest.mark.parametrize("kw,text", [
    (dict(offsets=torch.zeros(4, dtype=torch.int64)), "offsets must be"),
    (dict(offsets=torch.zeros(1, dtype=torch.int32)), "offsets must be"),
    (dict(offsets=torch.zeros((2, 2), dtype=torch.int32)), "offsets must be"),
    (dict(offsets=torch.zeros(3, dtype=torch.int32)), "qw must be|sw must be"),
    (dict(bias=torch.zeros(130, dtype=bf)), "bias must be"), (dict(), "GPU device"),
])
def test_fp8_grouped_linear_refuses(kw, text):
    a = dict(offsets=torch.zeros(4, dtype=torch.int32))
    a.update(_prod(groups=3))
    a.update(kw)
    with pytest.raises(ValueError, match=text):
        svdq.fp8_grouped_linear(a.pop("qx"), a.pop("sx"), a.pop("offsets"), a.pop("qw"), a.pop("sw"), **a)


@pytest.mark.parametrize("M", [1, 16, 400])
@pytest.mark.parametrize("kw,text", [
    (dict(x=torch.zeros((16, 128), dtype=bf)), "x must be"), (dict(x=torch.zeros((16, 144))), "x must be"),
    (dict(x=torch.zeros(144, dtype=bf)), "x must be"), (dict(x=torch.zeros((144, 16), dtype=bf).t()), "contiguous"),
    (dict(), "GPU device"),
])
def test_layer_refuses(M, kw, text):
    """The same words for few rows (one launch) and many."""
    a = _prod()
    x = kw.get("x", torch.zeros((M, 144), dtype=bf))
    if x.dim() == 2 and x.shape[0] == 16 and M > 16:
        x = x.repeat(M // 16, 1) if x.is_contiguous() else torch.zeros((144, M), dtype=bf).t()
    with pytest.raises(ValueError, match=text):
        svdq.Fp8Linear(a["qw"], a["sw"])(x)


@pytest.mark.parametrize("M", [2, 16, 400])
@pytest.mark.parametrize("kw,text", [
    (dict(offsets=torch.zeros(4, dtype=torch.int64)), "offsets must be"), (dict(offsets=torch.zeros(3, dtype=torch.int32)), "offsets must hold"),
    (dict(x=torch.zeros((2, 128), dtype=bf)), "x must be"), (dict(), "GPU device"),
])
def test_grouped_layer_refuses(M, kw, text):
    a = _prod(groups=3)
    a = dict(qw=a["qw"], sw=a["sw"], x=torch.zeros((M, 144), dtype=bf), offsets=torch.zeros(4, dtype=torch.int32)) | kw
    with pytest.raises(ValueError, match=text):
        svdq.Fp8GroupedLinear(a["qw"], a["sw"])(a["x"], a["offsets"])


def test_names_are_public():
    names = ("svdq_quantize_act_fp8", "svdq_quantize_weight_fp8", "svdq_gemm_fp8", "svdq_gemm_fp8_grouped",
             "svdq_linear_fp8", "svdq_linear_fp8_grouped", "svdq_linear_fp8_workspace_size", "svdq_rope_axes", "Fp8Linear", "Fp8GroupedLinear", "fp8_linear", "fp8_grouped_linear",
             "quantize_act_fp8", "quantize_fp8", "RopePlan", "rope_axes", "FusedQKV", "save_fp8_layer", "load_fp8_layer")
    assert all(n in svdq.__all__ and hasattr(svdq, n) for n in names)


def test_quantisers_refuse():
    for x in (torch.zeros((3, 32)), torch.zeros((3, 40), dtype=bf), torch.zeros((3, 0), dtype=bf),
              torch.zeros(32, dtype=bf), torch.zeros((32, 3), dtype=bf).t(), torch.zeros((3, 32), dtype=bf)):
        with pytest.raises(ValueError):
            svdq.quantize_act_fp8(x)
    for w in (torch.zeros((32, 8)), torch.zeros((40, 8), dtype=bf), torch.zeros((32, 0), dtype=bf),
              torch.zeros((0, 32, 8), dtype=bf), torch.zeros((8, 32), dtype=bf).t(), torch.zeros((32, 8), dtype=bf)):
        with pytest.raises(ValueError):
            svdq.quantize_fp8(w)
    with pytest.raises(ValueError, match="bias"):
        svdq.quantize_fp8(torch.zeros((32, 8), dtype=bf), bias=torch.zeros(9, dtype=bf))


def _layer(groups=0, N=192):
    a = _prod(groups)
    lead = (groups,) if groups else ()
    cls = svdq.Fp8GroupedLinear if groups else svdq.Fp8Linear
    return cls(torch.zeros((*lead, N, 144), dtype=torch.uint8).view(E4M3), torch.ones((*lead, 2, 2)))


def test_layers_and_qkv_block_refuse():
    with pytest.raises(ValueError, match="x must be"):
        _layer()(torch.zeros((3, 128), dtype=bf))
    with pytest.raises(ValueError, match="offsets"):
        _layer(2)(torch.zeros((3, 144), dtype=bf), torch.zeros(2, dtype=torch.int32))
    plan = svdq.RopePlan((16, 16), device="cpu")
    with pytest.raises(ValueError, match="outputs"):
        svdq.FusedQKV(_layer(N=96), plan, 2)
    with pytest.raises(ValueError, match="heads"):
        svdq.FusedQKV(_layer(), plan, 0)
    with pytest.raises(ValueError, match="q_norm"):
        svdq.FusedQKV(_layer(), plan, 2, q_norm=torch.zeros(32))
    block = svdq.FusedQKV(_layer(), plan, 2)
    with pytest.raises(ValueError, match="offsets"):
        block(torch.zeros((3, 144), dtype=bf), torch.zeros((3, 2), dtype=torch.int32), offsets=torch.zeros(2))
    with pytest.raises(ValueError, match="offsets"):
        svdq.FusedQKV(_layer(2), plan, 2)(torch.zeros((3, 144), dtype=bf), torch.zeros((3, 2), dtype=torch.int32))


def test_packaged_layers(tmp_path):
    from safetensors.torch import load_file, save_file
    path = str(tmp_path / "l.safetensors")
    for groups in (0, 3):
        lay = _layer(groups)
        lay.qw.view(torch.uint8).random_(0, 0x7F)
        meta = svdq.save_fp8_layer(path, lay, source="test")
        assert meta["groups"] == str(groups)
        got = svdq.load_fp8_layer(path, device="cpu")
        assert type(got) is type(lay) and got.bias is None
        assert torch.equal(got.qw.view(torch.uint8), lay.qw.view(torch.uint8)) and torch.equal(got.sw, lay.sw)
    ts, meta = load_file(path), svdq.read_metadata(path)
    for change, text in ((dict(groups="2"), "expected"), (dict(K="160"), "expected"), (dict(K="20"), "malformed"),
                         (dict(group="64"), "group"), (dict(format="x"), "format"), (dict(N="x"), "integer")):
        save_file(ts, path, metadata={**meta, **change})
        with pytest.raises(ValueError, match=text):
            svdq.load_fp8_layer(path, device="cpu")
    save_file({"qw": ts["qw"]}, path, metadata=meta)
    with pytest.raises(ValueError, match="missing"):
        svdq.load_fp8_layer(path, device="cpu")
    save_file({**ts, "more": ts["sw"].clone()}, path, metadata=meta)
    with pytest.raises(ValueError, match="unexpected"):
        svdq.load_fp8_layer(path, device="cpu")
    with pytest.raises(ValueError, match="expected"):
        svdq.save_fp8_layer(path, svdq.Fp8Linear(lay.qw[0], lay.sw[0, :1]))
