"""The cases of the 8-bit layers and of the multi-axis rotary positions: their
inputs, their plain forms, the framework's calls and what each has to move
and compute.

Kinds of a case:
  act      svdq.quantize_act_fp8: bf16 activations [M, K] -> E4M3 codes and an
           fp32 scale per (row, 128 channels)
  gemm     svdq.fp8_linear: codes and scales in hand -> act(X W^T + bias)
  layer    svdq.Fp8Linear: bf16 activations -> act(X W^T + bias), both steps
  grouped  svdq.fp8_grouped_linear: rows sorted by group, group g's rows meet
           weight g (experts, or the streams of a joint block)
  rope     svdq.rope_axes: queries and keys rotated by positions on several
           axes, optionally after an RMS norm of each head
"""
import math

import torch

own = False

BLOCK = 128
E4M3_MAX = 448.0
SCALE_MIN = 2.0 ** -120        # least block scale (a block of zeros has it)


# ---------------------------------------------------------------- cases

def listed():
    return [
        # one token's modulation input on its way into an 8-bit layer: latency
        dict(name="act_one_row", op="act", M=1, K=4096),
        # the GELU output of a 1024 x 1024 image with its text tokens, before the MLP's second layer
        dict(name="act_image", op="act", M=4608, K=12288),
        # modulation projection of a single conditioning vector: the weights' bytes count
        dict(name="gemm_one_row", op="gemm", M=1, K=4096, N=18432, act="none", bias=True, out="bf16"),
        # a short ragged prompt in a narrow model, odd in every size, full-precision output
        dict(name="gemm_odd", op="gemm", M=77, K=2064, N=1001, act="none", bias=True, out="f32"),
        # text tokens of a prompt through an MLP's first layer, from bf16 activations
        dict(name="layer_text", op="layer", M=512, K=4096, N=12288, act="gelu_tanh", bias=True, out="bf16"),
        # image and text tokens through an MLP's second layer: the matrix pipe counts
        dict(name="gemm_image", op="gemm", M=4608, K=12288, N=4096, act="none", bias=True, out="bf16"),
        # the same tokens through a whole first layer
        dict(name="layer_image", op="layer", M=4608, K=4096, N=12288, act="gelu_tanh", bias=True, out="bf16"),
        # few tokens over many experts, some without any
        dict(name="grouped_few", op="grouped", M=48, K=2048, N=4096, E=32, spread=1.0, act="none", bias=False,
             out="bf16"),
        # many tokens over experts whose shares differ
        dict(name="grouped_many", op="grouped", M=8200, K=4096, N=4096, E=16, spread=0.6, act="gelu_tanh",
             bias=True, out="bf16"),
        # one token's query and key: latency
        dict(name="rope_one", op="rope", T=1, hq=24, hk=24, D=128, dims="16,56,56", pairing="interleaved",
             norm=True, dtype="bf16", fused=True, inverse=False),
        # queries and keys inside the fused [Q | K | V] output of an image with its text tokens
        dict(name="rope_image", op="rope", T=4608, hq=24, hk=24, D=128, dims="16,56,56", pairing="interleaved",
             norm=True, dtype="bf16", fused=True, inverse=False),
        # a video's tokens (time, height, width), an odd number, shared key heads, half-split pairs
        dict(name="rope_video", op="rope", T=32761, hq=16, hk=4, D=128, dims="44,42,42", pairing="half",
             norm=False, dtype="bf16", fused=False, inverse=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    """One more case of the listed ones' ranges."""
    op = rng.choice(["act", "gemm", "layer", "grouped", "rope"])
    if op == "act":
        M = _log(rng, 1, 8192)
        K = 16 * _log(rng, 1, 768)
        return dict(op=op, M=min(M, max(1, 4608 * 12288 // K)), K=K)
    if op == "rope":
        D, dims = rng.choice([(64, "64"), (64, "16,24,24"), (96, "32,32,32"), (128, "16,56,56"), (128, "44,42,42"),
                              (128, "64,64"), (128, "32,32"), (72, "24,24,24"), (256, "64,96,96")])
        hq = rng.choice([1, 3, 8, 16, 24, 40])
        hk = rng.choice([h for h in (1, 2, 8, 24) if h <= hq])
        T = _log(rng, 1, 32768)
        T = min(T, max(1, 32761 * 20 * 128 // ((hq + hk) * D)))
        return dict(op=op, T=T, hq=hq, hk=hk, D=D, dims=dims, pairing=rng.choice(["interleaved", "half"]),
                    norm=rng.random() < 0.5, dtype=rng.choice(["bf16", "bf16", "f32"]), fused=rng.random() < 0.5,
                    inverse=rng.random() < 0.2)
    M = _log(rng, 1, 8200 if op == "grouped" else 4608)
    K = 16 * _log(rng, 4, 768)
    N = _log(rng, 8, 12288)
    E = _log(rng, 1, 48) if op == "grouped" else 1
    while E * N * K > 32 * 2048 * 4096 and E > 1:       # bytes of the weights
        E = max(1, E // 2)
    M = min(M, max(1, 4608 * 12288 * 4096 // (N * K)))
    case = dict(op=op, M=M, K=K, N=N, act=rng.choice(["none", "gelu_tanh"]), bias=rng.random() < 0.7,
                out=rng.choice(["bf16", "bf16", "f32"]))
    if op == "grouped":
        case.update(E=E, spread=round(rng.uniform(0.0, 1.5), 2))
    return case


# ---------------------------------------------------------------- inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) & 0x7FFFFFFFFFFF)
    return g


def _activations(M, K, g):
    """Normal values with a few channels that stand out, as a DiT's
    activations have them."""
    x = torch.randn((M, K), generator=g, device="cuda", dtype=torch.float32)
    loud = torch.rand((K,), generator=g, device="cuda") < 0.01
    return (x * torch.where(loud, 20.0, 1.0)).to(torch.bfloat16)


def _scale(amax):
    """max(amax / 448, 2^-120) with the fp32 quotient rounded correctly (a
    quotient by a number is computed as a product with its reciprocal, so it
    is taken in 64 bits)."""
    return torch.clamp((amax.double() / E4M3_MAX).float(), min=SCALE_MIN)


def _reciprocal(s):
    return (1.0 / s.double()).float()


def _codes_by_row(x):
    """E4M3 codes of x [M, K] and fp32 scales [ceil(K / 128), M]: per row and
    128 channels s = max(amax / 448, 2^-120), code = e4m3(x * (1 / s))."""
    M, K = x.shape
    kb = -(-K // BLOCK)
    xf = torch.nn.functional.pad(x.float(), (0, kb * BLOCK - K)).view(M, kb, BLOCK)
    s = _scale(xf.abs().amax(dim=2))
    q = torch.clamp(xf * _reciprocal(s)[:, :, None], -E4M3_MAX, E4M3_MAX).view(M, kb * BLOCK)[:, :K]
    return q.to(torch.float8_e4m3fn).contiguous(), s.t().contiguous()


def _codes_by_block(w):
    """E4M3 codes of w [N, K] and fp32 scales [ceil(N / 128), ceil(K / 128)]."""
    N, K = w.shape
    nb, kb = -(-N // BLOCK), -(-K // BLOCK)
    wf = torch.nn.functional.pad(w.float(), (0, kb * BLOCK - K, 0, nb * BLOCK - N)).view(nb, BLOCK, kb, BLOCK)
    s = _scale(wf.abs().amax(dim=(1, 3)))
    q = torch.clamp(wf * _reciprocal(s)[:, None, :, None], -E4M3_MAX, E4M3_MAX).view(nb * BLOCK, kb * BLOCK)
    return q[:N, :K].to(torch.float8_e4m3fn).contiguous(), s.contiguous()


def _group_sizes(case, seed):
    """Rows of each group: shares e^(spread z), z normal; they add up to M."""
    E, M = case["E"], case["M"]
    z = torch.randn(E, generator=torch.Generator().manual_seed(int(seed) * 7 + 1), dtype=torch.float64)
    share = torch.exp(case["spread"] * z)
    cuts = torch.floor(torch.cumsum(share, 0) / share.sum() * M).long()
    cuts[-1] = M
    return [int(b - a) for a, b in zip([0] + cuts[:-1].tolist(), cuts.tolist())]


def _axis_of_pairs(case):
    """(axis, inverse frequency) of every pair of a head: axis a of width d
    has the frequencies 10000^(-2 i / d), i = 0 .. d / 2 - 1."""
    axis, freq = [], []
    for a, d in enumerate(int(v) for v in case["dims"].split(",")):
        for i in range(d // 2):
            axis.append(a)
            freq.append(10000.0 ** (-2.0 * i / d))
    return axis, freq


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    st = dict(case=case)
    if own:
        import bit_quantized_diffusion_svdq_amd as svdq
        st["svdq"] = svdq
    if op == "act":
        st["x"] = _activations(case["M"], case["K"], g)
        return st
    if op == "rope":
        T, hq, hk, D = case["T"], case["hq"], case["hk"], case["D"]
        dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
        heads = hq + (2 * hk if case["fused"] else hk)
        flat = torch.randn((T, heads * D), generator=g, device="cuda").to(dt)
        if case["fused"]:            # views of the fused projection's output
            st["q"] = flat[:, :hq * D].view(T, hq, D)
            st["k"] = flat[:, hq * D:(hq + hk) * D].view(T, hk, D)
        else:
            st["q"] = flat[:, :hq * D].contiguous().view(T, hq, D)
            st["k"] = flat[:, hq * D:].contiguous().view(T, hk, D)
        dims = [int(v) for v in case["dims"].split(",")]
        st["pos"] = torch.randint(0, 4096, (T, len(dims)), generator=g, device="cuda", dtype=torch.int32)
        st["qn"] = st["kn"] = None
        if case["norm"]:
            st["qn"] = (1 + 0.2 * torch.randn(D, generator=g, device="cuda")).to(dt)
            st["kn"] = (1 + 0.2 * torch.randn(D, generator=g, device="cuda")).to(dt)
        if own:
            st["plan"] = st["svdq"].RopePlan(dims, head_dim=D, pairing=case["pairing"], device="cuda")
        else:
            axis, freq = _axis_of_pairs(case)
            st["axis"] = torch.tensor(axis, device="cuda")
            st["freq"] = torch.tensor(freq, device="cuda", dtype=torch.float64)
        return st
    M, K, N = case["M"], case["K"], case["N"]
    x = _activations(M, K, g)
    if op == "layer":
        st["x"] = x
    else:
        st["qx"], st["sx"] = _codes_by_row(x)
    E = case.get("E", 1)
    ws = [_codes_by_block(torch.randn((N, K), generator=g, device="cuda") * 0.02) for _ in range(E)]
    st["bias"] = (torch.randn((E, N), generator=g, device="cuda") * 0.1).to(torch.bfloat16) if case["bias"] else None
    if op == "grouped":
        st["qw"] = torch.stack([w.view(torch.uint8) for w, _ in ws]).view(torch.float8_e4m3fn)
        st["sw"] = torch.stack([s for _, s in ws])
        st["sizes"] = _group_sizes(case, seed)
        st["offsets"] = torch.tensor([0] + torch.tensor(st["sizes"]).cumsum(0).tolist(), dtype=torch.int32,
                                     device="cuda")
    else:
        st["qw"], st["sw"] = ws[0]
        st["bias"] = None if st["bias"] is None else st["bias"][0]
        if own and op == "layer":
            st["layer"] = st["svdq"].Fp8Linear(st["qw"], st["sw"], st["bias"])
    return st


# ---------------------------------------------------------------- one pass

def _out_dtype(case):
    return torch.bfloat16 if case["out"] == "bf16" else torch.float32


def _activation(y, act):
    if act == "none":
        return y
    return 0.5 * y * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (y + 0.044715 * y * y * y)))


def _by_row_values(q, s, dtype=torch.float32):
    K = q.shape[1]
    return q.to(dtype) * s.to(dtype).t().repeat_interleave(BLOCK, dim=1)[:, :K]


def _by_block_values(q, s, dtype=torch.float32):
    N, K = q.shape
    return q.to(dtype) * s.to(dtype).repeat_interleave(BLOCK, 0)[:N].repeat_interleave(BLOCK, 1)[:, :K]


def _linear(qx, sx, qw, sw, bias, act, dtype=torch.float32):
    y = _by_row_values(qx, sx, dtype) @ _by_block_values(qw, sw, dtype).t()
    if bias is not None:
        y = y + bias.to(dtype)
    return _activation(y, act)


def _grouped(st, dtype=torch.float32):
    case, out, m0 = st["case"], [], 0
    for e, m in enumerate(st["sizes"]):
        if m:
            out.append(_linear(st["qx"][m0:m0 + m], st["sx"][:, m0:m0 + m], st["qw"][e], st["sw"][e],
                               None if st["bias"] is None else st["bias"][e], case["act"], dtype))
        m0 += m
    return torch.cat(out)


def _rotate(x, norm, st, dtype):
    """The heads of x [T, H, D] rotated, in `dtype`."""
    case = st["case"]
    T, H, D = x.shape
    v = x.to(dtype)
    if norm is not None:
        v = v * torch.rsqrt((v * v).mean(dim=2, keepdim=True) + 1e-6) * norm.to(dtype)
    angle = st["pos"].double()[:, st["axis"]] * st["freq"]
    if case["inverse"]:
        angle = -angle
    c, s = torch.cos(angle).to(dtype)[:, None, :], torch.sin(angle).to(dtype)[:, None, :]
    R = 2 * c.shape[2]
    y = v.clone()
    if case["pairing"] == "interleaved":
        a, b = v[:, :, 0:R:2], v[:, :, 1:R:2]
        y[:, :, 0:R:2], y[:, :, 1:R:2] = a * c - b * s, a * s + b * c
    else:
        a, b = v[:, :, :R // 2], v[:, :, R // 2:R]
        y[:, :, :R // 2], y[:, :, R // 2:R] = a * c - b * s, a * s + b * c
    return y


def run(st):
    case = st["case"]
    op = case["op"]
    if own:
        svdq = st["svdq"]
        if op == "act":
            return svdq.quantize_act_fp8(st["x"])
        if op == "gemm":
            return svdq.fp8_linear(st["qx"], st["sx"], st["qw"], st["sw"], st["bias"], act=case["act"],
                                   out_dtype=_out_dtype(case))
        if op == "layer":
            return st["layer"](st["x"], act=case["act"], out_dtype=_out_dtype(case))
        if op == "grouped":
            return svdq.fp8_grouped_linear(st["qx"], st["sx"], st["offsets"], st["qw"], st["sw"], st["bias"],
                                           act=case["act"], out_dtype=_out_dtype(case))
        return svdq.rope_axes(st["q"], st["k"], st["pos"], st["plan"], q_norm=st["qn"], k_norm=st["kn"], eps=1e-6,
                              inverse=case["inverse"])
    if op == "act":
        return _codes_by_row(st["x"])
    if op == "gemm":
        return _linear(st["qx"], st["sx"], st["qw"], st["sw"], st["bias"], case["act"]).to(_out_dtype(case))
    if op == "layer":
        qx, sx = _codes_by_row(st["x"])
        return _linear(qx, sx, st["qw"], st["sw"], st["bias"], case["act"]).to(_out_dtype(case))
    if op == "grouped":
        return _grouped(st).to(_out_dtype(case))
    return (_rotate(st["q"], st["qn"], st, torch.float32).to(st["q"].dtype),
            _rotate(st["k"], st["kn"], st, torch.float32).to(st["k"].dtype))


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    op = case["op"]
    kb = -(-case.get("K", 0) // BLOCK)
    if op == "act":
        M, K = case["M"], case["K"]
        return dict(bytes=M * K * 3 + M * kb * 4, flops=M * K * 4)
    if op == "rope":
        el = 2 if case["dtype"] == "bf16" else 4
        n = case["T"] * (case["hq"] + case["hk"]) * case["D"]
        return dict(bytes=2 * n * el + case["T"] * 4 * len(case["dims"].split(",")), flops=n * (7 if case["norm"] else 3))
    M, K, N = case["M"], case["K"], case["N"]
    nb = -(-N // BLOCK)
    weights = N * K + nb * kb * 4 + (2 * N if case["bias"] else 0)
    experts = min(case.get("E", 1), M)
    x = M * K * 2 if op == "layer" else M * K + M * kb * 4
    return dict(bytes=x + experts * weights + M * N * (2 if case["out"] == "bf16" else 4), flops=2 * M * N * K)


# ---------------------------------------------------------------- the definition in 64 bits

def exact(case, seed):
    """What run() returns, in 64 bits (the codes and scales of the quantiser
    are defined by their fp32 roundings: those are kept)."""
    global own
    kept, own = own, False
    try:
        st = prepare(case, seed)
    finally:
        own = kept
    f64 = torch.float64

    def codes(x):
        """By the definition, a block of 128 channels at a time: every
        fp32 step is its 64-bit value rounded to 32 bits."""
        qs, ss = [], []
        for k0 in range(0, x.shape[1], BLOCK):
            v = x[:, k0:k0 + BLOCK].to(f64)
            s = (v.abs().max(dim=1).values / E4M3_MAX).float().to(f64)
            s = torch.where(s < SCALE_MIN, torch.full_like(s, SCALE_MIN), s)
            r = (1.0 / s).float().to(f64)
            t = (v * r[:, None]).float().to(f64).clamp(-E4M3_MAX, E4M3_MAX)
            # E4M3 by its grid: steps of 2^(e - 3), e = floor(log2 |t|) >= -6, ties to even
            e = torch.frexp(t).exponent.sub(1).clamp(min=-6).to(f64)
            step = torch.exp2(e - 3)
            qs.append(torch.round(t / step) * step)
            ss.append(s)
        return torch.cat(qs, dim=1), torch.stack(ss)

    def product(q, s, qw, sw, bias):
        y = torch.zeros((q.shape[0], qw.shape[0]), dtype=f64, device="cuda")
        rows = torch.arange(qw.shape[0], device="cuda") // BLOCK
        for b, k0 in enumerate(range(0, q.shape[1], BLOCK)):
            part = torch.mm(q[:, k0:k0 + BLOCK].to(f64), qw[:, k0:k0 + BLOCK].to(f64).t())
            y += part * s[b].to(f64)[:, None] * sw[:, b].to(f64)[rows][None, :]
        if bias is not None:
            y += bias.to(f64)
        if case["act"] == "gelu_tanh":
            u = math.sqrt(2.0 / math.pi) * (y + 0.044715 * y ** 3)
            y = y * torch.sigmoid(2.0 * u)
        return y

    op = case["op"]
    if op == "act":
        return codes(st["x"])
    if op == "gemm":
        return product(st["qx"], st["sx"], st["qw"], st["sw"], st["bias"])
    if op == "layer":
        q, s = codes(st["x"])
        return product(q, s, st["qw"], st["sw"], st["bias"])
    if op == "grouped":
        out, m0 = [], 0
        for e, m in enumerate(st["sizes"]):
            if m:
                out.append(product(st["qx"][m0:m0 + m], st["sx"][:, m0:m0 + m], st["qw"][e], st["sw"][e],
                                   None if st["bias"] is None else st["bias"][e]))
            m0 += m
        return torch.cat(out)
    # rotation as multiplication by e^(i angle)
    outs = []
    for x, w in ((st["q"], st["qn"]), (st["k"], st["kn"])):
        v = x.to(f64)
        if w is not None:
            v = v / torch.sqrt((v ** 2).sum(dim=2, keepdim=True) / x.shape[2] + 1e-6) * w.to(f64)
        angle = torch.stack([st["pos"][:, a].to(f64) * f for a, f in zip(st["axis"].tolist(), st["freq"].tolist())], 1)
        turn = torch.polar(torch.ones_like(angle), -angle if case["inverse"] else angle)[:, None, :]
        R = 2 * angle.shape[1]
        head = v[:, :, :R]
        if case["pairing"] == "interleaved":
            z = torch.view_as_complex(head.reshape(*head.shape[:2], R // 2, 2).contiguous()) * turn
            head = torch.view_as_real(z).flatten(2)
        else:
            z = torch.complex(head[:, :, :R // 2].contiguous(), head[:, :, R // 2:].contiguous()) * turn
            head = torch.cat([z.real, z.imag], dim=2)
        outs.append(torch.cat([head, v[:, :, R:]], dim=2))
    return tuple(outs)
