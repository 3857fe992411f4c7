"""The cases of the cached attention: keys and values appended to a paged cache
in 8 bits, attention over that cache, and the 8-bit layers whose epilogue joins
the block's residual stream. Their inputs, their plain forms, the framework's
calls and what each has to move and compute.

Kinds of a case:
  append   svdq.KVCache.append: a fused projection's keys (normed and rotated
           on the way) and values into the pages of their sequences, as E4M3
           codes with a power of two per 16 tokens and head; the queries
           rotated in the same call
  attend   svdq.KVCache.attend: softmax(scale q k^T) v over those pages, one
           token a sequence, ragged prompts or whole chunks
  layer    svdq.Fp8Linear: residual + gate * act(x W^T + bias), from bf16
           activations
  grouped  svdq.Fp8GroupedLinear: the same with a weight per group of rows
           (the streams of a joint block, experts)

The cache: data [pages, heads, page / 64, 2 (keys, values), 4, C, 1024] bytes,
C = ceil(D / 64): a block of 16 tokens of one head is C runs of 1024 codes.
Code j of run c is, among the keys, channel 64 c + 16 (j / 256) + j % 16 of
token (j / 16) % 16; among the values, channel 64 c + 16 (j / 4 % 4) +
j / 16 % 16 of token 4 (j / 256) + j % 4. Channels past D hold zeros. scales
[pages, heads, page / 64, 2, 4]: the blocks' exponents + 127.
"""
import math
import random

import torch

own = False

E4M3_MAX = 448.0
BLOCK = 128                    # channels of an 8-bit layer's scale
SCALE_MIN = 2.0 ** -120        # its least scale
EXP_MIN = -120                 # least exponent of a cache block's scale


# ---------------------------------------------------------------- cases

def listed():
    return [
        # one new token of one stream: latency
        dict(name="append_one", op="append", B=1, T=1, past=77, hq=24, hk=24, D=128, dims="16,56,56", pairing="interleaved",
             norm=True, page=64),
        # a step of a served batch, shared key heads, lengths of their own
        dict(name="append_step", op="append", B=64, T=64, past=1024, hq=32, hk=8, D=128, dims="128", pairing="half",
             norm=False, page=64),
        # the tokens of a video chunk behind the chunks before it
        dict(name="append_chunk", op="append", B=1, T=4608, past=9216, hq=24, hk=24, D=128, dims="16,56,56",
             pairing="interleaved", norm=True, page=128),
        # ragged prompts, an odd number of tokens, narrow heads
        dict(name="append_prompts", op="append", B=13, T=8003, past=500, hq=16, hk=4, D=64, dims="64", pairing="half",
             norm=False, page=64),
        # one token over a prompt's length of keys: latency
        dict(name="attend_one", op="attend", B=1, T=1, past=77, hq=24, hk=24, D=128, causal=True, window=0, page=64),
        # a step of a served batch over ragged lengths: the cache's bytes count
        dict(name="attend_step", op="attend", B=64, T=64, past=8192, hq=32, hk=8, D=128, causal=True, window=0, page=64),
        # one token of two streams over a long cache: few rows, much to read
        dict(name="attend_long", op="attend", B=2, T=2, past=131072, hq=24, hk=8, D=128, causal=True, window=0, page=128),
        # ragged prompts behind a shared length, causal: the matrix pipe counts
        dict(name="attend_prompts", op="attend", B=5, T=8003, past=1000, hq=32, hk=8, D=128, causal=True, window=0, page=64),
        # a video chunk's tokens see all chunks so far and their own
        dict(name="attend_chunk", op="attend", B=1, T=4608, past=18432, hq=24, hk=24, D=128, causal=False, window=0,
             page=128),
        # one token's attention output projected and added to its stream
        dict(name="layer_one_row", op="layer", M=1, K=4096, N=4096, act="none", bias=True, gate=False, out="bf16"),
        # the image's tokens through the output projection, gated
        dict(name="layer_image", op="layer", M=4608, K=4096, N=4096, act="none", bias=True, gate=True, out="bf16"),
        # text and image streams through their MLPs' second layers, gated
        dict(name="grouped_streams", op="grouped", M=5120, K=12288, N=4096, E=2, act="none", bias=True, gate=True,
             out="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    """One more case of the listed ones' ranges."""
    op = rng.choice(["append", "append", "attend", "attend", "attend", "layer", "grouped"])
    if op in ("layer", "grouped"):
        K, N = 16 * _log(rng, 4, 768), _log(rng, 8, 8192)
        E = _log(rng, 1, 16) if op == "grouped" else 1
        while E * N * K > 2 * 12288 * 4096:
            E = max(1, E // 2)
            N = N if E > 1 else min(N, 8192)
        M = min(_log(rng, 1, 5120), max(1, 5120 * 12288 * 4096 // (N * K)))
        case = dict(op=op, M=M, K=K, N=N, act=rng.choice(["none", "none", "gelu_tanh"]), bias=rng.random() < 0.7,
                    gate=rng.random() < 0.6, out=rng.choice(["bf16", "bf16", "f32"]))
        if op == "grouped":
            case["E"] = E
        return case
    D, dims = rng.choice([(64, "64"), (64, "16,24,24"), (128, "128"), (128, "16,56,56"), (128, "64"), (96, "32,32,32"),
                          (72, "24,24,24"), (256, "64,96,96")])
    hk = rng.choice([1, 2, 3, 8, 8, 24])
    hq = hk * rng.choice([1, 1, 3, 4, 8])
    B = _log(rng, 1, 64)
    page = rng.choice([64, 64, 128, 256])
    past = _log(rng, 1, 32768)
    past = min(past, max(16, 64 * 8192 * 8 * 128 // (B * hk * D) - 64))
    T = B if rng.random() < 0.4 else B + _log(rng, 1, 4608)
    if op == "append":
        T = min(T, max(B, 4608 * 72 * 128 // ((hq + 2 * hk) * D)))
        past = min(past, max(16, 16384 * 24 * 128 // (B * hk * D)))        # (the outputs are the whole cache)
        return dict(op=op, B=B, T=T, past=past, hq=hq, hk=hk, D=D, dims=dims, pairing=rng.choice(["interleaved", "half"]),
                    norm=rng.random() < 0.5, page=page)
    most = 4608 * 23040 * 24 * 128 // 2            # (queries x keys x channels)
    T = min(T, max(B, most // (hq * D * (past + 4608))))
    return dict(op=op, B=B, T=T, past=past, hq=hq, hk=hk, D=D, causal=rng.random() < 0.7,
                window=rng.choice([0, 0, 0, 1, 100, 1024]), page=page)


def _lengths(case):
    """(tokens of the call, tokens of the cache with them) of every sequence."""
    B, T, past = case["B"], case["T"], case["past"]
    r = random.Random(B * 1000003 + T * 10007 + past)
    counts = [1] * B
    if T > B:
        share = [r.uniform(0.2, 1.0) for _ in range(B)]
        cuts = [0] + [int(sum(share[:b + 1]) / sum(share) * (T - B)) for b in range(B)]
        cuts[-1] = T - B
        counts = [1 + cuts[b + 1] - cuts[b] for b in range(B)]
    before = [past] if B == 1 else [r.randint(past // 4, past) for _ in range(B)]
    return counts, [p + n for p, n in zip(before, counts)]


# ---------------------------------------------------------------- inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) & 0x7FFFFFFFFFFF)
    return g


def _activations(M, K, g):
    """Normal values with a few channels that stand out."""
    x = torch.randn((M, K), generator=g, device="cuda", dtype=torch.float32)
    loud = torch.rand((K,), generator=g, device="cuda") < 0.01
    return (x * torch.where(loud, 20.0, 1.0)).to(torch.bfloat16)


def _exponent(amax):
    """The least e with amax <= 448 2^e, at least EXP_MIN."""
    m, x = torch.frexp(amax)                             # 448 = 0.875 2^9
    e = torch.where(m <= 0.875, x - 9, x - 8)
    return torch.where(amax > 0, e, torch.full_like(e, EXP_MIN)).clamp(min=EXP_MIN)


def _cache(case, g):
    """A cache filled with random tokens (keys with a few loud channels), its
    pages in any order, and the sequences' page tables (-1: no page)."""
    H, D, page = case["hk"], case["D"], case["page"]
    C = -(-D // 64)
    lens = _lengths(case)[1]
    need = [-(-n // page) for n in lens]
    pages, wide = sum(need) + 2, max(need) + 1
    order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    row = torch.tensor([b for b, n in enumerate(need) for _ in range(n)], device="cuda")
    col = torch.tensor([i for n in need for i in range(n)], device="cuda")
    table = torch.full((len(lens), wide), -1, dtype=torch.int32, device="cuda")
    table[row, col] = order[:row.numel()]
    j = torch.arange(1024, device="cuda")
    d = torch.stack([16 * (j // 256) + j % 16, 16 * (j // 4 % 4) + j // 16 % 16])         # keys, values
    d = d[:, None, :] + 64 * torch.arange(C, device="cuda")[None, :, None]                # [2, C, 1024]
    loud = torch.where(torch.rand((2, H, D), generator=g, device="cuda") < 0.02, 6.0, 1.0)
    loud[1] = 1.0
    loud = torch.nn.functional.pad(loud, (0, 64 * C - D))                                 # channels past D: 0
    loud = torch.stack([loud[0][:, d[0]], loud[1][:, d[1]]], dim=1)                       # [H, 2, C, 1024]
    data = torch.empty((pages, H, page // 64, 2, 4, C, 1024), dtype=torch.uint8, device="cuda")
    scales = torch.empty((pages, H, page // 64, 2, 4), dtype=torch.uint8, device="cuda")
    step = max(1, (1 << 28) // (H * page * 2 * 64 * C))
    for p in range(0, pages, step):
        x = torch.randn(data[p:p + step].shape, generator=g, device="cuda") * loud[None, :, None, :, None]
        e = _exponent(x.abs().amax(dim=(5, 6)))
        data[p:p + step] = torch.ldexp(x, -e[..., None, None]).to(torch.float8_e4m3fn).view(torch.uint8)
        scales[p:p + step] = (e + 127).to(torch.uint8)
    return data, scales, table


def _group_sizes(case):
    """Rows of each group: one text and one image stream, or uneven shares."""
    E, M = case["E"], case["M"]
    r = random.Random(E * 1000003 + M)
    share = [1.0, 9.0] if E == 2 else [r.uniform(0.0, 1.0) for _ in range(E)]
    cuts = [0] + [int(sum(share[:e + 1]) / sum(share) * M) for e in range(E)]
    cuts[-1] = M
    return [b - a for a, b in zip(cuts, cuts[1:])]


def _weight_codes(w):
    """E4M3 codes of w [E, N, K] and an fp32 scale per 128 x 128 block."""
    E, N, K = w.shape
    nb, kb = -(-N // BLOCK), -(-K // BLOCK)
    wf = torch.nn.functional.pad(w, (0, kb * BLOCK - K, 0, nb * BLOCK - N)).view(E, nb, BLOCK, kb, BLOCK)
    s = torch.clamp((wf.abs().amax(dim=(2, 4)).double() / E4M3_MAX).float(), min=SCALE_MIN)
    q = torch.clamp(wf / s[:, :, None, :, None], -E4M3_MAX, E4M3_MAX).view(E, nb * BLOCK, kb * BLOCK)
    return q[:, :N, :K].to(torch.float8_e4m3fn).contiguous(), s.contiguous()


def _out_dtype(case):
    return torch.bfloat16 if case["out"] == "bf16" else torch.float32


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    st = dict(case=case)
    if op in ("layer", "grouped"):
        M, K, N, E = case["M"], case["K"], case["N"], case.get("E", 1)
        st["x"] = _activations(M, K, g)
        st["qw"], st["sw"] = _weight_codes(torch.randn((E, N, K), generator=g, device="cuda") * 0.02)
        st["bias"] = (torch.randn((E, N), generator=g, device="cuda") * 0.1).to(torch.bfloat16) if case["bias"] else None
        st["gate"] = torch.randn((E, N), generator=g, device="cuda").to(torch.bfloat16) if case["gate"] else None
        st["res"] = (torch.randn((M, N), generator=g, device="cuda") * 2.0).to(_out_dtype(case))
        sizes = _group_sizes(case) if op == "grouped" else [M]
        st["offsets"] = torch.tensor([0] + torch.tensor(sizes).cumsum(0).tolist(), dtype=torch.int32, device="cuda")
        if own:
            import bit_quantized_diffusion_svdq_amd as svdq
            make = svdq.Fp8GroupedLinear if op == "grouped" else svdq.Fp8Linear
            one = (lambda t: t) if op == "grouped" else (lambda t: None if t is None else t[0])
            st["layer"], st["own_gate"] = make(one(st["qw"]), one(st["sw"]), one(st["bias"])), one(st["gate"])
        return st
    hq, hk, D = case["hq"], case["hk"], case["D"]
    T = case["T"]
    counts, lens = _lengths(case)
    st["data"], st["scales"], st["table"] = _cache(case, g)
    st["lengths"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    st["offsets"] = torch.tensor([0] + torch.tensor(counts).cumsum(0).tolist(), dtype=torch.int32, device="cuda")
    st["ragged"] = st["offsets"] if case["T"] > case["B"] else None       # a token a sequence needs none
    st["most"] = max(counts)
    if op == "append":
        # the fused projection's output, whose queries the rotation leaves where it is told to
        flat = torch.randn((T, (hq + 2 * hk) * D), generator=g, device="cuda").to(torch.bfloat16)
        st["q"], st["k"], st["v"] = flat.view(T, hq + 2 * hk, D).split((hq, hk, hk), dim=1)
        dims = [int(n) for n in case["dims"].split(",")]
        st["pos"] = torch.randint(0, 4096, (T, len(dims)), generator=g, device="cuda", dtype=torch.int32)
        st["qn"] = st["kn"] = None
        if case["norm"]:
            st["qn"] = (1 + 0.2 * torch.randn(D, generator=g, device="cuda")).to(torch.bfloat16)
            st["kn"] = (1 + 0.2 * torch.randn(D, generator=g, device="cuda")).to(torch.bfloat16)
        # every pair's axis and angular frequency 10000^(-2 i / d)
        st["axis"] = torch.tensor([a for a, n in enumerate(dims) for _ in range(n // 2)], device="cuda")
        st["freq"] = torch.tensor([10000.0 ** (-2.0 * i / n) for n in dims for i in range(n // 2)], device="cuda",
                                  dtype=torch.float64)
    else:
        st["q"] = (torch.randn((T, hq, D), generator=g, device="cuda") * 1.5).to(torch.bfloat16)
    if own:
        import bit_quantized_diffusion_svdq_amd as svdq
        st["cache"] = svdq.KVCache(st["data"].shape[0], hk, D, page_size=case["page"], data=st["data"], scales=st["scales"])
        if op == "append":
            st["plan"] = svdq.RopePlan(dims, head_dim=D, pairing=case["pairing"])
            st["said"] = (st["data"].view(torch.float8_e4m3fn), st["scales"].view(torch.float8_e8m0fnu))
    return st


# ---------------------------------------------------------------- one pass

def _sequences(st):
    """(sequence, place among its tokens, position in the cache) of every token."""
    off, T = st["offsets"].long(), st["case"]["T"]
    t = torch.arange(T, device=off.device)
    b = torch.searchsorted(off, t, right=True) - 1
    i = t - off[b]
    return b, i, st["lengths"].long()[b] - (off[b + 1] - off[b]) + i


def _rotated(x, norm, st):
    case = st["case"]
    v = x.float()
    if norm is not None:
        v = v * torch.rsqrt((v * v).mean(dim=2, keepdim=True) + 1e-6) * norm.float()
    angle = st["pos"].double()[:, st["axis"]] * st["freq"]
    c, s = torch.cos(angle).float()[:, None, :], torch.sin(angle).float()[:, None, :]
    R = 2 * c.shape[2]
    if case["pairing"] == "interleaved":
        a, b = v[:, :, 0:R:2], v[:, :, 1:R:2]
        turned = torch.stack([a * c - b * s, a * s + b * c], dim=3).flatten(2)
    else:
        a, b = v[:, :, :R // 2], v[:, :, R // 2:R]
        turned = torch.cat([a * c - b * s, a * s + b * c], dim=2)
    return torch.cat([turned, v[:, :, R:]], dim=2)


def _by_token(data):
    """Keys and values [pages, page / 64, 4, 16, heads, 64 C] of a cache's bytes."""
    p, H, t, _, _, C, _ = data.shape
    k = data[:, :, :, 0].reshape(p, H, t, 4, C, 4, 16, 16).permute(0, 2, 3, 6, 1, 4, 5, 7).reshape(p, t, 4, 16, H, 64 * C)
    v = data[:, :, :, 1].reshape(p, H, t, 4, C, 4, 16, 4, 4).permute(0, 2, 3, 5, 8, 1, 4, 7, 6).reshape(p, t, 4, 16, H, 64 * C)
    return k, v


def _append_side(old, old_exp, x, block, slot):
    """One side's codes [blocks, 16, H, 64 C] and exponents [blocks, H] after
    the call: a block's exponent is the least that holds its new values, and
    not below the old one unless the call writes the block from its start; the
    tokens from before are rounded again to it; slots past the last token hold
    zeros."""
    n, _, H, W = old.shape
    dev = x.device
    amax = torch.zeros((n, H), device=dev).index_reduce_(0, block, x.abs().amax(dim=2), "amax")
    first = torch.full((n,), 16, device=dev).index_reduce_(0, block, slot, "amin")
    need = _exponent(amax)
    exp = torch.where((first == 0)[:, None], need, torch.maximum(need, old_exp))
    before = torch.arange(16, device=dev)[None, :] < first[:, None]
    was = torch.ldexp(old.view(torch.float8_e4m3fn).float(), (old_exp - exp)[:, None, :, None])
    codes = torch.where(before[:, :, None, None], was, torch.zeros_like(was))
    new = torch.ldexp(x, -exp[block][:, :, None]).clamp(-E4M3_MAX, E4M3_MAX)
    codes[block, slot] = torch.nn.functional.pad(new, (0, W - x.shape[2]))
    return codes.to(torch.float8_e4m3fn).view(torch.uint8), exp


def _append(st):
    case = st["case"]
    page, H = case["page"], case["hk"]
    data, scales = st["data"], st["scales"]
    tiles, C = page // 64, data.shape[5]
    _, _, at = sequence = _sequences(st)
    block = st["table"].long()[sequence[0], at // page] * (tiles * 4) + at % page // 16
    touched, block = torch.unique(block, return_inverse=True)
    n = touched.numel()
    where = (touched // (4 * tiles), slice(None), touched // 4 % tiles, slice(None), touched % 4)
    old, exp = data[where], scales[where].int() - 127                    # [n, H, 2, C, 1024], [n, H, 2]
    k = old[:, :, 0].reshape(n, H, C, 4, 16, 16).permute(0, 4, 1, 2, 3, 5).reshape(n, 16, H, 64 * C)
    v = old[:, :, 1].reshape(n, H, C, 4, 16, 4, 4).permute(0, 3, 6, 1, 2, 5, 4).reshape(n, 16, H, 64 * C)
    k, ke = _append_side(k, exp[:, :, 0], _rotated(st["k"], st["kn"], st), block, at % 16)
    v, ve = _append_side(v, exp[:, :, 1], st["v"].float(), block, at % 16)
    k = k.view(n, 16, H, C, 4, 16).permute(0, 2, 3, 4, 1, 5).reshape(n, H, C, 1024)
    v = v.view(n, 4, 4, H, C, 4, 16).permute(0, 3, 4, 1, 6, 5, 2).reshape(n, H, C, 1024)
    data[where] = torch.stack([k, v], dim=2)
    scales[where] = (torch.stack([ke, ve], dim=2) + 127).to(torch.uint8)
    q = _rotated(st["q"], st["qn"], st).to(torch.bfloat16)
    return q, data.view(torch.float8_e4m3fn), scales.view(torch.float8_e8m0fnu)


def _attend(st):
    case = st["case"]
    hq, hk, D, page = case["hq"], case["hk"], case["D"], case["page"]
    B, n, T = case["B"], st["most"], case["T"]
    table = st["table"].long().clamp(min=0)
    data, scales = st["data"][table], st["scales"][table]                # [B, wide, H, tiles, 2, 4, ...]
    wide = table.shape[1]
    k, v = (t.reshape(B, -1, hk, t.shape[-1])[..., :D] for t in _by_token(data.flatten(0, 1)))
    s = torch.ldexp(torch.ones((), device=k.device), scales.int() - 127).view(B, wide, hk, page // 64, 2, 4)
    s = s.permute(4, 0, 1, 3, 5, 2).reshape(2, B, -1, hk).repeat_interleave(16, dim=2)[..., None]
    k = (k.view(torch.float8_e4m3fn).float() * s[0]).permute(0, 2, 1, 3)
    v = (v.view(torch.float8_e4m3fn).float() * s[1]).permute(0, 2, 1, 3)   # [B, hk, L, D]
    L = k.shape[2]
    b, i, at = _sequences(st)
    q = torch.zeros((B, n, hq, D), device=k.device)
    q[b, i] = st["q"].float() * (1.0 / math.sqrt(D))
    q = q.view(B, n, hk, hq // hk, D).permute(0, 2, 1, 3, 4).reshape(B, hk, n * (hq // hk), D)
    p = torch.matmul(q, k.transpose(2, 3).contiguous()).view(B, hk, n, hq // hk, L)
    place = torch.zeros((B, n), dtype=torch.int64, device=k.device)
    place[b, i] = at
    key = torch.arange(L, device=k.device)
    seen = (key[None, :] < st["lengths"].long()[:, None])[:, None, :].expand(B, n, L)
    if case["causal"]:
        seen = seen & (key[None, None, :] <= place[:, :, None])
    if case["window"]:
        seen = seen & (key[None, None, :] > place[:, :, None] - case["window"])
    p.masked_fill_(~seen[:, None, :, None, :], -math.inf)
    p.sub_(p.amax(dim=4, keepdim=True).clamp(min=-3e38)).exp_()
    total = p.sum(dim=4, keepdim=True)
    o = torch.matmul(p.view(B, hk, -1, L), v).view(B, hk, n, hq // hk, D) / torch.where(total > 0, total, torch.ones_like(total))
    return o.permute(0, 2, 1, 3, 4).reshape(B, n, hq, D)[b, i].to(torch.bfloat16)


def _activation(y, act):
    if act == "none":
        return y
    return 0.5 * y * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (y + 0.044715 * y * y * y)))


def _linear(st):
    """residual + gate * act(x W^T + bias) with x turned into E4M3 codes and a
    scale per row and 128 channels first."""
    case = st["case"]
    x, qw, sw = st["x"], st["qw"], st["sw"]
    (M, K), (E, N, _) = x.shape, qw.shape
    kb = -(-K // BLOCK)
    xf = torch.nn.functional.pad(x.float(), (0, kb * BLOCK - K)).view(M, kb, BLOCK)
    s = torch.clamp((xf.abs().amax(dim=2).double() / E4M3_MAX).float(), min=SCALE_MIN)
    r = (1.0 / s.double()).float()
    q = torch.clamp(xf * r[:, :, None], -E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn).float() * s[:, :, None]
    q = q.view(M, kb * BLOCK)[:, :K]
    w = qw.float() * sw.repeat_interleave(BLOCK, 1)[:, :N].repeat_interleave(BLOCK, 2)[:, :, :K]
    if E == 1:
        y = q @ w[0].t()
        group = torch.zeros(M, dtype=torch.int64, device=x.device)
    else:
        group = torch.searchsorted(st["offsets"].long(), torch.arange(M, device=x.device), right=True) - 1
        y = torch.cat([q[a:z] @ w[e].t() for e, (a, z) in enumerate(_ranges(case))])
    if st["bias"] is not None:
        y = y + st["bias"].float()[group]
    y = _activation(y, case["act"])
    if st["gate"] is not None:
        y = y * st["gate"].float()[group]
    return (st["res"].float() + y).to(_out_dtype(case))


def _ranges(case):
    ends = torch.tensor(_group_sizes(case)).cumsum(0).tolist()
    return list(zip([0] + ends[:-1], ends))


def run(st):
    case = st["case"]
    op = case["op"]
    if own:
        if op == "append":
            q = st["cache"].append(st["k"], st["v"], st["table"], st["lengths"], offsets=st["ragged"], pos=st["pos"],
                                   plan=st["plan"], k_norm=st["kn"], q=st["q"], q_norm=st["qn"])
            return (q, *st["said"])
        if op == "attend":
            return st["cache"].attend(st["q"], st["table"], st["lengths"], offsets=st["ragged"], causal=case["causal"],
                                      window=case["window"])
        if op == "layer":
            return st["layer"](st["x"], act=case["act"], residual=st["res"], gate=st["own_gate"], out_dtype=_out_dtype(case))
        return st["layer"](st["x"], st["offsets"], act=case["act"], residual=st["res"], gate=st["own_gate"],
                           out_dtype=_out_dtype(case))
    if op == "append":
        return _append(st)
    if op == "attend":
        return _attend(st)
    return _linear(st)


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    op = case["op"]
    if op in ("layer", "grouped"):
        M, K, N, E = case["M"], case["K"], case["N"], case.get("E", 1)
        nb, kb = -(-N // BLOCK), -(-K // BLOCK)
        used = sum(n > 0 for n in _group_sizes(case)) if op == "grouped" else 1
        weights = N * K + nb * kb * 4 + 2 * N * (case["bias"] + case["gate"])
        return dict(bytes=M * K * 2 + used * weights + 2 * M * N * (2 if case["out"] == "bf16" else 4), flops=2 * M * N * K)
    hq, hk, D, T = case["hq"], case["hk"], case["D"], case["T"]
    counts, lens = _lengths(case)
    if op == "append":
        # heads in, rotated queries and codes out, and the scales of the blocks; the old tokens of a
        # block that the call begins inside of need not be read while its scales hold
        blocks = sum((n - 1) // 16 - (n - c) // 16 + 1 for c, n in zip(counts, lens))
        return dict(bytes=T * (2 * hq * 2 + hk * 2 * 3) * D + T * 4 * len(case["dims"].split(",")) + blocks * hk * 4,
                    flops=T * ((hq + hk) * (7 if case["norm"] else 3) + hk * 4) * D)
    keys = pairs = 0
    for c, n in zip(counts, lens):
        first = max(0, n - c - case["window"] + 1) if case["window"] else 0
        keys += n - first
        for i in range(c):
            at = n - c + i
            hi = at + 1 if case["causal"] else n
            pairs += hi - (max(0, at - case["window"] + 1) if case["window"] else 0)
    return dict(bytes=keys * hk * 2 * D + keys * hk // 8 + 4 * T * hq * D, flops=4 * pairs * hq * D)


# ---------------------------------------------------------------- the definition in 64 bits

def _grid(t):
    """t to the nearest E4M3 value, ties to even: steps of 2^(e - 3), e =
    floor(log2 |t|) >= -6."""
    e = torch.frexp(t).exponent.sub(1).clamp(min=-6).to(torch.float64)
    step = torch.exp2(e - 3)
    return (torch.round(t / step) * step).clamp(-E4M3_MAX, E4M3_MAX)


def _addresses(tokens, C, page, H, pages_of):
    """Byte of every (token, head, channel) of keys and values, and of its
    scale; tokens: positions of one sequence."""
    dev = tokens.device
    h = torch.arange(H, device=dev)[None, :, None]
    d = torch.arange(64 * C, device=dev)[None, None, :]
    t = tokens[:, None, None]
    tile = (pages_of[tokens // page][:, None, None] * H + h) * (page // 64) + t % page // 64
    blk, key = t % 64 // 16, t % 16
    c, r = d // 64, d % 64
    kj = r // 16 * 256 + key * 16 + r % 16
    vj = key // 4 * 256 + r % 16 * 16 + r // 16 * 4 + key % 4
    return (((tile * 2) * 4 + blk) * C + c) * 1024 + kj, (((tile * 2 + 1) * 4 + blk) * C + c) * 1024 + vj, tile * 8 + blk


def exact(case, seed):
    """What run() returns, in 64 bits (a code is defined by its rounding: that
    is kept)."""
    global own
    kept, own = own, False
    try:
        st = prepare(case, seed)
    finally:
        own = kept
    f64 = torch.float64
    op = case["op"]
    if op in ("layer", "grouped"):
        x = st["x"].to(f64)
        M, K = x.shape
        N = case["N"]
        out = torch.empty((M, N), dtype=f64, device="cuda")
        rows = torch.arange(N, device="cuda") // BLOCK
        for e, (a, z) in enumerate(_ranges(case) if op == "grouped" else [(0, M)]):
            y = torch.zeros((z - a, N), dtype=f64, device="cuda")
            for kb, k0 in enumerate(range(0, K, BLOCK)):
                v = x[a:z, k0:k0 + BLOCK]
                if z > a:
                    s = (v.abs().max(dim=1).values / E4M3_MAX).float().to(f64).clamp(min=SCALE_MIN)
                    r = (1.0 / s).float().to(f64)
                    q = _grid((v * r[:, None]).float().to(f64))
                    y += torch.mm(q, st["qw"][e][:, k0:k0 + BLOCK].to(f64).t()) * s[:, None] * st["sw"][e][:, kb].to(f64)[rows]
            if st["bias"] is not None:
                y += st["bias"][e].to(f64)
            if case["act"] == "gelu_tanh":
                y = y * torch.sigmoid(2.0 * math.sqrt(2.0 / math.pi) * (y + 0.044715 * y ** 3))
            if st["gate"] is not None:
                y *= st["gate"][e].to(f64)
            out[a:z] = st["res"][a:z].to(f64) + y
        return out

    hq, hk, D, page = case["hq"], case["hk"], case["D"], case["page"]
    counts, lens = _lengths(case)
    C = -(-D // 64)
    flat, exps = st["data"].view(-1).clone(), st["scales"].view(-1).clone()
    if op == "append":
        def turned(x, w):
            v = x.to(f64)
            if w is not None:
                v = v / torch.sqrt((v ** 2).sum(dim=2, keepdim=True) / D + 1e-6) * w.to(f64)
            angle = torch.stack([st["pos"][:, a].to(f64) * f for a, f in zip(st["axis"].tolist(), st["freq"].tolist())], 1)
            turn = torch.polar(torch.ones_like(angle), angle)[:, None, :]
            R = 2 * angle.shape[1]
            head = v[:, :, :R]
            if case["pairing"] == "interleaved":
                z = torch.view_as_complex(head.reshape(*head.shape[:2], R // 2, 2).contiguous()) * turn
                head = torch.view_as_real(z).flatten(2)
            else:
                z = torch.complex(head[:, :, :R // 2].contiguous(), head[:, :, R // 2:].contiguous()) * turn
                head = torch.cat([z.real, z.imag], dim=2)
            return torch.cat([head, v[:, :, R:]], dim=2)

        sides = [turned(st["k"], st["kn"]), st["v"].to(f64)]
        t0 = 0
        for b, (c, n) in enumerate(zip(counts, lens)):
            pages_of = st["table"][b].long()
            b0 = (n - c) // 16 * 16                               # the first block's first token
            tokens = torch.arange(b0, -(-n // 16) * 16, device="cuda")
            new = (tokens >= n - c) & (tokens < n)
            ka, va, sa = _addresses(tokens, C, page, hk, pages_of)
            for side, (addr, off) in enumerate(((ka, 0), (va, 4))):
                x = torch.zeros((tokens.numel(), hk, 64 * C), dtype=f64, device="cuda")
                x[new, :, :D] = sides[side][t0:t0 + c]
                amax = x.abs().amax(dim=2).view(-1, 16, hk).amax(dim=1)           # [blocks, heads]
                e = torch.ceil(torch.log2(amax / E4M3_MAX))
                e = torch.where(amax > E4M3_MAX * torch.exp2(e), e + 1, e)        # (log2 may round)
                e = torch.where(amax <= E4M3_MAX * torch.exp2(e - 1), e - 1, e).clamp(min=EXP_MIN)
                was = exps[sa[::16, :, 0] + off].to(f64) - 127
                if n - c > b0:
                    e[0] = torch.maximum(e[0], was[0])
                old = flat[addr].view(torch.float8_e4m3fn).to(f64) * torch.exp2(was - e).repeat_interleave(16, 0)[:, :, None]
                x = torch.where(new[:, None, None], x * torch.exp2(-e).repeat_interleave(16, 0)[:, :, None],
                                torch.where((tokens < n - c)[:, None, None], old, torch.zeros_like(old)))
                flat[addr] = _grid(x).to(torch.float8_e4m3fn).view(torch.uint8)
                exps[sa[::16, :, 0] + off] = (e + 127).to(torch.uint8)
            t0 += c
        return (turned(st["q"], st["qn"]), flat.view(torch.float8_e4m3fn).to(f64).view(st["data"].shape),
                torch.exp2(exps.to(f64) - 127).view(st["scales"].shape))
    # attention, a sequence and a key head at a time
    out = torch.zeros((case["T"], hq, D), dtype=f64, device="cuda")
    G, t0 = hq // hk, 0
    for b, (c, n) in enumerate(zip(counts, lens)):
        tokens = torch.arange(n, device="cuda")
        pages_of = st["table"][b].long()
        at = torch.arange(n - c, n, device="cuda")
        seen = torch.ones((c, n), dtype=torch.bool, device="cuda")
        if case["causal"]:
            seen &= tokens[None, :] <= at[:, None]
        if case["window"]:
            seen &= tokens[None, :] + case["window"] > at[:, None]
        for h in range(hk):
            part = torch.arange(0, n, 1 << 16, device="cuda").tolist()
            ks, vs = [], []
            for p0 in part:                                       # (addresses of a long cache a piece at a time)
                ka, va, sa = _addresses(tokens[p0:p0 + (1 << 16)], C, page, hk, pages_of)
                s = torch.exp2(exps[sa[:, h, 0]].to(f64) - 127)[:, None]
                ks.append(flat[ka[:, h, :D]].view(torch.float8_e4m3fn).to(f64) * s)
                s = torch.exp2(exps[sa[:, h, 0] + 4].to(f64) - 127)[:, None]
                vs.append(flat[va[:, h, :D]].view(torch.float8_e4m3fn).to(f64) * s)
            k, v = torch.cat(ks), torch.cat(vs)
            for g in range(G):
                q = st["q"][t0:t0 + c, h * G + g].to(f64)
                score = torch.mm(q, k.t().contiguous()) / math.sqrt(D)
                score = torch.where(seen, score, torch.full_like(score, -math.inf))
                w = torch.softmax(score, dim=1)
                out[t0:t0 + c, h * G + g] = torch.mm(w, v)
        t0 += c
    return out
