"""The paged 8-bit cache and its attention off the common path: batches that
lie (falling offsets, missing pages, lengths of any sign), graphs, streams,
strided and in-place buffers, inputs that are not finite, very long caches."""
import numpy as np
import pytest
import torch

from gpu_util import note
from kv_util import attend_bound, bf16, cum, paged, random_state
from test_gpu_kv import cache_of, check_append, dev, run_attend, state_of

pytestmark = pytest.mark.gpu

import bit_quantized_diffusion_svdq_amd as svdq
from oracle import kv as okv


def i32(*v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def both(rng, state, hq, H, D, page, table, lengths, offsets, T, causal=True, window=0, q_scale=1.0):
    """append then attend, both against the oracle; returns the cache."""
    cache = cache_of(state, H, D, page)
    k, kv = bf16(rng, (T, H, D))
    v, vv = bf16(rng, (T, H, D))
    assert cache.append(k.cuda(), v.cuda(), dev(table), dev(np.asarray(lengths, np.int32)), dev(offsets)) is None
    torch.cuda.synchronize()
    check_append(cache, state, kv, np.zeros_like(kv), vv, table, np.clip(lengths, 0, None), offsets)
    q, qv = bf16(rng, (T, hq, D), q_scale)
    out = torch.full((T, hq, D), 7.0, dtype=torch.bfloat16, device="cuda")
    run_attend(cache, state_of(cache), q.cuda(), qv, table, lengths, offsets, causal, window, out=out)
    off = okv.rising(offsets, T)
    owned = np.zeros(T, bool)
    owned[off[0]:off[-1]] = True
    assert (out.cpu()[~torch.from_numpy(owned)] == 7.0).all()
    return cache


@pytest.mark.parametrize("hq", [2, 24])                   # few rows, many
@pytest.mark.parametrize("offsets", [[0, 5, 3, 9], [-4, 2, 2, 7], [3, 3, 8, 40], [2, 1, 0, -5], [9, 9, 9, 9]])
def test_offsets_that_lie(offsets, hq):
    note(f"kv offsets {offsets} {hq}")
    rng = np.random.default_rng(5)
    H, D, page = 1, 64, 64
    lengths = [70, 20, 130]
    pages, table = paged(rng, lengths, page, width=3)
    both(rng, random_state(rng, pages, page, H, D), hq, H, D, page, table, lengths, np.asarray(offsets, np.int32), 12)


@pytest.mark.parametrize("hq", [2, 24])
def test_lengths_of_any_sign(hq):
    """Sequences shorter than their tokens, empty, negative, longer than the table; missing and
    impossible pages."""
    note(f"kv lengths {hq}")
    rng = np.random.default_rng(6)
    H, D, page = 2, 72, 64
    lengths = [3, 0, -7, 200, 400, 2 ** 31 - 1, -2 ** 31]
    pages, table = paged(rng, [3, 0, 0, 200, 256, 128, 0], page, width=4)
    table[3, 1], table[4, 0], table[4, 2] = -1, pages, -2 ** 31
    state = random_state(rng, pages, page, H, D)
    T = 7 * 5
    for window in (0, 66):
        both(rng, state, hq, H, D, page, table, lengths, cum([5] * 7), T, window=window)
    # no pages at all
    table = np.empty((7, 0), np.int32)
    cache = cache_of(state, H, D, page)
    q = torch.ones(T, hq, D, dtype=torch.bfloat16, device="cuda")
    cache.append(q[:, :H], q[:, :H], dev(table), i32(*lengths))
    assert (cache.attend(q, dev(table), i32(*lengths)) == 0).all()
    for a, b in zip(state_of(cache), state):
        np.testing.assert_array_equal(a, b)


@pytest.mark.parametrize("hq", [2, 24])
@pytest.mark.parametrize("causal", [True, False])
def test_widest_window(hq, causal):
    """The largest window hides nothing, from tokens before position 0 neither."""
    note(f"kv widest window {hq} {causal}")
    H, D = 2, 64
    cache = svdq.KVCache(4, H, D)
    x = torch.randn(20, H, D, device="cuda").bfloat16()
    q = torch.randn(20, hq, D, device="cuda").bfloat16()
    table, lengths = i32(0, 1, 2, 3).reshape(2, 2), i32(4, 100)
    cache.append(x, x, table, lengths)
    a, b = (cache.attend(q, table, lengths, causal=causal, window=w) for w in (0, 2 ** 31 - 1))
    assert torch.equal(a, b) and (a[:6] == 0).all() == causal


def test_no_tokens():
    note("kv no tokens")
    c = svdq.KVCache(2, 2, 64)
    x = torch.empty(0, 2, 64, dtype=torch.bfloat16, device="cuda")
    table, lengths = i32(0, 1).reshape(2, 1), i32(5, 0)
    q = c.append(x, x, table, lengths, q=x)
    assert q.shape == (0, 2, 64) and c.attend(q, table, lengths).shape == (0, 2, 64)
    assert (c.data == 0).all() and (c.scales == 7).all()


@pytest.mark.parametrize("counts,before,hq,H,causal", [
    ([1] * 300, None, 4, 2, True), (None, None, 2, 2, True), (None, None, 9, 1, True), ([0] * 70 + [40] + [0] * 70, None, 3, 1, False)])
def test_many_sequences(counts, before, hq, H, causal):
    """More sequences than lanes, ragged, with empty ones among them."""
    rng = np.random.default_rng(hq)
    if counts is None:
        counts = (rng.integers(0, 9, 150) * (rng.random(150) < 0.7)).tolist()
    note(f"kv many sequences {hq} {H}")
    D, page = 64, 64
    lengths = [int(n + rng.integers(0, 150)) for n in counts]
    pages, table = paged(rng, lengths, page)
    both(rng, random_state(rng, pages, page, H, D), hq, H, D, page, table, lengths, cum(counts), sum(counts), causal)


@pytest.mark.parametrize("T,hq,H,D,window", [
    (1, 2, 1, 64, 0), (1, 2, 1, 256, 0), (2, 15, 1, 128, 0), (2, 15, 1, 128, 5000), (40, 2, 1, 64, 0), (40, 1, 1, 200, 0),
    (130, 3, 3, 128, 0), (130, 3, 3, 128, 4000)])
def test_long_and_split(T, hq, H, D, window):
    """Few row tiles and many keys: the work is cut into pieces and joined."""
    note(f"kv long {T} {hq} {D} {window}")
    rng = np.random.default_rng(T + D)
    n, page = 9000 + T, 128
    pages, table = paged(rng, [n], page)
    state = random_state(rng, pages, page, H, D)
    q, qv = bf16(rng, (T, hq, D))
    if T > 2:                                             # (the oracle's time: some rows of the many)
        keep = [0, T // 2, T - 1]
        got = cache_of(state, H, D, page).attend(q.cuda(), dev(table), i32(n), window=window)
        for i in keep:
            y, mag, rss, peak = okv.attend(state, qv[i:i + 1], table, [n - T + 1 + i], [0, 1], True, window)
            d = np.abs(got[i:i + 1].double().cpu().numpy() - y)
            assert (d <= attend_bound(y, mag, rss, peak)).all(), f"row {i}"
    else:
        run_attend(cache_of(state, H, D, page), state, q.cuda(), qv, table, [n], cum([T]), True, window)


def test_causal_rows_of_a_split_tile():
    """Pieces that some of a row tile's queries do not reach: early queries of a long call."""
    note("kv split causal")
    rng = np.random.default_rng(1)
    T, D, page = 400, 64, 64
    pages, table = paged(rng, [T], page)
    state = random_state(rng, pages, page, 1, D)
    q, qv = bf16(rng, (T, 1, D))
    run_attend(cache_of(state, 1, D, page), state, q.cuda(), qv, table, [T], cum([T]), True, 0)


@pytest.mark.parametrize("T,hq", [(1, 1), (3, 2), (50, 1), (150, 1)])
def test_very_long(T, hq):
    """Millions of tokens: one page over and over gives what the page gives once."""
    note(f"kv very long {T} {hq}")
    rng = np.random.default_rng(T)
    D, page, width = 64, 64, 50000
    state = random_state(rng, 2, page, 1, D)
    cache = cache_of(state, 1, D, page)
    q, qv = bf16(rng, (T, hq, D))
    table = torch.ones(1, width, dtype=torch.int32, device="cuda")
    got = cache.attend(q.cuda(), table, i32(width * page), causal=False).double().cpu().numpy()
    y, mag, rss, peak = okv.attend(state, qv, np.ones((1, 1), np.int32), [page], [0, T], causal=False)
    assert (np.abs(got - y) <= attend_bound(y, mag, rss, peak)).all()


@pytest.mark.parametrize("T", [1, 40, 200])
def test_positions_near_31_bits(T):
    note(f"kv 31 bits {T}")
    rng = np.random.default_rng(T)
    D, page, width, window = 64, 65536, 32767, 1000
    n = width * page - 3
    state = random_state(rng, 1, page, 1, D)
    cache = cache_of(state, 1, D, page)
    q, qv = bf16(rng, (T, 1, D))
    table = torch.full((1, width), -1, dtype=torch.int32, device="cuda")
    table[0, -1] = 0
    got = cache.attend(q.cuda(), table, i32(n), window=window)
    want = cache.attend(q.cuda(), i32(0).reshape(1, 1), i32(page - 3), window=window)
    for i in {0, T // 2, T - 1}:                          # (their pieces may be cut elsewhere)
        y, mag, rss, peak = okv.attend(state, qv[i:i + 1], np.zeros((1, 1), np.int32), [page - 3 - T + 1 + i], [0, 1], True, window)
        for x in (got, want):
            assert (np.abs(x[i:i + 1].double().cpu().numpy() - y) <= attend_bound(y, mag, rss, peak)).all()
    # past the table: what there is of the window
    assert (cache.attend(q.cuda(), table, i32(2 ** 31 - 1), window=window) == 0).all()
    k, v = (bf16(rng, (T, 1, D))[0].cuda() for _ in range(2))
    small = cache_of(state, 1, D, page)
    cache.append(k, v, table, i32(n))
    small.append(k, v, i32(0).reshape(1, 1), i32(page - 3))
    assert torch.equal(cache.data, small.data) and torch.equal(cache.scales, small.scales)
    cache.append(k, v, table, i32(2 ** 31 - 1))
    assert torch.equal(cache.data, small.data)


def test_cache_past_32_bits():
    """Pages beyond 4 GiB of codes behave as the first ones."""
    note("kv 4 GiB")
    rng = np.random.default_rng(2)
    D, page, H = 256, 65536, 1
    big, small = svdq.KVCache(140, H, D, page_size=page), svdq.KVCache(3, H, D, page_size=page)
    assert big.data.numel() > 1 << 32
    for T, n in ((65536 + 90, 65536 + 90), (5, 65536 + 95), (150, 65536 + 245)):
        q = torch.randn(T, 2 + 2 * H, D, device="cuda").bfloat16()
        a, b, c = q.split((2, 1, 1), dim=1)
        got = []
        for cache, pages in ((big, (139, 131)), (small, (0, 2))):
            table = i32(*pages).reshape(1, 2)
            cache.append(b, c, table, i32(n))
            got.append(cache.attend(a[-200:], table, i32(n), window=300))
        assert torch.equal(*got) and got[0].abs().amax() > 0
    for i, j in ((139, 0), (131, 2)):
        assert torch.equal(big.data[i], small.data[j]) and torch.equal(big.scales[i], small.scales[j])
    big.data[139].zero_(), big.data[131].zero_()
    assert not big.data.any()


@pytest.mark.parametrize("T,hq", [(1, 4), (3, 30), (50, 4), (300, 2)])
def test_unwritten_blocks(T, hq):
    """A cache of arbitrary bytes (NaN codes, NaN scales): what no call wrote never shows."""
    note(f"kv unwritten {T} {hq}")
    H, D = 2, 128
    clean, dirty = svdq.KVCache(9, H, D), svdq.KVCache(9, H, D)
    dirty.data.fill_(0x7F)
    dirty.scales.fill_(0xFF)
    table = i32(*range(9)).reshape(1, 9)
    holes = table.clone()
    holes[0, 0] = holes[0, 2] = -1                        # (what stands for a missing page is hidden as well)
    k = torch.randn(330, 2 * H, D, device="cuda").bfloat16()
    q = torch.randn(T, hq, D, device="cuda").bfloat16()
    for n in (1, 17, 33, 330):
        n = max(n, T)
        for cache in (clean, dirty):
            cache.append(k[:n, :H], k[:n, H:], table, i32(n))
        for causal, window in ((True, 0), (False, 0), (True, 13)):
            a, b = (cache.attend(q, table, i32(n), causal=causal, window=window) for cache in (clean, dirty))
            assert torch.equal(a, b) and a.isfinite().all()
    dirty.data[0].fill_(0x7F), dirty.data[2].fill_(0xFF)
    dirty.scales[0].fill_(0xFF), dirty.scales[2].fill_(0xFF)
    a, b = (cache.attend(q, holes, i32(330)) for cache in (clean, dirty))
    assert torch.equal(a, b) and a.isfinite().all()


@pytest.mark.parametrize("D", [64, 72])
def test_append_not_finite(D):
    """NaN stays where it is, an infinity saturates, neither moves the exponent."""
    note(f"kv append NaN {D}")
    rng = np.random.default_rng(D)
    H, page, T = 2, 64, 40
    k, _ = bf16(rng, (T, H, D))
    v, _ = bf16(rng, (T, H, D))
    inf, nan = float("inf"), float("nan")
    k[3, 0, 5], k[4, 0, 6], k[5, 0, 7], v[3, 1, 5], v[4, 1, 6], v[5, 1, 7] = inf, -inf, nan, inf, -inf, nan
    k[16:32, 1], v[16:32, 0] = nan, inf                   # whole blocks
    k[33, 0], v[33, 0] = 0.0, 0.0
    k[34, 0], v[34, 0] = 3.3e38, -3.3e38
    k[35, 1], v[35, 1] = 1e-40, -1e-40
    state = random_state(rng, 2, page, H, D)
    cache = cache_of(state, H, D, page)
    table = np.asarray([[1]], np.int32)
    cache.append(k.cuda(), v.cuda(), dev(table), i32(T + 5))
    ref = [a.copy() for a in state]
    okv.append(ref, k.double().numpy(), v.double().numpy(), table, [T + 5], [0, T])
    for a, b in zip(state_of(cache), ref):
        np.testing.assert_array_equal(a, b)
    # through the norm: a row that is not finite spoils itself only
    w = torch.ones(D, dtype=torch.bfloat16, device="cuda")
    good = torch.where(k.isfinite() & (k.abs() < 1e30), k, torch.zeros_like(k)).cuda()
    bad = good.clone()
    bad[7, 0, 1], bad[20, 1, 0] = nan, inf
    a, b = svdq.KVCache(1, H, D), svdq.KVCache(1, H, D)
    qa = a.append(good, good, i32(0).reshape(1, 1), i32(T), k_norm=w, q=good, q_norm=w)
    qb = b.append(bad, bad, i32(0).reshape(1, 1), i32(T), k_norm=w, q=bad, q_norm=w)
    sa, sb = state_of(a), state_of(b)
    assert np.isnan(sb[0][0, 7, 0, :D]).all()             # (a NaN's root is one)
    assert np.isnan(sb[0][0, 20, 1, 0]) and (sb[0][0, 20, 1, 1:] == 0).all()     # (over an infinite one)
    there = np.ones(sa[0].shape, bool)
    there[0, 7, 0], there[0, 20, 1] = False, False
    there[0, 0:16, 0], there[0, 16:32, 1] = False, False  # (their block's exponent may be another)
    np.testing.assert_array_equal(sa[0][there], sb[0][there])
    keep = torch.ones(T, H, dtype=torch.bool, device="cuda")
    keep[7, 0] = keep[20, 1] = False
    assert torch.equal(qa[keep], qb[keep]) and not qb[7, 0].isfinite().all()


def test_token_by_token():
    """One token after another, each call's rounding included, for three sequences in turn."""
    note("kv token by token")
    rng = np.random.default_rng(8)
    H, D, page = 3, 136, 64
    state = random_state(rng, 4, page, H, D)
    cache = cache_of(state, H, D, page)
    table = np.asarray([[2], [0], [3]], np.int32)
    lengths = np.asarray([0, 9, 30], np.int32)
    for step in range(40):
        k, kv = bf16(rng, (3, H, D), float(2.0 ** rng.integers(-6, 7)))
        v, vv = bf16(rng, (3, H, D), float(2.0 ** rng.integers(-6, 7)))
        lengths += 1
        cache.append(k.cuda(), v.cuda(), dev(table), dev(np.minimum(lengths, 64)))
        okv.append(state, kv, vv, table, np.minimum(lengths, 64), [0, 1, 2, 3])
    for a, b in zip(state_of(cache), state):
        np.testing.assert_array_equal(a, b)


@pytest.mark.parametrize("T,hq", [(4, 6), (40, 6), (300, 2)])
def test_views_and_places(T, hq):
    """Strided sources and outputs, in place, another stream: the same bits; what lies between stays."""
    note(f"kv views {T} {hq}")
    H, D, page = 2, 72, 64
    plan = svdq.RopePlan((24, 24, 24), head_dim=D)
    pos = torch.randint(0, 500, (T, 3), device="cuda", dtype=torch.int32)
    w = (1 + 0.1 * torch.randn(D, device="cuda")).bfloat16()
    pages = 6
    table = torch.arange(pages, device="cuda", dtype=torch.int32).reshape(1, pages)
    start = 3
    lengths = i32(T + start)

    def run(q, k, v, q_out=None, out=None, stream=None):
        cache = svdq.KVCache(pages, H, D, page_size=page)
        torch.cuda.synchronize()
        qr = cache.append(k, v, table, lengths, pos=pos, plan=plan, k_norm=w, q=q, q_norm=w, q_out=q_out, stream=stream)
        y = cache.attend(qr, table, lengths, out=out, stream=stream)
        torch.cuda.synchronize()
        return cache.data, qr, y

    q, k, v = (torch.randn(T, h, D, device="cuda").bfloat16() for h in (hq, H, H))
    want = run(q, k, v)
    assert torch.equal(run(q, k, v)[2], want[2])
    wide = torch.full((T + 1, hq + 3, D + 8), 3.0, dtype=torch.bfloat16, device="cuda")
    outs = [torch.full((T + 2, hq + 1, D + 16), 5.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    views = [o[1:-1, :hq, 8:D + 8] for o in outs]
    qs = wide[:T, 2:2 + hq, :D]
    qs.copy_(q)
    hm = [torch.empty(H, T, D, dtype=torch.bfloat16, device="cuda").copy_(x.transpose(0, 1)).transpose(0, 1) for x in (k, v)]
    flat = torch.cat([q, k, v], dim=1)
    a, b, c = flat.split((hq, H, H), dim=1)
    tries = [run(qs, *hm, *views), run(a, b, c, q_out=a, out=a), run(q, k, v, stream=torch.cuda.Stream())]
    for got in tries:
        assert torch.equal(got[0], want[0]) and torch.equal(got[2], want[2])
    assert torch.equal(tries[0][1], want[1])
    assert torch.equal(flat[:, hq:], torch.cat([k, v], dim=1)) and torch.equal(flat[:, :hq], want[2])
    for o, x in zip(outs, (want[1], want[2])):
        o[1:-1, :hq, 8:D + 8] -= x
        o[1:-1, :hq, 8:D + 8] += 5.0
        assert (o == 5.0).all()
    wide[:T, 2:2 + hq, :D] = 3.0
    assert (wide == 3.0).all()
    # torch's current stream is the one that is used, and the workspace belongs to it
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = run(q * 2 / 2, k, v)
    assert torch.equal(got[2], want[2])


@pytest.mark.parametrize("hq,T", [(2, 3), (8, 24)])
def test_graphs(hq, T):
    """Captured once, replayed over changing tables, lengths and offsets, with eager work and a
    second graph between the replays; every replay against the eager calls."""
    note(f"kv graphs {hq} {T}")
    H, D, page, B, width = 2, 128, 64, 3, 12
    plan = svdq.RopePlan((128,), head_dim=D)
    w = torch.ones(D, device="cuda").bfloat16()
    rng = np.random.default_rng(T)

    class Side:
        def __init__(self):
            self.cache = svdq.KVCache(B * width, H, D, page_size=page)
            self.flat = torch.zeros(T, hq + 2 * H, D, dtype=torch.bfloat16, device="cuda")
            self.table = torch.zeros(B, width, dtype=torch.int32, device="cuda")
            self.lengths = torch.zeros(B, dtype=torch.int32, device="cuda")
            self.offsets = torch.zeros(B + 1, dtype=torch.int32, device="cuda")
            self.pos = torch.zeros(T, 1, dtype=torch.int32, device="cuda")
            self.out = torch.zeros(T, hq, D, dtype=torch.bfloat16, device="cuda")

        def step(self):
            q, k, v = self.flat.split((hq, H, H), dim=1)
            q = self.cache.append(k, v, self.table, self.lengths, self.offsets, pos=self.pos, plan=plan, k_norm=w, q=q,
                                  q_norm=w)
            self.cache.attend(q, self.table, self.lengths, self.offsets, out=self.out)

        def load(self, data):
            for dst, src in zip((self.flat, self.table, self.lengths, self.offsets, self.pos), data):
                dst.copy_(src)
            self.out.fill_(9.0)

    eager, sides = Side(), [Side(), Side()]
    graphs = []
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for s in sides:
            s.step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    pool = None
    for s in sides:
        s.cache.data.zero_(), s.cache.scales.fill_(7)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, pool=pool):
            s.step()
        pool = g.pool()                                   # the second graph's workspaces in the first one's memory
        graphs.append(g)
    lengths = np.zeros(B, np.int64)
    order = rng.permutation(B * width).astype(np.int32).reshape(B, width)
    for it in range(6):
        cut = np.sort(rng.integers(0, T + 1, B - 1))
        off = np.concatenate([[0], cut, [T]]).astype(np.int32)
        lengths += np.diff(off) + (rng.integers(0, 90, B) if it % 2 else 0)
        data = (torch.randn(T, hq + 2 * H, D).bfloat16(), torch.from_numpy(order), torch.from_numpy(lengths.astype(np.int32)),
                torch.from_numpy(off), torch.from_numpy(rng.integers(0, 900, (T, 1)).astype(np.int32)))
        eager.load(data)
        eager.step()
        for s, g in zip(sides, graphs):
            s.load(data)
            g.replay()
            torch.randn(1000, 1000, device="cuda").sum().item()
        for s in sides:
            assert torch.equal(s.out, eager.out) and torch.equal(s.cache.data, eager.cache.data)
            assert torch.equal(s.cache.scales, eager.cache.scales)
        assert not (eager.out == 9.0).all(dim=2).any()


@pytest.mark.parametrize("T,hq", [(2, 6), (50, 6)])
def test_two_streams_at_once(T, hq):
    """Calls that overlap on one cache: each has a workspace of its own."""
    note(f"kv two streams {T} {hq}")
    H, D, n = 2, 128, 20000
    cache = svdq.KVCache(n // 64 + 1, H, D)
    table = torch.arange(n // 64 + 1, dtype=torch.int32, device="cuda").reshape(1, -1)
    kv = torch.randn(n, 2 * H, D, device="cuda").bfloat16()
    cache.append(kv[:, :H], kv[:, H:], table, i32(n))
    qs = [torch.randn(T, hq, D, device="cuda").bfloat16() for _ in range(4)]
    want = [cache.attend(q, table, i32(n)) for q in qs]
    streams = [torch.cuda.Stream() for _ in qs]
    lengths = i32(n)
    torch.cuda.synchronize()
    got = [[] for _ in qs]
    for _ in range(5):
        for out, q, s in zip(got, qs, streams):
            out.append(cache.attend(q, table, lengths, stream=s))
    torch.cuda.synchronize()
    for out, w in zip(got, want):
        assert all(torch.equal(y, w) for y in out)


def test_rewound():
    """Lengths may go back: tokens that were given up are written over, in place and at once as the oracle has it."""
    note("kv rewound")
    rng = np.random.default_rng(13)
    H, D, page = 2, 64, 64
    state = random_state(rng, 2, page, H, D)
    cache = cache_of(state, H, D, page)
    table = np.asarray([[1, 0]], np.int32)
    for n, length in ((40, 40), (3, 20), (30, 35), (60, 95), (1, 1)):
        k, kv = bf16(rng, (n, H, D), float(2.0 ** rng.integers(-3, 4)))
        v, vv = bf16(rng, (n, H, D))
        cache.append(k.cuda(), v.cuda(), dev(table), i32(length))
        okv.append(state, kv, vv, table, [length], [0, n])
        for a, b in zip(state_of(cache), state):
            np.testing.assert_array_equal(a, b)


def test_scales_and_heads():
    """A scale of one's own, loud scores (one key takes all), equal scores, and a group of many heads."""
    note("kv scales")
    rng = np.random.default_rng(11)
    for hq, H, D, scale, loud in ((3, 3, 64, 1.0, 4.0), (70, 1, 64, 0.01, 1.0), (5, 1, 128, 30.0, 40.0), (2, 1, 8, 1e-30, 1.0)):
        for T in (1, 37):
            n = T + 100
            pages, table = paged(rng, [n], 64)
            state = random_state(rng, pages, 64, H, D, loud=loud)
            q, qv = bf16(rng, (T, hq, D))
            run_attend(cache_of(state, H, D, 64), state, q.cuda(), qv, table, [n], cum([T]), True, 0, scale=scale)


def test_shared_pages():
    """Two sequences over the same first pages, each with pages of its own behind them."""
    note("kv shared pages")
    rng = np.random.default_rng(12)
    H, D, page = 2, 64, 64
    state = random_state(rng, 5, page, H, D)
    table = np.asarray([[4, 0, 1], [4, 0, 2]], np.int32)
    both(rng, state, 4, H, D, page, table, [150, 133], cum([3, 2]), 5)


@pytest.mark.parametrize("kw,word", [
    (dict(k_norm=(32, torch.bfloat16)), "k_norm"), (dict(q_norm=(64, torch.float32)), "q_norm"), (dict(q=None, q_norm=(64, torch.bfloat16)), "need q"),
    (dict(q=None, q_out=((4, 6, 64), torch.bfloat16)), "need q"), (dict(q_out=((4, 5, 64), torch.bfloat16)), "q_out"),
    (dict(q=((4, 0, 64), torch.bfloat16)), "at least one"), (dict(q=((4, 6, 64), torch.float16)), "q must"),
])
def test_append_refuses(kw, word):
    c = svdq.KVCache(3, 2, 64)
    made = {n: None if a is None else torch.zeros(a[0], dtype=a[1], device="cuda") for n, a in kw.items()}
    a = dict(q=torch.zeros(4, 6, 64, dtype=torch.bfloat16, device="cuda"), **{n: x for n, x in made.items() if n != "q"})
    if "q" in made:
        a["q"] = made["q"]
    k = torch.zeros(4, 2, 64, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ValueError, match=word):
        c.append(k, k, i32(0, 1).reshape(2, 1), i32(1, 1), **a)


def test_refuses_overlap_and_other_devices():
    c = svdq.KVCache(3, 2, 64)
    flat = torch.zeros(4, 10, 64, dtype=torch.bfloat16, device="cuda")
    q, k, v = flat.split((6, 2, 2), dim=1)
    table, lengths = i32(0, 1).reshape(2, 1), i32(2, 2)
    for bad in (k, v):                                    # the queries' output over the call's own sources
        with pytest.raises(svdq.SvdqError):
            c.append(k, v, table, lengths, q=q[:, :2], q_out=bad)
    with pytest.raises(svdq.SvdqError):                   # in place with other strides
        c.append(k, v, table, lengths, q=q[:, ::2], q_out=q[:, :3])
    with pytest.raises(svdq.SvdqError):
        c.attend(q[:, ::3], table, lengths, out=q[:, :2])
    for bad in (dict(k=k.cpu()), dict(v=v.cpu()), dict(table=table.cpu()), dict(lengths=lengths.cpu()), dict(q=q.cpu()),
                dict(q_out=torch.zeros(4, 6, 64, dtype=torch.bfloat16))):
        a = dict(k=k, v=v, table=table, lengths=lengths, q=q) | bad
        with pytest.raises(ValueError, match="is on|is not on"):
            c.append(a.pop("k"), a.pop("v"), a.pop("table"), a.pop("lengths"), **a)
    for bad in (dict(q=q.cpu()), dict(table=table.cpu()), dict(out=torch.zeros(4, 6, 64, dtype=torch.bfloat16))):
        a = dict(q=q, table=table, lengths=lengths) | bad
        with pytest.raises(ValueError, match="is on|is not on"):
            c.attend(a.pop("q"), a.pop("table"), a.pop("lengths"), **a)
    with pytest.raises(ValueError, match="multiple of 2"):
        c.attend(flat[:, :5], table, lengths)
