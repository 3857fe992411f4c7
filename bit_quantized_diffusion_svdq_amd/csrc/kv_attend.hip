// svdq_kv_attend: attention over a paged cache of keys and values in 8 bits,
//
//   s_j = scale q . k_j,   y = sum_j exp(s_j - m) v_j / sum_j exp(s_j - m),   m = max_j s_j
//
// over the keys j that a query sees (its sequence's length, causal order, a
// window), in one pass: a running maximum m and sum per query, the sums so far
// rescaled where m rises. A query that sees no key gives zeros.
//
// Transposed products keep everything in registers. S^T = K Q^T leaves a lane
// with scores of one query (its column) and four keys of each block of 16, so
// maxima and sums are the lane's own but for one exchange over four lanes, and
// the probabilities, rounded to bf16 in pairs, are the operand of O^T = V^T P^T as
// they stand: the values' layout follows the order of keys that this gives.
//
// S: one v_mfma_scale_f32_16x16x128_f8f6f4 takes the keys' codes as they lie in
// memory, their block's exponent as the instruction's scale. The queries' 8
// significant bits are the sum of two E4M3 numbers of 4 (what the first leaves
// is exact in the second): two instructions at twice bf16's rate, and no key is
// ever converted. Q's row exponent is the other scale. (The instruction drops
// what falls 13 bits below the largest of 8 products: some 1e-4 of a score's
// larger terms, where P's rounding to bf16 is 2e-3 of a weight.)
// O: bf16 instructions; four values of a lane are two conversions with the
// block's exponent as scale.
#include "kv.h"

namespace {

typedef __attribute__((address_space(3))) void lds_void;
typedef __bf16 v2bf __attribute__((ext_vector_type(2)));

constexpr float kNone = -1e30f;      // a maximum of nothing

template <int BLK>
DEV v4f mfma_scores(const uint4& k0, const uint4& k1, const v8i& q, const v4f& c, int ks, int qs) {
    const v8i k{(int)k0.x, (int)k0.y, (int)k0.z, (int)k0.w, (int)k1.x, (int)k1.y, (int)k1.z, (int)k1.w};
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(k, q, c, 0, 0, BLK, ks, 0, qs);
}

// four codes of two blocks, each with its block's scale
DEV v8bf widen(uint32_t a, float sa, uint32_t b, float sb) {
    const v2bf v0 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((int)a, sa, false);
    const v2bf v1 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((int)a, sa, true);
    const v2bf v2 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((int)b, sb, false);
    const v2bf v3 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((int)b, sb, true);
    return v8bf{v0[0], v0[1], v1[0], v1[1], v2[0], v2[1], v3[0], v3[1]};
}

DEV v8bf bf16x8(const v4f& a, const v4f& b) {
    return v8bf{(__bf16)a[0], (__bf16)a[1], (__bf16)a[2], (__bf16)a[3],
                (__bf16)b[0], (__bf16)b[1], (__bf16)b[2], (__bf16)b[3]};
}

// the bytes of w that hold a NaN code (0x7f, 0xff), 0x80 each
DEV uint32_t nan_codes(uint32_t w) { return ~(((w & 0x7f7f7f7fu) ^ 0x7f7f7f7fu) + 0x7f7f7f7fu) & 0x80808080u; }

// 0x80 marks to bf16 ones, two at a time
DEV uint32_t ones2(uint32_t m, int at) {
    return ((m >> (8 * at + 7)) & 1u) * 0x3f80u | ((m >> (8 * at + 15)) & 1u) * 0x3f800000u;
}

// What a workgroup works on: rows row0 .. row0 + rows - 1 (row = token of the
// sequence * G + head of the group) against the tiles of keys [ta, tb).
struct Work {
    int b, t0, n, len, room, row0, rows, ta, tb;
};

// Keys that row `r` of the sequence sees: [lo, hi)
struct Span {
    int lo, hi;
};
DEV Span span_of(const KvAttendArgs& a, const Work& w, int r) {
    const int pos = w.len - w.n + (int)((uint32_t)r / (uint32_t)a.G);
    Span s;
    s.hi = a.causal ? (pos + 1 < 0 ? 0 : pos + 1) : w.len;
    if (s.hi > w.room) s.hi = w.room;
    s.lo = a.window && pos - a.window + 1 > 0 ? pos - a.window + 1 : 0;
    return s;
}

template <int R>
DEV bool find_work(const KvAttendArgs& a, int item, int split, Work& w) {
    KvItem it;
    const int G = a.G;
    if (!kv_find(a.s, item, [&](int o, int b) { return (int)((int64_t)o * G / R) + b; },
                 [&](int n) { return (int)(((int64_t)n * G + R - 1) / R); }, it))
        return false;
    w.b = it.b;
    w.t0 = it.t0;
    w.n = it.n;
    const int len = __builtin_amdgcn_readfirstlane(a.s.lengths[it.b]);
    w.len = len < 0 ? 0 : len;
    w.room = (int)kv_room(a.s, a.c);
    w.row0 = it.part * R;
    const int left = it.n * G - w.row0;
    w.rows = left < R ? left : R;
    const Span first = span_of(a, w, w.row0), last = span_of(a, w, w.row0 + w.rows - 1);
    const int ta = first.lo / 64, tb = (last.hi + 63) / 64, nt = tb > ta ? tb - ta : 0;
    int per = (nt + a.S - 1) / a.S;
    if (per < a.least) per = a.least;
    w.ta = ta + split * per < ta + nt ? ta + split * per : ta + nt;
    w.tb = w.ta + per < ta + nt ? w.ta + per : ta + nt;
    return true;
}

// Up to 64 page numbers of a sequence, one a lane, for the tiles t0, t0 + step, ...
struct Pages {
    int mine, left;
    DEV void load(const KvAttendArgs& a, int b, int t0, int step, int tb) {
        const int t = t0 + step * (int)(threadIdx.x & 63);
        mine = t < tb ? a.s.table[(int64_t)b * a.s.width + t / a.c.tiles] : -1;
    }
    DEV int at(int i) const { return __builtin_amdgcn_readlane(mine, i); }
};

template <int C, int QT>
struct Flash {
    v8i qf[QT][C];                   // query operands, in the order of the products
    int qs[QT];                      // their exponents (E8M0)
    Span see[QT];
    float m[QT], l[QT];              // maximum of the scores, the lane's sum
    v4f o[QT][4 * C];                // O^T: channels 16 i + 4 (lane / 16) + 0..3 of the lane's query

    DEV void clear() {
#pragma unroll
        for (int t = 0; t < QT; ++t) {
            m[t] = kNone;
            l[t] = 0.0f;
#pragma unroll
            for (int i = 0; i < 4 * C; ++i) o[t][i] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
        }
    }

    // The lane's 16 C channels of a query (16 (lane / 16) + 0..15 of each 64; p NULL: zeros) as two
    // E4M3 numbers each. A query with an infinity or a NaN becomes NaN.
    DEV void load_query(int t, const uint16_t* p, int D) {
        const int g = (threadIdx.x & 63) >> 4;
        float v[16 * C];
        float amax = 0.0f, odd = 0.0f;
#pragma unroll
        for (int c = 0; c < C; ++c)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int d = c * 64 + g * 16 + h * 8;
                uint4 w = make_uint4(0u, 0u, 0u, 0u);
                if (p && d < D) w = *(const uint4*)(p + d);
                const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float x = (e & 1) ? bf16_hi_to_f32(u[e >> 1]) : bf16_lo_to_f32(u[e >> 1]);
                    const float ax = fabsf(x);
                    v[c * 16 + h * 8 + e] = x;
                    if (ax < __builtin_inff()) amax = fmaxf(amax, ax);
                    else odd = 1.0f;
                }
            }
        amax = rows4_max(amax);
        odd = rows4_max(odd);
        const int e = kv_exponent(amax);
        const float r = odd > 0.0f ? __builtin_nanf("") : exp2i(-e);
        uint32_t hi[C][4], lo[C][4];
#pragma unroll
        for (int c = 0; c < C; ++c)
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                float s[4];
                int h = 0, lw = 0;
#pragma unroll
                for (int j = 0; j < 4; ++j) s[j] = v[c * 16 + k * 4 + j] * r;
                h = __builtin_amdgcn_cvt_pk_fp8_f32(s[0], s[1], h, false);
                h = __builtin_amdgcn_cvt_pk_fp8_f32(s[2], s[3], h, true);
                const auto b0 = __builtin_amdgcn_cvt_pk_f32_fp8(h, false);
                const auto b1 = __builtin_amdgcn_cvt_pk_f32_fp8(h, true);
                lw = __builtin_amdgcn_cvt_pk_fp8_f32(s[0] - b0[0], s[1] - b0[1], lw, false);
                lw = __builtin_amdgcn_cvt_pk_fp8_f32(s[2] - b1[0], s[3] - b1[1], lw, true);
                hi[c][k] = (uint32_t)h;
                lo[c][k] = (uint32_t)lw;
            }
        qs[t] = e + 127;
#pragma unroll
        for (int i = 0; i < C; ++i)
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                if (i + 1 < C || C % 2 == 0) {           // a pair of runs: first parts, then what they leave
                    qf[t][i][k] = (int)(i % 2 == 0 ? hi[i & ~1][k] : lo[i & ~1][k]);
                    qf[t][i][4 + k] = (int)(i % 2 == 0 ? hi[i | 1][k] : lo[i | 1][k]);
                } else {                                 // a run alone: both parts against its codes twice
                    qf[t][i][k] = (int)hi[i][k];
                    qf[t][i][4 + k] = (int)lo[i][k];
                }
            }
    }

    // scores of block BLK of a tile: the small second parts first
    template <int BLK, class KEY>
    DEV void scores(v4f (&s)[QT][4], uint32_t ks, KEY key) const {
        uint4 k[C];
#pragma unroll
        for (int c = 0; c < C; ++c) k[c] = key(BLK, c);
#pragma unroll
        for (int t = 0; t < QT; ++t) {
            v4f x = v4f{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int i = C - 1; i >= 0; --i) {
                const bool pair = i + 1 < C || C % 2 == 0;
                x = mfma_scores<BLK>(k[pair ? i & ~1 : i], k[pair ? i | 1 : i], qf[t][i], x, (int)ks, qs[t]);
            }
            s[t][BLK] = x;
        }
    }

    // Tile of 64 keys from k0. key(blk, c), value(blk, c): the lane's 16 codes; sc: the blocks'
    // exponents. masked: some of its keys are not seen by some query; keys outside [zlo, zhi) by none
    // (what lies there may be anything).
    template <class KEY, class VALUE>
    DEV void tile(const KvAttendArgs& a, int k0, uint2 sc, bool masked, int zlo, int zhi, KEY key, VALUE value) {
        const int g4 = ((threadIdx.x & 63) >> 4) * 4;
        v4f s[QT][4];
        scores<0>(s, sc.x, key);
        scores<1>(s, sc.x, key);
        scores<2>(s, sc.x, key);
        scores<3>(s, sc.x, key);
        if (masked) {
#pragma unroll
            for (int t = 0; t < QT; ++t)
#pragma unroll
                for (int b = 0; b < 4; ++b)
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const int k = k0 + b * 16 + g4 + r;
                        s[t][b][r] = k >= see[t].lo && k < see[t].hi ? s[t][b][r] : -__builtin_inff();
                    }
        }
        v8bf p[QT][2];
        float alpha[QT];
        bool rises = false;
#pragma unroll
        for (int t = 0; t < QT; ++t) {
            float mx = s[t][0][0];
#pragma unroll
            for (int b = 0; b < 4; ++b)
#pragma unroll
                for (int r = 0; r < 4; ++r) mx = fmaxf(mx, s[t][b][r]);
            mx = fmaxf(rows4_max(mx), m[t]);
            alpha[t] = __builtin_amdgcn_exp2f((m[t] - mx) * a.scale2);
            rises |= mx > m[t];
            m[t] = mx;
            const float off = -mx * a.scale2;
            float sum = 0.0f;
#pragma unroll
            for (int b = 0; b < 4; ++b)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    s[t][b][r] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[t][b][r], a.scale2, off));
                    sum += s[t][b][r];
                }
            l[t] = __builtin_fmaf(l[t], alpha[t], sum);
            p[t][0] = bf16x8(s[t][0], s[t][1]);
            p[t][1] = bf16x8(s[t][2], s[t][3]);
        }
        if (__ballot(rises)) {
#pragma unroll
            for (int t = 0; t < QT; ++t)
#pragma unroll
                for (int i = 0; i < 4 * C; ++i)
#pragma unroll
                    for (int e = 0; e < 4; ++e) o[t][i][e] *= alpha[t];
        }
        float vs[4];
#pragma unroll
        for (int b = 0; b < 4; ++b) vs[b] = __uint_as_float(((sc.y >> (8 * b)) & 0xffu) << 23);
        uint32_t keep[4] = {~0u, ~0u, ~0u, ~0u};         // the bytes of keys that some query sees
        if (masked) {
#pragma unroll
            for (int b = 0; b < 4; ++b) {
                const int first = k0 + b * 16 + g4;
                int lo = zlo - first, hi = zhi - first;
                lo = lo < 0 ? 0 : lo > 4 ? 4 : lo;
                hi = hi < 0 ? 0 : hi > 4 ? 4 : hi;
                const uint32_t below_hi = hi > 3 ? ~0u : (1u << (8 * hi)) - 1u;
                const uint32_t below_lo = lo > 3 ? ~0u : (1u << (8 * lo)) - 1u;
                keep[b] = below_hi & ~below_lo;
            }
        }
#pragma unroll
        for (int c = 0; c < C; ++c) {
            uint32_t v[4][4];
#pragma unroll
            for (int b = 0; b < 4; ++b) {
                const uint4 w = value(b, c);
                v[b][0] = w.x;
                v[b][1] = w.y;
                v[b][2] = w.z;
                v[b][3] = w.w;
            }
            if (masked) {
                uint32_t any = 0;
#pragma unroll
                for (int b = 0; b < 4; ++b)
#pragma unroll
                    for (int u = 0; u < 4; ++u) {
                        v[b][u] &= keep[b];
                        any |= nan_codes(v[b][u]);
                    }
                if (__ballot(any != 0)) nans(a, k0, c, v);
            }
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const v8bf v01 = widen(v[0][u], vs[0], v[1][u], vs[1]);
                const v8bf v23 = widen(v[2][u], vs[2], v[3][u], vs[3]);
#pragma unroll
                for (int t = 0; t < QT; ++t) {
                    o[t][c * 4 + u] = mfma_bf16_16x16x32(v01, p[t][0], o[t][c * 4 + u]);
                    o[t][c * 4 + u] = mfma_bf16_16x16x32(v23, p[t][1], o[t][c * 4 + u]);
                }
            }
        }
    }

    // A tile that not every query sees whole holds NaN values: they would reach the queries that do not
    // see them too (0 * NaN). Counted by a product of ones, they go to those that do, and leave v.
    DEV void nans(const KvAttendArgs& a, int k0, int c, uint32_t (&v)[4][4]) {
        const int g4 = ((threadIdx.x & 63) >> 4) * 4;
#pragma unroll 1
        for (int u = 0; u < 4; ++u) {
            uint32_t mark[4];
#pragma unroll
            for (int b = 0; b < 4; ++b) {
                const uint32_t w = u == 0 ? v[b][0] : u == 1 ? v[b][1] : u == 2 ? v[b][2] : v[b][3];
                mark[b] = nan_codes(w);
            }
#pragma unroll
            for (int t = 0; t < QT; ++t) {
                v4f n = v4f{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    uint32_t wa[4], wb[4];
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
                        const int b = 2 * h + x / 2, at = 2 * (x & 1), k = k0 + b * 16 + g4 + at;
                        wa[x] = ones2(mark[b], at);
                        wb[x] = (k >= see[t].lo && k < see[t].hi ? 0x3f80u : 0u) |
                                (k + 1 >= see[t].lo && k + 1 < see[t].hi ? 0x3f800000u : 0u);
                    }
                    n = mfma_bf16_16x16x32(__builtin_bit_cast(v8bf, make_uint4(wa[0], wa[1], wa[2], wa[3])),
                                           __builtin_bit_cast(v8bf, make_uint4(wb[0], wb[1], wb[2], wb[3])), n);
                }
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (i == u)
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            o[t][c * 4 + i][e] = n[e] > 0.0f ? __builtin_nanf("") : o[t][c * 4 + i][e];
            }
        }
#pragma unroll
        for (int b = 0; b < 4; ++b)
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const uint32_t x = nan_codes(v[b][u]) >> 7;
                v[b][u] &= ~(x * 0xffu);
            }
    }
};

// row r of the sequence: its token and query head
struct Row {
    int64_t t;
    int h;
};
DEV Row row_of(const KvAttendArgs& a, const Work& w, int h, int r) {
    const int i = (int)((uint32_t)r / (uint32_t)a.G);
    return Row{(int64_t)w.t0 + i, h * a.G + (r - i * a.G)};
}

DEV float* part_sums(const KvAttendArgs& a, const Row& r, int split, int W) {
    return a.part + ((r.t * (a.G * a.c.H) + r.h) * a.S + split) * W;
}
DEV float* part_stats(const KvAttendArgs& a, const Row& r, int split, int W) {
    return a.part + a.s.T * (a.G * a.c.H) * (int64_t)a.S * W + ((r.t * (a.G * a.c.H) + r.h) * a.S + split) * 2;
}

// ---------------------------------------------------------------- few rows

// 16 QT rows a workgroup; its four waves take its tiles of keys in turn,
// straight from memory into the operands (every key is used once), and join
// their sums in LDS.
template <int C, int QT>
__global__ __launch_bounds__(256, C <= 2 && QT == 1 ? 2 : 1) void attend_few_kernel(KvAttendArgs a) {
    constexpr int R = 16 * QT, W = 64 * C;
    __shared__ __attribute__((aligned(16))) float red[4][R][68];
    __shared__ float stat[4][R][2];
    const int tid = threadIdx.x, lane = tid & 63, l16 = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int split = blockIdx.x % a.S, rest = blockIdx.x / a.S, h = rest % a.c.H, item = rest / a.c.H;
    Work w;
    if (!find_work<R>(a, item, split, w)) return;
    Flash<C, QT> f;
    f.clear();
#pragma unroll
    for (int t = 0; t < QT; ++t) {
        const int i = t * 16 + l16, r = w.row0 + (i < w.rows ? i : w.rows - 1);
        const Row x = row_of(a, w, h, r);
        f.load_query(t, a.q + x.t * a.qts + x.h * a.qhs, a.c.D);
        f.see[t] = span_of(a, w, r);
    }
    const Span first = span_of(a, w, w.row0), last = span_of(a, w, w.row0 + w.rows - 1);
    const int64_t tile_bytes = 8 * C * 1024;
    uint4 kr[4][C], vr[4][C];
    uint2 sc, nsc;
    Pages pages;
    const int t0 = w.ta + wave;
    const int mine = w.tb > t0 ? (w.tb - t0 + 3) / 4 : 0;
    auto where = [&](int i, bool& ok) __attribute__((always_inline)) {       // the wave's i-th tile
        const int page = pages.at(i & 63), t = t0 + 4 * i;
        ok = (uint32_t)page < (uint64_t)a.c.pages;
        return ((int64_t)(ok ? page : 0) * a.c.H + h) * a.c.tiles + t % a.c.tiles;
    };
    auto load_k = [&](int64_t at) __attribute__((always_inline)) {
        const uint8_t* p = a.c.data + at * tile_bytes;
#pragma unroll
        for (int b = 0; b < 4; ++b)
#pragma unroll
            for (int c = 0; c < C; ++c) kr[b][c] = *(const uint4*)(p + (b * C + c) * 1024 + lane * 16);
        nsc = *(const uint2*)(a.c.scales + at * 8);
    };
    auto load_v = [&](int64_t at) __attribute__((always_inline)) {
        const uint8_t* p = a.c.data + at * tile_bytes + tile_bytes / 2;
#pragma unroll
        for (int b = 0; b < 4; ++b)
#pragma unroll
            for (int c = 0; c < C; ++c) vr[b][c] = *(const uint4*)(p + (b * C + c) * 1024 + lane * 16);
    };
    bool ok = false;
    int64_t at = 0;
    if (mine > 0) {
        pages.load(a, w.b, t0, 4, w.tb);
        at = where(0, ok);
        load_k(at);
        load_v(at);
    }
    for (int i = 0; i < mine; ++i) {
        const int k0 = (t0 + 4 * i) * 64;
        const bool masked = k0 < last.lo || k0 + 64 > first.hi;
        const bool seen = ok;
        sc = nsc;
        // the next tile's page; past the last one, this tile again
        if (((i + 1) & 63) == 0 && i + 1 < mine) pages.load(a, w.b, t0 + 4 * (i + 1), 4, w.tb);
        int64_t next = at;
        if (i + 1 < mine) next = where(i + 1, ok);
        if (seen)
            f.tile(a, k0, sc, masked, first.lo, last.hi, [&](int b, int c) __attribute__((always_inline)) { return kr[b][c]; },
                   [&](int b, int c) __attribute__((always_inline)) { return vr[b][c]; });
        at = next;
        if (i + 1 < mine) {
            load_k(at);
            load_v(at);
        }
    }
    // the waves' maxima and sums, then their outputs 64 channels at a time
#pragma unroll
    for (int t = 0; t < QT; ++t) {
        const float l = rows4_sum(f.l[t]);
        if (g == 0) {
            stat[wave][t * 16 + l16][0] = f.m[t];
            stat[wave][t * 16 + l16][1] = l;
        }
    }
    const int row = tid >> 4, c4 = (tid & 15) * 4;       // of the joined outputs
#pragma unroll
    for (int c = 0; c < C; ++c) {
        if (c) __syncthreads();
#pragma unroll
        for (int t = 0; t < QT; ++t)
#pragma unroll
            for (int u = 0; u < 4; ++u) *(v4f*)&red[wave][t * 16 + l16][u * 16 + g * 4] = f.o[t][c * 4 + u];
        __syncthreads();
#pragma unroll
        for (int t = 0; t < QT; ++t) {
            const int r = t * 16 + row;
            float m = stat[0][r][0];
#pragma unroll
            for (int k = 1; k < 4; ++k) m = fmaxf(m, stat[k][r][0]);
            float sum = 0.0f;
            v4f y = v4f{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const float s = __builtin_amdgcn_exp2f((stat[k][r][0] - m) * a.scale2);
                sum = __builtin_fmaf(s, stat[k][r][1], sum);
                const v4f v = *(const v4f*)&red[k][r][c4];
#pragma unroll
                for (int e = 0; e < 4; ++e) y[e] = __builtin_fmaf(s, v[e], y[e]);
            }
            if (r < w.rows) {
                const Row x = row_of(a, w, h, w.row0 + r);
                const int d = c * 64 + c4;
                if (a.S > 1) {
                    *(v4f*)(part_sums(a, x, split, W) + d) = y;
                    if (c == 0 && c4 == 0) *(float2*)part_stats(a, x, split, W) = make_float2(m, sum);
                } else if (d < a.c.D) {
                    const float n = sum != 0.0f ? 1.0f / sum : 0.0f;
                    *(uint2*)(a.y + x.t * a.yts + x.h * a.yhs + d) =
                        make_uint2(bf16x2(y[0] * n, y[1] * n), bf16x2(y[2] * n, y[3] * n));
                }
            }
        }
    }
}

// ---------------------------------------------------------------- many rows

// 128 rows a workgroup, 32 a wave; the tiles of keys come through LDS (two
// slots, loaded straight from memory: the cache's order is the operands'), one
// meeting of the waves a tile.
template <int C>
__global__ __launch_bounds__(256, C <= 2 ? 2 : 1) void attend_many_kernel(KvAttendArgs a) {
    constexpr int QT = 2, R = 128, W = 64 * C, TILE = 8 * C * 1024;
    __shared__ __attribute__((aligned(16))) char slot0[TILE + 256], slot1[TILE + 256];
    const int tid = threadIdx.x, lane = tid & 63, l16 = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    // Workgroup b runs on XCD b % 8: each takes a contiguous run of the row
    // tiles, key head by key head, so that those in flight share keys in its L2;
    // later row tiles, which see more keys where order counts, go first.
    const int all = gridDim.x, x8 = blockIdx.x & 7, q8 = all >> 3, r8 = all & 7;
    const int t8 = x8 * q8 + (x8 < r8 ? x8 : r8) + (blockIdx.x >> 3);
    const int split = t8 % a.S, rest = t8 / a.S, h = rest / a.items, item = a.items - 1 - rest % a.items;
    Work w;
    if (!find_work<R>(a, item, split, w)) return;
    Flash<C, QT> f;
    f.clear();
    const int wr = wave * 32;                            // the wave's first row; past the end it has none
#pragma unroll
    for (int t = 0; t < QT; ++t) {
        const int i = wr + t * 16 + l16, r = w.row0 + (i < w.rows ? i : w.rows - 1);
        const Row x = row_of(a, w, h, r);
        f.load_query(t, a.q + x.t * a.qts + x.h * a.qhs, a.c.D);
        f.see[t] = span_of(a, w, r);
    }
    const int rl = wr + 31 < w.rows ? wr + 31 : w.rows - 1;
    const Span first = span_of(a, w, w.row0 + (wr < w.rows ? wr : w.rows - 1)), last = span_of(a, w, w.row0 + rl);
    Pages pages;
    const int nt = w.tb - w.ta;
    auto fetch = [&](char* s, int i) __attribute__((always_inline)) {
        if ((i & 63) == 0) pages.load(a, w.b, w.ta + i, 1, w.tb);
        const int page = pages.at(i & 63);
        const bool ok = (uint32_t)page < (uint64_t)a.c.pages;
        const int64_t at = ((int64_t)(ok ? page : 0) * a.c.H + h) * a.c.tiles + (w.ta + i) % a.c.tiles;
        const rsrc_t rt = make_rsrc(a.c.data + at * TILE, TILE), rs = make_rsrc(a.c.scales + at * 8, 8);
#pragma unroll
        for (int k = 0; k < 2 * C; ++k) {
            const int p = (k * 4 + wave) * 1024;
            __builtin_amdgcn_raw_ptr_buffer_load_lds(rt, (lds_void*)(s + p), 16, lane * 16, p, 0, 0);
        }
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (lds_void*)(s + TILE), 4, lane * 4, 0, 0, 0);
        return ok;
    };
    bool ok = false, next = false;
    auto step = [&](const char* s, char* other, int i) __attribute__((always_inline)) {
        // this tile has landed, and nobody reads the other slot any more
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        lds_barrier();
        next = false;
        if (i + 1 < nt) next = fetch(other, i + 1);
        const int k0 = (w.ta + i) * 64;
        if (ok && wr < w.rows && k0 < last.hi && k0 + 64 > first.lo) {
            const bool masked = k0 < last.lo || k0 + 64 > first.hi;
            f.tile(a, k0, *(const uint2*)(s + TILE), masked, first.lo, last.hi,
                   [&](int b, int c) __attribute__((always_inline)) { return *(const uint4*)(s + (b * C + c) * 1024 + lane * 16); },
                   [&](int b, int c) __attribute__((always_inline)) {
                       return *(const uint4*)(s + TILE / 2 + (b * C + c) * 1024 + lane * 16);
                   });
        }
        ok = next;
    };
    if (nt > 0) ok = fetch(slot0, 0);
    for (int i = 0; i < nt; i += 2) {
        step(slot0, slot1, i);
        if (i + 1 < nt) step(slot1, slot0, i + 1);
    }
#pragma unroll
    for (int t = 0; t < QT; ++t) {
        const float l = rows4_sum(f.l[t]);
        const int i = wr + t * 16 + l16;
        if (i < w.rows) {
            const Row x = row_of(a, w, h, w.row0 + i);
            if (a.S > 1) {
                float* p = part_sums(a, x, split, W);
#pragma unroll
                for (int k = 0; k < 4 * C; ++k) *(v4f*)(p + k * 16 + g * 4) = f.o[t][k];
                if (g == 0) *(float2*)part_stats(a, x, split, W) = make_float2(f.m[t], l);
            } else {
                const float n = l != 0.0f ? 1.0f / l : 0.0f;
                uint16_t* p = a.y + x.t * a.yts + x.h * a.yhs;
#pragma unroll
                for (int k = 0; k < 4 * C; ++k) {
                    const int d = k * 16 + g * 4;
                    const v4f y = f.o[t][k];
                    if (d < a.c.D) *(uint2*)(p + d) = make_uint2(bf16x2(y[0] * n, y[1] * n), bf16x2(y[2] * n, y[3] * n));
                }
            }
        }
    }
}

// ---------------------------------------------------------------- splits joined

// A wave per (token, query head): the splits' sums, weighted by their maxima.
template <int C>
__global__ __launch_bounds__(256) void attend_join_kernel(KvAttendArgs a) {
    constexpr int W = 64 * C;
    const int lane = threadIdx.x & 63, heads = a.G * a.c.H;
    const int64_t row = (int64_t)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    if (row >= a.s.T * heads) return;
    const int64_t t = row / heads;
    const int h = (int)(row - t * heads);
    if (a.s.offs) {                                      // tokens of no sequence are left as they are
        KvItem it;
        if (!kv_find(a.s, (int)t, [](int o, int) { return o; }, [](int n) { return n; }, it)) return;
    }
    const Row x{t, h};
    const float* p = part_sums(a, x, 0, W);
    const float2 st = lane < a.S ? *(const float2*)part_stats(a, x, lane, W) : make_float2(kNone, 0.0f);
    float m = st.x;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) m = fmaxf(m, __shfl_xor(m, d));
    const float wgt = __builtin_amdgcn_exp2f((st.x - m) * a.scale2);
    float sum = st.y * wgt;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) sum += __shfl_xor(sum, d);
    const unsigned long long some = __ballot(lane < a.S && st.y != 0.0f);
    float y[C];
#pragma unroll
    for (int c = 0; c < C; ++c) y[c] = 0.0f;
    for (unsigned long long left = some; left; left &= left - 1) {
        const int s = __builtin_ctzll(left);
        const float ws = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(wgt), s));
#pragma unroll
        for (int c = 0; c < C; ++c) y[c] = __builtin_fmaf(ws, p[(int64_t)s * W + lane * C + c], y[c]);
    }
    const float n = sum != 0.0f ? 1.0f / sum : 0.0f;
    uint16_t* out = a.y + t * a.yts + h * a.yhs;
#pragma unroll
    for (int c = 0; c < C; ++c)
        if (lane * C + c < a.c.D) out[lane * C + c] = f32_to_bf16_bits(y[c] * n);
}

// ---------------------------------------------------------------- which kernel, how many splits

struct Plan {
    int many, qt, items, S, least;
};

Plan plan_of(const KvBatch& s, const KvCache& c, int G, int cus) {
    Plan p{};
    const int64_t rows = s.T * G;
    const int64_t most = s.offs ? (rows + s.B - 1) / s.B : (int64_t)s.n * G;      // of a sequence, on the average
    p.many = most > 32;
    p.qt = most > 16 ? 2 : 1;
    const int R = p.many ? 128 : 16 * p.qt;
    p.items = (int)(s.offs ? rows / R + s.B : s.B * (((int64_t)s.n * G + R - 1) / R));
    const int64_t groups = (int64_t)p.items * c.H, tiles = (int64_t)s.width * c.tiles;
    p.least = p.many ? 8 : 4;
    const int64_t want = (int64_t)cus * (p.many ? 2 : 4);
    int64_t S = groups > 0 ? (want + groups - 1) / groups : 1;
    const int64_t top = (tiles + p.least - 1) / p.least;
    if (S > top) S = top;
    if (S > 64) S = 64;
    p.S = S < 1 ? 1 : (int)S;
    return p;
}

template <int C>
hipError_t launch(const KvAttendArgs& a, const Plan& p, hipStream_t stream) {
    const dim3 grid((unsigned)((int64_t)p.items * a.c.H * p.S));
    if (p.many) hipLaunchKernelGGL((attend_many_kernel<C>), grid, dim3(256), 0, stream, a);
    else if (p.qt == 2) hipLaunchKernelGGL((attend_few_kernel<C, 2>), grid, dim3(256), 0, stream, a);
    else hipLaunchKernelGGL((attend_few_kernel<C, 1>), grid, dim3(256), 0, stream, a);
    if (p.S > 1) {
        const int64_t rows = a.s.T * a.G * a.c.H;
        hipLaunchKernelGGL((attend_join_kernel<C>), dim3((unsigned)((rows + 3) / 4)), dim3(256), 0, stream, a);
    }
    return hipGetLastError();
}

}  // namespace

int64_t kv_attend_workspace(const KvBatch& s, const KvCache& c, int G, int cus) {
    const Plan p = plan_of(s, c, G, cus);
    return p.S > 1 ? s.T * G * c.H * (int64_t)p.S * ((c.D + 63) / 64 * 64 + 2) * 4 : 0;
}

hipError_t launch_kv_attend(KvAttendArgs a, int cus, hipStream_t stream) {
    const Plan p = plan_of(a.s, a.c, a.G, cus);
    a.items = p.items;
    a.S = p.S;
    a.least = p.least;
    switch ((a.c.D + 63) / 64) {
        case 1: return launch<1>(a, p, stream);
        case 2: return launch<2>(a, p, stream);
        case 3: return launch<3>(a, p, stream);
        default: return launch<4>(a, p, stream);
    }
}
