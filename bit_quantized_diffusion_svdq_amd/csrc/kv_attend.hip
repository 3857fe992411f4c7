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

// the bytes of w that hold a NaN code (0x7f, 0xff), 0x80 each
DEV uint32_t nan_codes(uint32_t w) { return ~(((w & 0x7f7f7f7fu) ^ 0x7f7f7f7fu) + 0x7f7f7f7fu) & 0x80808080u; }

// a range of keys, [lo, hi)
struct Span {
    int lo, hi;
};

// A value that all lanes have alike, told to the compiler: quotients come from the
// vector unit, and what follows from them (branches, addresses, buffer
// descriptors) would stay there, with a loop around every load.
DEV int uni(int x) { return __builtin_amdgcn_readfirstlane(x); }
DEV Span uni(const Span& s) { return Span{uni(s.lo), uni(s.hi)}; }

// What a workgroup works on: rows row0 .. row0 + rows - 1 (row = token of the
// sequence * G + head of the group) against the tiles of keys [ta, tb).
struct Work {
    int b, t0, n, len, room, row0, rows, ta, tb;
};

// Keys that row `r` of the sequence sees
DEV Span span_of(const KvAttendArgs& a, const Work& w, int r) {
    const int pos = w.len - w.n + (int)((uint32_t)r / (uint32_t)a.G);
    Span s;
    s.hi = a.causal ? (pos + 1 < 0 ? 0 : pos + 1) : w.len;
    if (s.hi > w.room) s.hi = w.room;
    s.lo = a.window && pos - a.window + 1 > 0 ? pos - a.window + 1 : 0;
    return s;
}

template <int R>
DEV bool find_work(const KvAttendArgs& a, int item, int split, int splits, Work& w) {
    KvItem it;
    const int G = a.G;
    if (!kv_find(a.s, item, [&](int o, int b) { return (int)((int64_t)o * G / R) + b; },
                 [&](int n) { return (int)(((int64_t)n * G + R - 1) / R); }, it))
        return false;
    w.b = uni(it.b);
    w.t0 = uni(it.t0);
    w.n = uni(it.n);
    const int len = uni(a.s.lengths[w.b]);
    w.len = len < 0 ? 0 : len;
    w.room = (int)kv_room(a.s, a.c);
    w.row0 = uni(it.part) * R;
    const int left = w.n * G - w.row0;
    w.rows = left < R ? left : R;
    const Span first = uni(span_of(a, w, w.row0)), last = uni(span_of(a, w, w.row0 + w.rows - 1));
    const int ta = first.lo / 64, tb = (last.hi + 63) / 64, nt = tb > ta ? tb - ta : 0;
    int per = uni((nt + splits - 1) / splits);
    if (per < a.least) per = a.least;
    w.ta = ta + split * per < ta + nt ? ta + split * per : ta + nt;
    w.tb = w.ta + per < ta + nt ? w.ta + per : ta + nt;
    return true;
}

// Where the tiles t0, t0 + STEP, ... of a sequence lie, asked for in turn: up to 64
// page numbers at a time, one a lane.
template <int STEP>
struct Tiles {
    int mine, sub, next, tb;         // the lane's page; place in its page, number, and end of the next tile
    DEV void start(const KvAttendArgs& a, int t0, int end) {
        next = 0;
        tb = end;
        sub = uni(t0 % a.c.tiles);
    }
    // the index (of 64 tokens of head h) in the cache, 0 where the tile is past the end or on no page
    DEV int64_t take(const KvAttendArgs& a, int b, int h, int t0, bool& ok) {
        const int t = t0 + STEP * next;
        if ((next & 63) == 0) {
            const int u = t + STEP * (int)(threadIdx.x & 63);
            mine = u < tb ? a.s.table[(int64_t)b * a.s.width + u / a.c.tiles] : -1;
        }
        const int page = __builtin_amdgcn_readlane(mine, next & 63);
        ok = t < tb && (uint32_t)page < (uint64_t)a.c.pages;
        const int64_t at = ok ? ((int64_t)page * a.c.H + h) * a.c.tiles + sub : 0;
        ++next;
        sub += STEP;
        while (sub >= a.c.tiles) sub -= a.c.tiles;
        return at;
    }
};

template <int C, int QT>
struct Flash {
    v8i qf[QT][C];                   // query operands, in the order of the products
    int qs[QT];                      // their exponents (E8M0)
    Span see[QT];
    float m[QT];                     // what the scores are taken from before their exponential
    v4f l[QT];                       // the weights' sum, four times over
    v4f o[QT][4 * C];                // O^T: channels 16 i + 4 (lane / 16) + 0..3 of the lane's query

    DEV void clear() {
#pragma unroll
        for (int t = 0; t < QT; ++t) {
            m[t] = kNone;
            l[t] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
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

    // The scores' reference rises to their maximum, and the sums follow. Only where
    // some score is more than 8 above it (in powers of two): until then weights of up
    // to 2^8 are as exact as those of up to 1, and the sums have room. So the usual
    // tile asks one question of the lanes' own maxima, which need not meet.
    DEV void raise(const KvAttendArgs& a, const float (&top)[QT]) {
#pragma unroll
        for (int t = 0; t < QT; ++t) {
            const float mx = fmaxf(rows4_max(top[t]), m[t]);
            const float alpha = __builtin_amdgcn_exp2f((m[t] - mx) * a.scale2);
            m[t] = mx;
#pragma unroll
            for (int e = 0; e < 4; ++e) l[t][e] *= alpha;
#pragma unroll
            for (int i = 0; i < 4 * C; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[t][i][e] *= alpha;
        }
    }

    // A tile of 64 keys from k0 goes through these in turn. key(blk, c), value(blk, c): the lane's 16
    // codes; ks, vs: the exponents of its four blocks.
    template <class KEY>
    DEV void score_tile(v4f (&s)[QT][4], uint32_t ks, KEY key) const {
        scores<0>(s, ks, key);
        scores<1>(s, ks, key);
        scores<2>(s, ks, key);
        scores<3>(s, ks, key);
    }

    // some of the tile's keys are not seen by some query
    DEV void mask(v4f (&s)[QT][4], int k0) const {
        const int g4 = ((threadIdx.x & 63) >> 4) * 4;
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

    DEV void settle(const KvAttendArgs& a, const v4f (&s)[QT][4]) {
        float top[QT];
        bool rises = false;
#pragma unroll
        for (int t = 0; t < QT; ++t) {
            top[t] = s[t][0][0];
#pragma unroll
            for (int b = 0; b < 4; ++b)
#pragma unroll
                for (int r = 0; r < 4; ++r) top[t] = fmaxf(top[t], s[t][b][r]);
            rises |= (top[t] - m[t]) * a.scale2 > 8.0f;
        }
        if (__ballot(rises)) raise(a, top);
    }

    // weights of two of the lane's four keys of block b, t / 2-th query
    DEV void weight2(const KvAttendArgs& a, const v4f (&s)[QT][4], uint32_t (&p)[QT][8], int b, int i) const {
        const int t = i >> 1, r = 2 * (i & 1);
        const float off = -m[t] * a.scale2;
        const float e0 = __builtin_amdgcn_exp2f(__builtin_fmaf(s[t][b][r], a.scale2, off));
        const float e1 = __builtin_amdgcn_exp2f(__builtin_fmaf(s[t][b][r + 1], a.scale2, off));
        p[t][2 * b + (i & 1)] = bf16x2(e0, e1);
    }
    DEV static v8bf weight_operand(const uint32_t (&p)[8], int h) {
        return __builtin_bit_cast(v8bf, make_uint4(p[4 * h], p[4 * h + 1], p[4 * h + 2], p[4 * h + 3]));
    }

    DEV void weights(const KvAttendArgs& a, const v4f (&s)[QT][4], uint32_t (&p)[QT][8]) const {
#pragma unroll
        for (int b = 0; b < 4; ++b)
#pragma unroll
            for (int i = 0; i < 2 * QT; ++i) weight2(a, s, p, b, i);
    }

    // The next tile's scores of block BLK in the place of this one's, whose weights are formed, and
    // beside them the weights of the next block.
    template <int BLK, class KEY>
    DEV void exchange(const KvAttendArgs& a, v4f (&s)[QT][4], uint32_t (&p)[QT][8], uint32_t ks, uint4 (&k)[C], KEY key) const {
        uint4 next[C];                                   // the next block's, on their way
#pragma unroll
        for (int c = 0; c < C; ++c)
            if (BLK < 3) next[c] = key(BLK + 1, c);
#pragma unroll
        for (int j = 0; j < QT * (C > 2 ? C : 2); ++j) {
            const int i = C - 1 - j / QT, t = j % QT;
            if (i >= 0) {
                const bool pair = i + 1 < C || C % 2 == 0;
                const v4f x = i == C - 1 ? v4f{0.0f, 0.0f, 0.0f, 0.0f} : s[t][BLK];
                s[t][BLK] = mfma_scores<BLK>(k[pair ? i & ~1 : i], k[pair ? i | 1 : i], qf[t][i], x, (int)ks, qs[t]);
            }
            if (BLK < 3 && j < 2 * QT) weight2(a, s, p, BLK + 1, j);
            __builtin_amdgcn_sched_barrier(0);
        }
#pragma unroll
        for (int c = 0; c < C; ++c)
            if (BLK < 3) k[c] = next[c];
    }

    // Weights of a tile from its scores, the next tile's scores in their place, block by block: one
    // matrix instruction and a few of the vector unit in turn, which run side by side (a bf16 product
    // of 16 cycles leaves its SIMD 8 for others, the keys' of 32 leaves 16).
    template <class KEY, class VALUE>
    DEV void exchange_tile(const KvAttendArgs& a, v4f (&s)[QT][4], uint32_t (&p)[QT][8], uint32_t ks, KEY key, VALUE value,
                           uint32_t (&v)[4][4]) const {
        uint4 k[C];
#pragma unroll
        for (int c = 0; c < C; ++c) k[c] = key(0, c);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int i = 0; i < 2 * QT; ++i) weight2(a, s, p, 0, i);
        __builtin_amdgcn_sched_barrier(0);
        exchange<0>(a, s, p, ks, k, key);
        exchange<1>(a, s, p, ks, k, key);
        exchange<2>(a, s, p, ks, k, key);
        read_values(v, 0, value);                        // (on their way for sums())
        exchange<3>(a, s, p, ks, k, key);
    }

    // the lane's values of 64 channels: of four rows of the operand each, a word a block
    template <class VALUE>
    DEV static void read_values(uint32_t (&v)[4][4], int c, VALUE value) {
#pragma unroll
        for (int b = 0; b < 4; ++b) {
            const uint4 w = value(b, c);
            v[b][0] = w.x;
            v[b][1] = w.y;
            v[b][2] = w.z;
            v[b][3] = w.w;
        }
    }

    // The weights' and the weighted values' sums; v: read_values(0).
    template <class VALUE>
    DEV void sums(uint32_t ve, const uint32_t (&p)[QT][8], VALUE value, uint32_t (&v)[4][4]) {
        float vs[4];
        const uint32_t e4 = __builtin_amdgcn_readfirstlane(ve);
#pragma unroll
        for (int b = 0; b < 4; ++b) vs[b] = __uint_as_float(((e4 >> (8 * b)) & 0xffu) << 23);
        // two values of the operand of rows u: 8 make it (blocks 0 and 1, then 2 and 3)
        auto widen2 = [&](uint32_t (&f)[8], int u, int j) __attribute__((always_inline)) {
            const int b = j / 2;
            f[j] = __builtin_bit_cast(uint32_t, j % 2 ? __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((int)v[b][u], vs[b], true)
                                                      : __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((int)v[b][u], vs[b], false));
        };
        uint32_t f[2][8];
        const uint32_t one2 = 0x3f803f80u;
        const v8bf ones = __builtin_bit_cast(v8bf, make_uint4(one2, one2, one2, one2));
#pragma unroll
        for (int j = 0; j < 2 * QT; ++j) {
            l[j % QT] = mfma_bf16_16x16x32(ones, weight_operand(p[j % QT], j / QT), l[j % QT]);
#pragma unroll
            for (int x = 0; x < 4 / QT; ++x) widen2(f[0], 0, j * 4 / QT + x);
            __builtin_amdgcn_sched_barrier(0);
        }
#pragma unroll
        for (int c = 0; c < C; ++c)
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                if (u == 3 && c + 1 < C) read_values(v, c + 1, value);
                const uint32_t(&now)[8] = f[u & 1];
#pragma unroll
                for (int j = 0; j < 2 * QT; ++j) {
                    const int t = j % QT, h = j / QT;
                    o[t][c * 4 + u] = mfma_bf16_16x16x32(weight_operand(now, h), weight_operand(p[t], h), o[t][c * 4 + u]);
                    if (u < 3 || c + 1 < C) {
#pragma unroll
                        for (int x = 0; x < 4 / QT; ++x) widen2(f[(u + 1) & 1], (u + 1) & 3, j * 4 / QT + x);
                    }
                    __builtin_amdgcn_sched_barrier(0);
                }
            }
    }

    // NaN values among 64 channels of a tile that not every query sees whole: a product would take them
    // to the queries that do not see them as well (0 * NaN), so they are taken out, and the sums of those
    // that do see them become NaN here: bf16's largest number, squared, makes them infinite, and o * 0 + o
    // leaves what is finite.
    DEV void nan_values(int k0, int c, const uint32_t (&v)[4][4]) {
        const int g4 = ((threadIdx.x & 63) >> 4) * 4;
#pragma unroll
        for (int t = 0; t < QT; ++t) {
            uint32_t sees[8];
#pragma unroll
            for (int x = 0; x < 8; ++x) {
                const int k = k0 + (x >> 1) * 16 + g4 + 2 * (x & 1);
                sees[x] = (k >= see[t].lo && k < see[t].hi ? 0x7f7fu : 0u) |
                          (k + 1 >= see[t].lo && k + 1 < see[t].hi ? 0x7f7f0000u : 0u);
            }
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                uint32_t mark[8];
#pragma unroll
                for (int x = 0; x < 8; ++x) {
                    const uint32_t n = nan_codes(v[x >> 1][u]) >> (16 * (x & 1));
                    mark[x] = (n >> 7 & 1u) * 0x7f7fu | (n >> 15 & 1u) * 0x7f7f0000u;
                }
#pragma unroll
                for (int i = 0; i < 4 * C; ++i) {
                    if (i != c * 4 + u) continue;
#pragma unroll
                    for (int h = 0; h < 2; ++h) o[t][i] = mfma_bf16_16x16x32(weight_operand(mark, h), weight_operand(sees, h), o[t][i]);
#pragma unroll
                    for (int e = 0; e < 4; ++e) o[t][i][e] = __builtin_fmaf(o[t][i][e], 0.0f, o[t][i][e]);
                }
            }
        }
    }
};

// The bytes of a word of block b's values (tokens 4 g .. 4 g + 3 of it) whose keys lie in [lo, hi)
DEV uint32_t kept_bytes(int k0, int b, int lo, int hi) {
    const int first = k0 + b * 16 + ((threadIdx.x & 63) >> 4) * 4;
    lo -= first;
    hi -= first;
    lo = lo < 0 ? 0 : lo > 4 ? 4 : lo;
    hi = hi < 0 ? 0 : hi > 4 ? 4 : hi;
    const uint32_t below_hi = hi > 3 ? ~0u : (1u << (8 * hi)) - 1u, below_lo = lo > 3 ? ~0u : (1u << (8 * lo)) - 1u;
    return below_hi & ~below_lo;
}

DEV uint4 and4(const uint4& v, uint32_t m) { return make_uint4(v.x & m, v.y & m, v.z & m, v.w & m); }
DEV uint32_t nan_codes4(const uint4& v) { return nan_codes(v.x) | nan_codes(v.y) | nan_codes(v.z) | nan_codes(v.w); }
DEV uint32_t without_nan(uint32_t w) { return w & ~((nan_codes(w) >> 7) * 0xffu); }
DEV uint4 without_nan(const uint4& v) {
    return make_uint4(without_nan(v.x), without_nan(v.y), without_nan(v.z), without_nan(v.w));
}

// row r of the sequence: its token and query head
struct Row {
    int64_t t;
    int h;
};
DEV Row row_of(const KvAttendArgs& a, const Work& w, int h, int r) {
    const int i = (int)((uint32_t)r / (uint32_t)a.G);
    return Row{(int64_t)w.t0 + i, h * a.G + (r - i * a.G)};
}

// Sums and (reference, weights' sum) of row i of the n-th split row tile of R rows, by one split
DEV float* part_sums(const KvAttendArgs& a, int n, int R, int i, int split, int W) {
    return a.part + (((int64_t)n * R + i) * a.S + split) * W;
}
DEV float* part_stats(const KvAttendArgs& a, int n, int R, int i, int split, int W) {
    const int64_t rows = ((int64_t)a.items * a.c.H - a.whole) * R;
    return a.part + rows * a.S * W + (((int64_t)n * R + i) * a.S + split) * 2;
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
    const int rest = uni(blockIdx.x / a.S), split = blockIdx.x - rest * a.S, item = uni(rest / a.c.H), h = rest - item * a.c.H;
    Work w;
    if (!find_work<R>(a, item, split, a.S, w)) return;
    Flash<C, QT> f;
    f.clear();
#pragma unroll
    for (int t = 0; t < QT; ++t) {
        const int i = t * 16 + l16, r = w.row0 + (i < w.rows ? i : w.rows - 1);
        const Row x = row_of(a, w, h, r);
        f.load_query(t, a.q + x.t * a.qts + x.h * a.qhs, a.c.D);
        f.see[t] = span_of(a, w, r);
    }
    const Span first = uni(span_of(a, w, w.row0)), last = uni(span_of(a, w, w.row0 + w.rows - 1));
    const int64_t tile_bytes = 8 * C * 1024;
    uint4 kr[4][C], vr[4][C];
    uint2 sc, nsc;
    const int t0 = w.ta + wave;
    const int mine = w.tb > t0 ? (w.tb - t0 + 3) / 4 : 0;
    Tiles<4> tiles;
    tiles.start(a, t0, w.tb);
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
        at = tiles.take(a, w.b, h, t0, ok);
        load_k(at);
        load_v(at);
    }
    for (int i = 0; i < mine; ++i) {
        const int k0 = (t0 + 4 * i) * 64;
        const bool masked = k0 < last.lo || k0 + 64 > first.hi;
        const bool seen = ok;
        sc = nsc;
        if (i + 1 < mine) at = tiles.take(a, w.b, h, t0, ok);
        const auto key = [&](int b, int c) __attribute__((always_inline)) { return kr[b][c]; };
        const auto value = [&](int b, int c) __attribute__((always_inline)) { return vr[b][c]; };
        if (seen) {
            v4f s[QT][4];
            uint32_t p[QT][8];
            f.score_tile(s, sc.x, key);
            if (masked) {
                f.mask(s, k0);
                uint32_t any = 0;
#pragma unroll
                for (int b = 0; b < 4; ++b)
#pragma unroll
                    for (int c = 0; c < C; ++c) {
                        vr[b][c] = and4(vr[b][c], kept_bytes(k0, b, first.lo, last.hi));
                        any |= nan_codes4(vr[b][c]);
                    }
                if (__ballot(any != 0)) {
#pragma unroll
                    for (int c = 0; c < C; ++c) {
                        uint32_t v[4][4];
#pragma unroll
                        for (int b = 0; b < 4; ++b) {
                            v[b][0] = vr[b][c].x;
                            v[b][1] = vr[b][c].y;
                            v[b][2] = vr[b][c].z;
                            v[b][3] = vr[b][c].w;
                            vr[b][c] = without_nan(vr[b][c]);
                        }
                        f.nan_values(k0, c, v);
                    }
                }
            }
            f.settle(a, s);
            f.weights(a, s, p);
            uint32_t v[4][4];
            f.read_values(v, 0, value);
            f.sums(sc.y, p, value, v);
        }
        if (i + 1 < mine) {
            load_k(at);
            load_v(at);
        }
    }
    // the waves' maxima and sums, then their outputs 64 channels at a time
#pragma unroll
    for (int t = 0; t < QT; ++t) {
        const float l = f.l[t][0];
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
                    *(v4f*)(part_sums(a, rest, R, r, split, W) + d) = y;
                    if (c == 0 && c4 == 0) *(float2*)part_stats(a, rest, R, r, split, W) = make_float2(m, sum);
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

// 128 rows a workgroup, 32 a wave; the tiles of keys come through LDS, loaded
// straight from memory (the cache's order is the operands'), keys a tile before
// their values: the scores of a tile are formed beside the weights of the one
// before, matrix work beside vector work. One meeting of the waves a tile.
template <int C>
__global__ __launch_bounds__(256, C <= 2 ? 2 : 1) void attend_many_kernel(KvAttendArgs a) {
    constexpr int QT = 2, R = 128, W = 64 * C, HALF = 4 * C * 1024;
    __shared__ __attribute__((aligned(16))) char key0[HALF], key1[HALF], value0[HALF], value1[HALF];
    const int tid = threadIdx.x, lane = tid & 63, l16 = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    // Row tiles in the order of the key heads, later ones, which see more keys where order counts, first.
    // The first a.whole of them are a workgroup's each, the rest a.S workgroups'. Workgroup b runs on XCD b %
    // 8: of either part an XCD takes a contiguous run, so that those in flight share keys in its L2.
    const bool whole = (int)blockIdx.x < a.whole;
    const int all = whole ? a.whole : gridDim.x - a.whole, b8 = whole ? blockIdx.x : blockIdx.x - a.whole;
    const int x8 = b8 & 7, q8 = all >> 3, r8 = all & 7, splits = whole ? 1 : a.S;
    const int t8 = x8 * q8 + (x8 < r8 ? x8 : r8) + (b8 >> 3);
    const int of = uni(t8 / splits), split = t8 - of * splits, rest = whole ? of : a.whole + of;
    const int h = uni(rest / a.items), item = a.items - 1 - (rest - h * a.items);
    Work w;
    if (!find_work<R>(a, item, split, splits, w)) return;
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
    const Span first = uni(span_of(a, w, w.row0 + (wr < w.rows ? wr : w.rows - 1))), last = uni(span_of(a, w, w.row0 + rl));
    const Span wfirst = uni(span_of(a, w, w.row0)), wlast = uni(span_of(a, w, w.row0 + w.rows - 1));
    const int nt = w.tb - w.ta;

    Tiles<1> tiles;
    tiles.start(a, w.ta, w.tb);
    auto find = [&](bool& ok) __attribute__((always_inline)) { return tiles.take(a, w.b, h, w.ta, ok); };
    // one side of a tile into LDS, a quarter a wave (zeros if it is not there)
    auto fetch = [&](char* s, int64_t at, int side, bool ok) __attribute__((always_inline)) {
        const rsrc_t r = make_rsrc(a.c.data + (2 * at + side) * HALF, ok ? HALF : 0);
#pragma unroll
        for (int k = 0; k < C; ++k) {
            const int p = (k * 4 + wave) * 1024;
            __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_void*)(s + p), 16, lane * 16, p, 0, 0);
        }
    };
    auto landed = [&]() __attribute__((always_inline)) {
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        lds_barrier();
    };
    bool ok0, ok1, ok2;                                  // of tiles i, i + 1, i + 2
    v4f s[QT][4];
    uint2 sc0, sc1;                                      // exponents of tiles i, i + 1
    auto codes = [&](const char* k) __attribute__((always_inline)) {
        return [=](int b, int c) __attribute__((always_inline)) { return *(const uint4*)(k + (b * C + c) * 1024 + lane * 16); };
    };
    auto is_masked = [&](int i, bool ok) __attribute__((always_inline)) {
        const int k0 = (w.ta + i) * 64;
        return !ok || k0 < last.lo || k0 + 64 > first.hi;
    };
    auto hide = [&](int i, bool ok) __attribute__((always_inline)) {
        if (is_masked(i, ok)) f.mask(s, ok ? (w.ta + i) * 64 : INT32_MIN / 2);
        f.settle(a, s);
    };
    // Values of a tile that not all rows of the workgroup see whole: keys that none of them sees may
    // hold anything, and become zeros in LDS, as do NaN values once the sums have them.
    auto clean = [&](char* v, int k0) __attribute__((always_inline)) {
        uint32_t any = 0;
#pragma unroll 1
        for (int q = 0; q < 4 * C; ++q)
            any |= nan_codes4(and4(*(const uint4*)(v + q * 1024 + lane * 16), kept_bytes(k0, q / C, wfirst.lo, wlast.hi)));
        if (__ballot(any != 0)) {
#pragma unroll
            for (int c = 0; c < C; ++c) {
                uint32_t x[4][4];
#pragma unroll
                for (int b = 0; b < 4; ++b) {
                    const uint4 y = and4(codes(v)(b, c), kept_bytes(k0, b, wfirst.lo, wlast.hi));
                    x[b][0] = y.x;
                    x[b][1] = y.y;
                    x[b][2] = y.z;
                    x[b][3] = y.w;
                }
                f.nan_values(k0, c, x);
            }
        }
        lds_barrier();
#pragma unroll 1
        for (int q = wave; q < 4 * C; q += 4) {
            uint4* x = (uint4*)(v + q * 1024 + lane * 16);
            *x = without_nan(and4(*x, kept_bytes(k0, q / C, wfirst.lo, wlast.hi)));
        }
        lds_barrier();
    };
    // Tile i, whose scores are in s: its weights, beside them the next tile's scores; then its sums.
    int64_t at1 = 0;                                     // tile i + 1
    auto step = [&](char* knext, char* kfree, char* v, char* vfree, int i) __attribute__((always_inline)) {
        landed();                                        // keys of i + 1, values of i; nobody reads the others
        const int k0 = (w.ta + i) * 64;
        if (ok0 && (k0 < wlast.lo || k0 + 64 > wfirst.hi)) clean(v, k0);
        const int64_t at2 = find(ok2);
        fetch(kfree, at2, 0, ok2);
        fetch(vfree, at1, 1, ok1);
        const uint2 sc2 = *(const uint2*)(a.c.scales + at2 * 8);
        if (wr < w.rows) {
            uint32_t p[QT][8];
            uint32_t v0[4][4];
            f.exchange_tile(a, s, p, sc1.x, codes(knext), codes(v), v0);
            f.sums(sc0.y, p, codes(v), v0);
#pragma unroll
            for (int t = 0; t < QT; ++t)                 // (or the compiler moves the scores behind the branch)
#pragma unroll
                for (int b = 0; b < 4; ++b) order_point(s[t][b]);
            hide(i + 1, ok1);
        }
        ok0 = ok1;
        ok1 = ok2;
        sc0 = sc1;
        sc1 = sc2;
        at1 = at2;
    };
    if (nt > 0) {
        const int64_t at0 = find(ok0);
        at1 = find(ok1);
        fetch(key0, at0, 0, ok0);
        sc0 = *(const uint2*)(a.c.scales + at0 * 8);
        sc1 = *(const uint2*)(a.c.scales + at1 * 8);
        landed();
        fetch(value0, at0, 1, ok0);
        fetch(key1, at1, 0, ok1);
        if (wr < w.rows) {
            f.score_tile(s, sc0.x, codes(key0));
            hide(0, ok0);
        }
        for (int i = 0; i < nt; i += 2) {
            step(key1, key0, value0, value1, i);
            if (i + 1 < nt) step(key0, key1, value1, value0, i + 1);
        }
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory"); // (loads into LDS end before the workgroup does)
    }
#pragma unroll
    for (int t = 0; t < QT; ++t) {
        const float l = f.l[t][0];
        const int i = wr + t * 16 + l16;
        if (i < w.rows) {
            const Row x = row_of(a, w, h, w.row0 + i);
            if (splits > 1) {
                float* p = part_sums(a, rest - a.whole, R, i, split, W);
#pragma unroll
                for (int k = 0; k < 4 * C; ++k) *(v4f*)(p + k * 16 + g * 4) = f.o[t][k];
                if (g == 0) *(float2*)part_stats(a, rest - a.whole, R, i, split, W) = make_float2(f.m[t], l);
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
    KvItem it;                                           // tokens of no sequence are left as they are
    if (!kv_find(a.s, (int)t, [](int o, int) { return o; }, [](int n) { return n; }, it)) return;
    const int kh = h / a.G, r = ((int)t - it.t0) * a.G + h - kh * a.G, of = r / a.rows, i = r - of * a.rows;
    const int item = of + (a.s.offs ? (int)((int64_t)it.t0 * a.G / a.rows) + it.b : it.b * ((a.s.n * a.G + a.rows - 1) / a.rows));
    const int tile = a.rows == 128 ? kh * a.items + a.items - 1 - item - a.whole : item * a.c.H + kh;     // the kernels' orders
    if (tile < 0) return;                                   // not split
    const float* p = part_sums(a, tile, a.rows, i, 0, W);
    const float2 st = lane < a.S ? *(const float2*)part_stats(a, tile, a.rows, i, lane, W) : make_float2(kNone, 0.0f);
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
    int many, rows, items, whole, S, least;
};

// Few rows a sequence (up to 32, on the average): keys are split until there
// are four workgroups a CU, at least 4 tiles each. More rows: workgroups come in
// rounds of the CUs' places, and the row tiles of a last round that is not full are
// split where that takes less time: a tile of 64 keys takes 1.75 us with the
// places taken, a row tile's sums 26 ns a split and 128 channels to write and
// read, the launch that joins them 5 us (4608 queries over 23040 keys of 24 heads:
// 864 row tiles on 512 places).
Plan plan_of(const KvBatch& s, const KvCache& c, int G, int cus) {
    Plan p{};
    const int64_t rows = s.T * G;
    const int64_t most = s.offs ? (rows + s.B - 1) / s.B : (int64_t)s.n * G;      // of a sequence, on the average
    p.many = most > 32;
    const int R = p.rows = p.many ? 128 : most > 16 ? 32 : 16;
    p.items = (int)(s.offs ? rows / R + s.B : s.B * (((int64_t)s.n * G + R - 1) / R));
    const int64_t groups = (int64_t)p.items * c.H, tiles = (int64_t)s.width * c.tiles;
    p.least = p.many ? 8 : 4;
    p.S = 1;
    const int64_t top = (tiles + p.least - 1) / p.least < 64 ? (tiles + p.least - 1) / p.least : 64;
    if (!p.many) {
        const int64_t S = groups > 0 ? ((int64_t)cus * 4 + groups - 1) / groups : 1;
        p.S = (int)(S < top ? S : top);
        if (p.S < 1) p.S = 1;
        return p;
    }
    const int C = (c.D + 63) / 64;
    const int64_t places = (int64_t)cus * (C <= 2 ? 2 : 1), rest = groups % places;
    const double tile = 1.75 * (C <= 2 ? C / 2.0 : C / 4.0), io = 0.026 * C / 2.0;
    double least = (double)tiles * tile;                 // of the last round
    for (int S = 2; S <= top && rest; ++S) {
        const double t = (double)((rest * S + places - 1) / places) / S * (double)tiles * tile + (double)(rest * S) * io + 5.0;
        if (t < least) least = t, p.S = S;
    }
    p.whole = (int)(p.S > 1 ? groups - rest : groups);
    return p;
}

template <int C>
hipError_t launch(const KvAttendArgs& a, const Plan& p, hipStream_t stream) {
    const int64_t groups = (int64_t)p.items * a.c.H;
    const dim3 grid((unsigned)(p.whole + (groups - p.whole) * p.S));
    if (p.many) hipLaunchKernelGGL((attend_many_kernel<C>), grid, dim3(256), 0, stream, a);
    else if (p.rows == 32) hipLaunchKernelGGL((attend_few_kernel<C, 2>), grid, dim3(256), 0, stream, a);
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
    return p.S > 1 ? ((int64_t)p.items * c.H - p.whole) * p.rows * p.S * ((c.D + 63) / 64 * 64 + 2) * 4 : 0;
}

hipError_t launch_kv_attend(KvAttendArgs a, int cus, hipStream_t stream) {
    const Plan p = plan_of(a.s, a.c, a.G, cus);
    a.items = p.items;
    a.whole = p.whole;
    a.rows = p.rows;
    a.S = p.S;
    a.least = p.least;
    switch ((a.c.D + 63) / 64) {
        case 1: return launch<1>(a, p, stream);
        case 2: return launch<2>(a, p, stream);
        case 3: return launch<3>(a, p, stream);
        default: return launch<4>(a, p, stream);
    }
}
