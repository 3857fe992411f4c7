// What a wave does with tiles of 64 keys (kv_attend_few.hip, kv_attend_many.hip):
// attention over a paged cache of keys and values in 8 bits,
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
// significant bits are the sum of two E4M3 numbers of 4: two instructions at twice
// bf16's rate, and no key is ever converted. Q's row exponent is the other scale.
// What the first number leaves is exact in the second for channels from 1/896 of the
// row's largest on; E4M3's least step, 2^-9 where that largest is over 224, leaves
// smaller ones off by up to 2^-10 / 224 of it (2^-17.8; a bf16 product would keep their
// own 8 bits, in twice the time). The instruction drops what falls 13 bits below the
// largest of 8 products: at most 9e-4 of a score's larger terms, some 1e-4 as a rule,
// where P's rounding to bf16 is 2e-3 of a weight.
// O: bf16 instructions; four values of a lane are two conversions with the
// block's exponent as scale.
#pragma once
#include "kv.h"

namespace {

typedef __attribute__((address_space(3))) void lds_void;
typedef __bf16 v2bf __attribute__((ext_vector_type(2)));

constexpr float kNone = -__builtin_inff();       // a maximum of nothing
constexpr int kNowhere = -(1 << 30); // the first key of a tile that is not there

template <int BLK>
DEV v4f mfma_scores(const uint4& k0, const uint4& k1, const v8i& q, const v4f& c, int ks, int qs) {
    const v8i k{(int)k0.x, (int)k0.y, (int)k0.z, (int)k0.w, (int)k1.x, (int)k1.y, (int)k1.z, (int)k1.w};
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(k, q, c, 0, 0, BLK, ks, 0, qs);
}

// the bytes of w that hold a NaN code (0x7f, 0xff), 0x80 each
DEV uint32_t nan_codes(uint32_t w) { return ~(((w & 0x7f7f7f7fu) ^ 0x7f7f7f7fu) + 0x7f7f7f7fu) & 0x80808080u; }

// Values are taken over 64 and the outputs times 64: the largest (bf16's own go to code 256 at exponent
// 120, 2^128) stay finite in bf16, where a hidden key's weight of 0 times an infinity would be a NaN, and
// a weight of up to 2^8 times a value below 2^126 stays finite in fp32. Powers of two, so nothing changes but
// the finest steps: bf16 has none below 2^-133, so values have none below 2^-127 (blocks of exponents
// -119 and -120 go down to 2^-129).
constexpr int kValueShift = 6;
constexpr float kValueUnit = 1 << kValueShift;
// the scale of a block with the exponent byte e. (Bytes that no append writes count as the nearest one.)
DEV float value_scale(uint32_t e) {
    e = e < kKvExpMin + 127 ? kKvExpMin + 127 : e > kKvExpMax + 127 ? kKvExpMax + 127 : e;
    return __uint_as_float((e - kValueShift) << 23);
}

// What sums taken from `ref` count among those taken from `top` >= ref. (Alike: all, also where both are of
// nothing, whose difference is none.)
DEV float share_of(float ref, float top, float scale2) {
    return ref == top ? 1.0f : __builtin_amdgcn_exp2f((ref - top) * scale2);
}

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
    s.lo = a.window && pos >= a.window ? pos - a.window + 1 : 0;
    return s;
}

// Where the tiles t0, t0 + STEP, ... of a sequence lie, asked for in turn. The page of the
// one after is read meanwhile, by the scalar unit: a vector load now and then would
// have the compiler wait for all loads in flight.
template <int STEP>
struct Tiles {
    const int* row;                  // the sequence's pages
    int t, tb, pg, sub, last;        // the next tile, the end; its page's place in the row and its own in the page
    int dpg, dsub, page;
    DEV void start(const KvAttendArgs& a, int b, int t0, int end) {
        row = a.s.table + (int64_t)b * a.s.width;
        t = t0;
        tb = end;
        pg = uni(t0 / a.c.tiles);
        sub = t0 - pg * a.c.tiles;
        last = uni((end - 1) / a.c.tiles);
        dpg = uni(STEP / a.c.tiles);
        dsub = STEP - dpg * a.c.tiles;
        page = row[pg];
    }
    // its index (of 64 tokens of head h) in the cache, 0 where it is past the end or on no page
    DEV int64_t take(const KvAttendArgs& a, int h, bool& ok) {
        ok = t < tb && (uint32_t)page < (uint64_t)a.c.pages;
        const int64_t at = ok ? ((int64_t)page * a.c.H + h) * a.c.tiles + sub : 0;
        t += STEP;
        pg += dpg;
        sub += dsub;
        if (sub >= a.c.tiles) {
            sub -= a.c.tiles;
            ++pg;
        }
        page = row[pg < last ? pg : last];
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

    // The lane's 16 C channels of a query: 16 (lane / 16) + 0..15 of each 64
    DEV static void fetch_query(uint4 (&q)[2 * C], const uint16_t* p, int D) {
        const int g = (threadIdx.x & 63) >> 4;
#pragma unroll
        for (int c = 0; c < C; ++c)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int d = c * 64 + g * 16 + h * 8;
                q[2 * c + h] = make_uint4(0u, 0u, 0u, 0u);
                if (d < D) q[2 * c + h] = *(const uint4*)(p + d);
            }
    }

    // as two E4M3 numbers each. A query with an infinity or a NaN becomes NaN.
    DEV void take_query(int t, const uint4 (&q)[2 * C]) {
        float v[16 * C];
        float amax = 0.0f, odd = 0.0f;
#pragma unroll
        for (int c = 0; c < 2 * C; ++c) {
            const uint32_t u[4] = {q[c].x, q[c].y, q[c].z, q[c].w};
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float x = (e & 1) ? bf16_hi_to_f32(u[e >> 1]) : bf16_lo_to_f32(u[e >> 1]);
                const float ax = fabsf(x);
                v[c * 8 + e] = x;
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

    // The i-th of a block's C products, from the last: the queries' small second parts first.
    template <int BLK>
    DEV void product(v4f (&s)[QT][4], uint32_t ks, const uint4 (&k)[C], int t, int i) const {
        const bool pair = i + 1 < C || C % 2 == 0;
        const v4f x = i == C - 1 ? v4f{0.0f, 0.0f, 0.0f, 0.0f} : s[t][BLK];
        s[t][BLK] = mfma_scores<BLK>(k[pair ? i & ~1 : i], k[pair ? i | 1 : i], qf[t][i], x, (int)ks, qs[t]);
    }

    // The scores' reference rises to their maximum, and the sums follow. Only where
    // some score is more than 8 above it (in powers of two): until then weights of up
    // to 2^8 are as exact as those of up to 1, and the sums have room. So the usual
    // tile asks one question of the lanes' own maxima, which need not meet.
    DEV void raise(const KvAttendArgs& a, const float (&top)[QT]) {
#pragma unroll
        for (int t = 0; t < QT; ++t) {
            const float mx = fmaxf(rows4_max(top[t]), m[t]);
            const float alpha = share_of(m[t], mx, a.scale2);
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
        uint4 k[4][C];
#pragma unroll
        for (int b = 0; b < 4; ++b)
#pragma unroll
            for (int c = 0; c < C; ++c) k[b][c] = key(b, c);
#pragma unroll
        for (int i = C - 1; i >= 0; --i)
#pragma unroll
            for (int t = 0; t < QT; ++t) {
                product<0>(s, ks, k[0], t, i);
                product<1>(s, ks, k[1], t, i);
                product<2>(s, ks, k[2], t, i);
                product<3>(s, ks, k[3], t, i);
            }
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
        const float off = m[t] == kNone ? 0.0f : -m[t] * a.scale2;       // (nothing seen so far: the scores are -inf)
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
            if (i >= 0) product<BLK>(s, ks, k, t, i);
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
    template <class KEY>
    DEV void exchange_tile(const KvAttendArgs& a, v4f (&s)[QT][4], uint32_t (&p)[QT][8], uint32_t ks, KEY key) const {
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
        for (int b = 0; b < 4; ++b) vs[b] = value_scale((e4 >> (8 * b)) & 0xffu);
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

    // The same from operands that are ready: ready(i, h) of 16 channels (rows of the operand) and two
    // blocks of keys. meanwhile(i): other work of the wave, beside the products of channels 16 i.
    template <class READY, class MEANWHILE>
    DEV void ready_sums(const uint32_t (&p)[QT][8], READY ready, MEANWHILE meanwhile) {
        uint4 v[3][2];                                   // two on their way
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int h = 0; h < 2; ++h) v[i][h] = ready(i, h);
        const uint32_t one2 = 0x3f803f80u;
        const v8bf ones = __builtin_bit_cast(v8bf, make_uint4(one2, one2, one2, one2));
#pragma unroll
        for (int j = 0; j < 2 * QT; ++j) l[j % QT] = mfma_bf16_16x16x32(ones, weight_operand(p[j % QT], j / QT), l[j % QT]);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int i = 0; i < 4 * C; ++i) {
#pragma unroll
            for (int h = 0; h < 2; ++h)
                if (i + 2 < 4 * C) v[(i + 2) % 3][h] = ready(i + 2, h);
#pragma unroll
            for (int j = 0; j < 2 * QT; ++j) {
                const int t = j % QT, h = j / QT;
                o[t][i] = mfma_bf16_16x16x32(__builtin_bit_cast(v8bf, v[i % 3][h]), weight_operand(p[t], h), o[t][i]);
                if (j == 0) meanwhile(i);
            }
            __builtin_amdgcn_sched_barrier(0);
        }
    }

    // NaN values of a tile that not every query sees whole: a product would take them to the queries that
    // do not see them as well (0 * NaN), so they are taken out of it, and in the end, where there were any,
    // the sums of those that do see them become NaN here: bf16's largest number, squared, makes them
    // infinite, and o * 0 + o leaves what is finite.
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

// The bytes of a tile's exponents whose blocks have a key in [lo, hi): those of the others may be any
// (255 is a NaN, and times the zeros that stand for their values one again)
DEV uint32_t kept_blocks(int k0, int lo, int hi) {
    uint32_t w = 0;
#pragma unroll
    for (int b = 0; b < 4; ++b) w |= k0 + b * 16 < hi && k0 + b * 16 + 16 > lo ? 0xffu << (8 * b) : 0u;
    return w;
}

DEV uint4 and4(const uint4& v, uint32_t m) { return make_uint4(v.x & m, v.y & m, v.z & m, v.w & m); }
DEV uint32_t nan_codes4(const uint4& v) { return nan_codes(v.x) | nan_codes(v.y) | nan_codes(v.z) | nan_codes(v.w); }
DEV uint32_t without_nan(uint32_t w) { return w & ~((nan_codes(w) >> 7) * 0xffu); }
DEV uint4 without_nan(const uint4& v) {
    return make_uint4(without_nan(v.x), without_nan(v.y), without_nan(v.z), without_nan(v.w));
}

// nan_values() of the tile whose values lie at p, keys [lo, hi) of it
template <int C, int QT>
DEV void nan_tile(Flash<C, QT>& f, const uint8_t* p, int k0, int lo, int hi) {
#pragma unroll
    for (int c = 0; c < C; ++c) {
        uint32_t v[4][4], any = 0;
#pragma unroll
        for (int b = 0; b < 4; ++b) {
            const uint4 w = and4(*(const uint4*)(p + (b * C + c) * 1024 + (threadIdx.x & 63) * 16), kept_bytes(k0, b, lo, hi));
            v[b][0] = w.x;
            v[b][1] = w.y;
            v[b][2] = w.z;
            v[b][3] = w.w;
            any |= nan_codes4(w);
        }
        if (__ballot(any != 0)) f.nan_values(k0, c, v);
    }
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

}  // namespace
