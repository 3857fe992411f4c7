// svdq_kv_append: a call's keys (optionally normed and rotated on the way) and
// values into a paged cache in 8 bits, and its queries normed and rotated in
// the same launch.
//
// Per block of 16 tokens, key head and side: e = the least exponent with amax
// <= 448 * 2^e over the call's finite values, code = e4m3(x * 2^-e), nearest even,
// infinities saturate, a NaN keeps a NaN code. A block that an earlier call
// began keeps its exponent if that is larger; where it grows, the codes from
// before are rounded again to the new one: by powers of two only what becomes
// subnormal loses bits, so appending token by token costs no more than at once. Codes
// of the block past the last token become zeros.
//
// A workgroup takes one block of one sequence and some of its key heads, a
// wave the keys or the values of one head at a time. The waves work the
// block's cosines and sines out once, in LDS, while their first head is on its
// way. Keys: a lane holds 16 channels of one token in each 64, which is 16
// bytes of the cache; their norm and rotation are in 64 bits and their only rounding is that to
// the code (a code is one of few, so a rounding on the way shows where a key lies next to a
// border: of 14 million codes 27 are not the 64-bit key's in 32 bits, 7 with the rotation in 64, 3 with one
// rounding, none with the squares' sum in 64 as well; the last two take 1.3 us of 36). Values: a lane holds 4 channels of 4 tokens, which is four
// words of it; the words meet in LDS and leave 16 bytes a lane. A block is
// written by its two waves, so nothing is atomic.
//
// Bound by memory and, as a block of work is short, its latency: 4608 tokens of 24 + 2 x 24 heads of 128 with
// norms and three axes take 32.5 us in a graph (4.4 TB/s), 8003 of 16 + 2 x 4 of 64 15 (3.1).
#include "fp8.h"
#include "kv.h"
#include "rope_body.h"

namespace {

constexpr int kPairs = 128;          // of a head of 256

// four codes times 2^d, d <= 0
DEV uint32_t rescale4(uint32_t w, float f) {
    const auto a = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, false);
    const auto b = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, true);
    return e4m3_x4(a[0] * f, a[1] * f, b[0] * f, b[1] * f);
}
DEV uint4 rescale16(const uint4& v, float f) {
    return make_uint4(rescale4(v.x, f), rescale4(v.y, f), rescale4(v.z, f), rescale4(v.w, f));
}

// x * 2^-e as the conversion takes it: infinities at +-448, NaN as it is
DEV float fit(float x, float r) {
    const float v = x * r, c = __builtin_amdgcn_fmed3f(v, -kE4m3Max, kE4m3Max);
    return v == v ? c : v;
}

// the largest of a wave's values (>= 0), in all lanes
DEV float wave_max(float v) {
    v = fmaxf(v, lane16_other<0>(v));
    v = fmaxf(v, lane16_other<1>(v));
    v = fmaxf(v, lane16_other<2>(v));
    v = fmaxf(v, lane16_other<3>(v));
    return rows4_max(v);
}

template <bool F>
struct Finite {
    static constexpr bool value = F;
};

// bits of a magnitude that is no infinity and no NaN in any lane of the wave
DEV bool all_finite(uint32_t m) { return __ballot(m >= 0x7f800000u) == 0; }

// four values times r to four codes. FINITE: none is an infinity or a NaN, and so none passes 448 (r is
// the power of two that their largest allows)
template <bool FINITE>
DEV uint32_t codes4(float a, float b, float c, float d, float r) {
    if constexpr (FINITE) return e4m3_x4(a * r, b * r, c * r, d * r);
    else return e4m3_x4(fit(a, r), fit(b, r), fit(c, r), fit(d, r));
}

template <int STEP>
DEV double lane16_other64(double v) {
    const uint2 u = __builtin_bit_cast(uint2, v);
    return __builtin_bit_cast(double, make_uint2(__float_as_uint(lane16_other<STEP>(__uint_as_float(u.x))),
                                                 __float_as_uint(lane16_other<STEP>(__uint_as_float(u.y)))));
}

// A number in 64 bits to one in 32 that rounds to the code that the first one rounds to: 20 bits of its
// fraction and, in the last place, whether there was more (so what lies beside a border does not come to
// lie on it).
DEV float to_odd(double v) {
    const unsigned long long u = __builtin_bit_cast(unsigned long long, v);
    const uint32_t lo = (uint32_t)u;
    return (float)__builtin_bit_cast(double, (u & 0xffffffff00000000ull) | ((unsigned long long)((lo < 1u ? lo : 1u) << 29)));
}

DEV float bf16_at(const uint32_t* w, int e) { return (e & 1) ? bf16_hi_to_f32(w[e >> 1]) : bf16_lo_to_f32(w[e >> 1]); }

// Cosine and sine of pos * turns turns, 2^-29 off at the most: within an eighth of a turn of a multiple
// of a quarter by their series.
DEV double2 near_turn_of(double pos, double turns) {
    const double turn = pos * turns, quarters = rint(4.0 * turn);
    const double z = 6.283185307179586477 * __builtin_fma(-0.25, quarters, turn), z2 = z * z;
    const double c = __builtin_fma(z2, __builtin_fma(z2, __builtin_fma(z2, __builtin_fma(z2, __builtin_fma(z2, -1.0 / 3628800,
                     1.0 / 40320), -1.0 / 720), 1.0 / 24), -0.5), 1.0);
    const double s = z * __builtin_fma(z2, __builtin_fma(z2, __builtin_fma(z2, __builtin_fma(z2, 1.0 / 362880, -1.0 / 5040),
                         1.0 / 120), -1.0 / 6), 1.0);
    const int q = (int)(quarters - 4.0 * rint(0.25 * quarters));         // -2 .. 2
    const double x = q & 1 ? s : c, y = q & 1 ? c : s;                   // a quarter: (-s, c), half: (-c, -s)
    return make_double2((q + 1) & 2 ? -x : x, q & 2 ? -y : y);
}

// Cosines and sines of the block's tokens, slots [s0, s1): a wave takes every fourth slot, a lane a
// pair; the positions of its four slots are read at once.
DEV void block_angles(const KvAppendArgs& a, double2* cs, int pitch, int s0, int s1, int64_t t_at0, int wave) {
    const int lane = threadIdx.x & 63;
    for (int p = lane; p < a.pairs; p += 64) {
        int ax = a.axis[p];
        const double turns = a.turns[p];
        ax = ax < 0 ? 0 : ax >= a.axes ? a.axes - 1 : ax;
        int bits[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int s = s0 + wave + 4 * i;
            bits[i] = 0;
            if (s < s1) bits[i] = ((const int*)a.pos)[(t_at0 + s) * a.axes + ax];
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int s = s0 + wave + 4 * i;
            if (s < s1) cs[s * pitch + p] = near_turn_of(a.pos_f32 ? (double)__int_as_float(bits[i]) : (double)bits[i], turns);
        }
    }
}

// The values of heads hn, hn + 2, ... of a block, by one wave: a lane has 4 channels of each 64 of its
// four tokens, and of the cache's order a row of four words of 4 tokens.
template <int C, class MEANWHILE>
DEV void append_values(const KvAppendArgs& a, int page, int tile, int blk, int s0, int s1, int64_t t_at0, int hn, int hend,
                       uint8_t (&turn)[C][4 * 272], MEANWHILE meanwhile) {
    const int lane = threadIdx.x & 63, quad = lane >> 4, j = lane & 15, D = a.c.D;
    uint32_t isnew = 0, isold = 0;                       // bytes of the quad's words from the call, from before
#pragma unroll
    for (int s = 0; s < 4; ++s) {
        const int slot = quad * 4 + s;
        isnew |= slot >= s0 && slot < s1 ? 0xffu << (8 * s) : 0u;
        isold |= slot < s0 ? 0xffu << (8 * s) : 0u;
    }
    uint2 w[C][4];
    uint4 old[C];
    int e0 = kKvExpMin;
    uint8_t *vd = a.c.data, *sc = a.c.scales;
    auto fetch = [&](int h) __attribute__((always_inline)) {
        const int64_t at = ((int64_t)page * a.c.H + h) * a.c.tiles + tile;
        vd = a.c.data + at * (8 * C * 1024) + (4 + blk) * C * 1024 + lane * 16;
        sc = a.c.scales + at * 8 + 4 + blk;
#pragma unroll
        for (int c = 0; c < C; ++c) {
#pragma unroll
            for (int s = 0; s < 4; ++s) {
                const int slot = quad * 4 + s, d = c * 64 + j * 4;
                w[c][s] = make_uint2(0u, 0u);
                if (slot >= s0 && slot < s1 && d < D) w[c][s] = *(const uint2*)(a.v + (t_at0 + slot) * a.vts + h * a.vhs + d);
            }
            old[c] = make_uint4(0u, 0u, 0u, 0u);
            if (isold) old[c] = *(const uint4*)(vd + c * 1024);
        }
        if (s0 > 0) e0 = kv_old_exponent(sc[0]);
    };
    if (hn < hend) fetch(hn);
    meanwhile();
    for (int h = hn; h < hend; h += 2) {
        uint32_t m2 = 0;                                 // magnitudes of bf16 pairs, ordered as integers
#pragma unroll
        for (int c = 0; c < C; ++c)
#pragma unroll
            for (int s = 0; s < 4; ++s) m2 = max_u16x2(m2, max_u16x2(w[c][s].x & 0x7fff7fffu, w[c][s].y & 0x7fff7fffu));
        const uint32_t m = (m2 >> 16 > (m2 & 0xffffu) ? m2 >> 16 : m2 & 0xffffu) << 16;
        const bool finite = all_finite(m);
        float amax = __uint_as_float(m);
        if (!finite) {
            amax = 0.0f;
#pragma unroll
            for (int c = 0; c < C; ++c)
#pragma unroll
                for (int s = 0; s < 4; ++s) {
                    const uint32_t x[2] = {w[c][s].x, w[c][s].y};
#pragma unroll
                    for (int i = 0; i < 4; ++i) amax = fmaxf(amax, finite_abs(bf16_at(x, i)));
                }
        }
        int e = kv_exponent(wave_max(amax));
        e = e < e0 ? e0 : e;
        if (lane == 0) sc[0] = (uint8_t)(e + 127);
        const float rv = exp2i(-e);
        auto turned = [&](auto fin) __attribute__((always_inline)) {
#pragma unroll
            for (int c = 0; c < C; ++c)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    float t[4];
#pragma unroll
                    for (int s = 0; s < 4; ++s) {
                        const uint32_t x[2] = {w[c][s].x, w[c][s].y};
                        t[s] = bf16_at(x, i);
                    }
                    // channel 64 c + 4 j + i: row 4 (j % 4) + i of the run, word j / 4
                    *(uint32_t*)&turn[c][quad * 272 + ((j & 3) * 4 + i) * 16 + (j >> 2) * 4] =
                        codes4<decltype(fin)::value>(t[0], t[1], t[2], t[3], rv);
                }
        };
        if (finite) turned(Finite<true>{});
        else turned(Finite<false>{});
        __builtin_amdgcn_wave_barrier();
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
#pragma unroll
        for (int c = 0; c < C; ++c) {
            if (isold == ~0u && e == e0) continue;       // four tokens from before, as they are
            uint4 x = *(const uint4*)&turn[c][quad * 272 + j * 16];
            x = make_uint4(x.x & isnew, x.y & isnew, x.z & isnew, x.w & isnew);
            if (isold) {
                uint4 o = old[c];
                if (e != e0) o = rescale16(o, exp2i(e0 - e < -126 ? -126 : e0 - e));
                x = make_uint4(x.x | (o.x & isold), x.y | (o.y & isold), x.z | (o.z & isold), x.w | (o.w & isold));
            }
            *(uint4*)(vd + c * 1024) = x;
        }
        __builtin_amdgcn_wave_barrier();
        if (h + 2 < hend) fetch(h + 2);
    }
}

template <int C, int HALF, int U>
__global__ __launch_bounds__(256) void kv_append_kernel(KvAppendArgs a, RopeArgs q) {
    __shared__ double2 cs[16 * (kPairs + 2)];            // a token's pairs, rows apart by two more
    __shared__ __attribute__((aligned(16))) uint8_t turn[2][C][4 * 272];
    static_assert(sizeof cs >= sizeof(float2) * 4 * kMaxPairs, "the queries' angles fit");
    const int blocks = a.items * a.groups;
    if ((int)blockIdx.x >= blocks) {
        const int64_t b = (int)blockIdx.x - blocks;
        rope_axes_body<0, HALF, U, true, true>(q, b % a.qx, (int)(b / a.qx), (float2(*)[kMaxPairs])cs);
        return;
    }
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int item = blockIdx.x / a.groups, h0 = blockIdx.x % a.groups * a.per;
    KvItem it;
    if (!kv_find(a.s, item, [](int o, int b) { return o / 16 + 2 * b; }, [](int n) { return n > 0 ? (n + 14) / 16 + 1 : 0; }, it))
        return;
    // The block's tokens: slots [s0, s1) of it are the call's, those before s0 are there already.
    // What has no place (before 0, past the table, on no page) is left out.
    const int raw = __builtin_amdgcn_readfirstlane(a.s.lengths[it.b]);
    const int len = raw < 0 ? 0 : raw, start = len - it.n, begin = start < 0 ? 0 : start;
    const int64_t first = ((int64_t)(begin / 16) + it.part) * 16;                 // the block's first token
    if (first >= len || first >= kv_room(a.s, a.c)) return;
    const int page = a.s.table[(int64_t)it.b * a.s.width + first / (a.c.tiles * 64)];
    if ((uint32_t)page >= (uint64_t)a.c.pages) return;
    const int s0 = begin > first ? (int)(begin - first) : 0, s1 = len - first < 16 ? (int)(len - first) : 16;
    const int64_t t_at0 = (int64_t)it.t0 + (first - start);                       // the call's token in slot 0
    const int tile = (int)(first / 64 % a.c.tiles), blk = (int)(first / 16 % 4);

    const int P = a.pairs, pitch = P + 2;
    const int D = a.c.D;
    const int hend = h0 + a.per < a.c.H ? h0 + a.per : a.c.H;
    const int hn = h0 + (wave >> 1);                     // the wave's heads: hn, hn + 2, ...; waves 0 and 2 their keys
    if (wave & 1) {
        append_values<C>(a, page, tile, blk, s0, s1, t_at0, hn, hend, turn[wave >> 1], [&]() __attribute__((always_inline)) {
            block_angles(a, cs, pitch, s0, s1, t_at0, wave);
            __syncthreads();                             // (with the keys' waves)
        });
        return;
    }

    // ---- keys
    const int key = lane >> 2, part = lane & 3;          // the lane's token, its 16 channels of each 64
    const bool knew = key >= s0 && key < s1;
    uint4 kw[C][2], pw[HALF ? C : 1][2];
    int e0 = kKvExpMin;
    uint8_t *kd = a.c.data, *sc = a.c.scales;
    auto fetch = [&](int h) __attribute__((always_inline)) {
        const int64_t at = ((int64_t)page * a.c.H + h) * a.c.tiles + tile;
        kd = a.c.data + at * (8 * C * 1024) + blk * C * 1024 + (part * 16 + key) * 16;
        sc = a.c.scales + at * 8 + blk;
        const uint16_t* kp = a.k + (t_at0 + key) * a.kts + h * a.khs;
#pragma unroll
        for (int c = 0; c < C; ++c)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int d = c * 64 + part * 16 + e * 8;
                kw[c][e] = make_uint4(0u, 0u, 0u, 0u);
                if (knew && d < D) kw[c][e] = *(const uint4*)(kp + d);
                if constexpr (HALF) {                    // the other channels of their pairs, 4 at a time
                    const int o0 = d < P ? d + P : d - P, o1 = d + 4 < P ? d + 4 + P : d + 4 - P;
                    uint2 x = make_uint2(0u, 0u), y = x;
                    if (knew && d < 2 * P) x = *(const uint2*)(kp + o0);
                    if (knew && d + 4 < 2 * P) y = *(const uint2*)(kp + o1);
                    pw[c][e] = make_uint4(x.x, x.y, y.x, y.y);
                }
            }
        if (s0 > 0) e0 = kv_old_exponent(sc[0]);
    };
    if (hn < hend) fetch(hn);                            // on its way while the angles are worked out
    block_angles(a, cs, pitch, s0, s1, t_at0, wave);
    // the norm's weights of the lane's channels and of the others of their pairs
    uint4 nw[C][2], mw[HALF ? C : 1][2];
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int d = c * 64 + part * 16 + e * 8;
            nw[c][e] = make_uint4(0u, 0u, 0u, 0u);
            if (a.norm && d < D) nw[c][e] = *(const uint4*)(a.norm + d);
            if constexpr (HALF) {
                uint2 x = make_uint2(0u, 0u), y = x;
                if (a.norm && d < 2 * P) x = *(const uint2*)(a.norm + (d < P ? d + P : d - P));
                if (a.norm && d + 4 < 2 * P) y = *(const uint2*)(a.norm + (d + 4 < P ? d + 4 + P : d + 4 - P));
                mw[c][e] = make_uint4(x.x, x.y, y.x, y.y);
            }
        }
    const double inv_d = 1.0 / D;
    __syncthreads();
    auto keep = [](uint4& w) __attribute__((always_inline)) { asm volatile("" : "+v"(w.x), "+v"(w.y), "+v"(w.z), "+v"(w.w)); };
    for (int h = hn; h < hend; h += 2) {
        if (a.norm) {
#pragma unroll
            for (int c = 0; c < C; ++c)
#pragma unroll
                for (int e = 0; e < 2; ++e) {            // (or they are widened before the loop, in twice the registers)
                    keep(nw[c][e]);
                    if constexpr (HALF) keep(mw[c][e]);
                }
        }
        double r = 1.0;
        if (a.norm) {
            double sum[2] = {0.0, 0.0};
#pragma unroll
            for (int c = 0; c < C; ++c)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const uint32_t w[4] = {kw[c][e].x, kw[c][e].y, kw[c][e].z, kw[c][e].w};
#pragma unroll
                    for (int i = 0; i < 8; i += 4) {     // (four squares, each exact, in 32 bits: 2^-28 of the root)
                        const float s0 = __builtin_fmaf(bf16_at(w, i), bf16_at(w, i), bf16_at(w, i + 1) * bf16_at(w, i + 1));
                        const float s1 = __builtin_fmaf(bf16_at(w, i + 2), bf16_at(w, i + 2), bf16_at(w, i + 3) * bf16_at(w, i + 3));
                        sum[i / 4] += (double)(s0 + s1);
                    }
                }
            double ss = sum[0] + sum[1];
            ss += lane16_other64<0>(ss);
            ss += lane16_other64<1>(ss);
            const double var = __builtin_fma(ss, inv_d, (double)a.eps);
            r = (double)__builtin_amdgcn_rsqf((float)var);
            if (r > 0.0) r = __builtin_fma(0.5 * r, __builtin_fma(-var * r, r, 1.0), r);     // (0: an infinite sum)
            r = knew && (float)ss != __builtin_inff() ? r : 0.0;         // (past 32 bits: 0, as the queries')
        }
        float x[C][16];
        uint32_t m = 0;                                  // magnitudes, ordered as integers
#pragma unroll
        for (int c = 0; c < C; ++c)
#pragma unroll
            for (int f = 0; f < 4; ++f) {                // 4 channels from d
                const int d = c * 64 + part * 16 + f * 4;
                const uint4 ow = kw[c][f >> 1], tw = pw[HALF ? c : 0][HALF ? f >> 1 : 0];
                const uint32_t o[2] = {f & 1 ? ow.z : ow.x, f & 1 ? ow.w : ow.y};
                const uint32_t p[2] = {f & 1 ? tw.z : tw.x, f & 1 ? tw.w : tw.y};
                float x32[4], y32[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    x32[i] = bf16_at(o, i);
                    y32[i] = HALF ? bf16_at(p, i) : 0.0f;
                }
                const bool first_half = d < P, turned = d < 2 * P;
                if (a.norm) {                            // (the products with the weights are exact)
                    const uint4 ww = nw[c][f >> 1], vw = mw[HALF ? c : 0][HALF ? f >> 1 : 0];
                    const uint32_t n[2] = {f & 1 ? ww.z : ww.x, f & 1 ? ww.w : ww.y};
                    const uint32_t o2[2] = {f & 1 ? vw.z : vw.x, f & 1 ? vw.w : vw.y};
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        x32[i] *= bf16_at(n, i);
                        if (HALF) y32[i] *= bf16_at(o2, i);
                    }
                }
                double own[4], other[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) own[i] = x32[i], other[i] = y32[i];
                if (turned && knew) {
                    if constexpr (HALF) {
                        const int p0 = first_half ? d : d - P;
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const double2 t = cs[key * pitch + p0 + i];
                            own[i] = __builtin_fma(own[i], t.x, first_half ? -(other[i] * t.y) : other[i] * t.y);
                        }
                    } else {
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const double2 t = cs[key * pitch + d / 2 + i];
                            const double u = own[2 * i], v = own[2 * i + 1];
                            own[2 * i] = __builtin_fma(u, t.x, -(v * t.y));
                            own[2 * i + 1] = __builtin_fma(u, t.y, v * t.x);
                        }
                    }
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    x[c][f * 4 + i] = to_odd(own[i] * r);
                    const uint32_t b = __float_as_uint(x[c][f * 4 + i]) & 0x7fffffffu;
                    m = m > b ? m : b;
                }
                __builtin_amdgcn_sched_barrier(0);       // (four channels' 64-bit values at a time: registers)
            }
        const bool finite = all_finite(m);
        float amax = __uint_as_float(m);
        if (!finite) {
            amax = 0.0f;
#pragma unroll
            for (int c = 0; c < C; ++c)
#pragma unroll
                for (int i = 0; i < 16; ++i) amax = fmaxf(amax, finite_abs(x[c][i]));
        }
        int e = kv_exponent(wave_max(amax));
        e = e < e0 ? e0 : e;
        if (lane == 0) sc[0] = (uint8_t)(e + 127);
        const float rk = exp2i(-e);
#pragma unroll
        for (int c = 0; c < C; ++c) {
            if (key >= s0) {                             // the call's tokens; zeros past them
                uint32_t w[4];
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    w[i] = finite ? codes4<true>(x[c][4 * i], x[c][4 * i + 1], x[c][4 * i + 2], x[c][4 * i + 3], rk)
                                  : codes4<false>(x[c][4 * i], x[c][4 * i + 1], x[c][4 * i + 2], x[c][4 * i + 3], rk);
                if (c == C - 1 && !finite) {             // past the head: 0 times a root that is a NaN
                    const int past = c * 64 + part * 16 + 16 - D;
                    if (past > 0) w[2] = w[3] = 0u;      // (a multiple of 8)
                    if (past > 8) w[0] = w[1] = 0u;
                }
                *(uint4*)(kd + c * 1024) = make_uint4(w[0], w[1], w[2], w[3]);
            } else if (e != e0) {
                *(uint4*)(kd + c * 1024) = rescale16(*(const uint4*)(kd + c * 1024), exp2i(e0 - e < -126 ? -126 : e0 - e));
            }
        }
        if (h + 2 < hend) fetch(h + 2);
    }
}

template <int C, int HALF, int U>
void run(const KvAppendArgs& a, const RopeArgs& q, unsigned grid, hipStream_t stream) {
    hipLaunchKernelGGL((kv_append_kernel<C, HALF, U>), dim3(grid), dim3(256), 0, stream, a, q);
}

template <int C>
hipError_t launch(KvAppendArgs a, RopeArgs q, int half, int cus, hipStream_t stream) {
    const int U = a.s.T <= 2 * (int64_t)cus ? 1 : 4;     // as launch_rope_axes has it
    int64_t gx = 0, gy = 0;
    if (q.heads[0]) rope_shares(q, U, cus, gx, gy);
    a.qx = gx ? (int)gx : 1;
    const int64_t grid = (int64_t)a.items * a.groups + gx * gy;
    if (!grid) return hipSuccess;
    if (half) U == 1 ? run<C, 1, 1>(a, q, (unsigned)grid, stream) : run<C, 1, 4>(a, q, (unsigned)grid, stream);
    else U == 1 ? run<C, 0, 1>(a, q, (unsigned)grid, stream) : run<C, 0, 4>(a, q, (unsigned)grid, stream);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_kv_append(KvAppendArgs a, RopeArgs q, int half, int cus, hipStream_t stream) {
    a.items = (int)(a.s.offs ? a.s.T / 16 + 2 * (int64_t)a.s.B : a.s.n > 0 ? (int64_t)a.s.B * ((a.s.n + 14) / 16 + 1) : 0);
    // The heads of a block share its angles, and more workgroups share the chip: as few of a block as make
    // three for each two CUs, with as many heads each, in twos. (Tokens of 24 heads of 128, us with 2 heads a
    // workgroup, 4, 8, 12, 24, the rule's in brackets: 512 [9.0] 9.7 13.8 18.0 30.3; 1152 14.6 [12.7] 15.6 19.9
    // 33.2; 2304 26.4 22.5 [20.1] 23.4 35.0; 4608 46.1 39.4 34.3 [32.5] 40.4; 9216 92.3 76.0 66.7 64.8 [62.4]. 2048
    // of 8 heads 17.9 [16.4] 16.8.)
    const int64_t blocks = a.s.T / 16 + a.s.B;           // (about: sequences begin and end inside of blocks)
    int64_t groups = (3 * (int64_t)cus / 2 + blocks - 1) / blocks;
    if (groups > a.c.H) groups = a.c.H;
    a.per = (int)((a.c.H + groups - 1) / groups + 1) & ~1;
    a.groups = (a.c.H + a.per - 1) / a.per;
    switch ((a.c.D + 63) / 64) {
        case 1: return launch<1>(a, q, half, cus, stream);
        case 2: return launch<2>(a, q, half, cus, stream);
        case 3: return launch<3>(a, q, half, cus, stream);
        default: return launch<4>(a, q, half, cus, stream);
    }
}
