// The rotation of one token's heads by a wave (rope.hip: what it computes, and
// why it is done so; kv_append.hip rotates the queries beside the keys it
// stores).
#pragma once
#include "lanes.h"
#include "rope.h"

namespace {

// a lane's eight values as they lie in memory
template <int F32>
struct Raw {
    uint4 v[F32 ? 2 : 1];
};

template <int F32, int HALF>
DEV Raw<F32> load8(const void* p, int64_t at, int e0, int e1) {
    Raw<F32> r;
    if constexpr (F32) {
        r.v[0] = *(const uint4*)((const float*)p + at + e0);
        r.v[1] = *(const uint4*)((const float*)p + at + e1);
    } else if constexpr (HALF) {
        const uint2 a = *(const uint2*)((const uint16_t*)p + at + e0), b = *(const uint2*)((const uint16_t*)p + at + e1);
        r.v[0] = make_uint4(a.x, a.y, b.x, b.y);
    } else {
        r.v[0] = *(const uint4*)((const uint16_t*)p + at + e0);          // e1 = e0 + 4
    }
    return r;
}

template <int F32>
DEV void unpack(const Raw<F32>& r, float* v) {
    const uint32_t w[4] = {r.v[0].x, r.v[0].y, r.v[0].z, r.v[0].w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (F32) {
            const uint32_t w1[4] = {r.v[F32].x, r.v[F32].y, r.v[F32].z, r.v[F32].w};
            v[i] = __uint_as_float(w[i]);
            v[4 + i] = __uint_as_float(w1[i]);
        } else {
            v[2 * i] = bf16_lo_to_f32(w[i]);
            v[2 * i + 1] = bf16_hi_to_f32(w[i]);
        }
    }
}

template <int F32, int HALF>
DEV void store8(void* p, int64_t at, int e0, int e1, const float* v) {
    if constexpr (F32) {
        *(float4*)((float*)p + at + e0) = make_float4(v[0], v[1], v[2], v[3]);
        *(float4*)((float*)p + at + e1) = make_float4(v[4], v[5], v[6], v[7]);
    } else if constexpr (HALF) {
        *(uint2*)((uint16_t*)p + at + e0) = make_uint2(bf16x2(v[0], v[1]), bf16x2(v[2], v[3]));
        *(uint2*)((uint16_t*)p + at + e1) = make_uint2(bf16x2(v[4], v[5]), bf16x2(v[6], v[7]));
    } else {
        *(uint4*)((uint16_t*)p + at + e0) = make_uint4(bf16x2(v[0], v[1]), bf16x2(v[2], v[3]),
                                                       bf16x2(v[4], v[5]), bf16x2(v[6], v[7]));
    }
}

// cosine and sine of pos * turns turns: the product and its whole turns in 64 bits
DEV float2 turn_of(double pos, double turns) {
    const double turn = pos * turns;
    const float part = (float)(turn - rint(turn));
    float s, c;
    sincospif(2.0f * part, &s, &c);
    return make_float2(c, s);
}

constexpr int kMaxPairs = 256;

// Whether some offset is past token t (the same for all lanes). Where offsets fall, each counts as the
// largest before it, so the last token of a group is before the largest of them all, not before the last.
DEV bool some_past(const int* offs, int groups, int64_t t) {
    for (int i = threadIdx.x & 63; __ballot(i <= groups); i += 64)
        if (__ballot(i <= groups && offs[i < groups ? i : groups] > t)) return true;
    return false;
}

// HALF 0: pairs are neighbours (2i, 2i + 1); 1: pair i is (i, i + pairs). U:
// loads of a wave in flight (16 bytes a lane each, bf16). EDGES: heads may have
// channels past their pairs and tokens may be of no group (kept apart: the
// selects and the look at the offsets take 0.1 of 2.9 us for one token and 0.5
// of 21.0 for 4608 of 24 + 24 heads of 128)
// A workgroup of 256: tokens 4 bx .. 4 bx + 3, the by-th run of their loads. RISING: offsets may fall and
// are made to rise, as the cache's are; else a token from the last one on is of no group.
template <int F32, int HALF, int U, bool EDGES, bool RISING = false>
DEV void rope_axes_body(const RopeArgs& a, int64_t bx, int by, float2 (*cs)[kMaxPairs]) {
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t t = bx * 4 + wave;            // the wave's token
    if (t >= a.T) return;
    const int per = 64 / a.lp;                                   // heads per load
    // its share of the token's loads, of which the first lq are the queries'
    const int lq = (a.heads[0] + per - 1) / per, loads = lq + (a.heads[1] + per - 1) / per;
    const int first = by * a.chunk, last = first + a.chunk < loads ? first + a.chunk : loads;
    const int u = lane & (a.lp - 1), slot = lane / a.lp;
    const bool in = u * 8 < a.D, turned = u * 4 < a.pairs;
    // the lane's values: e0 .. e0 + 3 and e1 .. e1 + 3 of the head
    const int e0 = HALF && turned ? 4 * u : 8 * u, e1 = HALF && turned ? a.pairs + 4 * u : 8 * u + 4;
    // a group: up to U loads of one side
    auto side_of = [&](int l) __attribute__((always_inline)) { return l >= lq ? 1 : 0; };
    auto end_of = [&](int l) __attribute__((always_inline)) {
        const int stop = l < lq && lq < last ? lq : last;
        return l + U < stop ? l + U : stop;
    };
    Raw<F32> raw[U];
    auto fetch = [&](int l0) __attribute__((always_inline)) {
        const int side = side_of(l0), end = end_of(l0);
        const int64_t hs = a.hs[side], at0 = t * a.ts[side] + (int64_t)slot * hs;
        const int h0 = (side ? l0 - lq : l0) * per;
#pragma unroll
        for (int k = 0; k < U; ++k) {
            const int h = h0 + k * per;
            raw[k] = Raw<F32>{};
            if (l0 + k < end && in && h + slot < a.heads[side]) raw[k] = load8<F32, HALF>(a.x[side], at0 + h * hs, e0, e1);
        }
    };
    if (first < last) fetch(first);                              // on its way while the angles are worked out
    if (EDGES && a.offs && (t < a.offs[0] || (t >= a.offs[a.groups] && !(RISING && some_past(a.offs, a.groups, t)))))
        return;                                                  // of no group: left as it is

    // the token's positions, one a lane (no pairs: there may be none)
    const int pv = a.pairs > 0 && lane < a.axes ? ((const int*)a.pos)[t * a.axes + lane] : 0;
    for (int p0 = 0; p0 < a.pairs; p0 += 64) {
        const int p = p0 + lane < a.pairs ? p0 + lane : a.pairs - 1;
        int ax = a.axis[p];
        ax = ax < 0 ? 0 : ax >= a.axes ? a.axes - 1 : ax;
        const int bits = __shfl(pv, ax);
        const float2 turn = turn_of(a.pos_f32 ? (double)__int_as_float(bits) : (double)bits, a.turns[p]);
        cs[wave][p] = make_float2(turn.x, a.inverse ? -turn.y : turn.y);
    }
    __builtin_amdgcn_wave_barrier();
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    const float inv_d = 1.0f / (float)a.D;
    float m[4][4];
    for (int l0 = first; l0 < last;) {
        const int side = side_of(l0), end = end_of(l0);
        if (l0 == first || l0 == lq) {
            // Pair i of the lane, with the side's norm weights taken in:
            //   x' = (x r) (w_x cos) - (y r) (w_y sin),  y' = (x r) (w_x sin) + (y r) (w_y cos)
            float w[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) w[e] = 1.0f;
            if (in && a.norm[side]) unpack<F32>(load8<F32, HALF>(a.norm[side], 0, e0, e1), w);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 v = turned ? cs[wave][4 * u + i] : make_float2(1.0f, 0.0f);
                const float wx = w[HALF ? i : 2 * i], wy = w[HALF ? 4 + i : 2 * i + 1];
                m[i][0] = wx * v.x;
                m[i][1] = EDGES && !turned ? 0.0f : wy * v.y;
                m[i][2] = EDGES && !turned ? 0.0f : wx * v.y;
                m[i][3] = wy * v.x;
            }
        }
        Raw<F32> now[U];
#pragma unroll
        for (int k = 0; k < U; ++k) now[k] = raw[k];
        if (end < last) fetch(end);
        const int64_t hs = a.yhs[side], at0 = t * a.yts[side] + (int64_t)slot * hs;
        const int h0 = (side ? l0 - lq : l0) * per;
#pragma unroll
        for (int k = 0; k < U; ++k) {
            if (l0 + k >= end) break;                             // the same for all lanes
            float v[8], o[8];
            unpack<F32>(now[k], v);
            if (a.norm[side]) {
                float ss = 0.0f;
#pragma unroll
                for (int e = 0; e < 8; ++e) ss = __builtin_fmaf(v[e], v[e], ss);
                if (a.lp > 1) ss += lane16_other<0>(ss);
                if (a.lp > 2) ss += lane16_other<1>(ss);
                if (a.lp > 4) ss += lane16_other<2>(ss);
                if (a.lp > 8) ss += lane16_other<3>(ss);
                if (a.lp > 16) ss += __shfl_xor(ss, 16);
                if (a.lp > 32) ss += __shfl_xor(ss, 32);
                const float r = __builtin_amdgcn_rsqf(__builtin_fmaf(ss, inv_d, a.eps));   // within an ulp
#pragma unroll
                for (int e = 0; e < 8; ++e) v[e] *= r;
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int ex = HALF ? i : 2 * i, ey = HALF ? 4 + i : 2 * i + 1;
                // channels past the pairs: with a sine of 0 alone, an infinity or a NaN would
                // still get into the other one
                const float x = EDGES && !turned ? 0.0f : v[ex], y = EDGES && !turned ? 0.0f : v[ey];
                o[ex] = __builtin_fmaf(v[ex], m[i][0], -(y * m[i][1]));
                o[ey] = __builtin_fmaf(x, m[i][2], v[ey] * m[i][3]);
            }
            const int h = h0 + k * per;
            if (in && h + slot < a.heads[side]) store8<F32, HALF>(a.y[side], at0 + h * hs, e0, e1, o);
        }
        l0 = end;
    }
}

}  // namespace
