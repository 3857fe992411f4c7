// svdq_rope_axes: rotary positions with several axes on query and key heads,
// optionally after an RMS norm of each head.
//
// Pair i of a head belongs to axis a(i) and turns by the angle
// pos[t, a(i)] f(i):
//
//   (x, y) -> (x cos - y sin, x sin + y cos)     (inverse: angle negated)
//
// The plan holds f(i) / 2 pi in 64 bits, so an angle is a number of turns:
// the product, and taking off its whole turns, run in 64 bits and lose
// nothing at far positions; sine and cosine of the remaining part of a turn
// run in 32 bits (sinpi / cospi). Everything else is 32-bit, with one rounding
// of the output.
//
// Bound by memory: every head is read and written once. A wave owns one
// token and a run of its heads: it computes the token's cosines and sines
// once (one pair per lane, shared through LDS, while its first loads are on
// their way) and reuses them, multiplied by the norm's weights, for all its
// heads. A lane owns four pairs of a head (8 values, 16 bytes of bf16), so a
// 128-wide head is 16 lanes and a load instruction covers four heads; the
// norm's sum of squares is a butterfly over a head's lanes without LDS. The
// vector work counts beside the memory's: folding the weights into the
// rotation, uniform sides and the hardware's reciprocal root took 4608 tokens
// of 24 + 24 heads of 128 (normed) from 47.6 to 27.1 us, loads ahead of the
// angles and less work a pair to 21.1, 5.4 TB/s; 32761 of 16 + 4 without a norm
// run in 64.3 us, 5.2 TB/s (fp32: 41.8 and 127.7, 5.4 and 5.3; a plain copy: 5.5).
// All figures of this file are kernels in a graph.
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

constexpr int kMaxPairs = 256;

// HALF 0: pairs are neighbours (2i, 2i + 1); 1: pair i is (i, i + pairs). U:
// loads of a wave in flight (16 bytes a lane each, bf16). EDGES: heads may have
// channels past their pairs and tokens may be of no group (kept apart: the
// selects and the look at the offsets take 0.1 of 2.9 us for one token and 0.5
// of 21.0 for 4608 of 24 + 24 heads of 128)
template <int F32, int HALF, int U, bool EDGES>
__global__ __launch_bounds__(256) void rope_axes_kernel(RopeArgs a) {
    __shared__ float2 cs[4][kMaxPairs];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t t = (int64_t)blockIdx.x * 4 + wave;            // the wave's token
    if (t >= a.T) return;
    const int per = 64 / a.lp;                                   // heads per load
    // its share of the token's loads, of which the first lq are the queries'
    const int lq = (a.heads[0] + per - 1) / per, loads = lq + (a.heads[1] + per - 1) / per;
    const int first = blockIdx.y * a.chunk, last = first + a.chunk < loads ? first + a.chunk : loads;
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
    if (EDGES && a.offs && (t < a.offs[0] || t >= a.offs[a.groups])) return;   // of no group: left as it is

    // the token's positions, one a lane (no pairs: there may be none)
    const int pv = a.pairs > 0 && lane < a.axes ? ((const int*)a.pos)[t * a.axes + lane] : 0;
    for (int p0 = 0; p0 < a.pairs; p0 += 64) {
        const int p = p0 + lane < a.pairs ? p0 + lane : a.pairs - 1;
        int ax = a.axis[p];
        const double turns = a.turns[p];
        ax = ax < 0 ? 0 : ax >= a.axes ? a.axes - 1 : ax;
        const int bits = __shfl(pv, ax);
        const double turn = (a.pos_f32 ? (double)__int_as_float(bits) : (double)bits) * turns;
        const float part = (float)(turn - rint(turn));
        float s, co;
        sincospif(2.0f * part, &s, &co);
        cs[wave][p] = make_float2(co, a.inverse ? -s : s);
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

template <int F32, int HALF, int U, bool EDGES>
void run(const RopeArgs& a, dim3 grid, hipStream_t stream) {
    hipLaunchKernelGGL((rope_axes_kernel<F32, HALF, U, EDGES>), grid, dim3(256), 0, stream, a);
}

}  // namespace

template <int U>
static hipError_t launch(RopeArgs a, int f32, int half, int cus, hipStream_t stream) {
    a.lp = 1;
    while (a.lp * 8 < a.D) a.lp *= 2;
    const int per = 64 / a.lp, loads = (a.heads[0] + per - 1) / per + (a.heads[1] + per - 1) / per;
    // A wave takes all of its token's heads where the tokens fill the chip (12
    // waves a CU), else a share of them, U loads at the least, and works the
    // angles out again (1024 tokens of 24 + 24 heads of 128 take 7.3 us in three
    // waves a token, 7.9 in two, 10.7 in one; 32761 of 16 + 4 69 in two and 64.3 in
    // one).
    int64_t chunks = ((int64_t)cus * 12 + a.T - 1) / a.T;
    if (chunks > (loads + U - 1) / U) chunks = (loads + U - 1) / U;
    a.chunk = (int)((loads + chunks - 1) / chunks);
    const dim3 grid((unsigned)((a.T + 3) / 4), (unsigned)((loads + a.chunk - 1) / a.chunk));
    const bool edges = a.offs || 2 * a.pairs < a.D;
    if (f32) {
        if (half) edges ? run<1, 1, U, true>(a, grid, stream) : run<1, 1, U, false>(a, grid, stream);
        else edges ? run<1, 0, U, true>(a, grid, stream) : run<1, 0, U, false>(a, grid, stream);
    } else {
        if (half) edges ? run<0, 1, U, true>(a, grid, stream) : run<0, 1, U, false>(a, grid, stream);
        else edges ? run<0, 0, U, true>(a, grid, stream) : run<0, 0, U, false>(a, grid, stream);
    }
    return hipGetLastError();
}

hipError_t launch_rope_axes(RopeArgs a, int f32, int half, int cus, hipStream_t stream) {
    // Few tokens: one load a wave at a time, more waves (24 + 24 heads of 128: 1 token 3.0 us, 4.5
    // with four loads; 77 tokens 3.5, 5.3; 512 5.5, 6.1). More tokens: four loads in flight (1024
    // tokens 7.3, 8.1 with one; 4608 of 32 + 8 heads, half-split 17.1, 18.6).
    return a.T <= 2 * (int64_t)cus ? launch<1>(a, f32, half, cus, stream) : launch<4>(a, f32, half, cus, stream);
}
