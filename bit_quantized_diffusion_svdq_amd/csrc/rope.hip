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
// once (one pair per lane, shared through LDS) and reuses them for all its
// heads. A lane owns four pairs of a head (8 values, 16 bytes of bf16), so a
// 128-wide head is 16 lanes and a load instruction covers four heads; the
// norm's sum of squares is a butterfly over a head's lanes.
#include "common.h"
#include "rope.h"

namespace {

template <int F32>
DEV void load4(const void* p, int64_t at, float* v) {
    if constexpr (F32) {
        const float4 u = *(const float4*)((const float*)p + at);
        v[0] = u.x; v[1] = u.y; v[2] = u.z; v[3] = u.w;
    } else {
        const uint2 u = *(const uint2*)((const uint16_t*)p + at);
        v[0] = bf16_lo_to_f32(u.x); v[1] = bf16_hi_to_f32(u.x);
        v[2] = bf16_lo_to_f32(u.y); v[3] = bf16_hi_to_f32(u.y);
    }
}

template <int F32>
DEV void store4(void* p, int64_t at, const float* v) {
    if constexpr (F32) *(float4*)((float*)p + at) = make_float4(v[0], v[1], v[2], v[3]);
    else *(uint2*)((uint16_t*)p + at) = make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
}

constexpr int kMaxPairs = 256;

// HALF 0: pairs are neighbours (2i, 2i + 1); 1: pair i is (i, i + pairs)
template <int F32, int HALF>
__global__ __launch_bounds__(256) void rope_axes_kernel(RopeArgs a) {
    __shared__ float2 cs[4][kMaxPairs];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int per = 64 / a.lp;                                   // heads per load
    const int H = a.heads[0] + a.heads[1];
    const int loads = (H + per - 1) / per, chunks = (loads + a.chunk - 1) / a.chunk;
    const int64_t item = (int64_t)blockIdx.x * 4 + wave;
    const int64_t t = item / chunks;
    if (t >= a.T) return;
    const int c = (int)(item - t * chunks);

    for (int p = lane; p < a.pairs; p += 64) {
        int ax = a.axis[p];
        ax = ax < 0 ? 0 : ax >= a.axes ? a.axes - 1 : ax;
        const int64_t at = t * a.axes + ax;
        const double pos = a.pos_f32 ? (double)((const float*)a.pos)[at] : (double)((const int*)a.pos)[at];
        const double turn = pos * a.turns[p];
        const float part = (float)(turn - rint(turn));
        float s, co;
        sincospif(2.0f * part, &s, &co);
        cs[wave][p] = make_float2(co, a.inverse ? -s : s);
    }
    __builtin_amdgcn_wave_barrier();
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");

    const int u = lane & (a.lp - 1), slot = lane / a.lp;
    const bool in = u * 8 < a.D, turned = u * 4 < a.pairs;
    // the lane's values: e0 .. e0 + 3 and e1 .. e1 + 3 of the head
    const int e0 = HALF && turned ? 4 * u : 8 * u, e1 = HALF && turned ? a.pairs + 4 * u : 8 * u + 4;
    float co[4], si[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 v = turned ? cs[wave][4 * u + i] : make_float2(1.0f, 0.0f);
        co[i] = v.x;
        si[i] = v.y;
    }
    const int first = c * a.chunk, last = first + a.chunk < loads ? first + a.chunk : loads;
    constexpr int U = 4;
    for (int l0 = first; l0 < last; l0 += U) {
        float v[U][8];
        int hd[U], side[U];
        bool ok[U];
#pragma unroll
        for (int k = 0; k < U; ++k) {
            const int h = (l0 + k) * per + slot;
            ok[k] = in && l0 + k < last && h < H;
            side[k] = h >= a.heads[0];
            hd[k] = side[k] ? h - a.heads[0] : h;
#pragma unroll
            for (int e = 0; e < 8; ++e) v[k][e] = 0.0f;
            if (ok[k]) {
                const int64_t at = t * a.ts[side[k]] + hd[k] * a.hs[side[k]];
                load4<F32>(a.x[side[k]], at + e0, v[k]);
                load4<F32>(a.x[side[k]], at + e1, v[k] + 4);
            }
        }
#pragma unroll
        for (int k = 0; k < U; ++k) {
            if (l0 + k >= last) break;                            // the same for all lanes
            if (a.norm[0] || a.norm[1]) {
                float ss = 0.0f;
#pragma unroll
                for (int e = 0; e < 8; ++e) ss = __builtin_fmaf(v[k][e], v[k][e], ss);
                for (int d = 1; d < a.lp; d <<= 1) ss += __shfl_xor(ss, d);
                if (ok[k] && a.norm[side[k]]) {
                    const float r = 1.0f / sqrtf(ss / (float)a.D + a.eps);
                    float w[8];
                    load4<F32>(a.norm[side[k]], e0, w);
                    load4<F32>(a.norm[side[k]], e1, w + 4);
#pragma unroll
                    for (int e = 0; e < 8; ++e) v[k][e] = v[k][e] * r * w[e];
                }
            }
            float o[8];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int ex = HALF ? i : 2 * i, ey = HALF ? 4 + i : 2 * i + 1;
                o[ex] = v[k][ex] * co[i] - v[k][ey] * si[i];
                o[ey] = v[k][ex] * si[i] + v[k][ey] * co[i];
            }
            if (ok[k]) {
                const int64_t at = t * a.yts[side[k]] + hd[k] * a.yhs[side[k]];
                store4<F32>(a.y[side[k]], at + e0, o);
                store4<F32>(a.y[side[k]], at + e1, o + 4);
            }
        }
    }
}

}  // namespace

hipError_t launch_rope_axes(RopeArgs a, int f32, int half, int cus, hipStream_t stream) {
    a.lp = 1;
    while (a.lp * 8 < a.D) a.lp *= 2;
    const int per = 64 / a.lp, loads = (a.heads[0] + a.heads[1] + per - 1) / per;
    // all of a token's heads in one wave once that fills the chip (8 waves a SIMD), else one load each
    a.chunk = a.T >= (int64_t)cus * 8 ? loads : 1;
    const int64_t items = a.T * ((loads + a.chunk - 1) / a.chunk);
    const dim3 grid((unsigned)((items + 3) / 4)), block(256);
    if (f32) {
        if (half) hipLaunchKernelGGL((rope_axes_kernel<1, 1>), grid, block, 0, stream, a);
        else hipLaunchKernelGGL((rope_axes_kernel<1, 0>), grid, block, 0, stream, a);
    } else {
        if (half) hipLaunchKernelGGL((rope_axes_kernel<0, 1>), grid, block, 0, stream, a);
        else hipLaunchKernelGGL((rope_axes_kernel<0, 0>), grid, block, 0, stream, a);
    }
    return hipGetLastError();
}
