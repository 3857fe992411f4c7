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
// wave one head at a time. It works the block's cosines and sines out once, in
// LDS. Keys: a lane holds 16 channels of one token in each 64, which is 16
// bytes of the cache. Values: a lane holds 4 channels of 4 tokens, which is four
// words of it; the words meet in LDS and leave 16 bytes a lane. A block is
// written by one wave, so nothing is atomic.
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

// the largest of a wave's values, in all lanes
DEV float wave_max(float v) {
    v = fmaxf(v, lane16_other<0>(v));
    v = fmaxf(v, lane16_other<1>(v));
    v = fmaxf(v, lane16_other<2>(v));
    v = fmaxf(v, lane16_other<3>(v));
    return rows4_max(v);
}

DEV float bf16_at(const uint32_t* w, int e) { return (e & 1) ? bf16_hi_to_f32(w[e >> 1]) : bf16_lo_to_f32(w[e >> 1]); }

template <int C, int HALF, int U>
__global__ __launch_bounds__(256) void kv_append_kernel(KvAppendArgs a, RopeArgs q) {
    __shared__ float2 cs[16 * (kPairs + 2)];             // a token's pairs, rows apart by two more
    __shared__ __attribute__((aligned(16))) uint8_t turn[4][C][4 * 272];
    static_assert(sizeof cs >= sizeof(float2) * 4 * kMaxPairs, "the queries' angles fit");
    const int blocks = a.items * a.groups;
    if ((int)blockIdx.x >= blocks) {
        const int64_t b = (int)blockIdx.x - blocks;
        rope_axes_body<0, HALF, U, true>(q, b % a.qx, (int)(b / a.qx), (float2(*)[kMaxPairs])cs);
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
    for (int i = tid; i < (s1 - s0) * P; i += 256) {
        const int s = s0 + i / P, p = i - (s - s0) * P;
        int ax = a.axis[p];
        ax = ax < 0 ? 0 : ax >= a.axes ? a.axes - 1 : ax;
        const int bits = ((const int*)a.pos)[(t_at0 + s) * a.axes + ax];
        cs[s * pitch + p] = turn_of(a.pos_f32 ? (double)__int_as_float(bits) : (double)bits, a.turns[p]);
    }
    __syncthreads();

    const int key = lane >> 2, part = lane & 3;          // keys: the lane's token, its 16 channels of each 64
    const int quad = lane >> 4, j = lane & 15;           // values: its 4 tokens, its 4 channels of each 64
    const bool knew = key >= s0 && key < s1;
    uint32_t vnew = 0, vold = 0;                         // bytes of the quad's words from the call, from before
#pragma unroll
    for (int s = 0; s < 4; ++s) {
        const int slot = quad * 4 + s;
        vnew |= slot >= s0 && slot < s1 ? 0xffu << (8 * s) : 0u;
        vold |= slot < s0 ? 0xffu << (8 * s) : 0u;
    }
    const int D = a.c.D;
    const int hend = h0 + a.per < a.c.H ? h0 + a.per : a.c.H;
    for (int h = h0 + wave; h < hend; h += 4) {
        const int64_t at = ((int64_t)page * a.c.H + h) * a.c.tiles + tile;
        uint8_t* kd = a.c.data + at * (8 * C * 1024) + blk * C * 1024 + (part * 16 + key) * 16;
        uint8_t* vd = a.c.data + at * (8 * C * 1024) + (4 + blk) * C * 1024 + lane * 16;
        uint8_t* sc = a.c.scales + at * 8 + blk;
        // everything that the head needs, on its way
        uint4 kw[C][2], pw[C][2];
        uint2 vw[C][4];
        const uint16_t* kp = a.k + (t_at0 + key) * a.kts + h * a.khs;
#pragma unroll
        for (int c = 0; c < C; ++c) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int d = c * 64 + part * 16 + e * 8;
                kw[c][e] = pw[c][e] = make_uint4(0u, 0u, 0u, 0u);
                if (knew && d < D) kw[c][e] = *(const uint4*)(kp + d);
                if (HALF && knew) {                      // the other channels of their pairs, 4 at a time
                    const int o0 = d < P ? d + P : d - P, o1 = d + 4 < P ? d + 4 + P : d + 4 - P;
                    uint2 x = make_uint2(0u, 0u), y = x;
                    if (d < 2 * P) x = *(const uint2*)(kp + o0);
                    if (d + 4 < 2 * P) y = *(const uint2*)(kp + o1);
                    pw[c][e] = make_uint4(x.x, x.y, y.x, y.y);
                }
            }
#pragma unroll
            for (int s = 0; s < 4; ++s) {
                const int slot = quad * 4 + s, d = c * 64 + j * 4;
                vw[c][s] = make_uint2(0u, 0u);
                if (slot >= s0 && slot < s1 && d < D) vw[c][s] = *(const uint2*)(a.v + (t_at0 + slot) * a.vts + h * a.vhs + d);
            }
        }
        int ek0 = kKvExpMin, ev0 = kKvExpMin;
        if (s0 > 0) {
            ek0 = (int)sc[0] - 127;
            ev0 = (int)sc[4] - 127;
        }

        // ---- keys
        float r = 1.0f;
        if (a.norm) {
            float ss = 0.0f;
#pragma unroll
            for (int c = 0; c < C; ++c)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const uint32_t w[4] = {kw[c][e].x, kw[c][e].y, kw[c][e].z, kw[c][e].w};
#pragma unroll
                    for (int i = 0; i < 8; ++i) ss = __builtin_fmaf(bf16_at(w, i), bf16_at(w, i), ss);
                }
            ss += lane16_other<0>(ss);
            ss += lane16_other<1>(ss);
            r = __builtin_amdgcn_rsqf(__builtin_fmaf(ss, 1.0f / (float)D, a.eps));
        }
        float x[C][16], amax = 0.0f;
#pragma unroll
        for (int c = 0; c < C; ++c)
#pragma unroll
            for (int f = 0; f < 4; ++f) {                // 4 channels from d
                const int d = c * 64 + part * 16 + f * 4;
                const uint4 ow = kw[c][f >> 1], tw = pw[c][f >> 1];
                const uint32_t o[2] = {f & 1 ? ow.z : ow.x, f & 1 ? ow.w : ow.y};
                const uint32_t p[2] = {f & 1 ? tw.z : tw.x, f & 1 ? tw.w : tw.y};
                float own[4], other[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    own[i] = bf16_at(o, i);
                    other[i] = HALF ? bf16_at(p, i) : 0.0f;
                }
                const bool first_half = d < P, turned = d < 2 * P;
                if (a.norm && knew && d < D) {
                    const uint2 nw = *(const uint2*)(a.norm + d);
                    const uint32_t n[2] = {nw.x, nw.y};
#pragma unroll
                    for (int i = 0; i < 4; ++i) own[i] *= r * bf16_at(n, i);
                    if (HALF && turned) {
                        const uint2 mw = *(const uint2*)(a.norm + (first_half ? d + P : d - P));
                        const uint32_t m[2] = {mw.x, mw.y};
#pragma unroll
                        for (int i = 0; i < 4; ++i) other[i] *= r * bf16_at(m, i);
                    }
                }
                if (turned && knew) {
                    if constexpr (HALF) {
                        const int p0 = first_half ? d : d - P;
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const float2 t = cs[key * pitch + p0 + i];
                            own[i] = __builtin_fmaf(own[i], t.x, first_half ? -(other[i] * t.y) : other[i] * t.y);
                        }
                    } else {
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const float2 t = cs[key * pitch + d / 2 + i];
                            const float u = own[2 * i], v = own[2 * i + 1];
                            own[2 * i] = __builtin_fmaf(u, t.x, -(v * t.y));
                            own[2 * i + 1] = __builtin_fmaf(u, t.y, v * t.x);
                        }
                    }
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    x[c][f * 4 + i] = own[i];
                    amax = fmaxf(amax, finite_abs(own[i]));
                }
            }
        int e = kv_exponent(wave_max(amax));
        e = e < ek0 ? ek0 : e;
        if (lane == 0) sc[0] = (uint8_t)(e + 127);
        const float rk = exp2i(-e);
        const float fk = exp2i(ek0 - e < -126 ? -126 : ek0 - e);
#pragma unroll
        for (int c = 0; c < C; ++c) {
            if (key >= s0) {                             // the call's tokens; zeros past them
                uint32_t w[4];
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    w[i] = e4m3_x4(fit(x[c][4 * i], rk), fit(x[c][4 * i + 1], rk), fit(x[c][4 * i + 2], rk), fit(x[c][4 * i + 3], rk));
                *(uint4*)(kd + c * 1024) = make_uint4(w[0], w[1], w[2], w[3]);
            } else if (e != ek0) {
                *(uint4*)(kd + c * 1024) = rescale16(*(const uint4*)(kd + c * 1024), fk);
            }
        }

        // ---- values
        amax = 0.0f;
#pragma unroll
        for (int c = 0; c < C; ++c)
#pragma unroll
            for (int s = 0; s < 4; ++s) {
                const uint32_t w[2] = {vw[c][s].x, vw[c][s].y};
#pragma unroll
                for (int i = 0; i < 4; ++i) amax = fmaxf(amax, finite_abs(bf16_at(w, i)));
            }
        e = kv_exponent(wave_max(amax));
        e = e < ev0 ? ev0 : e;
        if (lane == 0) sc[4] = (uint8_t)(e + 127);
        const float rv = exp2i(-e);
        const float fv = exp2i(ev0 - e < -126 ? -126 : ev0 - e);
        __builtin_amdgcn_wave_barrier();
#pragma unroll
        for (int c = 0; c < C; ++c)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float t[4];
#pragma unroll
                for (int s = 0; s < 4; ++s) {
                    const uint32_t w[2] = {vw[c][s].x, vw[c][s].y};
                    t[s] = fit(bf16_at(w, i), rv);
                }
                // channel 64 c + 4 j + i: row 4 (j % 4) + i of the run, word j / 4
                *(uint32_t*)&turn[wave][c][quad * 272 + ((j & 3) * 4 + i) * 16 + (j >> 2) * 4] = e4m3_x4(t[0], t[1], t[2], t[3]);
            }
        __builtin_amdgcn_wave_barrier();
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
#pragma unroll
        for (int c = 0; c < C; ++c) {
            if (vold == ~0u && e == ev0) continue;       // four tokens from before, as they are
            uint4 w = *(const uint4*)&turn[wave][c][quad * 272 + j * 16];
            w = make_uint4(w.x & vnew, w.y & vnew, w.z & vnew, w.w & vnew);
            if (vold) {
                uint4 o = *(const uint4*)(vd + c * 1024);
                if (e != ev0) o = rescale16(o, fv);
                w = make_uint4(w.x | (o.x & vold), w.y | (o.y & vold), w.z | (o.z & vold), w.w | (o.w & vold));
            }
            *(uint4*)(vd + c * 1024) = w;
        }
        __builtin_amdgcn_wave_barrier();
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
    // Four heads a workgroup, one a wave; more, which share the angles, once there are four
    // workgroups a CU without.
    a.per = 4;
    while (a.per < a.c.H && (int64_t)a.items * ((a.c.H + 2 * a.per - 1) / (2 * a.per)) >= 4 * (int64_t)cus) a.per *= 2;
    a.groups = (a.c.H + a.per - 1) / a.per;
    switch ((a.c.D + 63) / 64) {
        case 1: return launch<1>(a, q, half, cus, stream);
        case 2: return launch<2>(a, q, half, cus, stream);
        case 3: return launch<3>(a, q, half, cus, stream);
        default: return launch<4>(a, q, half, cus, stream);
    }
}
