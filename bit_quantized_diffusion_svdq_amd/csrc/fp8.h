// bf16 values to E4M3 codes with one fp32 scale per block of 128, bit by bit
// the same wherever it is done (the activation pass, the few-rows layer, the
// weights).
//
// Per block: amax = max |v| over its finite values; s = max(amax / 448,
// 2^-120) (the fp32 quotient; 448 is the largest E4M3 value, and the floor
// keeps 1 / s finite, so a block of zeros has zero codes without a branch);
// code = e4m3(clamp(v * fp32(1 / s), -448, 448)), nearest, ties to even.
// Infinities saturate at +-448, a NaN keeps a NaN code (0x7f).
#pragma once
#include "lanes.h"

constexpr float kE4m3Max = 448.0f;
constexpr float kScaleMin = 7.52316384526264e-37f;      // 2^-120

// |v| where v is finite, else 0: infinities and NaN leave the scale to the
// block's other values
DEV float finite_abs(float v) {
    const float a = fabsf(v);
    return a < __builtin_inff() ? a : 0.0f;
}

// max(amax / 448, 2^-120), the quotient rounded correctly: a first one from
// the rounded reciprocal, then its exact remainder (fma) brought back in.
// (Quotients small enough for the remainder to lose bits are below 2^-120.)
DEV float block_scale(float amax) {
    const float inv = 1.0f / kE4m3Max;
    const float q = amax * inv;
    return fmaxf(__builtin_fmaf(__builtin_fmaf(-q, kE4m3Max, amax), inv, q), kScaleMin);
}

// 1 / s rounded correctly (s in [2^-120, 2^120], no step leaves the normal
// numbers): two Newton steps on the hardware reciprocal, each remainder exact.
DEV float reciprocal(float s) {
    float y = __builtin_amdgcn_rcpf(s);
    y = __builtin_fmaf(__builtin_fmaf(-s, y, 1.0f), y, y);
    return __builtin_fmaf(__builtin_fmaf(-s, y, 1.0f), y, y);
}

// four values to four E4M3 bytes (the conversion rounds to nearest even)
DEV uint32_t e4m3_x4(float a, float b, float c, float d) {
    int w = 0;
    w = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, w, false);
    w = __builtin_amdgcn_cvt_pk_fp8_f32(c, d, w, true);
    return (uint32_t)w;
}

// Eight bf16 values times r to eight codes. FINITE: none is an infinity or a
// NaN, so the clamp (against a product rounded past 448) need not keep NaN.
template <bool FINITE>
DEV uint2 codes8(const uint32_t (&w)[4], float r) {
    float t[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const float v = ((e & 1) ? bf16_hi_to_f32(w[e >> 1]) : bf16_lo_to_f32(w[e >> 1])) * r;
        const float c = __builtin_amdgcn_fmed3f(v, -kE4m3Max, kE4m3Max);
        t[e] = FINITE || v == v ? c : v;
    }
    return make_uint2(e4m3_x4(t[0], t[1], t[2], t[3]), e4m3_x4(t[4], t[5], t[6], t[7]));
}

typedef unsigned short v2u16 __attribute__((ext_vector_type(2)));

// the larger of two magnitudes in each half (bf16 without sign: ordered as integers)
DEV uint32_t max_u16x2(uint32_t a, uint32_t b) {
    return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(v2u16, a), __builtin_bit_cast(v2u16, b)));
}

// A block of 128 values held by 16 lanes (8 each): its scale and the lane's
// eight codes. All 16 lanes take part.
DEV uint2 block_codes(const uint4& v, float& s) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    const uint32_t m = max_u16x2(max_u16x2(w[0] & 0x7fff7fffu, w[1] & 0x7fff7fffu),
                                 max_u16x2(w[2] & 0x7fff7fffu, w[3] & 0x7fff7fffu));
    float amax = __uint_as_float((m >> 16 > (m & 0xffffu) ? m >> 16 : m & 0xffffu) << 16);
    // an infinity or a NaN in the wave: the maximum of the others, value by value
    const bool finite = __ballot(!(amax < __builtin_inff())) == 0;
    if (!finite) {
        amax = 0.0f;
#pragma unroll
        for (int e = 0; e < 4; ++e)
            amax = fmaxf(amax, fmaxf(finite_abs(bf16_lo_to_f32(w[e])), finite_abs(bf16_hi_to_f32(w[e]))));
    }
    amax = fmaxf(amax, lane16_other<0>(amax));
    amax = fmaxf(amax, lane16_other<1>(amax));
    amax = fmaxf(amax, lane16_other<2>(amax));
    amax = fmaxf(amax, lane16_other<3>(amax));
    s = block_scale(amax);
    const float r = reciprocal(s);
    return finite ? codes8<true>(w, r) : codes8<false>(w, r);
}
