// svdq_quantize_act_fp8 / svdq_quantize_weight_fp8: bf16 values to E4M3 codes
// with one fp32 scale per block of 128 (activations: 128 channels of a row;
// weights: 128 output x 128 input channels).
//
// Per block: amax = max |v| over its finite values; s = max(amax / 448,
// 2^-120) (the fp32 quotient; 448 is the largest E4M3 value, and the floor
// keeps 1 / s finite, so a block of zeros has zero codes without a branch);
// code = e4m3(clamp(v * fp32(1 / s), -448, 448)), nearest, ties to even.
// Infinities saturate at +-448, a NaN keeps a NaN code (0x7f).
//
// The activation pass is bound by memory: 2 bytes in and 1 byte out per value
// (plus 4 bytes per 128). A wave takes four blocks of a row at a time (16
// lanes and 16 bytes per lane each: 1 KB contiguous) and walks `rpw`
// consecutive rows with eight rows' loads in flight, so the scales of its
// rows, which are stored block-major ([ceil(K / 128)][M]), leave as one
// contiguous run per block instead of one 4-byte store per row. Maxima are
// taken on the bf16 bits, two at a time, and across lanes without LDS; with
// that 4608 x 12288 went from 37.4 to 34.6 us, 4.9 TB/s (a plain copy: 5.5).
#include "lanes.h"

namespace {

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

constexpr int UNROLL = 8;                               // rows in flight per wave

__global__ __launch_bounds__(256) void quant_act_fp8_kernel(const uint16_t* __restrict__ x, int64_t M, int K,
                                                            int64_t ldx, int rpw, uint8_t* __restrict__ qx,
                                                            float* __restrict__ sx) {
    const int lane = threadIdx.x & 63, sub = lane >> 4, l16 = lane & 15;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int KB = (K + 127) / 128, QB = (KB + 3) / 4;   // blocks, quads of blocks
    const int64_t item = (int64_t)blockIdx.x * 4 + wave;
    const int64_t rg = item / QB;
    const int kb = (int)(item - rg * QB) * 4 + sub;
    const int64_t m0 = rg * rpw;
    if (m0 >= M) return;
    const int rows = (int)((M - m0) < rpw ? (M - m0) : rpw);
    const int k = kb * 128 + l16 * 8;
    const bool in = k < K;                              // K is a multiple of 16
    const uint16_t* xp = x + m0 * ldx + k;
    uint8_t* qp = qx + m0 * K + k;
    float mine = 0.0f;
    for (int r0 = 0; r0 < rows; r0 += UNROLL) {
        uint4 v[UNROLL];
#pragma unroll
        for (int u = 0; u < UNROLL; ++u) {
            v[u] = make_uint4(0u, 0u, 0u, 0u);
            if (in && r0 + u < rows) v[u] = *(const uint4*)(xp + (int64_t)(r0 + u) * ldx);
        }
#pragma unroll
        for (int u = 0; u < UNROLL; ++u) {
            if (r0 + u < rows) {
                const uint32_t w[4] = {v[u].x, v[u].y, v[u].z, v[u].w};
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
                const float s = block_scale(amax), r = reciprocal(s);
                const uint2 o = finite ? codes8<true>(w, r) : codes8<false>(w, r);
                if (((r0 + u) & 15) == l16) mine = s;
                if (in) *(uint2*)(qp + (int64_t)(r0 + u) * K) = o;
            }
        }
    }
    if (l16 < rows && kb < KB) sx[(int64_t)kb * M + m0 + l16] = mine;
}

// One workgroup per 128 x 128 block of W [K][N]: 16 lanes read 8 consecutive
// outputs of an input row, the block's maximum meets in LDS, and the codes
// are turned through LDS so that qw [N][K] is written 16 input channels at a
// time. Offline work: one pass over the weight.
__global__ __launch_bounds__(256) void quant_weight_fp8_kernel(const uint16_t* __restrict__ w, int64_t K, int64_t N,
                                                               int64_t ldw, uint8_t* __restrict__ qw,
                                                               float* __restrict__ sw) {
    __shared__ __attribute__((aligned(16))) uint8_t tile[128][144];   // [n][k], rows padded by 16 bytes
    __shared__ float red[4];
    const int tid = threadIdx.x, c = tid & 15, r = tid >> 4;
    const int64_t k0 = (int64_t)blockIdx.x * 128, n0 = (int64_t)blockIdx.y * 128;
    const int64_t KB = (K + 127) / 128;
    const int64_t n = n0 + c * 8;
    uint4 v[8];
    float amax = 0.0f;
#pragma unroll
    for (int p = 0; p < 8; ++p) {
        const int64_t k = k0 + p * 16 + r;
        v[p] = make_uint4(0u, 0u, 0u, 0u);
        if (k < K && n + 8 <= N) {
            v[p] = *(const uint4*)(w + k * ldw + n);
        } else if (k < K && n < N) {
            uint32_t t[4] = {0u, 0u, 0u, 0u};
            for (int e = 0; e < (int)(N - n); ++e) t[e >> 1] |= (uint32_t)w[k * ldw + n + e] << (16 * (e & 1));
            v[p] = make_uint4(t[0], t[1], t[2], t[3]);
        }
        const uint32_t t[4] = {v[p].x, v[p].y, v[p].z, v[p].w};
#pragma unroll
        for (int e = 0; e < 4; ++e)
            amax = fmaxf(amax, fmaxf(finite_abs(bf16_lo_to_f32(t[e])), finite_abs(bf16_hi_to_f32(t[e]))));
    }
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) amax = fmaxf(amax, __shfl_xor(amax, d));
    if ((tid & 63) == 0) red[tid >> 6] = amax;
    __syncthreads();
    const float s = block_scale(fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3]))), inv = reciprocal(s);
#pragma unroll
    for (int p = 0; p < 8; ++p) {
        const uint32_t t[4] = {v[p].x, v[p].y, v[p].z, v[p].w};
        const uint2 q = codes8<false>(t, inv);
#pragma unroll
        for (int e = 0; e < 8; ++e) tile[c * 8 + e][p * 16 + r] = (uint8_t)((e < 4 ? q.x : q.y) >> (8 * (e & 3)));
    }
    if (tid == 0) sw[(int64_t)blockIdx.y * KB + blockIdx.x] = s;
    __syncthreads();
#pragma unroll
    for (int p = 0; p < 4; ++p) {
        const int row = p * 32 + (tid >> 3), kc = (tid & 7) * 16;
        if (n0 + row < N && k0 + kc < K) *(uint4*)(qw + (n0 + row) * K + k0 + kc) = *(const uint4*)(&tile[row][kc]);
    }
}

}  // namespace

hipError_t launch_quant_act_fp8(const uint16_t* x, int64_t M, int64_t K, int64_t ldx, uint8_t* qx, float* sx, int cus,
                                hipStream_t stream) {
    const int64_t QB = (K + 511) / 512;
    // 16 rows per wave once that leaves every SIMD two waves (4608 x 4096: 12.9 us); fewer rows
    // fill the chip sooner (512 x 4096: 4.6 us with 4)
    const int rpw = (M + 15) / 16 * QB >= (int64_t)cus * 8 ? 16 : (M + 3) / 4 * QB >= (int64_t)cus * 8 ? 4 : 1;
    const int64_t items = (M + rpw - 1) / rpw * QB;
    hipLaunchKernelGGL(quant_act_fp8_kernel, dim3((unsigned)((items + 3) / 4)), dim3(256), 0, stream, x, M, (int)K, ldx,
                       rpw, qx, sx);
    return hipGetLastError();
}

hipError_t launch_quant_weight_fp8(const uint16_t* w, int64_t K, int64_t N, int64_t ldw, uint8_t* qw, float* sw,
                                   hipStream_t stream) {
    hipLaunchKernelGGL(quant_weight_fp8_kernel, dim3((unsigned)((K + 127) / 128), (unsigned)((N + 127) / 128)),
                       dim3(256), 0, stream, w, K, N, ldw, qw, sw);
    return hipGetLastError();
}
