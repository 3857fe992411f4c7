// svdq_quantize_act_fp8 / svdq_quantize_weight_fp8: bf16 values to E4M3 codes
// with one fp32 scale per block of 128 (activations: 128 channels of a row;
// weights: 128 output x 128 input channels).
//
// The activation pass is bound by memory: 2 bytes in and 1 byte out per value
// (plus 4 bytes per 128). A wave takes four blocks of a row at a time (16
// lanes and 16 bytes per lane each: 1 KB contiguous) and walks `rpw`
// consecutive rows two at a time, so the scales of its rows, which are stored
// block-major ([ceil(K / 128)][M]), leave as one contiguous run per block.
// Maxima are taken on the bf16 bits, two at a time, and across lanes without
// LDS. 4608 x 12288 takes 29.5 us, 5.8 TB/s with what the last-level cache
// keeps of the output (a plain copy: 5.5).
#include "fp8.h"

namespace {

// rows in flight per wave: few registers, many waves (with 8, 512 x 4096 took 4.2 us instead
// of 3.6, 64 x 4096 2.9 instead of 2.5; with 1, 4608 x 4096 13.3 instead of 12.4)
constexpr int UNROLL = 2;

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
                float s;
                const uint2 o = block_codes(v[u], s);
                if (r0 + u == l16) mine = s;
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
    // few rows a wave fill the chip sooner, more make fewer and longer runs of scales (1, 2, 4,
    // 8 rows: 512 x 4096 3.6, 3.8, 4.4, 5.9 us; 1024 x 4096 4.8, 4.6, 4.9, 6.3; 1024 x 12288
    // 10.2, 9.7, 9.0, 9.7; 4608 x 4096 13.7, 12.8, 12.4, 12.0)
    const int64_t waves = M * QB;
    const int rpw = waves > (int64_t)cus * 48 ? 4 : waves > (int64_t)cus * 16 ? 2 : 1;
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
