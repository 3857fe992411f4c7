// Arguments of the rotary kernel (rope.hip), filled by the C ABI's host side.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

struct RopeArgs {
    const void* x[2];               // q, k (k NULL: no keys)
    void* y[2];
    const void* norm[2];            // [D] or NULL
    int64_t ts[2], hs[2], yts[2], yhs[2];
    int heads[2];
    const void* pos;
    const double* turns;            // [pairs] turns per unit of position
    const int* axis;                // [pairs]
    int64_t T;
    int D, pairs, axes, pos_f32, inverse;
    float eps;
    int lp, chunk;                  // lanes per head (a power of two), loads of heads per wave
    const int* offs;                // rows in groups: [groups + 1] row offsets, else NULL
    int groups;
};

// Lanes per head, and how a token's loads are shared: a wave takes all of its
// token's heads where the tokens fill the chip (12 waves a CU), else a share of
// them, U loads at the least, and works the angles out again (1024 tokens of 24 +
// 24 heads of 128 take 7.3 us in three waves a token, 7.9 in two, 10.7 in one;
// 32761 of 16 + 4 69 in two and 64.3 in one). Returns the workgroups: x * y.
static inline void rope_shares(RopeArgs& a, int U, int cus, int64_t& x, int64_t& y) {
    a.lp = 1;
    while (a.lp * 8 < a.D) a.lp *= 2;
    const int per = 64 / a.lp, loads = (a.heads[0] + per - 1) / per + (a.heads[1] + per - 1) / per;
    int64_t chunks = ((int64_t)cus * 12 + a.T - 1) / a.T;
    if (chunks > (loads + U - 1) / U) chunks = (loads + U - 1) / U;
    a.chunk = (int)((loads + chunks - 1) / chunks);
    x = (a.T + 3) / 4;
    y = (loads + a.chunk - 1) / a.chunk;
}

hipError_t launch_rope_axes(RopeArgs a, int f32, int half, int cus, hipStream_t stream);
