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

hipError_t launch_rope_axes(RopeArgs a, int f32, int half, int cus, hipStream_t stream);
