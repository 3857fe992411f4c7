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
#include "rope_body.h"

namespace {

template <int F32, int HALF, int U, bool EDGES>
__global__ __launch_bounds__(256) void rope_axes_kernel(RopeArgs a) {
    __shared__ float2 cs[4][kMaxPairs];
    rope_axes_body<F32, HALF, U, EDGES>(a, blockIdx.x, blockIdx.y, cs);
}

template <int F32, int HALF, int U, bool EDGES>
void run(const RopeArgs& a, dim3 grid, hipStream_t stream) {
    hipLaunchKernelGGL((rope_axes_kernel<F32, HALF, U, EDGES>), grid, dim3(256), 0, stream, a);
}

}  // namespace

template <int U>
static hipError_t launch(RopeArgs a, int f32, int half, int cus, hipStream_t stream) {
    int64_t gx, gy;
    rope_shares(a, U, cus, gx, gy);
    const dim3 grid((unsigned)gx, (unsigned)gy);
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
