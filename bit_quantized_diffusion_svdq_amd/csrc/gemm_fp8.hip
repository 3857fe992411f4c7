// svdq_gemm_fp8, svdq_linear_fp8 and their grouped forms: E4M3 x E4M3 products with one fp32
// scale per block of 128 input channels,
//
//   Y[m, n] = act( sum_b sx[b, m] sw[n / 128, b] P_b[m, n] + bias[n] ),
//   P_b[m, n] = sum_{k in block b} qx[m, k] qw[n, k],
//
// dense or grouped (rows offs[g] .. offs[g + 1] meet weight g).
//
//  - One v_mfma_f32_16x16x128_f8f6f4 forms P_b of a 16 x 16 tile from a zero
//    accumulator; its four results per lane then join the fp32 sums with one
//    FMA each. The weights are the MFMA's row operand and the activations its
//    column operand, so a lane's four results belong to one row m and take
//    one scale, sx[b, m] sw[.., b], which a wave forms once per 16 rows.
//  - Block scales are fp32 with a mantissa, so they cannot ride on the matrix
//    pipe's E8M0 scales: the FMAs (4 of 64 lanes, 16 cycles of a SIMD) run
//    beside the MFMAs (32 cycles).
#include "fp8.h"

namespace {

typedef __attribute__((address_space(3))) void lds_void;

// byte offset past any buffer: a load there returns 0. (The range check takes
// the lane's and the wave's offset together, and their sum stays below 2^32:
// checked on gfx950 for loads into registers and into LDS.)
constexpr int kBeyond = 0x7ffffff0;

// D = A(16x128) * B(128x16) from zero, both E4M3: lane l holds 32 bytes of
// row (column) l % 16; which 32 of the 128 channels is free as long as both
// operands agree. D: column l % 16, rows 4 (l / 16) + 0..3.
DEV v4f mfma_fp8_16x16x128(const v8i& a, const v8i& b) {
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, v4f{0.0f, 0.0f, 0.0f, 0.0f}, 0, 0, 0, 0, 0, 0);
}

// An operand of a 16-row block and 128 channels: lane l holds 32 E4M3 bytes of
// row l % 16.
//
// PREC 0 keeps them for v_mfma_f32_16x16x128_f8f6f4. That instruction (as every
// E4M3 form of the matrix pipe) adds 8 products at a time after shifting them
// to the largest one's exponent, and drops what falls more than 13 bits below
// it; groups of 8 and the accumulator meet in fp32. The loss is at most
// 7 x 2^-13 of the largest product of each 8. Measured at K = 4096 and 12288 it
// has no bias and 1.4e-5 of the outputs' rms for normal operands, 3.1e-5 with 1 %
// of the channels 20 times as loud, and adds 0.02 % to what rounding to bf16
// leaves (1.658e-3). It is of one size for all outputs: those that cancel to
// under a twentieth of the median magnitude are 2.0e-3 off in the median
// (1.4e-3 by rounding alone), 7 % of them by more than a hundredth. Taken for
// bf16 outputs: sums in fp32 would halve the rate (4608 x 12288 x 4096 takes 426
// us instead of 211), beside operands that carry 4 significant bits.
//
// PREC 1 widens them to bf16 (exact) for v_mfma_f32_16x16x32_bf16, whose
// products and sums keep fp32: half the matrix rate, taken for fp32 outputs.
template <int PREC>
struct Frag;

template <>
struct Frag<0> {
    v8i v;
    DEV void set(const uint4& lo, const uint4& hi) {
        v = v8i{(int)lo.x, (int)lo.y, (int)lo.z, (int)lo.w, (int)hi.x, (int)hi.y, (int)hi.z, (int)hi.w};
    }
    static DEV v4f dot(const Frag& a, const Frag& b) { return mfma_fp8_16x16x128(a.v, b.v); }
};

typedef __bf16 v2bf __attribute__((ext_vector_type(2)));

template <>
struct Frag<1> {
    v8bf v[4];
    static DEV v8bf widen(uint32_t lo, uint32_t hi) {
        const v2bf a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((int)lo, 1.0f, false);
        const v2bf b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((int)lo, 1.0f, true);
        const v2bf c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((int)hi, 1.0f, false);
        const v2bf d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((int)hi, 1.0f, true);
        return v8bf{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
    }
    DEV void set(const uint4& lo, const uint4& hi) {
        v[0] = widen(lo.x, lo.y);
        v[1] = widen(lo.z, lo.w);
        v[2] = widen(hi.x, hi.y);
        v[3] = widen(hi.z, hi.w);
    }
    static DEV v4f dot(const Frag& a, const Frag& b) {
        v4f p = v4f{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int k = 0; k < 4; ++k) p = mfma_bf16_16x16x32(a.v[k], b.v[k], p);
        return p;
    }
};

// Workgroup -> tile of a dense product. Workgroup b runs on XCD b % 8 (dealt
// round-robin); each XCD takes a contiguous run of tiles, walked in bands of
// `band` tile rows, column by column, so the tiles in flight on an XCD share
// few rows of X and of W in its L2.
DEV void tile_coords(int b, int tiles_m, int tiles_n, int& tm, int& tn) {
    const int T = tiles_m * tiles_n, q = T >> 3, r = T & 7, x = b & 7;
    const int t = x * q + (x < r ? x : r) + (b >> 3);
    constexpr int band = 8;
    const int per = band * tiles_n, g = t / per, first = g * band;
    const int rows = tiles_m - first < band ? tiles_m - first : band;
    tm = first + (t - g * per) % rows;
    tn = (t - g * per) / rows;
}

// acc += p * s in the two-address form, which issues faster than the
// three-address one the compiler picks here. (The compiler does not see an
// MFMA result's read in it: callers put other MFMAs in between.)
DEV void fmac(v4f& acc, const v4f& p, float s) {
#pragma unroll
    for (int e = 0; e < 4; ++e) asm volatile("v_fmac_f32_e32 %0, %1, %2" : "+v"(acc[e]) : "v"(p[e]), "v"(s));
}

struct Args {
    const uint8_t* qx;
    const float* sx;
    const uint8_t* qw;
    const float* sw;
    const uint16_t* bias;
    void* y;
    const int* offs;                // grouped: [E + 1] row offsets, else NULL
    int64_t M, ldy;
    int N, K, E;
    int act, y_f32, vec;            // vec: rows of y take 16-byte stores
    const uint16_t* x;              // the layer of few rows: bf16 activations (qx, sx NULL), else NULL
    int64_t ldx;
};

// The rows a workgroup works on: m0 .. m0 + rows - 1 of group g (rows 0: none)
struct Rows {
    int64_t m0;
    int rows, g;
};

// Row tile `mt` of `bm` rows in the ragged groups, found by every wave on its
// own: 64 groups at a time, their tile counts are summed along the lanes.
// Offsets are clamped into [0, M], and one that falls counts as the largest
// before it: bad offsets lead nowhere outside the arrays, no row belongs to
// two groups (two workgroups would write it), and the tiles stay within the
// launch's. Returns the number of tiles in *total.
DEV Rows group_rows(const Args& a, int mt, int bm, int* total) {
    const int lane = threadIdx.x & 63;
    Rows r{0, 0, 0};
    int before = 0;
    int done = 0;                                        // the largest offset so far (M < 2^31)
    for (int g0 = 0; g0 < a.E; g0 += 64) {
        const int g = g0 + lane;
        int64_t lo = 0, hi = 0;
        if (g < a.E) {
            lo = a.offs[g];
            hi = a.offs[g + 1];
            lo = lo < 0 ? 0 : lo > a.M ? a.M : lo;
            hi = hi < 0 ? 0 : hi > a.M ? a.M : hi;
        }
        if (__builtin_amdgcn_readfirstlane((int)lo) < done || __ballot(hi < lo)) {
            // somewhere they fall: each becomes the largest up to it (never with good offsets)
            int top = (int)lo > done ? (int)lo : done;
#pragma unroll
            for (int d = 1; d < 64; d <<= 1) {
                const int o = __shfl_up(top, d);
                if (lane >= d && o > top) top = o;
            }
            lo = top;
            hi = hi < lo ? lo : hi;
        }
        done = __builtin_amdgcn_readlane((int)hi, 63);   // (nobody asks after the last 64)
        const int cnt = (int)((hi - lo + bm - 1) / bm);
        int inc = cnt;
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            const int o = __shfl_up(inc, d);
            if (lane >= d) inc += o;
        }
        const int start = before + inc - cnt;
        const unsigned long long hit = __ballot(mt >= start && mt < start + cnt);
        if (hit) {
            const int src = __builtin_ctzll(hit);
            const int64_t m0 = lo + (int64_t)(mt - start) * bm;
            const int64_t left = hi - m0;
            r.m0 = __shfl(m0, src);
            r.rows = __shfl((int)(left < bm ? left : bm), src);
            r.g = g0 + src;
        }
        before += __shfl(inc, 63);
    }
    r.m0 = ((int64_t)__builtin_amdgcn_readfirstlane((int)(r.m0 >> 32)) << 32) |
           (uint32_t)__builtin_amdgcn_readfirstlane((int)r.m0);
    r.rows = __builtin_amdgcn_readfirstlane(r.rows);
    r.g = __builtin_amdgcn_readfirstlane(r.g);
    *total = __builtin_amdgcn_readfirstlane(before);
    return r;
}

DEV float finish(float v, float b, int act) {
    v += b;
    return act ? gelu_tanh_f32(v) : v;
}

// one output element
DEV void store1(const Args& a, int64_t row, int col, float v) {
    if (a.y_f32) ((float*)a.y)[row * a.ldy + col] = v;
    else ((uint16_t*)a.y)[row * a.ldy + col] = f32_to_bf16_bits(v);
}

// four consecutive outputs of one row
DEV void store4(const Args& a, int64_t row, int col, const float* v) {
    if (a.vec && col + 4 <= a.N) {
        if (a.y_f32) *(float4*)((float*)a.y + row * a.ldy + col) = make_float4(v[0], v[1], v[2], v[3]);
        else *(uint2*)((uint16_t*)a.y + row * a.ldy + col) = make_uint2(bf16x2(v[0], v[1]), bf16x2(v[2], v[3]));
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (col + e < a.N) store1(a, row, col + e, v[e]);
    }
}

// ---------------------------------------------------------------- tiles

// BM x BN outputs per workgroup, WGM x WGN waves of (16 TM) x (16 TN) each, S
// slots (blocks of K in LDS or on their way). PREC 0: E4M3 matrix
// instructions, 1: exact products on the bf16 ones. WPE: waves per SIMD the
// registers are kept for. MID: where W's slot is given back (see block()).
template <int TM_, int TN_, int WGM_, int WGN_, int WPE_, int PREC_, int MID_, int S_>
struct Cfg {
    static constexpr int TM = TM_, TN = TN_, WGM = WGM_, WGN = WGN_, WPE = WPE_, PREC = PREC_, MID = MID_, S = S_;
    static constexpr int BM = 16 * TM * WGM, BN = 16 * TN * WGN;
    static constexpr int NW = WGM * WGN, NT = 64 * NW;
    static constexpr int XL = BM / 8, WL = BN / 8;                // 8-row loads per block of K
    static constexpr int XP = (XL + NW - 1) / NW, WP = (WL + NW - 1) / NW, SP = (BM + 63) / 64;
    static_assert(128 % (TN * 16) == 0, "a wave's outputs share one weight scale");
    static_assert(NW % 2 == 0, "a wave's loads have one parity");
    static_assert(SP <= NW, "one load of 64 row scales per wave");
    static constexpr int XSLOT = BM * 128 + SP * 256, WSLOT = BN * 128;
    static_assert(S >= 2 && S <= 4 && S * (XSLOT + WSLOT) * WPE * 4 / NW <= 160 * 1024, "LDS budget");
};

DEV void dma16(rsrc_t r, char* lds, int voff, int soff) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_void*)lds, 16, voff, soff, 0, 0);
}
DEV void dma4(rsrc_t r, char* lds, int voff, int soff) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_void*)lds, 4, voff, soff, 0, 0);
}

template <class C, bool GROUPED>
__global__ __launch_bounds__(C::NT, C::WPE) void gemm_fp8_kernel(Args a) {
    constexpr int BM = C::BM, BN = C::BN, TM = C::TM, TN = C::TN, NW = C::NW;
    // S slots of X's rows and row scales and S of W's rows, each a block of K;
    // separate objects, so that the compiler waits only for loads into the one
    // it reads
    constexpr int S = C::S, XB = C::XSLOT, WB = C::WSLOT;
    __shared__ __attribute__((aligned(16))) char xs0[XB], xs1[XB], xs2[S > 2 ? XB : 16], xs3[S > 3 ? XB : 16];
    __shared__ __attribute__((aligned(16))) char ws0[WB], ws1[WB], ws2[S > 2 ? WB : 16], ws3[S > 3 ? WB : 16];
    const int tid = threadIdx.x, lane = tid & 63, l16 = lane & 15, q4 = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave / C::WGN, wn = wave % C::WGN;
    auto xslot = [&](int s) __attribute__((always_inline)) {
        return s % S == 0 ? xs0 : s % S == 1 ? xs1 : s % S == 2 ? xs2 : xs3;
    };
    auto wslot = [&](int s) __attribute__((always_inline)) {
        return s % S == 0 ? ws0 : s % S == 1 ? ws1 : s % S == 2 ? ws2 : ws3;
    };
    const int tiles_n = (a.N + BN - 1) / BN;
    Rows rr;
    int tn;
    if constexpr (GROUPED) {
        const int t = blockIdx.x;
        int total;
        rr = group_rows(a, t / tiles_n, BM, &total);
        if (t / tiles_n >= total) return;
        tn = t % tiles_n;
    } else {
        const int tiles_m = (int)((a.M + BM - 1) / BM);
        int tm;
        tile_coords(blockIdx.x, tiles_m, tiles_n, tm, tn);
        rr.m0 = (int64_t)tm * BM;
        rr.rows = (int)((a.M - rr.m0) < BM ? (a.M - rr.m0) : BM);
        rr.g = 0;
    }
    const int n0 = tn * BN;
    const int K = a.K, KB = (K + 127) / 128, NB = (a.N + 127) / 128;
    const uint8_t* qw = a.qw + (int64_t)rr.g * a.N * K;
    const int nrows = a.N - n0 < BN ? a.N - n0 : BN;
    const rsrc_t rx = make_rsrc(a.qx + rr.m0 * K, (int64_t)rr.rows * K);
    const rsrc_t rw = make_rsrc(qw + (int64_t)n0 * K, (int64_t)nrows * K);

    // ---- loads into LDS: instruction p brings rows 8 p .. 8 p + 7 of a tile,
    // lane l the row l / 8 and the 16-byte chunk (l % 8) ^ f, f = (row / 2) % 8,
    // so chunk c of row r lands at 128 r + 16 (c ^ f(r)) and the MFMA's reads
    // find no bank conflicts. Instructions are dealt to the waves in turn
    // (p = wave, wave + NW, ...). Rows past the end and channels past K read 0.
    const int lr8 = lane >> 3;
    const int c_even = 16 * ((lane & 7) ^ (lr8 >> 1));             // byte of the chunk, even p
    const int cme = (wave & 1) ? c_even ^ 64 : c_even;             // NW is even: a wave's p have one parity
    const int vx = (wave * 8 + lr8) * K + cme;                     // step NW rows of 8: + 8 NW K
    // Loads of a block: XN of X's rows (the last: the row scales) and WP of
    // W's. A wave without a load in the last round repeats its first (the same
    // bytes to the same place), and waves past the row scales repeat those: no
    // branches.
    constexpr int XN = C::XP + 1;
    auto load_x = [&](char* xs, int kb, int d) __attribute__((always_inline)) {
        if (d < C::XP) {
            const int p = C::XL % NW == 0 || wave + d * NW < C::XL ? d : 0;
            dma16(rx, xs + (wave + p * NW) * 1024, kb * 128 + cme < K ? vx : kBeyond, kb * 128 + p * (8 * NW) * K);
        } else {
            const rsrc_t rs = make_rsrc(a.sx + (int64_t)kb * a.M + rr.m0, kb < KB ? (int64_t)rr.rows * 4 : 0);
            dma4(rs, xs + BM * 128 + (wave % C::SP) * 256, (wave % C::SP) * 256 + lane * 4, 0);
        }
    };
    auto load_w = [&](char* ws, int kb, int d) __attribute__((always_inline)) {
        const int p = C::WL % NW == 0 || wave + d * NW < C::WL ? d : 0;
        dma16(rw, ws + (wave + p * NW) * 1024, kb * 128 + cme < K ? vx : kBeyond, kb * 128 + p * (8 * NW) * K);
    };

    // the weight's scales of the wave's outputs, 64 blocks of K at a time, one per lane
    const int nb = (n0 + wn * TN * 16) / 128;
    const float* swp = a.sw + ((int64_t)rr.g * NB + (nb < NB ? nb : NB - 1)) * KB;
    float sw64 = 0.0f;
    int sw0 = 0;                                                   // the block of lane 0
    auto load_sw = [&](int kb) __attribute__((always_inline)) {
        sw0 = kb;
        sw64 = kb + lane < KB ? swp[kb + lane] : 0.0f;
        order_point(sw64);           // waited for here, not among the loads in flight later
    };

    // the sums start at the bias (its loads hide behind the first block's)
    v4f acc[TM][TN];
    const rsrc_t rb = make_rsrc(a.bias ? a.bias + (int64_t)rr.g * a.N : nullptr, a.bias ? (int64_t)a.N * 2 : 0);
#pragma unroll
    for (int j = 0; j < TN; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int col = n0 + wn * TN * 16 + j * 16 + q4 * 4 + e;
            acc[0][j][e] = bf16_lo_to_f32((uint16_t)__builtin_amdgcn_raw_buffer_load_b16(rb, col * 2, 0, 0));
        }
#pragma unroll
    for (int i = 1; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < TN; ++j) acc[i][j] = acc[0][j];

    // ---- operands: the lane's chunks q4 and q4 + 4 of its row in each 16-row block
    const int xo0 = (wm * TM * 16 + l16) * 128 + 16 * (q4 ^ ((l16 >> 1) & 7));
    const int wo0 = (wn * TN * 16 + l16) * 128 + 16 * (q4 ^ ((l16 >> 1) & 7));
    const int so0 = BM * 128 + wm * TM * 64 + l16 * 4;
    Frag<C::PREC> wf[TN], xf[2];
    float sx[2];
    auto read_x = [&](const char* xs, int i, int par) __attribute__((always_inline)) {
        xf[par].set(*(const uint4*)(xs + i * 2048 + xo0), *(const uint4*)(xs + i * 2048 + (xo0 ^ 64)));
        sx[par] = *(const float*)(xs + so0 + i * 64);
    };
    auto read_w = [&](const char* ws, int j) __attribute__((always_inline)) {
        wf[j].set(*(const uint4*)(ws + j * 2048 + wo0), *(const uint4*)(ws + j * 2048 + (wo0 ^ 64)));
    };

    // Block kb, whose W operands and first X operand are in registers. Each
    // MFMA is followed by the four FMAs that add the product of the same
    // columns 16 rows earlier (the last block's last rows for the first),
    // which is complete by then: alternating like this, the vector work runs
    // in the matrix pipe's shadow (an MFMA and its four FMAs take 14.1 ns of a
    // SIMD with two waves, the MFMA alone 14.3, while four MFMAs and then
    // sixteen FMAs take 16.6 a piece).
    //
    // Two meetings of the waves. At row block MID everybody has W's operands
    // of this block in registers, so W of block kb + S starts on its way into
    // their slot. At the last row block nobody reads X's slot any more: block
    // kb + 1 has landed (all but the loads begun after its own, AHEAD), its
    // first operands are read as this block's are used up, and X of block kb + S
    // starts. Loads go out one at a time between the MFMAs: in a burst they
    // hold the waves up at the vector memory unit.
    constexpr int MID = C::MID, PX = (MID + 1) * TN, PW_ = (TM - 1 - MID) * TN;   // places for loads of X and W
    static_assert(MID >= 0 && MID <= TM - 2, "the meetings follow each other");
    constexpr int GAP = PW_ >= 2 * C::WP && PX >= 2 * XN ? 2 : 1;                 // a load at every GAP-th place,
    constexpr int NX = (XN + PX - 1) / PX, NWL = (C::WP + PW_ - 1) / PW_;         // or several at each
    constexpr int AHEAD = C::WP + (S - 2) * (C::WP + XN);
    auto meet = [&](bool all) __attribute__((always_inline)) {
        if (all) asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        else asm volatile("s_waitcnt vmcnt(%0)" ::"n"(AHEAD) : "memory");
        lds_barrier();
    };
    v4f p[2][TN];
    float sp[2] = {0.0f, 0.0f};
#pragma unroll
    for (int j = 0; j < TN; ++j) p[0][j] = p[1][j] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
    auto block = [&](int s, int kb, int par0) __attribute__((always_inline)) {
        char *const xs = xslot(s), *const nxs = xslot(s + 1), *const pxs = xslot(s + S - 1);
        char *const ws = wslot(s), *const nws = wslot(s + 1);
        const float sw = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(sw64), kb - sw0));
#pragma unroll
        for (int i = 0; i < TM; ++i) {
            const int par = (par0 + i) & 1, before = (i + TM - 1) % TM;
            if (i == MID) lds_barrier();
            if (i + 1 < TM) {
                read_x(xs, i + 1, par ^ 1);
            } else {
                meet(false);
                read_x(nxs, 0, par ^ 1);
            }
            sp[par] = sx[par] * sw;
#pragma unroll
            for (int j = 0; j < TN; ++j) {
                p[par][j] = Frag<C::PREC>::dot(wf[j], xf[par]);
                __builtin_amdgcn_sched_barrier(0);
                fmac(acc[before][j], p[par ^ 1][j], sp[par ^ 1]);
                const int ax = (i + 1) % TM * TN + j, aw = (i - MID) * TN + j;   // places since the meetings
#pragma unroll
                for (int u = 0; u < NX; ++u) {
                    const int d = ax / GAP * NX + u;
                    if (ax % GAP == 0 && d < XN) {
                        if (i + 1 == TM) load_x(xs, kb + S, d);
                        else load_x(pxs, kb + S - 1, d);
                    }
                }
#pragma unroll
                for (int u = 0; u < NWL; ++u) {
                    const int d = aw / GAP * NWL + u;
                    if (aw >= 0 && aw % GAP == 0 && d < C::WP && i + 1 < TM) load_w(ws, kb + S, d);
                }
                if (i + 1 == TM) read_w(nws, j);
                __builtin_amdgcn_sched_barrier(0);
            }
        }
    };

    // Blocks run S (or twice an odd S) at a time, which keeps the loop free of
    // branches; blocks past the end of K are zeros.
#pragma unroll
    for (int d = 0; d < XN; ++d) load_x(xs0, 0, d);
#pragma unroll
    for (int s = 0; s < S; ++s) {
#pragma unroll
        for (int d = 0; d < C::WP; ++d) load_w(wslot(s), s, d);
#pragma unroll
        for (int d = 0; d < XN; ++d)
            if (s > 0 && s + 1 < S) load_x(xslot(s), s, d);
    }
    meet(false);
    constexpr int TURN = TM % 2 && S % 2 ? 2 * S : S;              // (the registers' roles repeat after these)
    if ((GROUPED || BM <= 128) && wm * TM * 16 >= rr.rows) {
        // A wave without rows brings its part of the operands and meets the others,
        // which then have the SIMD for themselves: 8200 rows of 16 ragged groups x
        // 4096 x 4096 with GELU take 165.5 us (168.6), 16 x 4096 x 12288 12.8 (13.2). (The large dense
        // tiles, with one such row of tiles at most, would lose 1 % to the branch.)
        for (int kb = 0; kb < KB; kb += TURN) {
#pragma unroll
            for (int s = 0; s < TURN; ++s) {
#pragma unroll
                for (int d = 0; d < XN; ++d) load_x(xslot(s + S - 1), kb + s + S - 1, d);
                lds_barrier();
#pragma unroll
                for (int d = 0; d < C::WP; ++d) load_w(wslot(s), kb + s + S, d);
                meet(false);
            }
        }
        meet(true);
        return;
    }
    read_x(xs0, 0, 0);
#pragma unroll
    for (int j = 0; j < TN; ++j) {
#pragma unroll
        for (int u = 0; u < NX; ++u)
            if (j % GAP == 0 && j / GAP * NX + u < XN) load_x(xslot(S - 1), S - 1, j / GAP * NX + u);
        read_w(ws0, j);
    }
    for (int kb = 0; kb < KB; kb += TURN) {
        if (kb == 0 || kb - sw0 + TURN > 64) load_sw(kb);
#pragma unroll
        for (int s = 0; s < TURN; ++s) block(s, kb + s, s * TM & 1);
    }
    meet(true);                                          // (the last products are complete)
#pragma unroll
    for (int j = 0; j < TN; ++j) fmac(acc[TM - 1][j], p[(TURN * TM - 1) & 1][j], sp[(TURN * TM - 1) & 1]);

    // ---- outputs, 16 rows at a time: activation in registers, one rounding, then
    // through LDS (free now) so that rows leave as 16-byte stores of whole
    // lines, the memory taking one run of rows while the next is worked on.
    // The 16-byte chunks of a staged row are XOR-swizzled against bank
    // conflicts; a wave reads back only what it wrote, in order.
    constexpr int ES = C::PREC ? 4 : 2;                            // bytes of an output
    constexpr int RB = TN * 16 * ES, CPR = RB / 16;                // bytes, 16-byte chunks of a staged row
    constexpr int PER = 16 / ES, CHUNKS = 16 * CPR / 64;           // outputs of a chunk, chunks of a lane
    static_assert(NW * 16 * RB <= C::XSLOT && 16 * CPR % 64 == 0, "the staged rows fit a slot");
    char* stg = xs0 + wave * (16 * RB);
#pragma unroll
    for (int i = 0; i < TM; ++i) {
#pragma unroll
        for (int j = 0; j < TN; ++j) {
            if (a.act) {
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[i][j][e] = gelu_tanh_f32(acc[i][j][e]);
            }
            const int at = (j * 16 + q4 * 4) * ES;
            char* d = stg + l16 * RB + ((((at >> 4) ^ l16) & (CPR - 1)) << 4) + (at & 15);
            if constexpr (C::PREC) *(float4*)d = make_float4(acc[i][j][0], acc[i][j][1], acc[i][j][2], acc[i][j][3]);
            else *(uint2*)d = make_uint2(bf16x2(acc[i][j][0], acc[i][j][1]), bf16x2(acc[i][j][2], acc[i][j][3]));
        }
#pragma unroll
        for (int k = 0; k < CHUNKS; ++k) {
            const int q = k * 64 + lane, r = q / CPR, c = q % CPR;
            const uint4 v = *(const uint4*)(stg + r * RB + (((c ^ r) & (CPR - 1)) << 4));
            const int row = (wm * TM + i) * 16 + r, col = n0 + wn * TN * 16 + c * PER;
            if (row < rr.rows && col < a.N) {
                char* d = (char*)a.y + ((rr.m0 + row) * a.ldy + col) * ES;
                if (a.vec && col + PER <= a.N) {
                    *(uint4*)d = v;
                } else {
                    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                    for (int e = 0; e < PER; ++e)
                        if (col + e < a.N) {
                            if constexpr (C::PREC) ((uint32_t*)d)[e] = w[e];
                            else ((uint16_t*)d)[e] = (uint16_t)(w[e >> 1] >> (16 * (e & 1)));
                        }
                }
            }
        }
    }
}

// ---------------------------------------------------------------- few rows

// Up to 16 MT rows: 16 NT outputs per workgroup, the K blocks dealt to its NW
// waves U at a time, the weights straight from memory into the MFMA operand
// (no reuse to stage for), the waves' sums joined in LDS in wave order.
template <int MT_, int NT_, int NW_, int U_, int PREC_>
struct FewCfg {
    static constexpr int MT = MT_, NT = NT_, NW = NW_, U = U_, PREC = PREC_;
};

// What its activations are: codes of one batch, codes of ragged groups, or bf16
// values of either, which every workgroup turns into codes in LDS for itself while
// its first weights are on their way (one launch instead of two). That
// costs rows x blocks of vector work per workgroup, so it is for few of them:
// 1 x 4096 x 18432 takes 16.3 us (20.2 in two launches, 16.9 their product
// alone), 1 x 18432 x 4096 18.2 (22.4), 16 x 1536 x 6144 7.3 (8.2); even at 256
// rows x blocks, 8 x 4096 x 18432 24.6 (24.9), 8 x 4096 x 4096 9.4 (9.1); behind
// at 384, 4 x 12288 x 4096 17.6 (16.1). Grouped, 2 rows of 8 groups x 2048 x 4096
// take 5.8 (8.4), 4 of 8 x 4096 x 4096 13.9 (14.7). The codes are the activation
// pass's.
enum { DENSE, GROUPS, LAYER, LAYER_GROUPS };

template <class C, int KIND>
__global__ __launch_bounds__(64 * C::NW) void gemm_fp8_few_kernel(Args a) {
    constexpr int MT = C::MT, NT = C::NT, NW = C::NW, U = C::U;
    constexpr bool OWN = KIND >= LAYER, RAGGED = KIND == GROUPS || KIND == LAYER_GROUPS;
    static_assert(!OWN || MT == 1, "up to 16 rows");
    constexpr int QB = 3;                                // blocks of activations in flight per 16 lanes
    __shared__ __attribute__((aligned(16))) v4f red[NW][MT * NT][64];
    extern __shared__ __attribute__((aligned(16))) char codes[];   // OWN: its rows of codes, then their scales
    const int tid = threadIdx.x, lane = tid & 63, l16 = lane & 15, q4 = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int tiles_n = (a.N + 16 * NT - 1) / (16 * NT);
    const int t = blockIdx.x;
    Rows rr;
    if constexpr (RAGGED) {
        int total;
        rr = group_rows(a, t / tiles_n, 16 * MT, &total);
        if (t / tiles_n >= total) return;
    } else {
        rr.m0 = (int64_t)(t / tiles_n) * (16 * MT);
        rr.rows = (int)((a.M - rr.m0) < 16 * MT ? (a.M - rr.m0) : 16 * MT);
        rr.g = 0;
    }
    const int n0 = (t % tiles_n) * 16 * NT;
    const int K = a.K, KB = (K + 127) / 128, NB = (a.N + 127) / 128;
    const int nrows = a.N - n0 < 16 * NT ? a.N - n0 : 16 * NT;
    const rsrc_t rx = make_rsrc(a.qx + rr.m0 * K, OWN ? 0 : (int64_t)rr.rows * K);
    const rsrc_t rw = make_rsrc(a.qw + ((int64_t)rr.g * a.N + n0) * K, (int64_t)nrows * K);
    const float* swp = a.sw + ((int64_t)rr.g * NB + n0 / 128) * KB;
    const float* sxp = a.sx + rr.m0;
    const int pitch = KB * 128 + 16;                     // of a row of codes: 16 rows fall on different banks
    float* scales = (float*)(codes + rr.rows * pitch);
    int ms[MT];
#pragma unroll
    for (int i = 0; i < MT; ++i) ms[i] = 16 * i + l16 < rr.rows ? 16 * i + l16 : rr.rows - 1;
    const int vo = l16 * K + 16 * q4;
    v4f acc[MT][NT];
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j) acc[i][j] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
    uint4 w[U][NT][2];
    float sw[U];
    auto load_w = [&](int kb0) __attribute__((always_inline)) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int kb = kb0 + u * NW;
            const int left = K - kb * 128 - 16 * q4;     // channels left at the lane's first chunk
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int v = 64 * h < left ? vo + 64 * h : kBeyond;
#pragma unroll
                for (int j = 0; j < NT; ++j)
                    w[u][j][h] = __builtin_bit_cast(uint4, __builtin_amdgcn_raw_buffer_load_b128(rw, v, kb * 128 + j * 16 * K, 0));
            }
            sw[u] = swp[kb < KB ? kb : KB - 1];
        }
    };
    if constexpr (OWN) {
        load_w(wave);                                    // on their way while the activations are turned
        const int pairs = rr.rows * KB;                  // (row, block): 16 lanes each
        for (int p0 = tid >> 4; p0 < pairs; p0 += QB * NW * 4) {
            uint4 v[QB];
#pragma unroll
            for (int b = 0; b < QB; ++b) {
                const int p = p0 + b * NW * 4, m = p / KB, k = (p - m * KB) * 128 + l16 * 8;
                v[b] = make_uint4(0u, 0u, 0u, 0u);
                if (p < pairs && k < K) v[b] = *(const uint4*)(a.x + (rr.m0 + m) * a.ldx + k);
            }
#pragma unroll
            for (int b = 0; b < QB; ++b) {
                const int p = p0 + b * NW * 4, m = p / KB, k = (p - m * KB) * 128 + l16 * 8;
                if (p < pairs) {
                    float s;
                    *(uint2*)(codes + m * pitch + k) = block_codes(v[b], s);
                    if (l16 == 0) scales[p] = s;
                }
            }
        }
        __syncthreads();
    }
    for (int kb0 = wave; kb0 < KB; kb0 += NW * U) {
        uint4 x[U][MT][2];
        float s[U][MT];
        if (!OWN || kb0 != wave) load_w(kb0);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int kb = kb0 + u * NW, kc = kb < KB ? kb : KB - 1;
            const int left = K - kb * 128 - 16 * q4;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int v = 64 * h < left ? vo + 64 * h : kBeyond;
#pragma unroll
                for (int i = 0; i < MT; ++i) {
                    if constexpr (OWN) x[u][i][h] = *(const uint4*)(codes + ms[i] * pitch + kc * 128 + 64 * h + 16 * q4);
                    else x[u][i][h] = __builtin_bit_cast(uint4, __builtin_amdgcn_raw_buffer_load_b128(rx, v, kb * 128 + i * 16 * K, 0));
                }
            }
#pragma unroll
            for (int i = 0; i < MT; ++i) s[u][i] = (OWN ? scales[ms[i] * KB + kc] : sxp[(int64_t)kc * a.M + ms[i]]) * sw[u];
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            Frag<C::PREC> wf[NT];
#pragma unroll
            for (int j = 0; j < NT; ++j) wf[j].set(w[u][j][0], w[u][j][1]);
#pragma unroll
            for (int i = 0; i < MT; ++i) {
                Frag<C::PREC> xf;
                xf.set(x[u][i][0], x[u][i][1]);
#pragma unroll
                for (int j = 0; j < NT; ++j) {
                    const v4f p = Frag<C::PREC>::dot(wf[j], xf);
#pragma unroll
                    for (int e = 0; e < 4; ++e) acc[i][j][e] = __builtin_fmaf(p[e], s[u][i], acc[i][j][e]);
                }
            }
        }
    }
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j) red[wave][i * NT + j][lane] = acc[i][j];
    __syncthreads();
    for (int b = wave; b < MT * NT; b += NW) {           // a 16 x 16 tile per wave
        v4f sum = red[0][b][lane];
#pragma unroll
        for (int k = 1; k < NW; ++k) {
            const v4f o = red[k][b][lane];
#pragma unroll
            for (int e = 0; e < 4; ++e) sum[e] += o[e];
        }
        const int row = b / NT * 16 + l16, col = n0 + b % NT * 16 + q4 * 4;
        float v[4];
#pragma unroll
        for (int e = 0; e < 4; ++e)
            v[e] = finish(sum[e], a.bias && col + e < a.N ? bf16_lo_to_f32(a.bias[(int64_t)rr.g * a.N + col + e]) : 0.0f,
                          a.act);
        if (row < rr.rows) store4(a, rr.m0 + row, col, v);
    }
}

// the most row tiles that M rows in E ragged groups (0: one batch) can need; each has a row
int64_t row_tiles(const Args& a, int bm) {
    const int64_t t = a.offs ? (a.M + (int64_t)a.E * (bm - 1)) / bm : (a.M + bm - 1) / bm;
    return t < a.M ? t : a.M;
}

template <class C, bool GROUPED>
void launch_tiles(const Args& a, hipStream_t stream) {
    const int64_t tm = row_tiles(a, C::BM);
    const int64_t tn = (a.N + C::BN - 1) / C::BN;
    hipLaunchKernelGGL((gemm_fp8_kernel<C, GROUPED>), dim3((unsigned)(tm * tn)), dim3(C::NT), 0, stream, a);
}

template <class C, bool GROUPED>
void launch_few(const Args& a, hipStream_t stream) {
    const int64_t tm = row_tiles(a, 16 * C::MT);
    const int64_t tn = (a.N + 16 * C::NT - 1) / (16 * C::NT);
    hipLaunchKernelGGL((gemm_fp8_few_kernel<C, GROUPED ? GROUPS : DENSE>), dim3((unsigned)(tm * tn)), dim3(64 * C::NW), 0, stream, a);
}

// 16 outputs a workgroup, or 32 where one trip of its waves' loads still covers
// K and the narrow ones would come in turns: 1 x 1536 x 6144 takes 5.1 us with
// 32 (5.6 with 16), but 1 x 4096 x 18432 21.4 (16.2) and 1 x 1024 x 1024, 64
// narrow workgroups, 4.1 (3.7).
template <int PREC, int KIND>
void launch_layer(const Args& a, int cus, hipStream_t stream) {
    const int KB = (a.K + 127) / 128;
    const size_t lds = (size_t)a.M * (KB * 128 + 16 + KB * 4);
    const int64_t tm = row_tiles(a, 16), narrow = tm * ((a.N + 15) / 16);
    if (KB <= 16 && narrow > cus) {
        typedef FewCfg<1, 2, 8, 2, PREC> C;
        hipLaunchKernelGGL((gemm_fp8_few_kernel<C, KIND>), dim3((unsigned)(tm * ((a.N + 31) / 32))), dim3(64 * C::NW), lds, stream, a);
    } else {
        typedef FewCfg<1, 1, 8, 4, PREC> C;
        hipLaunchKernelGGL((gemm_fp8_few_kernel<C, KIND>), dim3((unsigned)narrow), dim3(64 * C::NW), lds, stream, a);
    }
}

// ---------------------------------------------------------------- which kernel
//
// One estimate per variant, in microseconds, from times measured on MI355X at
// K = 4096 (32 blocks of 128; a launch of nothing takes 3):
//  - tiles: `full` per block of K with `per_cu` workgroups on a CU, `lone` with
//    one of two. Large tiles move fewer bytes and read LDS less per product:
//    4096 x 4096 x 8192 takes 121 us with 256 x 256, 132 with 192 x 256, 143
//    with 128 x 128 (two a CU), 184 with 64 x 128, 223 with 64 x 64. Which one
//    wins is decided by how its tiles fill rounds of the CUs: 4608 x 12288 x 4096
//    takes 211 us with 160 x 256 (1.8 rounds; 211 to 228 from run to run) and
//    272 with 256 x 256 (1.1),
//    4608 x 4096 x 12288 204 with 224 x 256 (3.9 rounds) and 233 with 160 x
//    256. Where the tiles do not fill the CUs once, memory latency counts, and
//    the small ones keep three or four slots: 256 x 4096 x 4096 takes 11.6 with
//    64 x 64 (256 tiles; 13.2 with two slots), 19.3 with 128 x 128 (64 tiles);
//    256 x 12288 x 4096 34 (46 with two slots); 1024 x 4096 x 4096 22 with
//    128 x 128 in eight waves and four slots, 23.5 in four waves and two, two
//    workgroups a CU, which take 512 x 4096 x 12288 in 37 (44 the other way,
//    33 with 256 x 128). Where M is small the weights count: `start` and then
//    `rate` MB a us (tiles of 64 rows hide most of it beside their loads).
//  - few rows: `lone` for a trip of a workgroup's loads, four workgroups a CU;
//    the operands at 29 KB a us and CU; the weights from memory. 1 x 4096 x 18432
//    takes 17.4 us (20.4 with 32 columns, best tile 20.5), 16 of its rows 23
//    (19.4 with 64 x 128), 16 x 1536 x 6144 6.6 with 16 columns and 5.1 with 32,
//    64 x 4096 x 12288 26 (15 in tiles); 48 rows of 32 groups x 2048 x 4096 37
//    with 32 columns, 43 in tiles.
// Measured sizes and how far the variant it picks is behind the best one: 648 of
// 1 to 64 rows 1.3 % on the average, 9 or more in one of 20, 23 at the worst; 467
// of 77 to 4608 rows 0.6, 4, 22; 810 with fp32 outputs 2.2, 13, 68; 532 grouped
// ones (half to 2300 rows a group, ragged) 4.1, 20, 46: it does not know the
// groups' sizes.
struct Variant {
    int rows, cols, few;             // outputs per workgroup; few: the few-rows kernel
    int per_cu, trip;                // workgroups on a CU; K blocks per trip of a few-rows workgroup
    double lone, full;
    double start, rate;              // of the weights
};

constexpr Variant kVariants[] = {
    {256, 256, 0, 1, 0, 0, 1.74, 1.2, 4.3},    {224, 256, 0, 1, 0, 0, 1.52, 1.2, 4.3},
    {192, 256, 0, 1, 0, 0, 1.36, 1.2, 4.3},    {160, 256, 0, 1, 0, 0, 1.18, 1.2, 4.3},
    {256, 128, 0, 1, 0, 0, 0.98, 1.2, 4.3},    {128, 128, 0, 2, 0, 0.60, 1.07, 1.2, 4.3},
    {128, 128, 0, 1, 0, 0, 0.56, 2.2, 5.1},    {64, 128, 0, 2, 0, 0.42, 0.76, 1.6, 8.5},
    {64, 64, 0, 2, 0, 0.30, 0.44, 1.3, 9.4},   {16, 16, 1, 4, 32, 2.2, 0, 2.0, 6.6},
    {16, 32, 1, 4, 16, 2.2, 0, 0.5, 5.3},      {32, 32, 1, 4, 16, 3.1, 0, 1.0, 5.4},
};

double estimate(const Variant& v, const Args& a, int cus) {
    const double M = (double)a.M, E = a.E, kb = (a.K + 127) / 128;
    // groups that have rows, if rows fall at random
    const double active = a.offs ? E * (1.0 - __builtin_exp(-M / E)) : 1.0;
    const double tn = (double)((a.N + v.cols - 1) / v.cols);
    // ragged groups: half a tile is lost at the end of each, on the average
    double tm = a.offs ? M / v.rows + 0.5 * active : (double)((a.M + v.rows - 1) / v.rows);
    if (tm < active) tm = active;
    const double tiles = tm * tn;
    // many groups' weights stream at one rate in the small variants
    const double weights = v.start + active * a.N * (double)a.K / (a.offs && v.rows < 128 ? 6.5e6 : v.rate * 1e6);
    double t;
    if (v.few) {
        const double g = __builtin_ceil(tiles / cus), turns = g < v.per_cu ? 1.0 : g / v.per_cu;
        const double rows = M < v.rows * tm ? M / tm : v.rows;
        const double trips = turns * v.lone * __builtin_ceil(kb / v.trip), reads = g * (v.cols + rows) * a.K / 2.9e4;
        t = trips > reads ? trips : reads;
    } else {
        // exact products for fp32 outputs take the bf16 instructions twice the time (over
        // 660 sizes 1.8 % behind the best variant, 2.2 without)
        const double kt = a.y_f32 ? 2.0 * kb : kb;
        const double slots = (double)cus * v.per_cu, rounds = __builtin_floor(tiles / slots);
        const double rest = __builtin_ceil((tiles - rounds * slots) / cus);
        const double share = v.full * rest / v.per_cu, out = 4.0 * v.rows * v.cols * v.per_cu / 65536.0;
        t = rounds * (kt * v.full + out) + (rest > 0 ? kt * (share > v.lone ? share : v.lone) + out * rest / v.per_cu : 0.0);
    }
    return 3.0 + (t > weights ? t : weights);
}

// lanes of a launch stay below 2^32
bool fits(const Variant& v, const Args& a) {
    const double tm = (double)a.M / v.rows + 1.0 + a.E, tn = (double)a.N / v.cols + 1.0;
    return tm * tn * 512.0 < 4294967296.0;
}

// The variant with the least estimate, or -1
int pick_variant(const Args& a, int prec, int cus) {
    int best = -1;
    double least = 0.0;
    for (int i = 0; i < (int)(sizeof kVariants / sizeof kVariants[0]); ++i) {
        // fp32 outputs have the two tile sizes whose operands fit the registers when widened
        if (prec == 1 && i < 9 && i != 5 && i != 8) continue;
        if (!fits(kVariants[i], a)) continue;
        const double t = estimate(kVariants[i], a, cus);
        if (best < 0 || t < least) best = i, least = t;
    }
    return best;
}

template <int PREC, bool GROUPED>
bool launch_variant(const Args& a, int cus, hipStream_t stream) {
    const int best = pick_variant(a, PREC, cus);
    switch (best) {
        case 0: if constexpr (PREC == 0) launch_tiles<Cfg<8, 4, 2, 4, 2, 0, 3, 2>, GROUPED>(a, stream); break;
        case 1: if constexpr (PREC == 0) launch_tiles<Cfg<7, 4, 2, 4, 2, 0, 3, 2>, GROUPED>(a, stream); break;
        case 2: if constexpr (PREC == 0) launch_tiles<Cfg<6, 4, 2, 4, 2, 0, 2, 2>, GROUPED>(a, stream); break;
        case 3: if constexpr (PREC == 0) launch_tiles<Cfg<5, 4, 2, 4, 2, 0, 2, 2>, GROUPED>(a, stream); break;
        case 4: if constexpr (PREC == 0) launch_tiles<Cfg<4, 4, 4, 2, 2, 0, 2, 2>, GROUPED>(a, stream); break;
        case 5: launch_tiles<Cfg<4, 4, 2, 2, 2, PREC, 2, 2>, GROUPED>(a, stream); break;
        case 6: if constexpr (PREC == 0) launch_tiles<Cfg<2, 4, 4, 2, 2, 0, 0, 4>, GROUPED>(a, stream); break;
        case 7: if constexpr (PREC == 0) launch_tiles<Cfg<2, 4, 2, 2, 2, 0, 0, 3>, GROUPED>(a, stream); break;
        case 8: launch_tiles<Cfg<2, 2, 2, 2, 2, PREC, 0, 4>, GROUPED>(a, stream); break;
        case 9: launch_few<FewCfg<1, 1, 8, 4, PREC>, GROUPED>(a, stream); break;
        case 10: launch_few<FewCfg<1, 2, 8, 2, PREC>, GROUPED>(a, stream); break;
        case 11: launch_few<FewCfg<2, 2, 8, 2, PREC>, GROUPED>(a, stream); break;
        default: return false;
    }
    return true;
}

}  // namespace

// whether some variant's grid fits a launch
bool gemm_fp8_fits(int64_t M, int64_t N, int E) {
    Args a{};
    a.M = M;
    a.N = (int)N;
    a.E = E;
    return fits(kVariants[5], a);
}

// what a product of these sizes runs
int gemm_fp8_variant(int64_t M, int64_t K, int64_t N, int groups, int y_f32, int cus) {
    static const int32_t ragged = 0;
    Args a{};
    a.M = M;
    a.K = (int)K;
    a.N = (int)N;
    a.E = groups;
    a.offs = groups ? &ragged : nullptr;                 // (only asked whether there are any)
    a.y_f32 = y_f32;
    return pick_variant(a, y_f32 ? 1 : 0, cus);
}

hipError_t launch_gemm_fp8(const uint8_t* qx, const float* sx, int64_t M, int64_t K, const uint8_t* qw, const float* sw,
                           int64_t N, const int32_t* offs, int E, const uint16_t* bias, int act, void* y, int y_f32,
                           int64_t ldy, int cus, hipStream_t stream) {
    const int vec = ldy % (y_f32 ? 4 : 8) == 0 && (uintptr_t)y % 16 == 0;
    const Args a{qx, sx, qw, sw, bias, y, offs, M, ldy, (int)N, (int)K, E, act, y_f32, vec, nullptr, 0};
    const bool ok = offs ? (y_f32 ? launch_variant<1, true>(a, cus, stream) : launch_variant<0, true>(a, cus, stream))
                         : (y_f32 ? launch_variant<1, false>(a, cus, stream) : launch_variant<0, false>(a, cus, stream));
    return ok ? hipGetLastError() : hipErrorInvalidValue;
}

hipError_t launch_linear_fp8(const uint16_t* x, int64_t M, int64_t K, int64_t ldx, const uint8_t* qw, const float* sw,
                             int64_t N, const int32_t* offs, int E, const uint16_t* bias, int act, void* y, int y_f32,
                             int64_t ldy, int cus, hipStream_t stream) {
    const int vec = ldy % (y_f32 ? 4 : 8) == 0 && (uintptr_t)y % 16 == 0;
    const Args a{nullptr, nullptr, qw, sw, bias, y, offs, M, ldy, (int)N, (int)K, E, act, y_f32, vec, x, ldx};
    if (offs) y_f32 ? launch_layer<1, LAYER_GROUPS>(a, cus, stream) : launch_layer<0, LAYER_GROUPS>(a, cus, stream);
    else y_f32 ? launch_layer<1, LAYER>(a, cus, stream) : launch_layer<0, LAYER>(a, cus, stream);
    return hipGetLastError();
}
