// svdq_kv_attend for sequences of many query rows (kv_flash.h has the mathematics):
// the matrix pipe counts. 4608 queries over 23040 keys of 24 heads of 128 take 1100 to 1136 us, 1.15 to
// 1.19 PFLOP/s where a large bf16 product reaches 1.48; the pipe is 59 % busy, the vector work (an
// exponential and its share of the rest a score) mostly in its shadow. 32 rows a wave fill the registers, two
// workgroups of four waves the CU: each key operand read from LDS serves two products, and one
// workgroup's vector work runs beside the other's products.
#include "kv_flash.h"

namespace {

typedef __attribute__((address_space(3))) void lds_void;

constexpr int kRows = 128;           // of a row tile
constexpr int kLeast = 8;            // tiles of 64 keys of a split

// Row tile `item`, the split-th of its splits of the keys
DEV bool find_work(const KvAttendArgs& a, int item, int split, int splits, Work& w) {
    KvItem it;
    const int G = a.G;
    if (!kv_find(a.s, item, [&](int o, int b) { return (int)((int64_t)o * G / kRows) + b; },
                 [&](int n) { return (int)(((int64_t)n * G + kRows - 1) / kRows); }, it))
        return false;
    w.b = uni(it.b);
    w.t0 = uni(it.t0);
    w.n = uni(it.n);
    const int len = uni(a.s.lengths[w.b]);
    w.len = len < 0 ? 0 : len;
    w.room = (int)kv_room(a.s, a.c);
    w.row0 = uni(it.part) * kRows;
    const int left = w.n * G - w.row0;
    w.rows = left < kRows ? left : kRows;
    const Span first = uni(span_of(a, w, w.row0)), last = uni(span_of(a, w, w.row0 + w.rows - 1));
    const int ta = first.lo / 64, tb = (last.hi + 63) / 64, nt = tb > ta ? tb - ta : 0;
    int per = uni((nt + splits - 1) / splits);
    if (per < kLeast) per = kLeast;
    w.ta = ta + split * per < ta + nt ? ta + split * per : ta + nt;
    w.tb = w.ta + per < ta + nt ? w.ta + per : ta + nt;
    return true;
}

// Sums and (reference, weights' sum) of row i of the n-th split row tile, by one split
DEV float* part_sums(const KvAttendArgs& a, int n, int i, int split, int W) {
    return a.part + (((int64_t)n * kRows + i) * a.S + split) * W;
}
DEV float* part_stats(const KvAttendArgs& a, int n, int i, int split, int W) {
    const int64_t rows = ((int64_t)a.items * a.c.H - a.whole) * kRows;
    return a.part + rows * a.S * W + (((int64_t)n * kRows + i) * a.S + split) * 2;
}

// ---------------------------------------------------------------- many rows

// 128 rows a workgroup, 32 a wave; the tiles of keys come through LDS, loaded
// straight from memory (the cache's order is the operands'), keys a tile before
// their values: the scores of a tile are formed beside the weights of the one
// before, matrix work beside vector work. One meeting of the waves a tile.
template <int C>
__global__ __launch_bounds__(256, C <= 2 ? 2 : 1) void attend_many_kernel(KvAttendArgs a) {
    constexpr int QT = 2, R = kRows, W = 64 * C, HALF = 4 * C * 1024;
    __shared__ __attribute__((aligned(16))) char key0[HALF], key1[HALF], raw0[HALF], raw1[HALF];
    __shared__ __attribute__((aligned(16))) char value0[2 * HALF], value1[2 * HALF];
    const int tid = threadIdx.x, lane = tid & 63, l16 = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    // Row tiles in the order of the key heads, later ones, which see more keys where order counts, first.
    // The first a.whole of them are a workgroup's each, the rest a.S workgroups'. Workgroup b runs on XCD b %
    // 8: of either part an XCD takes a contiguous run, so that those in flight share keys in its L2.
    const bool whole = (int)blockIdx.x < a.whole;
    const int all = whole ? a.whole : gridDim.x - a.whole, b8 = whole ? blockIdx.x : blockIdx.x - a.whole;
    const int x8 = b8 & 7, q8 = all >> 3, r8 = all & 7, splits = whole ? 1 : a.S;
    const int t8 = x8 * q8 + (x8 < r8 ? x8 : r8) + (b8 >> 3);
    const int of = uni(t8 / splits), split = t8 - of * splits, rest = whole ? of : a.whole + of;
    const int h = uni(rest / a.items), item = a.items - 1 - (rest - h * a.items);
    Work w;
    if (!find_work(a, item, split, splits, w)) return;
    Flash<C, QT> f;
    f.clear();
    const int wr = wave * 32;                            // the wave's first row; past the end it has none
#pragma unroll
    for (int t = 0; t < QT; ++t) {
        const int i = wr + t * 16 + l16, r = w.row0 + (i < w.rows ? i : w.rows - 1);
        const Row x = row_of(a, w, h, r);
        uint4 q[2 * C];
        f.fetch_query(q, a.q + x.t * a.qts + x.h * a.qhs, a.c.D);
        f.take_query(t, q);
        f.see[t] = span_of(a, w, r);
    }
    const int rl = wr + 31 < w.rows ? wr + 31 : w.rows - 1;
    const Span first = uni(span_of(a, w, w.row0 + (wr < w.rows ? wr : w.rows - 1))), last = uni(span_of(a, w, w.row0 + rl));
    const Span wfirst = uni(span_of(a, w, w.row0)), wlast = uni(span_of(a, w, w.row0 + w.rows - 1));
    const int nt = w.tb - w.ta;

    Tiles<1> tiles;
    auto find = [&](bool& ok) __attribute__((always_inline)) { return tiles.take(a, h, ok); };
    // one side of a tile into LDS, a quarter a wave (zeros if it is not there)
    auto fetch = [&](char* s, int64_t at, int side, bool ok) __attribute__((always_inline)) {
        const rsrc_t r = make_rsrc(a.c.data + (2 * at + side) * HALF, ok ? HALF : 0);
#pragma unroll
        for (int k = 0; k < C; ++k) {
            const int p = (k * 4 + wave) * 1024;
            __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_void*)(s + p), 16, lane * 16, p, 0, 0);
        }
    };
    auto landed = [&]() __attribute__((always_inline)) {
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        lds_barrier();
    };
    bool ok0, ok1, ok2;                                  // whether tiles 0, i + 1, i + 2 are there
    v4f s[QT][4];
    uint2 sc1;                                           // exponents of tile i + 1
    auto codes = [&](const char* k) __attribute__((always_inline)) {
        return [=](int b, int c) __attribute__((always_inline)) { return *(const uint4*)(k + (b * C + c) * 1024 + lane * 16); };
    };
    auto is_masked = [&](int i, bool ok) __attribute__((always_inline)) {
        const int k0 = (w.ta + i) * 64;
        return !ok || k0 < last.lo || k0 + 64 > first.hi;
    };
    auto hide = [&](int i, bool ok) __attribute__((always_inline)) {
        if (is_masked(i, ok)) f.mask(s, ok ? (w.ta + i) * 64 : kNowhere);
        f.settle(a, s);
    };
    // Values of a tile that not all rows of the workgroup see whole: keys that none of them sees may
    // hold anything, and become zeros in LDS, as do NaN values (which are seen to in the end).
    auto partly = [&](int k0) __attribute__((always_inline)) { return k0 < wlast.lo || k0 + 64 > wfirst.hi; };
    uint32_t nans = 0;
    auto clean = [&](char* v, int k0) __attribute__((always_inline)) {
#pragma unroll 1
        for (int q = wave; q < 4 * C; q += 4) {
            uint4* x = (uint4*)(v + q * 1024 + lane * 16);
            const uint4 y = and4(*x, kept_bytes(k0, q / C, wfirst.lo, wlast.hi));
            nans |= nan_codes4(y);
            *x = without_nan(y);
        }
        lds_barrier();
    };
    // The values of a tile as operands in bf16, a share of the workgroup's waves each: 64 channels (c) of
    // two blocks of keys (h) at a time, in eight steps.
    constexpr int SHARES = (2 * C + 3) / 4;
    uint4 rw[2];
    uint32_t half[8];
    auto widen = [&](const char* raw, char* out, uint32_t ve, int x) __attribute__((always_inline)) {
        const int q = wave + x / 8 * 4, hh = q / C, c = q - hh * C, u = x % 8 / 2, b = x % 2;
        if (2 * C % 4 && q >= 2 * C) return;
        if (x % 8 == 0) {
            rw[0] = *(const uint4*)(raw + (2 * hh * C + c) * 1024 + lane * 16);
            rw[1] = *(const uint4*)(raw + ((2 * hh + 1) * C + c) * 1024 + lane * 16);
        }
        const float vs = value_scale((ve >> (16 * hh + 8 * b)) & 0xffu);
        const uint4 r = rw[b];
        const uint32_t word = u == 0 ? r.x : u == 1 ? r.y : u == 2 ? r.z : r.w;
        half[2 * b] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((int)word, vs, false));
        half[2 * b + 1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((int)word, vs, true));
        if (b) *(uint4*)(out + ((c * 4 + u) * 2 + hh) * 1024 + lane * 16) = make_uint4(half[0], half[1], half[2], half[3]);
    };
    // Tile i, whose scores are in s: its weights, beside them the next tile's scores; then its sums,
    // beside them the next tile's values.
    auto step = [&](char* knext, char* kfree, char* rnext, char* rfree, char* v, char* vnext, int i) __attribute__((always_inline)) {
        landed();                                        // tile i + 1, and tile i's values; nobody reads the others
        const int k1 = (w.ta + i + 1) * 64;
        if (ok1 && partly(k1)) clean(rnext, k1);
        const int64_t at2 = find(ok2);
        fetch(kfree, at2, 0, ok2);
        fetch(rfree, at2, 1, ok2);
        const uint2 sc2 = *(const uint2*)(a.c.scales + at2 * 8);
        uint32_t ve = uni(sc1.y);
        if (!ok1 || partly(k1)) ve &= ok1 ? kept_blocks(k1, wfirst.lo, wlast.hi) : 0u;
        auto meanwhile = [&](int x) __attribute__((always_inline)) {
            constexpr int PER = (8 * SHARES + 4 * C - 1) / (4 * C);
#pragma unroll
            for (int y = 0; y < PER; ++y)
                if (x * PER + y < 8 * SHARES) widen(rnext, vnext, ve, x * PER + y);
        };
        if (wr < w.rows) {
            uint32_t p[QT][8];
            // Of a SIMD's two waves the one that is further goes first: its products then start as the other's
            // vector work leaves room for them (1225 us without, 1200 with the sums first, 1163 like this).
            __builtin_amdgcn_s_setprio(1);
            f.exchange_tile(a, s, p, sc1.x, codes(knext));
            __builtin_amdgcn_s_setprio(2);
            f.ready_sums(p, [&](int x, int hh) __attribute__((always_inline)) {
                return *(const uint4*)(v + (x * 2 + hh) * 1024 + lane * 16);
            }, meanwhile);
#pragma unroll
            for (int t = 0; t < QT; ++t)                 // (or the compiler moves the scores behind the branch)
#pragma unroll
                for (int b = 0; b < 4; ++b) order_point(s[t][b]);
            hide(i + 1, ok1);
            __builtin_amdgcn_s_setprio(0);
        } else {
#pragma unroll
            for (int x = 0; x < 4 * C; ++x) meanwhile(x);
        }
        ok1 = ok2;
        sc1 = sc2;
    };
    if (nt > 0) {
        tiles.start(a, w.b, w.ta, w.tb);
        const int64_t at0 = find(ok0), at1 = find(ok1);
        fetch(key0, at0, 0, ok0);
        fetch(raw0, at0, 1, ok0);
        const uint2 sc0 = *(const uint2*)(a.c.scales + at0 * 8);
        sc1 = *(const uint2*)(a.c.scales + at1 * 8);
        landed();
        const int k0 = w.ta * 64;
        if (ok0 && partly(k0)) clean(raw0, k0);
        fetch(key1, at1, 0, ok1);
        fetch(raw1, at1, 1, ok1);
        uint32_t ve = uni(sc0.y);
        if (!ok0 || partly(k0)) ve &= ok0 ? kept_blocks(k0, wfirst.lo, wlast.hi) : 0u;
#pragma unroll
        for (int x = 0; x < 8 * SHARES; ++x) widen(raw0, value0, ve, x);
        if (wr < w.rows) {
            f.score_tile(s, sc0.x, codes(key0));
            hide(0, ok0);
        }
        for (int i = 0; i < nt; i += 2) {
            step(key1, key0, raw1, raw0, value0, value1, i);
            if (i + 1 < nt) step(key0, key1, raw0, raw1, value1, value0, i + 1);
        }
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory"); // (loads into LDS end before the workgroup does)
        if (__syncthreads_or(nans != 0)) {
#pragma unroll 1
            for (int i = 0; i < nt; ++i) {
                const int t = w.ta + i, pg = uni(t / a.c.tiles), page = a.s.table[(int64_t)w.b * a.s.width + pg];
                if (!partly(t * 64) || (uint32_t)page >= (uint64_t)a.c.pages) continue;
                const int64_t at = ((int64_t)page * a.c.H + h) * a.c.tiles + t - pg * a.c.tiles;
                nan_tile(f, a.c.data + (2 * at + 1) * HALF, t * 64, wfirst.lo, wlast.hi);
            }
        }
    }
#pragma unroll
    for (int t = 0; t < QT; ++t) {
        const float l = f.l[t][0];
        const int i = wr + t * 16 + l16;
        if (i < w.rows) {
            const Row x = row_of(a, w, h, w.row0 + i);
            if (splits > 1) {
                float* p = part_sums(a, rest - a.whole, i, split, W);
#pragma unroll
                for (int k = 0; k < 4 * C; ++k) *(v4f*)(p + k * 16 + g * 4) = f.o[t][k];
                if (g == 0) *(float2*)part_stats(a, rest - a.whole, i, split, W) = make_float2(f.m[t], l);
            } else {
                const float n = l != 0.0f ? kValueUnit / l : 0.0f;
                uint16_t* p = a.y + x.t * a.yts + x.h * a.yhs;
#pragma unroll
                for (int k = 0; k < 4 * C; ++k) {
                    const int d = k * 16 + g * 4;
                    const v4f y = f.o[t][k];
                    if (d < a.c.D) *(uint2*)(p + d) = make_uint2(bf16x2(y[0] * n, y[1] * n), bf16x2(y[2] * n, y[3] * n));
                }
            }
        }
    }
}

// ---------------------------------------------------------------- splits joined

constexpr int kJoin = 4;             // rows of a wave

// The splits' sums of a row, weighted by their references: four rows a wave at a time, so that
// their loads are in flight together (4608 queries of 24 heads, 352 of 864 row tiles split: 35.6 us with a
// wave for every row of the call, 23.0 like this).
template <int C>
__global__ __launch_bounds__(256) void attend_many_join_kernel(KvAttendArgs a) {
    constexpr int W = 64 * C, PER = kRows / (4 * kJoin);
    const int lane = threadIdx.x & 63;
    const int n = blockIdx.x / PER, rest = a.whole + n;  // the split tile, in the kernel's order
    const int i0 = (blockIdx.x % PER * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6)) * kJoin;
    const int h = uni(rest / a.items), item = a.items - 1 - (rest - h * a.items);
    Work w;
    if (!find_work(a, item, 0, a.S, w) || i0 >= w.rows) return;
    float wgt[kJoin], sum[kJoin], y[kJoin][C];
    const float* p[kJoin];
#pragma unroll
    for (int j = 0; j < kJoin; ++j) {
        const int i = i0 + j < w.rows ? i0 + j : w.rows - 1;
        p[j] = part_sums(a, n, i, 0, W) + lane * C;
        const float2 st = lane < a.S ? *(const float2*)part_stats(a, n, i, lane, W) : make_float2(kNone, 0.0f);
        float m = st.x;
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) m = fmaxf(m, __shfl_xor(m, d));
        wgt[j] = lane < a.S ? share_of(st.x, m, a.scale2) : 0.0f;
        sum[j] = st.y * wgt[j];
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) sum[j] += __shfl_xor(sum[j], d);
#pragma unroll
        for (int c = 0; c < C; ++c) y[j][c] = 0.0f;
    }
#pragma unroll 2
    for (int s = 0; s < a.S; ++s)                        // (a split that a row sees nothing of left zeros)
#pragma unroll
        for (int j = 0; j < kJoin; ++j) {
            const float ws = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(wgt[j]), s));
#pragma unroll
            for (int c = 0; c < C; ++c) y[j][c] = __builtin_fmaf(ws, p[j][(int64_t)s * W + c], y[j][c]);
        }
#pragma unroll
    for (int j = 0; j < kJoin; ++j) {
        if (i0 + j >= w.rows) break;
        const Row x = row_of(a, w, h, w.row0 + i0 + j);
        const float k = sum[j] != 0.0f ? kValueUnit / sum[j] : 0.0f;
        uint16_t* out = a.y + x.t * a.yts + x.h * a.yhs;
#pragma unroll
        for (int c = 0; c < C; ++c)
            if (lane * C + c < a.c.D) out[lane * C + c] = f32_to_bf16_bits(y[j][c] * k);
    }
}

// ---------------------------------------------------------------- how many splits

struct Plan {
    int items, whole, S;
};

// Workgroups come in rounds of the CUs' places, and the row tiles of a last round
// that is not full are split where that takes less time: a tile of 64 keys takes 1.75 us
// with the places taken, a row tile's sums 26 ns a split and 128 channels to write
// and read, the launch that joins them 5 us (24 heads over 23040 keys, 512 places: 256 queries
// 442 us whole, 115 split; 3000 1024 and 714; 4608 1122 and 1076).
Plan plan_of(const KvBatch& s, const KvCache& c, int G, int cus) {
    Plan p{};
    p.items = (int)(s.offs ? s.T * G / kRows + s.B : s.B * (((int64_t)s.n * G + kRows - 1) / kRows));
    p.S = 1;
    const int64_t groups = (int64_t)p.items * c.H, tiles = (int64_t)s.width * c.tiles;
    const int64_t top = (tiles + kLeast - 1) / kLeast < 64 ? (tiles + kLeast - 1) / kLeast : 64;
    const int C = (c.D + 63) / 64;
    const int64_t places = (int64_t)cus * (C <= 2 ? 2 : 1), rest = groups % places;
    const double tile = 1.75 * (C <= 2 ? C / 2.0 : C / 4.0), io = 0.026 * C / 2.0;
    double least = (double)tiles * tile;                 // of the last round
    for (int S = 2; S <= top && rest; ++S) {
        const double t = (double)((rest * S + places - 1) / places) / S * (double)tiles * tile + (double)(rest * S) * io + 5.0;
        if (t < least) least = t, p.S = S;
    }
    p.whole = (int)(p.S > 1 ? groups - rest : groups);
    return p;
}

template <int C>
void launch(const KvAttendArgs& a, hipStream_t stream) {
    const int64_t groups = (int64_t)a.items * a.c.H;
    const dim3 grid((unsigned)(a.whole + (groups - a.whole) * a.S));
    hipLaunchKernelGGL((attend_many_kernel<C>), grid, dim3(256), 0, stream, a);
    if (a.S > 1)
        hipLaunchKernelGGL((attend_many_join_kernel<C>), dim3((unsigned)((groups - a.whole) * (kRows / (4 * kJoin)))), dim3(256), 0,
                           stream, a);
}

}  // namespace

int64_t kv_attend_many_workspace(const KvBatch& s, const KvCache& c, int G, int cus) {
    const Plan p = plan_of(s, c, G, cus);
    return p.S > 1 ? ((int64_t)p.items * c.H - p.whole) * kRows * p.S * ((c.D + 63) / 64 * 64 + 2) * 4 : 0;
}

hipError_t launch_kv_attend_many(KvAttendArgs a, int cus, hipStream_t stream) {
    const Plan p = plan_of(a.s, a.c, a.G, cus);
    a.items = p.items;
    a.whole = p.whole;
    a.S = p.S;
    switch ((a.c.D + 63) / 64) {
        case 1: launch<1>(a, stream); break;
        case 2: launch<2>(a, stream); break;
        case 3: launch<3>(a, stream); break;
        default: launch<4>(a, stream);
    }
    return hipGetLastError();
}
