// svdq_kv_attend for sequences of few query rows (kv_flash.h has the mathematics):
// the cache's bytes count. Every key is used once, straight from memory into the
// operands; the tiles of all sequences and key heads are dealt out evenly.
// 64 sequences to 8192 tokens, 32 heads over 8 of 128, take 118 us (5.9 TB/s), two of 131072 tokens, 24 heads
// over 8, 76 (5.8).
//
// The tiles of 64 keys of one key head of a row tile are padded to a multiple of four
// (one for each wave of a workgroup), those of all row tiles and key heads form one
// line, and workgroup w takes the `share` tiles from w * share on, of one row tile after
// the other. Lengths are known on the GPU only, so every workgroup adds them up for
// itself. A row tile that crosses a border leaves sums of its pieces, joined by a second
// launch: the first piece of a workgroup (which goes on what the one before began)
// in slot 2 w, the last in 2 w + 1.
#include "kv_flash.h"

namespace {

// a load that leaves no line behind for others (5.9 -> 6.8 TB/s over 690 MB)
DEV uint4 load_once(const uint8_t* p) {
    typedef uint32_t v4u __attribute__((ext_vector_type(4)));
    const v4u v = __builtin_nontemporal_load((const v4u*)p);
    return make_uint4(v[0], v[1], v[2], v[3]);
}

// sums over the lanes up to each
DEV int lanes_sum(int v) {
    v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xf, 0xf, true);       // one lane before, of the 16
    v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xf, 0xf, true);       // two
    v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xf, 0xf, true);
    v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xf, 0xf, true);
    v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xa, 0xf, true);       // the last of the 16 before, to rows 1 and 3
    v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xc, 0xf, true);       // lane 31, to rows 2 and 3
    return v;
}

// 64 sequences at a time, one a lane, and where their tiles lie on a key head's line
template <int R>
struct Line {
    int b0, done;                    // the first lane's sequence; the largest offset before it
    int before, sum;                 // tiles before it, of the 64 (the host has seen that all of them stay below 2^31)
    int lo, n, len, ta, nt, pad;     // the lane's: first token, tokens, length, first tile of keys, tiles, padded
    int units, start;                // row tiles * pad, and where they start

    DEV void restart() {
        b0 = -64;
        done = 0;
        before = sum = 0;
    }
    DEV void next(const KvAttendArgs& a) {
        const int lane = threadIdx.x & 63;
        b0 += 64;
        before += sum;
        const int b = b0 + lane;
        const bool in = b < a.s.B;
        lo = n = len = 0;
        if (in) len = a.s.lengths[b];
        if (a.s.offs) {
            kv_offsets(a.s, b0, done, lo, n);
        } else if (in) {
            lo = b * a.s.n;
            n = a.s.n;
        }
        const int room = (int)kv_room(a.s, a.c);
        len = len < 0 ? 0 : len;
        const int hi = len < room ? len : room, from = a.window && len - n >= a.window ? len - n - a.window + 1 : 0;
        ta = from / 64;
        nt = (hi + 63) / 64 - ta;
        nt = nt < 0 ? 0 : nt;
        pad = nt < 4 ? 4 : (nt + 3) & ~3;
        units = in ? (n * a.G + R - 1) / R * pad : 0;
        const int inc = lanes_sum(units);
        start = before + inc - units;
        sum = __builtin_amdgcn_readlane(inc, 63);
    }
    // tiles of a key head
    DEV int total(const KvAttendArgs& a) {
        restart();
        while (b0 + 64 < a.s.B) next(a);
        return before + sum;
    }
};

// A workgroup's tiles: a multiple of four
DEV int tiles_of(const KvAttendArgs& a, int total) {
    const uint32_t per = ((uint32_t)(total * a.c.H) + a.S - 1) / (uint32_t)a.S;
    return uni(per <= 4 ? 4 : (int)((per + 3) & ~3u));
}

// Sums and (reference, weights' sum) of row i of a piece
template <int R>
DEV float* part_sums(const KvAttendArgs& a, int64_t slot, int i, int W) { return a.part + (slot * R + i) * W; }
template <int R>
DEV float* part_stats(const KvAttendArgs& a, int64_t slot, int i, int W) {
    return a.part + 2 * (int64_t)a.S * R * W + (slot * R + i) * 2;
}

// One piece of a row tile: tiles [w.ta, w.tb) of it. slot: where its sums go; -1: it is whole.
template <int C, int QT>
DEV void piece(const KvAttendArgs& a, const Work& w, int h, int64_t slot, float (&red)[4][16 * QT][68], float (&stat)[4][16 * QT][2]) {
    constexpr int R = 16 * QT, W = 64 * C;
    const int tid = threadIdx.x, lane = tid & 63, l16 = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int t0 = w.ta + wave;
    const int mine = w.tb > t0 ? (w.tb - t0 + 3) / 4 : 0;
    Tiles<4> tiles;
    if (mine > 0) tiles.start(a, w.b, t0, w.tb);
    Flash<C, QT> f;
    uint4 q[QT][2 * C];
#pragma unroll
    for (int t = 0; t < QT; ++t) {
        const int i = t * 16 + l16, r = w.row0 + (i < w.rows ? i : w.rows - 1);
        const Row x = row_of(a, w, h, r);
        f.fetch_query(q[t], a.q + x.t * a.qts + x.h * a.qhs, a.c.D);
        f.see[t] = span_of(a, w, r);
    }
    const Span first = uni(span_of(a, w, w.row0)), last = uni(span_of(a, w, w.row0 + w.rows - 1));
    const int64_t tile_bytes = 8 * C * 1024;
    uint4 kr[4][C], vr[4][C];
    uint2 sc, nsc;
    auto load_k = [&](int64_t at) __attribute__((always_inline)) {
        const uint8_t* p = a.c.data + at * tile_bytes;
#pragma unroll
        for (int b = 0; b < 4; ++b)
#pragma unroll
            for (int c = 0; c < C; ++c) kr[b][c] = load_once(p + (b * C + c) * 1024 + lane * 16);
        nsc = *(const uint2*)(a.c.scales + at * 8);
    };
    auto load_v = [&](int64_t at) __attribute__((always_inline)) {
        const uint8_t* p = a.c.data + at * tile_bytes + tile_bytes / 2;
#pragma unroll
        for (int b = 0; b < 4; ++b)
#pragma unroll
            for (int c = 0; c < C; ++c) vr[b][c] = load_once(p + (b * C + c) * 1024 + lane * 16);
    };
    bool ok = false, next = false;
    int64_t at = 0;
    uint32_t nans = 0;
    if (mine > 0) {
        at = tiles.take(a, h, ok);
        load_k(at);
        load_v(at);
    }
    f.clear();
#pragma unroll
    for (int t = 0; t < QT; ++t) f.take_query(t, q[t]);
    const auto key = [&](int b, int c) __attribute__((always_inline)) { return kr[b][c]; };
    const auto value = [&](int b, int c) __attribute__((always_inline)) { return vr[b][c]; };
    for (int i = 0; i < mine; ++i) {
        const int k0 = (t0 + 4 * i) * 64;
        const bool masked = !ok || k0 < last.lo || k0 + 64 > first.hi;
        sc = nsc;
        at = tiles.take(a, h, next);            // the next tile (past the last one: any)
        v4f s[QT][4];
        uint32_t p[QT][8];
        f.score_tile(s, sc.x, key);
        __builtin_amdgcn_sched_barrier(0);
        load_k(at);                                      // in flight while this tile is worked on
        __builtin_amdgcn_sched_barrier(0);
        if (masked) {
            sc.y &= ok ? kept_blocks(k0, first.lo, last.hi) : 0u;
            f.mask(s, ok ? k0 : kNowhere);
#pragma unroll
            for (int b = 0; b < 4; ++b)
#pragma unroll
                for (int c = 0; c < C; ++c) {            // (NaN values are seen to in the end)
                    vr[b][c] = and4(vr[b][c], ok ? kept_bytes(k0, b, first.lo, last.hi) : 0u);
                    nans |= nan_codes4(vr[b][c]);
                    vr[b][c] = without_nan(vr[b][c]);
                }
        }
        f.settle(a, s);
        f.weights(a, s, p);
        uint32_t v[4][4];
        f.read_values(v, 0, value);
        f.sums(sc.y, p, value, v);
        __builtin_amdgcn_sched_barrier(0);
        load_v(at);
        ok = next;
    }
    if (__ballot(nans != 0)) {
#pragma unroll 1
        for (int i = 0; i < mine; ++i) {
            const int t = t0 + 4 * i, k0 = t * 64, pg = uni(t / a.c.tiles);
            const int page = a.s.table[(int64_t)w.b * a.s.width + pg];
            if ((k0 >= last.lo && k0 + 64 <= first.hi) || (uint32_t)page >= (uint64_t)a.c.pages) continue;
            const int64_t u = ((int64_t)page * a.c.H + h) * a.c.tiles + t - pg * a.c.tiles;
            nan_tile(f, a.c.data + u * tile_bytes + tile_bytes / 2, k0, first.lo, last.hi);
        }
    }
    // the waves' maxima and sums, then their outputs 64 channels at a time
#pragma unroll
    for (int t = 0; t < QT; ++t) {
        const float l = f.l[t][0];
        if (g == 0) {
            stat[wave][t * 16 + l16][0] = f.m[t];
            stat[wave][t * 16 + l16][1] = l;
        }
    }
    const int row = tid >> 4, c4 = (tid & 15) * 4;       // of the joined outputs
#pragma unroll
    for (int c = 0; c < C; ++c) {
        if (c) __syncthreads();
#pragma unroll
        for (int t = 0; t < QT; ++t)
#pragma unroll
            for (int u = 0; u < 4; ++u) *(v4f*)&red[wave][t * 16 + l16][u * 16 + g * 4] = f.o[t][c * 4 + u];
        __syncthreads();
#pragma unroll
        for (int t = 0; t < QT; ++t) {
            const int r = t * 16 + row;
            float m = stat[0][r][0];
#pragma unroll
            for (int k = 1; k < 4; ++k) m = fmaxf(m, stat[k][r][0]);
            float sum = 0.0f;
            v4f y = v4f{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const float s = share_of(stat[k][r][0], m, a.scale2);
                sum = __builtin_fmaf(s, stat[k][r][1], sum);
                const v4f v = *(const v4f*)&red[k][r][c4];
#pragma unroll
                for (int e = 0; e < 4; ++e) y[e] = __builtin_fmaf(s, v[e], y[e]);
            }
            if (r < w.rows) {
                const Row x = row_of(a, w, h, w.row0 + r);
                const int d = c * 64 + c4;
                if (slot >= 0) {
                    *(v4f*)(part_sums<R>(a, slot, r, W) + d) = y;
                    if (c == 0 && c4 == 0) *(float2*)part_stats<R>(a, slot, r, W) = make_float2(m, sum);
                } else if (d < a.c.D) {
                    const float n = sum != 0.0f ? kValueUnit / sum : 0.0f;
                    *(uint2*)(a.y + x.t * a.yts + x.h * a.yhs + d) =
                        make_uint2(bf16x2(y[0] * n, y[1] * n), bf16x2(y[2] * n, y[3] * n));
                }
            }
        }
    }
}

template <int C, int QT>
__global__ __launch_bounds__(256, C <= 2 && QT == 1 ? 2 : 1) void attend_few_kernel(KvAttendArgs a) {
    constexpr int R = 16 * QT;
    __shared__ __attribute__((aligned(16))) float red[4][R][68];
    __shared__ float stat[4][R][2];
    Line<R> line;
    const int total = line.total(a);
    if (total == 0) return;
    const int share = tiles_of(a, total), all = total * a.c.H;
    if ((int64_t)blockIdx.x * share >= all) return;
    int x = blockIdx.x * share;
    const int end = all - x < share ? all : x + share;
    int h = uni((uint32_t)x / (uint32_t)total);
    int at = x - h * total;                              // on head h's line
    if (a.s.B > 64) line.restart();
    for (bool again = false; x < end; again = true) {
        if (again) __syncthreads();                      // (the last piece's sums are read)
        if (at >= total) {
            at -= total;
            ++h;
            if (a.s.B > 64) line.restart();
        }
        while (at >= line.before + line.sum) {
            if (line.b0 + 64 >= a.s.B) return;           // lengths that fell since they were added up: no more tiles
            line.next(a);
        }
        const unsigned long long hit = __ballot(at >= line.start && at < line.start + line.units);
        const int src = __builtin_ctzll(hit);
        const int pad = __builtin_amdgcn_readlane(line.pad, src);
        const int into = at - __builtin_amdgcn_readlane(line.start, src);
        const int part = uni((uint32_t)into / (uint32_t)pad), from = into - part * pad;
        const int to = end - x < pad - from ? from + end - x : pad;
        Work w;
        w.b = line.b0 + src;
        w.t0 = __builtin_amdgcn_readlane(line.lo, src);
        w.n = __builtin_amdgcn_readlane(line.n, src);
        w.len = __builtin_amdgcn_readlane(line.len, src);
        w.room = (int)kv_room(a.s, a.c);
        w.row0 = part * R;
        const int left = w.n * a.G - w.row0;
        w.rows = left < R ? left : R;
        const int ta = __builtin_amdgcn_readlane(line.ta, src), tb = ta + __builtin_amdgcn_readlane(line.nt, src);
        w.ta = ta + from;
        w.tb = ta + to < tb ? ta + to : tb;
        const int64_t slot = from == 0 && to == pad ? -1 : 2 * (int64_t)blockIdx.x + (from == 0);
        piece<C, QT>(a, w, h, slot, red, stat);
        x += to - from;
        at += to - from;
    }
}

// ---------------------------------------------------------------- pieces joined

// A workgroup per (token, query head): its pieces' sums, weighted by their references,
// dealt to four waves and joined in LDS.
template <int C, int QT>
__global__ __launch_bounds__(256) void attend_few_join_kernel(KvAttendArgs a) {
    constexpr int R = 16 * QT, W = 64 * C;
    __shared__ float red[4][W], stat[4][2];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int t = blockIdx.x, h = blockIdx.y, kh = uni(h / a.G);
    Line<R> line;
    const int total = line.total(a), share = tiles_of(a, total);
    unsigned long long hit = 0;
    if (a.s.B > 64) line.restart();
    else hit = __ballot(t >= line.lo && t < line.lo + line.n);
    while (!hit) {
        if (line.b0 + 64 >= a.s.B) return;               // of no sequence: left as it is
        line.next(a);
        hit = __ballot(t >= line.lo && t < line.lo + line.n);
    }
    const int src = __builtin_ctzll(hit);
    const int r = (t - __builtin_amdgcn_readlane(line.lo, src)) * a.G + h - kh * a.G, i = r % R;
    const int pad = __builtin_amdgcn_readlane(line.pad, src);
    const uint32_t from = kh * total + __builtin_amdgcn_readlane(line.start, src) + r / R * pad;
    int w0 = uni(from / (uint32_t)share), w1 = uni((from + pad - 1) / (uint32_t)share);
    if (w0 == w1) return;                                // one piece: written already
    if (w1 >= a.S) w1 = a.S - 1;                         // (lengths that have changed since: in bounds all the same)
    if (w0 > w1) w0 = w1;
    // piece 0 is the last of workgroup w0, piece j > 0 the first of w0 + j
    const int pieces = w1 - w0 + 1;
    auto slot = [&](int j) __attribute__((always_inline)) { return (int64_t)(j ? 2 * (w0 + j) : 2 * w0 + 1); };
    float m = kNone;
    for (int j = lane; j < pieces; j += 64) m = fmaxf(m, part_stats<R>(a, slot(j), i, W)[0]);
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) m = fmaxf(m, __shfl_xor(m, d));
    float y[C], sum = 0.0f;
#pragma unroll
    for (int c = 0; c < C; ++c) y[c] = 0.0f;
#pragma unroll 4
    for (int j = wave; j < pieces; j += 4) {
        const float2 st = *(const float2*)part_stats<R>(a, slot(j), i, W);
        const float wgt = share_of(st.x, m, a.scale2);
        const float* p = part_sums<R>(a, slot(j), i, W);
        sum = __builtin_fmaf(wgt, st.y, sum);
#pragma unroll
        for (int c = 0; c < C; ++c) y[c] = __builtin_fmaf(wgt, p[c * 64 + lane], y[c]);
    }
#pragma unroll
    for (int c = 0; c < C; ++c) red[wave][c * 64 + lane] = y[c];
    if (lane == 0) stat[wave][0] = sum;
    __syncthreads();
    const float all = stat[0][0] + stat[1][0] + stat[2][0] + stat[3][0], n = all != 0.0f ? kValueUnit / all : 0.0f;
    uint16_t* out = a.y + t * a.yts + h * a.yhs;
    for (int d = threadIdx.x; d < a.c.D; d += 256) out[d] = f32_to_bf16_bits((red[0][d] + red[1][d] + red[2][d] + red[3][d]) * n);
}

// whether the tiles of all row tiles and key heads can be numbered
}  // namespace
bool kv_attend_few_fits(const KvBatch& s, const KvCache& c, int G, int rows) {
    const int64_t tiles = s.offs ? s.T * G / rows + s.B : s.B * (((int64_t)s.n * G + rows - 1) / rows);
    return (double)tiles * c.H * ((double)s.width * c.tiles + 4.0) < 2147483648.0;
}
namespace {

// workgroups: as many as stay on the chip at a time, or one for each four tiles if those are fewer
int64_t shares(const KvBatch& s, const KvCache& c, int G, int rows, int cus) {
    const int64_t pad = (((int64_t)s.width * c.tiles + 3) & ~(int64_t)3) < 4 ? 4 : ((int64_t)s.width * c.tiles + 3) & ~(int64_t)3;
    const int64_t tiles = s.offs ? s.T * G / rows + s.B : s.B * (((int64_t)s.n * G + rows - 1) / rows);
    const int64_t places = (int64_t)cus * ((c.D <= 128 && rows == 16) ? 2 : 1);
    const double most = (double)tiles * c.H * (double)pad / 4.0;
    return most < (double)places ? (int64_t)most : places;
}

template <int C, int QT>
void launch(const KvAttendArgs& a, hipStream_t stream) {
    hipLaunchKernelGGL((attend_few_kernel<C, QT>), dim3((unsigned)a.S), dim3(256), 0, stream, a);
    if (a.part) hipLaunchKernelGGL((attend_few_join_kernel<C, QT>), dim3((unsigned)a.s.T, (unsigned)(a.G * a.c.H)), dim3(256), 0, stream, a);
}

template <int C>
void launch(const KvAttendArgs& a, int rows, hipStream_t stream) {
    if constexpr (C <= 2)
        if (rows == 32) return launch<C, 2>(a, stream);
    launch<C, 1>(a, stream);
}

}  // namespace

// A cache of four tiles a sequence at the most whose workgroups take four each: no piece.
int64_t kv_attend_few_workspace(const KvBatch& s, const KvCache& c, int G, int rows, int cus) {
    const int64_t S = shares(s, c, G, rows, cus), items = s.offs ? s.T * G / rows + s.B : s.B * (((int64_t)s.n * G + rows - 1) / rows);
    if ((int64_t)s.width * c.tiles <= 4 && items * c.H <= S) return 0;
    return 2 * S * rows * ((c.D + 63) / 64 * 64 + 2) * 4;
}

hipError_t launch_kv_attend_few(KvAttendArgs a, int rows, int cus, hipStream_t stream) {
    a.S = (int)shares(a.s, a.c, a.G, rows, cus);
    if (!kv_attend_few_workspace(a.s, a.c, a.G, rows, cus)) a.part = nullptr;
    switch ((a.c.D + 63) / 64) {
        case 1: launch<1>(a, rows, stream); break;
        case 2: launch<2>(a, rows, stream); break;
        case 3: launch<3>(a, rows, stream); break;
        default: launch<4>(a, rows, stream);
    }
    return hipGetLastError();
}
