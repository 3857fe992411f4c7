// A paged cache of keys and values in 8 bits: its layout, and the sequences of
// a call. Filled by the C ABI's host side; shared by kv_append.hip (which
// writes the cache) and kv_attend_few.hip, kv_attend_many.hip (which read it).
//
// A page holds 64 `tiles` tokens of every key head; a tile (64 tokens of one
// head) is contiguous: 4 blocks of 16 tokens of keys, then 4 of values, C =
// ceil(D / 64) runs of 1024 E4M3 codes each. The codes of a block and side
// stand for code * 2^e with one exponent e, stored as the byte e + 127 (E8M0):
// the matrix pipe takes it as a block scale of the keys, the conversion
// v_cvt_scalef32_pk_bf16_fp8 as the scale of the values, both for nothing.
//
// The order within a run is the order in which a wave's lanes hold matrix
// operands, so both sides are read 16 bytes a lane, 1 KB contiguous, and used
// as they come:
//   keys    byte (g * 16 + key) * 16 + j = channel 16 g + j of token `key`: lane
//           16 g + key holds 16 channels of its key
//   values  byte (g * 16 + r) * 16 + 4 u + j = channel 16 u + r of token 4 g + j:
//           lane 16 g + r holds four tokens of four of the value operand's rows
#pragma once
#include "lanes.h"
#include "rope.h"

constexpr int kKvExpMin = -120;      // least exponent of a block (a block of zeros has it)
constexpr int kKvExpMax = 120;       // the largest: fp32's largest number is code 256 there

struct KvCache {
    uint8_t* data;                   // [pages][H][tiles][2][4][C][1024]
    uint8_t* scales;                 // [pages][H][tiles][2][4]
    int64_t pages;
    int H, D, tiles;
};

struct KvBatch {
    const int* table;                // [B][width] pages of each sequence, in order
    const int* lengths;              // [B] tokens in the cache, the call's own among them
    const int* offs;                 // [B + 1] the call's tokens by sequence, or NULL: n each
    int64_t T;
    int B, width, n;
};

// An item of work of a ragged batch: tokens t0 .. t0 + n - 1 belong to
// sequence b, and the item is the part-th of its items.
struct KvItem {
    int b, t0, n, part;
};

// The lane's tokens of 64 sequences from b0 on: n from lo. Offsets are clamped into [0, T], and one
// that falls counts as the largest before it (`done`, carried along), so no token belongs to two
// sequences.
DEV void kv_offsets(const KvBatch& s, int b0, int& done, int& lo, int& n) {
    const int lane = threadIdx.x & 63, T = (int)s.T, b = b0 + lane;
    int hi = 0;
    lo = 0;
    if (b < s.B) {
        lo = s.offs[b];
        hi = s.offs[b + 1];
        lo = lo < 0 ? 0 : lo > T ? T : lo;
        hi = hi < 0 ? 0 : hi > T ? T : hi;
    }
    if (__builtin_amdgcn_readfirstlane(lo) < done || __ballot(b < s.B && hi < lo)) {
        int top = lo > done ? lo : done;                 // somewhere they fall: each becomes the largest up to it
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            const int o = __shfl_up(top, d);
            if (lane >= d && o > top) top = o;
        }
        lo = top;
        hi = hi < lo ? lo : hi;
    }
    done = __builtin_amdgcn_readlane(hi, s.B - b0 < 64 ? s.B - b0 - 1 : 63);
    n = b < s.B ? hi - lo : 0;
}

// The sequence of item `item`, found by every wave on its own, 64 sequences at
// a time. base(o, b): the first item of sequence b whose tokens start at o;
// count(n): items of n tokens; base(o + n, b + 1) - base(o, b) >= count(n).
// False: no such item.
template <class BASE, class COUNT>
DEV bool kv_find(const KvBatch& s, int item, BASE base, COUNT count, KvItem& r) {
    if (!s.offs) {
        const int per = count(s.n);
        r.b = per ? item / per : s.B;
        r.part = item - r.b * per;
        r.t0 = r.b * s.n;
        r.n = s.n;
        return r.b < s.B;
    }
    int done = 0;                                        // the largest offset so far
    for (int b0 = 0; b0 < s.B; b0 += 64) {
        const int b = b0 + (threadIdx.x & 63);
        int lo, n;
        kv_offsets(s, b0, done, lo, n);
        const int first = base(lo, b);
        const unsigned long long hit = __ballot(b < s.B && item >= first && item < first + count(n));
        if (hit) {
            const int src = __builtin_ctzll(hit);
            r.b = b0 + src;
            r.t0 = __builtin_amdgcn_readlane(lo, src);
            r.n = __builtin_amdgcn_readlane(n, src);
            r.part = item - __builtin_amdgcn_readlane(first, src);
            return true;
        }
    }
    return false;
}

// tokens that a row of the table has room for
DEV int64_t kv_room(const KvBatch& s, const KvCache& c) { return (int64_t)s.width * c.tiles * 64; }

// the largest of the four lanes that share a column (lane % 16) of a 16 x 16
// result: two exchanges of rows of 16 lanes on the vector unit
DEV float rows4_max(float v) {
    const uint32_t x = __float_as_uint(v);
    const auto a = __builtin_amdgcn_permlane32_swap(x, x, false, false);
    v = fmaxf(__uint_as_float(a[0]), __uint_as_float(a[1]));
    const uint32_t y = __float_as_uint(v);
    const auto b = __builtin_amdgcn_permlane16_swap(y, y, false, false);
    return fmaxf(__uint_as_float(b[0]), __uint_as_float(b[1]));
}
// least e with amax <= 448 * 2^e, at least kKvExpMin (amax finite, >= 0)
DEV int kv_exponent(float amax) {
    // 448 = 1.75 * 2^8: by the exponent field, one more where the fraction is past .75
    const uint32_t u = __float_as_uint(amax);
    const int e = (int)(u >> 23) - 127 - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
    return e < kKvExpMin ? kKvExpMin : e;
}

// the exponent of a block that is there already (a byte past the largest that an append writes counts as it)
DEV int kv_old_exponent(uint8_t e) { return (e > kKvExpMax + 127 ? kKvExpMax + 127 : (int)e) - 127; }

// 2^e, e in [-126, 127]
DEV float exp2i(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

struct KvAppendArgs {
    KvCache c;
    KvBatch s;
    const uint16_t *k, *v, *norm;    // norm [D] or NULL
    int64_t kts, khs, vts, vhs;
    const void* pos;
    const double* turns;             // as RopeArgs has them
    const int* axis;
    int axes, pos_f32, pairs;
    float eps;
    int items, per, groups;          // blocks of tokens at the most; key heads a workgroup, workgroups a block
    int qx;                          // workgroups of the queries' tokens
};

struct KvAttendArgs {
    KvCache c;
    KvBatch s;
    const uint16_t* q;
    uint16_t* y;
    int64_t qts, qhs, yts, yhs;
    int G;                           // query heads of a key head
    int causal, window;              // window 0: none
    float scale2;                    // scale * log2(e)
    float* part;                     // pieces of rows: weighted sums, then references and weights' sums
    int S;                           // splits of a split row tile; workgroups (few rows)
    int items, whole;                // many rows: row tiles of a key head; those of all heads that are not split
};

hipError_t launch_kv_append(KvAppendArgs a, RopeArgs q, int half, int cus, hipStream_t stream);
bool kv_attend_few_fits(const KvBatch& s, const KvCache& c, int G, int rows);
int64_t kv_attend_few_workspace(const KvBatch& s, const KvCache& c, int G, int rows, int cus);
int64_t kv_attend_many_workspace(const KvBatch& s, const KvCache& c, int G, int cus);
hipError_t launch_kv_attend_few(KvAttendArgs a, int rows, int cus, hipStream_t stream);
hipError_t launch_kv_attend_many(KvAttendArgs a, int cus, hipStream_t stream);

// Query rows of a sequence (tokens * query heads of a key head), on the average, decide: up to 32 go to
// the few-rows kernel, in row tiles of 16 or 32 (wide heads: 16, whose sums and operands fit the
// registers), more (0) to the other. (64 sequences to 8192 tokens, 32 heads over 8:
// 1 token, 4 rows, 114 us with few rows, 193 with many; 32 rows 161 and 200; 36 rows 275 and 217.)
static inline int kv_attend_rows(const KvBatch& s, int D, int G) {
    const int64_t most = s.offs ? (s.T * G + s.B - 1) / s.B : (int64_t)s.n * G;
    return most > 32 ? 0 : most > 16 && D <= 128 ? 32 : 16;
}
