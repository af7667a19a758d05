// What the kernels of cache attention (fwd_cache.cu, fwd_cache_tile.cu) share: the
// tokens of a tile of rows, the line of all steps that a grid's blocks share out,
// and the conversion of codes to fp16.
#pragma once

#include "cache.cuh"
#include "sm100_ptx.cuh"

namespace spattn {
namespace cache_attn {

constexpr float kNone = -1e30f;      // reference of a row without a token so far
// Weights are stored in fp16: up to 2^16, in steps of 2^-24 when small. The largest is kept high, so
// that many light tokens are not lost beside a heavy one: a weight is off by at most 2^-33 of it.
// (With 2^10 for 2^8 the reference moves more often: 409 us for 390 on a chunk of 2 x 2048 tokens.)
constexpr float kRescaleAt = 15.f;   // largest exponent of a weight before the reference moves
constexpr float kHeadroom = 8.f;     // exponent of the largest weight after it moved
constexpr float kMinScale = 7.8886090522101181e-31f;  // 2^-100: a V scale below it counts as 0
// In place of the log2 of such a scale, and of 1 / scale. Its tokens count in l alone. A small
// substitute, so that they do not raise the reference above what the pages with values need (taken as
// 1, they left weights of V scales of 2^-24 no bits in fp16); not so small that their weights leave
// the range of fp32 beside V scales up to 2^30.
constexpr float kNoValues = -64.f, kNoValuesInv = 1.8446744073709552e19f;  // 2^64

constexpr long long kCacheWaitCycles = 2000000000LL;  // limit of a wait for a copy: about one second
constexpr int kUnread = -0x7fffffff; // page of a sub-block that needs none
constexpr float kNoPage = -1.f;      // in place of the K scale of a sub-block that has no page

// What a block leaves for the joining kernel: the segment that it began and later
// blocks went on with, if there is one (more = how many).
struct Begun {
    int more, b, first_row, rows, hk, pad[3];
};
// A (sequence, row tile): the tokens its rows attend to, as groups of GROUP tokens:
// na groups of the global tokens [0, a_hi), then the groups from b_first on that
// hold [b_lo, b_hi).
struct Tile {
    int b, first_row, rows;  // valid rows
    int base;                // pos of query 0
    int a_hi, b_lo, b_hi;
    int na, b_first, groups; // groups >= 1
    int full_hi, full_lo, full_a;  // every row attends to [full_lo, full_hi) of the second part, [0, full_a) of the first
};

template <int GROUP, int ROWS>
__device__ __forceinline__ Tile make_tile(const CacheFwdParams& p, int b, int rt) {
    Tile t;
    const int64_t cap = cache_capacity(p.c);
    int64_t n64 = p.seqlen[b];
    const int n = (int)(n64 < 0 ? 0 : n64 < cap ? n64 : cap);
    int nq = p.qlen ? p.qlen[b] : p.m;
    nq = nq < 0 ? 0 : nq < p.m ? nq : p.m;
    t.b = b;
    t.first_row = rt * ROWS;
    const int64_t left = (int64_t)nq * p.G - t.first_row;
    t.rows = (int)(left < 0 ? 0 : left < ROWS ? left : ROWS);
    t.base = n - nq;
    int lo_pos = t.base, hi_pos = t.base + (nq > 0 ? nq : 1) - 1;  // of a sequence's only tile
    if ((int64_t)p.m * p.G > ROWS) {
        lo_pos = t.base + t.first_row / p.G;
        hi_pos = t.base + (t.first_row + (t.rows > 0 ? t.rows : 1) - 1) / p.G;
    }
    t.b_hi = t.rows > 0 && hi_pos >= 0 ? hi_pos + 1 : 0;
    const int win = p.window < 0 ? 0x7fffffff : p.window;
    t.b_lo = lo_pos > win ? lo_pos - win : 0;
    t.a_hi = p.n_global < t.b_hi ? p.n_global : t.b_hi;
    if (p.window < 0 || t.b_lo <= t.a_hi) t.b_lo = t.a_hi = 0;  // one run
    t.na = (t.a_hi + GROUP - 1) / GROUP;
    t.b_first = t.b_lo / GROUP;
    const int end = (t.b_hi + GROUP - 1) / GROUP;
    t.groups = t.na + (end > t.b_first ? end - t.b_first : 0);
    if (t.groups < 1) t.groups = 1;
    t.full_hi = lo_pos + 1;
    t.full_lo = hi_pos > win ? hi_pos - win : 0;
    t.full_a = p.n_global < t.full_hi ? p.n_global : t.full_hi;
    return t;
}

template <int ROWS>
__host__ __device__ __forceinline__ int row_tiles(const CacheFwdParams& p) {
    return (int)(((int64_t)p.m * p.G + ROWS - 1) / ROWS);
}

// The line of all steps: entry e = (sequence, row tile) holds Hk segments one after
// the other, each of the tile's groups. Every warp works it out for itself (no
// barrier; a block's start counts in a token's step): lane x sums the entries
// [x per, (x + 1) per).
template <int GROUP, int ROWS>
struct Line {
    int64_t total;   // places
    int64_t before;  // places before this lane's entries
    int per, entries, rts;
    __device__ __forceinline__ int groups(const CacheFwdParams& p, int e) const {
        return rts == 1 ? make_tile<GROUP, ROWS>(p, e, 0).groups : make_tile<GROUP, ROWS>(p, e / rts, e % rts).groups;
    }
    __device__ __forceinline__ explicit Line(const CacheFwdParams& p) {
        rts = row_tiles<ROWS>(p);
        entries = p.B * rts;
        per = (entries + 31) >> 5;
        const int lane = threadIdx.x & 31;
        int64_t mine = 0;
        for (int e = lane * per; e < entries && e < (lane + 1) * per; ++e) mine += groups(p, e);
        mine *= p.c.Hk;
        int64_t x = mine;
#pragma unroll
        for (int y = 1; y < 32; y <<= 1) {
            const int64_t up = __shfl_up_sync(0xffffffffu, x, y);
            if (lane >= y) x += up;
        }
        before = x - mine;
        total = __shfl_sync(0xffffffffu, x, 31);
    }
    // The entry that holds place `at` < total, and its first place.
    __device__ __forceinline__ void find(const CacheFwdParams& p, int64_t at, int* entry, int64_t* first) const {
        // the last lane whose entries begin at or before it (lanes behind the entries begin at `total`)
        const int lane = 31 - __clz(__ballot_sync(0xffffffffu, before <= at));
        int64_t place = __shfl_sync(0xffffffffu, before, lane);
        int e = lane * per;
        while (true) {
            const int64_t len = (int64_t)groups(p, e) * p.c.Hk;
            if (place + len > at) break;
            place += len;
            ++e;
        }
        *entry = e;
        *first = place;
    }
};

// a / b for a >= 0, b > 0, in 32 bits where they fit (a fraction of the time).
__device__ __forceinline__ int64_t quotient(int64_t a, int64_t b) {
    return ((a | b) >> 32) == 0 ? (int64_t)((uint32_t)a / (uint32_t)b) : a / b;
}
// The line's blocks: the first `longer` of `blocks` hold share + 1 places, the others `share`.
struct Shares {
    int blocks;
    int64_t share, longer;
    __device__ __forceinline__ Shares(int64_t total, int grid) {
        blocks = total < grid ? (int)total : grid;
        share = quotient(total, blocks);
        longer = total - share * blocks;
    }
    __device__ __forceinline__ int64_t start(int x) const { return share * x + (x < longer ? x : longer); }
    __device__ __forceinline__ int block_of(int64_t place) const {
        const int64_t cut = (share + 1) * longer;
        return (int)(place < cut ? quotient(place, share + 1) : longer + quotient(place - cut, share));
    }
};

// A walk over the groups of a tile: group x, its first token j.
template <int GROUP>
struct Walk {
    int x, j;
    __device__ __forceinline__ void begin(const Tile& t, int x0) {
        x = x0;
        j = (x0 < t.na ? x0 : t.b_first + x0 - t.na) * GROUP;
    }
    __device__ __forceinline__ void next(const Tile& t) {
        ++x;
        j = x == t.na ? j + (t.b_first - t.na + 1) * GROUP : j + GROUP;
    }
    __device__ __forceinline__ int lo(const Tile& t) const { return x < t.na ? 0 : t.b_lo; }
    __device__ __forceinline__ int hi(const Tile& t) const { return x < t.na ? t.a_hi : t.b_hi; }
};

// A block's part of the line, segment by segment.
template <int GROUP, int ROWS>
struct Part {
    int64_t at, end, place;  // next step, one past the last, the entry's first
    int entry;
    Tile t;
    int hk, first, last;  // of the current segment
    __device__ __forceinline__ bool open(const CacheFwdParams& p, int rts) {  // the segment that holds `at`
        if (at >= end) return false;
        t = rts == 1 ? make_tile<GROUP, ROWS>(p, entry, 0) : make_tile<GROUP, ROWS>(p, entry / rts, entry % rts);
        hk = (int)quotient(at - place, t.groups);
        first = (int)(at - place - (int64_t)hk * t.groups);
        last = end - at < t.groups - first ? first + (int)(end - at) : t.groups;  // one past
        return true;
    }
    __device__ __forceinline__ void close(const CacheFwdParams& p) {  // on to the next one
        at += last - first;
        if (at >= place + (int64_t)t.groups * p.c.Hk) {
            place += (int64_t)t.groups * p.c.Hk;
            ++entry;
        }
    }
};

// Four codes of a word as two fp16 pairs. int8: 1024 + (c + 128) is the fp16
// number 0x6400 | (c ^ 0x80); subtracting 1152 is exact.
template <int CODE>
__device__ __forceinline__ void codes_to_half(uint32_t w, uint32_t& lo, uint32_t& hi) {
    if constexpr (CODE == kCodeI8) {
        w ^= 0x80808080u;
        const uint32_t a = __byte_perm(w, 0x64646464u, 0x4140), b = __byte_perm(w, 0x64646464u, 0x4342);
        asm("sub.f16x2 %0, %1, %2;" : "=r"(lo) : "r"(a), "r"(0x64806480u));
        asm("sub.f16x2 %0, %1, %2;" : "=r"(hi) : "r"(b), "r"(0x64806480u));
    } else {
        asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\t"
            "cvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
            : "=r"(lo), "=r"(hi)
            : "r"(w));
    }
}

__device__ __forceinline__ uint32_t half_pair(float a, float b) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
}

}  // namespace cache_attn
}  // namespace spattn
