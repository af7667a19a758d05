// Attention of a sequence's last tokens over its 8-bit key/value cache.
//
// Query t < qlen[b] of sequence b is token pos = seqlen[b] - qlen[b] + t. It
// attends to the tokens j <= pos, and with a window only to those with
// j >= pos - window or j < n_global:
//     s_j = scale <q, k_j>,  out = sum_j softmax_j(s) v_j,  lse = log sum_j exp(s_j)
//
// Rows. The m * G rows (query t, head g of the group) of a (sequence, K/V head)
// share its tokens and are cut into tiles of 16, the M of mma.m16n8k16 (fp16 in,
// fp32 out). A row tile of one K/V head is a segment. Codes are exact in fp16,
// and so are bf16 queries once a row is scaled by a power of two that brings its
// largest element to [2^14, 2^15) (elements 2^-28 below it lose bits): QK^T is
// exact up to fp32 accumulation. fp32 queries and their weights go in as the sum
// of two fp16 numbers (22 bits), at twice the products.
//
// Scales. A page's K scale multiplies its scores. Its V scale vs goes into the
// exponent: p' = 2^(x + log2 vs - m) with x the score in base 2, so that weights
// are largest where p v is, whatever the scales; O = sum p' c, l = sum p' / vs.
// Weights are rounded to fp16 for P V (11 bits; bf16 outputs have 8). m is a
// reference that moves only when some p' would pass 2^12 (it then becomes the
// largest exponent - 5), so that most steps need no exchange between lanes.
//
// Streaming. The kernel is bound by HBM at long caches: each code is read once,
// by cp.async of 16 (8, 4) bytes into a ring of kStages steps in shared memory.
// A lane copies exactly the bytes that its own mma fragments need (any order of
// d and of the output's columns does for a product as long as both sides use the
// same one), so that nothing is exchanged, transposed or synchronised: K
// fragments are 4 neighbouring codes of a token, V fragments byte columns of four
// tokens. A warp's step is 128 / D sub-blocks of 16 tokens, each inside one page.
//
// Work. All segments' steps form one line, which the grid's blocks share evenly
// (they know it from the lengths alone), so that one long sequence among short
// ones is spread over the GPU. A block that holds a whole segment writes its
// rows; pieces of a segment go to a workspace as (m, l, O), and k_fwd_cache_join
// adds them up by the running max / sum rule.
#include "cache.cuh"
#include "sm100_ptx.cuh"

#include <type_traits>

namespace spattn {
namespace {

using sm100::ex2;

constexpr int kWarps = 4;
constexpr float kNone = -1e30f;      // reference of a row without a token so far
constexpr float kRescaleAt = 12.f;   // largest exponent of a weight before the reference moves
constexpr float kHeadroom = 5.f;     // exponent of the largest weight after it moved
constexpr float kMinScale = 7.8886090522101181e-31f;  // 2^-100: a V scale below it counts as 0

constexpr float kNoPage = -1.f;      // in place of the K scale of a sub-block that has no page

// Sizes that follow from the head dim.
template <int D>
struct Geo {
    static constexpr int kSub = 128 / D;              // sub-blocks of 16 tokens a warp step
    static constexpr int kGroup = kWarps * kSub * 16; // tokens a block step
    static constexpr int kKBytes = D >= 64 ? 16 : 8;  // bytes a K copy
    static constexpr int kKCopies = D / (4 * kKBytes);// of each token, by a lane
    static constexpr int kNT = D / 8;                 // mma tiles over the head dim = bytes a V copy
    static constexpr int kSteps = D / 16;             // mma steps over the head dim
    static constexpr int kStage = 4096;               // bytes of a warp's ring stage: K, then V
    static constexpr int kPiece = 32 + 16 * D;        // floats of a stored piece
};

// A (sequence, row tile): the tokens its rows attend to, as groups of kGroup:
// na groups of the global tokens [0, a_hi), then the groups from b_first on that
// hold [b_lo, b_hi).
struct Tile {
    int b, first_row, rows;  // valid rows
    int base;                // pos of query 0
    int a_hi, b_lo, b_hi;
    int na, b_first, groups; // groups >= 1
    int full_hi, full_lo, full_a;  // every row attends to [full_lo, full_hi) of the second part, [0, full_a) of the first
};

template <int D>
__device__ __forceinline__ Tile make_tile(const CacheFwdParams& p, int b, int rt) {
    Tile t;
    const int64_t cap = cache_capacity(p.c);
    int64_t n64 = p.seqlen[b];
    const int n = (int)(n64 < 0 ? 0 : n64 < cap ? n64 : cap);
    int nq = p.qlen ? p.qlen[b] : p.m;
    nq = nq < 0 ? 0 : nq < p.m ? nq : p.m;
    t.b = b;
    t.first_row = rt * 16;
    const int64_t left = (int64_t)nq * p.G - t.first_row;
    t.rows = (int)(left < 0 ? 0 : left < 16 ? left : 16);
    t.base = n - nq;
    const int lo_pos = t.base + t.first_row / p.G;
    const int hi_pos = t.base + (t.first_row + (t.rows > 0 ? t.rows : 1) - 1) / p.G;
    t.b_hi = t.rows > 0 && hi_pos >= 0 ? hi_pos + 1 : 0;
    const int win = p.window < 0 ? 0x7fffffff : p.window;
    t.b_lo = lo_pos > win ? lo_pos - win : 0;
    t.a_hi = p.n_global < t.b_hi ? p.n_global : t.b_hi;
    if (p.window < 0 || t.b_lo <= t.a_hi) t.b_lo = t.a_hi = 0;  // one run
    t.na = (t.a_hi + Geo<D>::kGroup - 1) / Geo<D>::kGroup;
    t.b_first = t.b_lo / Geo<D>::kGroup;
    const int end = (t.b_hi + Geo<D>::kGroup - 1) / Geo<D>::kGroup;
    t.groups = t.na + (end > t.b_first ? end - t.b_first : 0);
    if (t.groups < 1) t.groups = 1;
    t.full_hi = lo_pos + 1;
    t.full_lo = hi_pos > win ? hi_pos - win : 0;
    t.full_a = p.n_global < t.full_hi ? p.n_global : t.full_hi;
    return t;
}

__host__ __device__ __forceinline__ int row_tiles(const CacheFwdParams& p) { return (int)(((int64_t)p.m * p.G + 15) / 16); }

// The line of all steps: entry e = (sequence, row tile) holds Hk segments one
// after the other. Finds the total, and the entry that holds place `at` (in
// steps of one head, times Hk) with its first place. Every thread of the block
// calls it.
struct Line {
    int64_t total;
};
template <int D>
__device__ Line line_total(const CacheFwdParams& p, int64_t (&sums)[kWarps * 32 + 1]) {
    const int entries = p.B * row_tiles(p), per = (entries + kWarps * 32 - 1) / (kWarps * 32);
    const int tid = threadIdx.x;
    int64_t mine = 0;
    for (int e = tid * per; e < entries && e < (tid + 1) * per; ++e)
        mine += make_tile<D>(p, e / row_tiles(p), e % row_tiles(p)).groups;
    // inclusive scan over the block
    int64_t x = mine;
#pragma unroll
    for (int y = 1; y < 32; y <<= 1) {
        const int64_t up = __shfl_up_sync(0xffffffffu, x, y);
        if ((tid & 31) >= y) x += up;
    }
    sums[tid + 1] = x;
    if (tid == 0) sums[0] = 0;
    __syncthreads();
    int64_t before = 0;
    for (int w = 0; w < (tid >> 5); ++w) before += sums[32 * (w + 1)];
    __syncthreads();
    sums[tid + 1] = x + before;
    __syncthreads();
    return Line{sums[kWarps * 32] * p.c.Hk};
}
// The entry that holds place `at` < total, and its first place.
template <int D>
__device__ void line_find(const CacheFwdParams& p, const int64_t (&sums)[kWarps * 32 + 1], int64_t at, int* entry,
                          int64_t* first) {
    const int per = (p.B * row_tiles(p) + kWarps * 32 - 1) / (kWarps * 32);
    int lo = 0, hi = kWarps * 32 - 1;  // the thread whose entries hold it
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (sums[mid + 1] * p.c.Hk > at) hi = mid;
        else lo = mid + 1;
    }
    int e = lo * per;
    int64_t place = sums[lo] * p.c.Hk;
    while (true) {
        const int64_t len = (int64_t)make_tile<D>(p, e / row_tiles(p), e % row_tiles(p)).groups * p.c.Hk;
        if (place + len > at) break;
        place += len;
        ++e;
    }
    *entry = e;
    *first = place;
}
// Blocks that take part, and the first place of block x of them.
__device__ __forceinline__ int line_blocks(int64_t total, int grid) { return total < grid ? (int)total : grid; }
__device__ __forceinline__ int64_t line_start(int64_t total, int blocks, int x) { return total * x / blocks; }

template <int N>
__device__ __forceinline__ void copy_async(uint32_t dst, const void* src, bool there) {
    const int bytes = there ? N : 0;  // 0: N zeros
    if constexpr (N == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(dst), "l"(src), "n"(N), "r"(bytes) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

template <int N>
__device__ __forceinline__ void load_words(uint32_t addr, uint32_t* w) {
    if constexpr (N == 16)
        asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "r"(addr) : "memory");
    else if constexpr (N == 8)
        asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "r"(addr) : "memory");
    else
        asm volatile("ld.shared.u32 %0, [%1];" : "=r"(w[0]) : "r"(addr) : "memory");
}

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

__device__ __forceinline__ void mma_f16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t half_pair(float a, float b) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
}
// What the fp16 pair `h` leaves of (a, b), as another one.
__device__ __forceinline__ uint32_t half_rest(float a, float b, uint32_t h) {
    const __half2 v = *reinterpret_cast<const __half2*>(&h);
    return half_pair(a - __low2float(v), b - __high2float(v));
}

// A tile's running state in one warp: lane (g = lane / 4, c = lane % 4) holds rows
// g and g + 8. o[j][2 r + e] is row g + 8 r, element NT (2 c + e) + j; m and l
// are the row's (l: this lane's part until it is summed over c).
template <int D>
struct State {
    float o[Geo<D>::kNT][4];
    float m[2], l[2];
    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int j = 0; j < Geo<D>::kNT; ++j) o[j][0] = o[j][1] = o[j][2] = o[j][3] = 0.f;
        m[0] = m[1] = kNone;
        l[0] = l[1] = 0.f;
    }
    __device__ __forceinline__ void scale(float a0, float a1) {
#pragma unroll
        for (int j = 0; j < Geo<D>::kNT; ++j) {
            o[j][0] *= a0;
            o[j][1] *= a0;
            o[j][2] *= a1;
            o[j][3] *= a1;
        }
        l[0] *= a0;
        l[1] *= a1;
    }
};

template <int D>
struct Join {
    float ml[kWarps][2][16];
    float4 o[2][Geo<D>::kNT][32];  // lane-linear
};

template <int D>
__device__ __forceinline__ float4 get4(const State<D>& s, int x) {  // x: constant after unrolling
    const int r = x / (Geo<D>::kNT / 2), e = x / (Geo<D>::kNT / 4) % 2, j = x % (Geo<D>::kNT / 4) * 4;
    return make_float4(s.o[j][2 * r + e], s.o[j + 1][2 * r + e], s.o[j + 2][2 * r + e], s.o[j + 3][2 * r + e]);
}
template <int D>
__device__ __forceinline__ void add4(State<D>& s, int x, const float4& v, float a) {
    const int r = x / (Geo<D>::kNT / 2), e = x / (Geo<D>::kNT / 4) % 2, j = x % (Geo<D>::kNT / 4) * 4;
    s.o[j][2 * r + e] += v.x * a;
    s.o[j + 1][2 * r + e] += v.y * a;
    s.o[j + 2][2 * r + e] += v.z * a;
    s.o[j + 3][2 * r + e] += v.w * a;
}

// The block's warps' states (l summed over the row's lanes) joined into warp 0's.
template <int D>
__device__ __forceinline__ void join_warps(State<D>& s, Join<D>& sh) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2;
    if ((lane & 3) == 0) {
        sh.ml[warp][0][g] = s.m[0];
        sh.ml[warp][0][g + 8] = s.m[1];
    }
    __syncthreads();
    float top[2];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
        top[r] = sh.ml[0][0][g + 8 * r];
#pragma unroll
        for (int w = 1; w < kWarps; ++w) top[r] = fmaxf(top[r], sh.ml[w][0][g + 8 * r]);
    }
    s.scale(ex2(s.m[0] - top[0]), ex2(s.m[1] - top[1]));
    s.m[0] = top[0];
    s.m[1] = top[1];
    if ((lane & 3) == 0) {
        sh.ml[warp][1][g] = s.l[0];
        sh.ml[warp][1][g + 8] = s.l[1];
    }
    if (warp >= 2) {
#pragma unroll
        for (int x = 0; x < Geo<D>::kNT; ++x) sh.o[warp - 2][x][lane] = get4<D>(s, x);
    }
    __syncthreads();
    if (warp < 2) {
#pragma unroll
        for (int x = 0; x < Geo<D>::kNT; ++x) add4<D>(s, x, sh.o[warp][x][lane], 1.f);
        if (warp == 1) {  // only this warp reads or wrote o[1] since the barrier
#pragma unroll
            for (int x = 0; x < Geo<D>::kNT; ++x) sh.o[1][x][lane] = get4<D>(s, x);
        }
    }
    __syncthreads();
    if (warp == 0) {
#pragma unroll
        for (int x = 0; x < Geo<D>::kNT; ++x) add4<D>(s, x, sh.o[1][x][lane], 1.f);
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            s.l[r] = 0.f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) s.l[r] += sh.ml[w][1][g + 8 * r];
        }
    }
    __syncthreads();  // the buffers may be written again
}

// Warp 0: the finished rows of a tile. Those behind the sequence's queries get
// zeros: the state holds what a query of zeros gave.
template <typename T, int D>
__device__ __forceinline__ void write_rows(const CacheFwdParams& p, const Tile& tile, int hk, State<D>& s) {
    const int lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
#pragma unroll
    for (int r = 0; r < 2; ++r) {
        const int row = tile.first_row + g + 8 * r;
        if (row >= p.m * p.G) continue;
        const int b = tile.b, t = row / p.G, h = hk * p.G + row % p.G;
        if (g + 8 * r >= tile.rows) {
            s.l[r] = 0.f;
#pragma unroll
            for (int j = 0; j < Geo<D>::kNT; ++j) s.o[j][2 * r] = s.o[j][2 * r + 1] = 0.f;
        }
        const float l = s.l[r], inv = l != 0.f ? 1.f / l : 0.f;
        T* out = static_cast<T*>(p.out) + b * p.o_sb + h * p.o_sh + t * p.o_sn + 2 * Geo<D>::kNT * c;
        if constexpr (std::is_same<T, float>::value) {
#pragma unroll
            for (int x = 0; x < Geo<D>::kNT / 2; ++x) {
                const float4 v = get4<D>(s, r * (Geo<D>::kNT / 2) + x);
                reinterpret_cast<float4*>(out)[x] = make_float4(v.x * inv, v.y * inv, v.z * inv, v.w * inv);
            }
        } else {
#pragma unroll
            for (int x = 0; x < Geo<D>::kNT / 4; ++x) {
                uint32_t u[4];
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                    const float4 v = get4<D>(s, r * (Geo<D>::kNT / 2) + 2 * x + y);
                    const __nv_bfloat162 a = __floats2bfloat162_rn(v.x * inv, v.y * inv),
                                         d = __floats2bfloat162_rn(v.z * inv, v.w * inv);
                    u[2 * y] = *reinterpret_cast<const uint32_t*>(&a);
                    u[2 * y + 1] = *reinterpret_cast<const uint32_t*>(&d);
                }
                reinterpret_cast<uint4*>(out)[x] = make_uint4(u[0], u[1], u[2], u[3]);
            }
        }
        if (p.lse && c == 0)
            p.lse[((int64_t)b * p.H + h) * p.m + t] = l != 0.f ? (s.m[r] + log2f(l)) * kLn2 : -INFINITY;
    }
}

// Pieces in the workspace: m and l of the 16 rows, then O lane-linear.
template <int D>
__device__ __forceinline__ void write_piece(float* ws, const State<D>& s, int rows) {
    const int lane = threadIdx.x & 31, g = lane >> 2;
#pragma unroll
    for (int r = 0; r < 2; ++r) {
        if (g + 8 * r >= rows) continue;
        if ((lane & 3) == 0) {
            ws[g + 8 * r] = s.m[r];
            ws[16 + g + 8 * r] = s.l[r];
        }
#pragma unroll
        for (int x = 0; x < Geo<D>::kNT / 2; ++x)
            reinterpret_cast<float4*>(ws + 32)[(r * (Geo<D>::kNT / 2) + x) * 32 + lane] =
                get4<D>(s, r * (Geo<D>::kNT / 2) + x);
    }
}
// Adds a piece to the state (whose l is complete in every lane of the row).
template <int D>
__device__ __forceinline__ void add_piece(const float* ws, State<D>& s, int rows) {
    const int lane = threadIdx.x & 31, g = lane >> 2;
#pragma unroll
    for (int r = 0; r < 2; ++r) {
        if (g + 8 * r >= rows) continue;
        const float m = ws[g + 8 * r], l = ws[16 + g + 8 * r];
        const float top = fmaxf(s.m[r], m), a = ex2(s.m[r] - top), w = ex2(m - top);
        s.m[r] = top;
        s.l[r] = s.l[r] * a + l * w;
#pragma unroll
        for (int j = 0; j < Geo<D>::kNT; ++j) {
            s.o[j][2 * r] *= a;
            s.o[j][2 * r + 1] *= a;
        }
#pragma unroll
        for (int x = 0; x < Geo<D>::kNT / 2; ++x) {
            const float4 v = reinterpret_cast<const float4*>(ws + 32)[(r * (Geo<D>::kNT / 2) + x) * 32 + lane];
            add4<D>(s, r * (Geo<D>::kNT / 2) + x, v, w);
        }
    }
}

// fp32: two fp16 parts.
template <typename T>
constexpr int parts() {
    return std::is_same<T, float>::value ? 2 : 1;
}
template <typename T>
constexpr int stages() {
    return std::is_same<T, float>::value ? 4 : 3;
}
template <typename T>
constexpr int blocks_per_sm() {  // registers: 168 a thread, or 255
    return std::is_same<T, float>::value ? 2 : 3;
}

template <typename T, int D>
struct Shared {
    uint8_t ring[kWarps][stages<T>()][Geo<D>::kStage];
    float scales[kWarps][stages<T>()][2 * Geo<D>::kSub];  // K, V of each sub-block
    Join<D> join;
    int64_t sums[kWarps * 32 + 1];
};

// Queries of a tile as mma A fragments: row g + 8 r of step x holds the elements
// that the lane's K bytes stand for.
template <typename T, int D>
struct Query {
    uint32_t a[parts<T>()][Geo<D>::kSteps][4];
    float factor[2];  // of a row's scores, to base 2
};
template <typename T, int D>
__device__ __forceinline__ void load_query(const CacheFwdParams& p, const Tile& t, int hk, Query<T, D>& q) {
    using G = Geo<D>;
    const int lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
#pragma unroll
    for (int r = 0; r < 2; ++r) {
        float x[D / 4];
        const int row = t.first_row + g + 8 * r;
        if (g + 8 * r < t.rows) {
            const T* src = static_cast<const T*>(p.q) + t.b * p.q_sb + (hk * p.G + row % p.G) * p.q_sh +
                           (row / p.G) * p.q_sn;
            constexpr int V = 16 / sizeof(T);
#pragma unroll
            for (int i = 0; i < G::kKCopies; ++i)
#pragma unroll
                for (int y = 0; y < G::kKBytes; y += V) {
                    const uint4 w = *reinterpret_cast<const uint4*>(src + (i * 4 + c) * G::kKBytes + y);
                    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                    for (int z = 0; z < V; ++z)
                        x[i * G::kKBytes + y + z] =
                            V == 4 ? __uint_as_float(u[z % 4])
                                   : __uint_as_float(z & 1 ? u[z / 2 % 4] & 0xffff0000u : u[z / 2 % 4] << 16);
                }
        } else {
#pragma unroll
            for (int y = 0; y < D / 4; ++y) x[y] = 0.f;
        }
        float top = 0.f;
#pragma unroll
        for (int y = 0; y < D / 4; ++y) top = fmaxf(top, fabsf(x[y]));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
        int up = 0;  // 2^up brings the largest element to [2^14, 2^15)
        if (top > 0.f && top < INFINITY) up = 14 - ilogbf(top);
        up = up > 120 ? 120 : up;
        const float by = exp2f((float)up);
        q.factor[r] = p.scale_log2 * exp2f((float)-up);
#pragma unroll
        for (int s = 0; s < G::kSteps; ++s) {
            const float v0 = x[4 * s] * by, v1 = x[4 * s + 1] * by, v2 = x[4 * s + 2] * by, v3 = x[4 * s + 3] * by;
            q.a[0][s][r] = half_pair(v0, v1);
            q.a[0][s][2 + r] = half_pair(v2, v3);
            if constexpr (parts<T>() == 2) {
                q.a[1][s][r] = half_rest(v0, v1, q.a[0][s][r]);
                q.a[1][s][2 + r] = half_rest(v2, v3, q.a[0][s][2 + r]);
            }
        }
    }
}

// The first token of a warp's step in group x of the tile, and the run it belongs to.
template <int D>
__device__ __forceinline__ int step_tokens(const Tile& t, int x, int warp, int& lo, int& hi) {
    const bool a = x < t.na;
    lo = a ? 0 : t.b_lo;
    hi = a ? t.a_hi : t.b_hi;
    return (a ? x : t.b_first + x - t.na) * Geo<D>::kGroup + warp * Geo<D>::kSub * 16;
}

template <typename T, int CODE, int D>
__global__ void __launch_bounds__(kWarps * 32, blocks_per_sm<T>()) k_fwd_cache(CacheFwdParams p, float* ws) {
    using G = Geo<D>;
    constexpr int kS = stages<T>(), kParts = parts<T>();
    extern __shared__ __align__(16) uint8_t smem_raw[];
    Shared<T, D>& sh = *reinterpret_cast<Shared<T, D>*>(smem_raw);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
    asm volatile("griddepcontrol.launch_dependents;");

    const Line line = line_total<D>(p, sh.sums);
    const int blocks = line_blocks(line.total, (int)gridDim.x);
    if ((int)blockIdx.x >= blocks) return;
    int64_t at = line_start(line.total, blocks, blockIdx.x);
    const int64_t end = line_start(line.total, blocks, blockIdx.x + 1);
    int entry;
    int64_t place;
    line_find<D>(p, sh.sums, at, &entry, &place);
    const int rts = row_tiles(p);

    const uint32_t ring = sm100::smem_u32(&sh.ring[warp][0][0]) ;
    const uint32_t scales = sm100::smem_u32(&sh.scales[warp][0][0]);
    const int page_mask = (1 << p.c.page_shift) - 1;

    while (at < end) {
        const Tile t = make_tile<D>(p, entry / rts, entry % rts);
        const int hk = (int)((at - place) / t.groups);
        const int first = (int)((at - place) % t.groups);
        const int last = end - at < t.groups - first ? first + (int)(end - at) : t.groups;  // one past
        Query<T, D> q;
        load_query<T, D>(p, t, hk, q);
        State<D> st;
        st.clear();

        // the page of this lane's sub-block (lane % kSub) in group x, -1 where none is needed
        auto page_of = [&](int x) -> int {
            if (x >= last) return -1;
            int lo, hi;
            const int j = step_tokens<D>(t, x, warp, lo, hi) + 16 * (lane % G::kSub);
            return j + 16 > lo && j < hi ? cache_page(p.c, t.b, j) : -1;
        };
        auto issue = [&](int x, int my_page) {
            if (x < last) {
                const int stage = x % kS;
                int lo, hi;
                const int j0 = step_tokens<D>(t, x, warp, lo, hi);
                const uint32_t kd = ring + stage * G::kStage, vd = kd + G::kStage / 2;
#pragma unroll
                for (int sb = 0; sb < G::kSub; ++sb) {
                    const int pid = __shfl_sync(0xffffffffu, my_page, sb);
                    const int j = j0 + 16 * sb;
                    const uint8_t* kp = p.c.k.codes + (pid < 0 ? 0 : pid * p.c.k.s_p + hk * p.c.k.s_h + (j & page_mask) * p.c.k.s_t);
                    const uint8_t* vp = p.c.v.codes + (pid < 0 ? 0 : pid * p.c.v.s_p + hk * p.c.v.s_h + (j & page_mask) * p.c.v.s_t);
#pragma unroll
                    for (int nt = 0; nt < 2; ++nt) {
                        const int o = 8 * nt + g;
                        const bool there = pid >= 0 && j + o >= lo && j + o < hi;
#pragma unroll
                        for (int i = 0; i < G::kKCopies; ++i)
                            copy_async<G::kKBytes>(kd + ((sb * 2 + nt) * G::kKCopies + i) * 32 * G::kKBytes + lane * G::kKBytes,
                                                   kp + (there ? o * p.c.k.s_t + (i * 4 + c) * G::kKBytes : 0), there);
                    }
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const int o = 2 * c + (r & 1) + 8 * (r >> 1);
                        const bool there = pid >= 0 && j + o >= lo && j + o < hi;
                        copy_async<G::kNT>(vd + (sb * 4 + r) * 32 * G::kNT + lane * G::kNT,
                                           vp + (there ? o * p.c.v.s_t + g * G::kNT : 0), there);
                    }
                }
                if (lane < 2 * G::kSub) {  // lane: sub-block lane % kSub, of K or V
                    const uint32_t dst = scales + (stage * 2 * G::kSub + lane) * 4;
                    if (my_page >= 0)
                        copy_async<4>(dst, (lane < G::kSub ? p.c.k.scale : p.c.v.scale) + (int64_t)my_page * p.c.Hk + hk, true);
                    else
                        asm volatile("st.shared.f32 [%0], %1;" ::"r"(dst), "f"(kNoPage) : "memory");
                }
            }
            copy_commit();
        };

        int page = page_of(first);
#pragma unroll
        for (int s = 0; s < kS - 1; ++s) {
            issue(first + s, page);
            page = page_of(first + s + 1);
        }
        for (int x = first; x < last; ++x) {
            copy_wait<kS - 2>();
            __syncwarp();  // the other lanes' scales are there, and every lane is done with the stage refilled next
            issue(x + kS - 1, page);
            page = page_of(x + kS);
            const int stage = x % kS;
            int lo, hi;
            const int j0 = step_tokens<D>(t, x, warp, lo, hi);
            const uint32_t kd = ring + stage * G::kStage, vd = kd + G::kStage / 2;
#pragma unroll
            for (int sb = 0; sb < G::kSub; ++sb) {
                const int j = j0 + 16 * sb;
                if (j + 16 <= lo || j >= hi) continue;
                float ks, vs;
                asm volatile("ld.shared.f32 %0, [%1];" : "=f"(ks) : "r"(scales + (stage * 2 * G::kSub + sb) * 4) : "memory");
                asm volatile("ld.shared.f32 %0, [%1];" : "=f"(vs) : "r"(scales + (stage * 2 * G::kSub + G::kSub + sb) * 4) : "memory");
                if (ks == kNoPage) continue;
                const bool no_v = vs < kMinScale;
                const float lv = no_v ? 0.f : log2f(vs), inv_vs = no_v ? 1.f : 1.f / vs;
                // S = Q K^T
                float s[2][4];
#pragma unroll
                for (int nt = 0; nt < 2; ++nt) {
                    s[nt][0] = s[nt][1] = s[nt][2] = s[nt][3] = 0.f;
#pragma unroll
                    for (int i = 0; i < G::kKCopies; ++i) {
                        uint32_t w[G::kKBytes / 4];
                        load_words<G::kKBytes>(kd + ((sb * 2 + nt) * G::kKCopies + i) * 32 * G::kKBytes + lane * G::kKBytes, w);
#pragma unroll
                        for (int y = 0; y < G::kKBytes / 4; ++y) {
                            uint32_t b0, b1;
                            codes_to_half<CODE>(w[y], b0, b1);
#pragma unroll
                            for (int a = 0; a < kParts; ++a) mma_f16(s[nt], q.a[a][i * (G::kKBytes / 4) + y], b0, b1);
                        }
                    }
                }
                // exponents x + log2 vs - m, -inf where the row does not attend
                const bool first_part = x < t.na;
                const bool full = first_part ? j + 16 <= t.full_a
                                             : j + 16 <= t.full_hi && (j >= t.full_lo || j + 16 <= t.full_a);
                const float f0 = ks * q.factor[0], f1 = ks * q.factor[1];
                float e[2][4];
                auto exponents = [&](float m0, float m1) {
                    const float a0 = lv - m0, a1 = lv - m1;
#pragma unroll
                    for (int nt = 0; nt < 2; ++nt) {
                        e[nt][0] = fmaf(s[nt][0], f0, a0);
                        e[nt][1] = fmaf(s[nt][1], f0, a0);
                        e[nt][2] = fmaf(s[nt][2], f1, a1);
                        e[nt][3] = fmaf(s[nt][3], f1, a1);
                    }
                    if (!full) {
#pragma unroll
                        for (int r = 0; r < 2; ++r) {
                            const int row = g + 8 * r;
                            const int pos = row < t.rows ? t.base + (t.first_row + row) / p.G : -1;
#pragma unroll
                            for (int nt = 0; nt < 2; ++nt)
#pragma unroll
                                for (int y = 0; y < 2; ++y) {
                                    const int tok = j + 8 * nt + 2 * c + y;
                                    const bool sees = tok <= pos && tok >= lo && tok < hi &&
                                                      (p.window < 0 || tok >= pos - p.window || tok < p.n_global);
                                    if (!sees) e[nt][2 * r + y] = -INFINITY;
                                }
                        }
                    }
                };
                auto top_of = [&](int r) {
                    return fmaxf(fmaxf(e[0][2 * r], e[0][2 * r + 1]), fmaxf(e[1][2 * r], e[1][2 * r + 1]));
                };
                exponents(st.m[0], st.m[1]);
                if (__any_sync(0xffffffffu, fmaxf(top_of(0), top_of(1)) > kRescaleAt)) {
                    exponents(0.f, 0.f);
                    float m[2];
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        float top = top_of(r);
                        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
                        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
                        m[r] = top - st.m[r] > kRescaleAt ? top - kHeadroom : st.m[r];
                    }
                    st.scale(ex2(st.m[0] - m[0]), ex2(st.m[1] - m[1]));
                    st.m[0] = m[0];
                    st.m[1] = m[1];
                    exponents(m[0], m[1]);
                }
                float sum0 = 0.f, sum1 = 0.f;
#pragma unroll
                for (int nt = 0; nt < 2; ++nt) {
#pragma unroll
                    for (int y = 0; y < 4; ++y) e[nt][y] = ex2(e[nt][y]);
                    sum0 += e[nt][0] + e[nt][1];
                    sum1 += e[nt][2] + e[nt][3];
                }
                st.l[0] = fmaf(sum0, inv_vs, st.l[0]);
                st.l[1] = fmaf(sum1, inv_vs, st.l[1]);
                if (no_v) continue;
                // O += P V
                uint32_t pa[kParts][4];
#pragma unroll
                for (int nt = 0; nt < 2; ++nt)
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        pa[0][2 * nt + r] = half_pair(e[nt][2 * r], e[nt][2 * r + 1]);
                        if constexpr (kParts == 2)
                            pa[1][2 * nt + r] = half_rest(e[nt][2 * r], e[nt][2 * r + 1], pa[0][2 * nt + r]);
                    }
                uint32_t v[4][(G::kNT + 3) / 4];
#pragma unroll
                for (int r = 0; r < 4; ++r) load_words<G::kNT>(vd + (sb * 4 + r) * 32 * G::kNT + lane * G::kNT, v[r]);
#pragma unroll
                for (int y = 0; y < G::kNT / 4; ++y) {
#pragma unroll
                    for (int z = 0; z < 2; ++z) {  // byte columns 4 y + 2 z, + 1
                        const unsigned pick = z ? 0x7362 : 0x5140;
                        uint32_t b[2][2];
                        codes_to_half<CODE>(__byte_perm(v[0][y], v[1][y], pick), b[0][0], b[1][0]);
                        codes_to_half<CODE>(__byte_perm(v[2][y], v[3][y], pick), b[0][1], b[1][1]);
#pragma unroll
                        for (int a = 0; a < kParts; ++a) {
                            mma_f16(st.o[4 * y + 2 * z], pa[a], b[0][0], b[0][1]);
                            mma_f16(st.o[4 * y + 2 * z + 1], pa[a], b[1][0], b[1][1]);
                        }
                    }
                }
            }
        }
        copy_wait<0>();
        __syncwarp();
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            st.l[r] += __shfl_xor_sync(0xffffffffu, st.l[r], 1);
            st.l[r] += __shfl_xor_sync(0xffffffffu, st.l[r], 2);
        }
        join_warps<D>(st, sh.join);
        if (warp == 0) {
            if (first == 0 && last == t.groups)
                write_rows<T, D>(p, t, hk, st);
            else  // slot 0: a segment that an earlier block began; slot 1: one that a later block goes on with
                write_piece<D>(ws + ((int64_t)blockIdx.x * 2 + (first == 0)) * G::kPiece, st, t.rows);
        }
        at += last - first;
        if (at >= place + (int64_t)t.groups * p.c.Hk) {
            place += (int64_t)t.groups * p.c.Hk;
            ++entry;
        }
    }
}

// Block x: segment x (entry x / Hk). The pieces of a segment that several blocks
// worked on are added up, each warp taking every fourth.
template <typename T, int D>
__global__ void __launch_bounds__(kWarps * 32) k_fwd_cache_join(CacheFwdParams p, const float* ws, int grid) {
    __shared__ Join<D> join;
    __shared__ int64_t sums[kWarps * 32 + 1];
    const int warp = threadIdx.x >> 5;
    const Line line = line_total<D>(p, sums);
    const int blocks = line_blocks(line.total, grid), rts = row_tiles(p);
    const int entry = blockIdx.x / p.c.Hk, hk = blockIdx.x % p.c.Hk;
    const int per = (p.B * rts + kWarps * 32 - 1) / (kWarps * 32);
    int64_t place = sums[entry / per];
    for (int e = entry / per * per; e < entry; ++e) place += make_tile<D>(p, e / rts, e % rts).groups;
    const Tile t = make_tile<D>(p, entry / rts, entry % rts);
    const int64_t s0 = place * p.c.Hk + (int64_t)hk * t.groups, s1 = s0 + t.groups - 1;
    // the block that holds place s: the last x with total x / blocks <= s
    auto block_of = [&](int64_t s) {
        int x = (int)((s * blocks + blocks - 1) / line.total);
        while (x > 0 && line_start(line.total, blocks, x) > s) --x;
        while (x + 1 < blocks && line_start(line.total, blocks, x + 1) <= s) ++x;
        return x;
    };
    const int x0 = block_of(s0), x1 = block_of(s1);
    asm volatile("griddepcontrol.wait;" ::: "memory");  // every block, so that this kernel ends after the first
    if (x0 == x1) return;
    State<D> st;
    st.clear();
    for (int x = x0 + warp; x <= x1; x += kWarps)
        add_piece<D>(ws + ((int64_t)x * 2 + (x == x0)) * Geo<D>::kPiece, st, t.rows);
    join_warps<D>(st, join);
    if (warp == 0) write_rows<T, D>(p, t, hk, st);
}

template <typename T, int CODE, int D>
cudaError_t fwd_d(const CacheFwdParams& p, int num_sms, float* ws, cudaStream_t s) {
    const int smem = (int)sizeof(Shared<T, D>);
    cudaError_t e = cudaFuncSetAttribute(k_fwd_cache<T, CODE, D>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    const int grid = num_sms * kCacheBlocksPerSm;
    const int use = grid / kCacheBlocksPerSm * blocks_per_sm<T>();
    k_fwd_cache<T, CODE, D><<<use, kWarps * 32, smem, counted(s)>>>(p, ws);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((int64_t)p.B * row_tiles(p) * p.c.Hk));
    cfg.blockDim = dim3(kWarps * 32);
    cfg.stream = counted(s);
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, k_fwd_cache_join<T, D>, p, (const float*)ws, use);
}

template <typename T, int CODE>
cudaError_t fwd_code(const CacheFwdParams& p, int d, int num_sms, float* ws, cudaStream_t s) {
    switch (d) {
        case 32: return fwd_d<T, CODE, 32>(p, num_sms, ws, s);
        case 64: return fwd_d<T, CODE, 64>(p, num_sms, ws, s);
        default: return fwd_d<T, CODE, 128>(p, num_sms, ws, s);
    }
}

}  // namespace

int64_t fwd_cache_workspace(int d, int num_sms) { return (int64_t)num_sms * kCacheBlocksPerSm * 2 * (32 + 16 * d); }

cudaError_t launch_fwd_cache(const CacheFwdParams& p, int real, int code, int d, int num_sms, float* ws,
                             cudaStream_t s) {
    if (real == 0)
        return code == kCodeI8 ? fwd_code<__nv_bfloat16, kCodeI8>(p, d, num_sms, ws, s)
                               : fwd_code<__nv_bfloat16, kCodeE4m3>(p, d, num_sms, ws, s);
    return code == kCodeI8 ? fwd_code<float, kCodeI8>(p, d, num_sms, ws, s)
                           : fwd_code<float, kCodeE4m3>(p, d, num_sms, ws, s);
}

}  // namespace spattn
