// Attention of a sequence's last tokens over its 8-bit key/value cache.
//
// Query t < qlen[b] of sequence b is token pos = seqlen[b] - qlen[b] + t. It
// attends to the tokens j <= pos, and with a window only to those with
// j >= pos - window or j < n_global:
//     s_j = scale <q, k_j>,  out = sum_j softmax_j(s) v_j,  lse = log sum_j exp(s_j)
//
// Rows. The m * G rows (query t, head g of the group) of a (sequence, K/V head)
// share its tokens and are cut into tiles of 8 R rows, R = 1..4 as the rows need:
// with tokens (then head dim elements) on the M side of mma.m16n8k16 and rows on
// its N = 8 side, the common case of up to 8 rows wastes no products and holds O
// in D / 4 registers, so that enough warps fit to keep HBM busy. A row tile of
// one K/V head is a segment. Codes are exact in fp16, and so are bf16 queries
// once a row is scaled by a power of two that brings its largest element to
// [2^14, 2^15) (elements 2^-28 below it lose bits): K Q^T is exact up to fp32
// accumulation.
//
// Scales. A page's K scale multiplies its scores. Its V scale vs goes into the
// exponent: p' = 2^(x + log2 vs - m) with x the score in base 2, so that weights
// are largest where p v is, whatever the scales; O = sum p' c, l = sum p' / vs. A page
// whose scale is 0 is taken to have a small one and no values.
// Weights are rounded to fp16 for P V (11 bits; bf16 outputs have 8). m is a
// reference that moves only when some p' would pass 2^15 (it then becomes the
// largest exponent - 8), so that most steps need no exchange between lanes.
//
// fp32. Queries and weights go in as the sum of two fp16 numbers (24 bits with their
// signs), at twice the products. A weight's second number is held 2^11 times as large
// and meets V codes 2^-11 times as large, so that light weights, whose first number has
// few bits left or none, keep theirs. The tensor cores' accumulation truncates, so the
// second parts' scores have sums of their own, and each 16 tokens' P V starts at 0 and
// is added to O by ordinary sums. m is a whole number, and of vs only the power of two
// goes into the exponent; the rest is a factor of the weight. The error against 64 bits
// is 0.2 to 0.3e-6 of out where torch operations in fp32 have 0.2 to 0.9e-6.
//
// Streaming. Each code is read once; HBM is what the kernel cannot do without. It
// gets 5.2 TB/s of it (two sequences of 131071 tokens, d = 128, int8: 104 us): 14
// computing warps an SM wait for loads from shared memory and for their own chains
// of conversions, products and exponentials, and issue slots are busy 53 % of the time.
// A producer warp fills a ring in shared memory by TMA: a copy brings 16 tokens
// of one page (4-D map {d, token, head, page}, any strides), swizzled so that the
// fragment loads meet few bank conflicts; a stage is kSub such sub-blocks of K and
// of V for each of the other warps. It reads the page table two stages ahead and
// the pages' scales one, and runs on over the ends of segments. Fragments need no
// exchange between lanes: any order of the head dim and of the tokens does for a
// product as long as both sides use the same, so K fragments are 4 neighbouring
// codes of a token, and V fragments byte columns of four tokens.
//
// Work. All segments' steps form one line, which the grid's blocks share evenly
// (they know it from the lengths alone), so that one long sequence among short
// ones is spread over the GPU. A block that holds a whole segment writes its
// rows; pieces of a segment go to a workspace as (m, l, O), and k_fwd_cache_join
// adds them up by the running max / sum rule.
#include "cache_attn.cuh"

#include <mutex>
#include <type_traits>

namespace spattn {
namespace {

using namespace cache_attn;
using sm100::ex2;

constexpr int kWarps = 7;                         // that compute
constexpr int kThreads = (kWarps + 1) * 32;       // and the producer
constexpr int kJoinThreads = 128;
// Sizes that follow from the head dim.
template <int D>
struct Geo {
    static constexpr int kSub = 128 / D;              // sub-blocks of 16 tokens a warp step
    static constexpr int kGroup = kWarps * kSub * 16; // tokens a block step
    static constexpr int kKBytes = D >= 64 ? 16 : 8;  // bytes of a K load
    static constexpr int kKLoads = D / (4 * kKBytes); // of each token, by a lane
    static constexpr int kVBytes = D / 8;             // bytes of a V load
    static constexpr int kSteps = D / 16;             // mma steps over the head dim; mma tiles of O
    static constexpr int kBox = 16 * D;               // bytes of a sub-block of K or V
    static constexpr int kSide = kSub * kBox;         // bytes of K (and of V) in a ring stage
    // The token of a sub-block's half that stands at row x of a product (D = 128:
    // neighbours differ in bit 2, so that the swizzle spreads their loads).
    static __device__ __forceinline__ int token(int x) { return D == 128 ? (0x37156240 >> (4 * x)) & 7 : x; }
    // Byte `at` of token o's row in a sub-block: the copy's swizzle exchanges 16-byte units.
    static __device__ __forceinline__ int byte(int o, int at) {
        const int x = D == 128 ? o & 7 : D == 64 ? (o >> 1) & 3 : (o >> 2) & 1;
        return o * D + (at ^ (16 * x));
    }
};
// Floats of a stored piece: m and l of the 8 R rows, then O.
template <int D, int R>
constexpr int piece_floats() {
    return 8 * R * (2 + D);
}

template <int N>
__device__ __forceinline__ void load_words(const uint8_t* p, uint32_t* w) {
    if constexpr (N == 16) {
        const uint4 v = *reinterpret_cast<const uint4*>(p);
        w[0] = v.x;
        w[1] = v.y;
        w[2] = v.z;
        w[3] = v.w;
    } else if constexpr (N == 8) {
        const uint2 v = *reinterpret_cast<const uint2*>(p);
        w[0] = v.x;
        w[1] = v.y;
    } else {
        w[0] = *reinterpret_cast<const uint32_t*>(p);
    }
}

__device__ __forceinline__ void mma_f16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// What the fp16 pair `h` leaves of (a, b), times `by`, as another one.
__device__ __forceinline__ uint32_t half_rest(float a, float b, uint32_t h, float by) {
    const __half2 v = *reinterpret_cast<const __half2*>(&h);
    return half_pair((a - __low2float(v)) * by, (b - __high2float(v)) * by);
}
constexpr float kRestScale = 2048.f;  // 2^11, of a weight's second part
// An fp16 pair of codes times 2^-11: exact (multiples of 2^-20).
__device__ __forceinline__ uint32_t rest_codes(uint32_t x) {
    uint32_t y;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(y) : "r"(x), "r"(0x10001000u));
    return y;
}

// Transposes an 8 x 8 matrix of fp16 held as lane (g, c): row g, columns 2 c, 2 c + 1.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
    uint32_t y;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

// fp32: two fp16 parts.
template <typename T>
constexpr int parts() {
    return std::is_same<T, float>::value ? 2 : 1;
}
// How far a weight's exponent may pass 0 before the reference moves, and what the weights are multiplied by
// on their way into P V (O is that much too large; m and l are not). fp32: the reference is the whole number
// below the largest exponent, since an exponent near 0 is rounded least, and the weights are lifted after the
// exponential; with the rest of vs they stay below 2^4 * 2 * 2^10.
template <typename T>
constexpr float kMoveAt = parts<T>() == 2 ? 4.f : kRescaleAt;
template <typename T>
constexpr float kLift = parts<T>() == 2 ? 1024.f : 1.f;

// A tile's running state in one warp: lane (g = lane / 4, c = lane % 4) holds rows
// 8 k + 2 c + e. o[k][i][2 x + e] is element kVBytes g + 2 i + x of that row; l is
// this lane's part of the row's sum until it is summed over g.
template <int D, int R>
struct State {
    float o[R][Geo<D>::kSteps][4];
    float m[R][2], l[R][2];
    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int k = 0; k < R; ++k) {
#pragma unroll
            for (int i = 0; i < Geo<D>::kSteps; ++i) o[k][i][0] = o[k][i][1] = o[k][i][2] = o[k][i][3] = 0.f;
            m[k][0] = m[k][1] = kNone;
            l[k][0] = l[k][1] = 0.f;
        }
    }
    __device__ __forceinline__ void scale(int k, float a0, float a1) {
#pragma unroll
        for (int i = 0; i < Geo<D>::kSteps; ++i) {
            o[k][i][0] *= a0;
            o[k][i][1] *= a1;
            o[k][i][2] *= a0;
            o[k][i][3] *= a1;
        }
        l[k][0] *= a0;
        l[k][1] *= a1;
    }
    __device__ __forceinline__ float4 get(int k, int i) const { return make_float4(o[k][i][0], o[k][i][1], o[k][i][2], o[k][i][3]); }
    __device__ __forceinline__ void add(int k, int i, const float4& v, float w0, float w1) {
        o[k][i][0] += v.x * w0;
        o[k][i][1] += v.y * w1;
        o[k][i][2] += v.z * w0;
        o[k][i][3] += v.w * w1;
    }
};

// Where the computing warps' states meet.
template <int D, int R>
struct JoinO {
    float4 o[3][R * Geo<D>::kSteps][32];
};
template <int R>
using JoinMl = float[kWarps][2][8 * R];

// The computing warps' states (l summed over the row's lanes) joined into warp 0's.
template <int D, int R>
__device__ __forceinline__ void join_warps(State<D, R>& s, JoinMl<R>& ml, JoinO<D, R>& sh) {
    constexpr int N = Geo<D>::kSteps;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, c = lane & 3;
    auto sync = []() { sm100::named_sync(1, kWarps * 32); };
    if (lane < 4) {
#pragma unroll
        for (int k = 0; k < R; ++k)
#pragma unroll
            for (int e = 0; e < 2; ++e) ml[warp][0][8 * k + 2 * c + e] = s.m[k][e];
    }
    sync();
#pragma unroll
    for (int k = 0; k < R; ++k) {
        float top[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int row = 8 * k + 2 * c + e;
            top[e] = ml[0][0][row];
#pragma unroll
            for (int w = 1; w < kWarps; ++w) top[e] = fmaxf(top[e], ml[w][0][row]);
        }
        s.scale(k, ex2(s.m[k][0] - top[0]), ex2(s.m[k][1] - top[1]));
        s.m[k][0] = top[0];
        s.m[k][1] = top[1];
        if (lane < 4) {
            ml[warp][1][8 * k + 2 * c] = s.l[k][0];
            ml[warp][1][8 * k + 2 * c + 1] = s.l[k][1];
        }
    }
    // 7 -> 4 -> 2 -> 1: after the first round a warp writes the buffer that only it has read
    auto give = [&](int buf) {
#pragma unroll
        for (int x = 0; x < R * N; ++x) sh.o[buf][x][lane] = s.get(x / N, x % N);
    };
    auto take = [&](int buf) {
#pragma unroll
        for (int x = 0; x < R * N; ++x) s.add(x / N, x % N, sh.o[buf][x][lane], 1.f, 1.f);
    };
    static_assert(kWarps == 7, "the rounds below");
    if (warp >= 4) give(warp - 4);
    sync();
    if (warp >= 1 && warp <= 3) take(warp - 1);
    if (warp == 2 || warp == 3) give(warp - 1);
    sync();
    if (warp <= 1) take(warp + 1);
    if (warp == 1) give(0);
    sync();
    if (warp == 0) take(0);
    if (warp == 0) {
#pragma unroll
        for (int k = 0; k < R; ++k)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                s.l[k][e] = 0.f;
#pragma unroll
                for (int w = 0; w < kWarps; ++w) s.l[k][e] += ml[w][1][8 * k + 2 * c + e];
            }
    }
    sync();  // the buffers may be written again
}

// Warp 0: the finished rows of a tile. Those behind the sequence's queries get
// zeros: the state holds what a query of zeros gave.
template <typename T, int D, int R>
__device__ __forceinline__ void write_rows(const CacheFwdParams& p, const Tile& tile, int hk, const State<D, R>& s) {
    constexpr int N = Geo<D>::kVBytes;
    const int lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
#pragma unroll
    for (int k = 0; k < R; ++k)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int in_tile = 8 * k + 2 * c + e, row = tile.first_row + in_tile;
            if (row >= p.m * p.G) continue;
            const int b = tile.b, t = row / p.G, h = hk * p.G + row % p.G;
            const bool there = in_tile < tile.rows && s.l[k][e] != 0.f;
            const float inv = 1.f / (kLift<T> * s.l[k][e]);
            T* out = static_cast<T*>(p.out) + b * p.o_sb + h * p.o_sh + t * p.o_sn + N * g;
            float v[N];
#pragma unroll
            for (int x = 0; x < N; ++x) v[x] = there ? s.o[k][x / 2][2 * (x & 1) + e] * inv : 0.f;
            if constexpr (std::is_same<T, float>::value) {
#pragma unroll
                for (int x = 0; x < N; x += 4) *reinterpret_cast<float4*>(out + x) = make_float4(v[x], v[x + 1], v[x + 2], v[x + 3]);
            } else {
                uint32_t u[N / 2];
#pragma unroll
                for (int x = 0; x < N / 2; ++x) {
                    const __nv_bfloat162 a = __floats2bfloat162_rn(v[2 * x], v[2 * x + 1]);
                    u[x] = *reinterpret_cast<const uint32_t*>(&a);
                }
                if constexpr (N >= 8) {
#pragma unroll
                    for (int x = 0; x < N / 2; x += 4) *reinterpret_cast<uint4*>(out + 2 * x) = make_uint4(u[x], u[x + 1], u[x + 2], u[x + 3]);
                } else {
                    *reinterpret_cast<uint2*>(out) = make_uint2(u[0], u[1]);
                }
            }
            if (p.lse && g == 0)
                p.lse[((int64_t)b * p.H + h) * p.m + t] = there ? (s.m[k][e] + log2f(s.l[k][e])) * kLn2 : -INFINITY;
        }
}

// Pieces in the workspace: m and l of the rows, then O by lane.
template <int D, int R>
__device__ __forceinline__ void write_piece(float* ws, const State<D, R>& s, int rows) {
    constexpr int N = Geo<D>::kSteps;
    const int lane = threadIdx.x & 31, c = lane & 3;
#pragma unroll
    for (int k = 0; k < R; ++k) {
        const int row = 8 * k + 2 * c;
        if (row >= rows) continue;
        if (lane < 4) {
            *reinterpret_cast<float2*>(ws + row) = make_float2(s.m[k][0], s.m[k][1]);
            *reinterpret_cast<float2*>(ws + 8 * R + row) = make_float2(s.l[k][0], s.l[k][1]);
        }
#pragma unroll
        for (int i = 0; i < N; ++i) reinterpret_cast<float4*>(ws + 16 * R)[(k * N + i) * 32 + lane] = s.get(k, i);
    }
}
// Blocks an SM holds: with 128 registers a thread two, else one. O, Q and the
// scores take `held` of them. Two blocks are faster up to 68, though some of those
// builds spill (the second number: one block; 16 sequences of 8192 tokens at d = 128,
// of 16384 below): bf16 d = 64 R = 2 83 / 113 us, d = 32 R = 2 70 / 95 us, fp32 d = 128
// R = 1 74 / 82 us, d = 32 R = 2 85 / 103 us. From 80 on they are not: fp32 d = 64
// R = 2 75 / 72 us, bf16 d = 32 R = 3 120 / 103 us, d = 64 R = 3 123 / 119 us.
template <typename T, int D, int R>
constexpr int blocks_per_sm() {
    const int held = (D / 4 + parts<T>() * D / 8 + 4 * Geo<D>::kSub) * R;
    return held <= 68 ? 2 : 1;
}
template <typename T, int D, int R>
constexpr int stages() {  // of the ring, 28 KB each
    return blocks_per_sm<T, D, R>() == 2 ? 3 : 5;
}

template <int D, int R, int S>
struct Shared {
    uint8_t ring[S][kWarps][2 * Geo<D>::kSide];  // a warp's part of a stage: K, then V
    JoinO<D, R> join;
    float scales[S][2][kWarps * Geo<D>::kSub];  // K, V of each sub-block
    uint64_t full[S], empty[S];
    JoinMl<R> ml;
};
constexpr int kRingAlign = 1024;  // the swizzle's period

// Queries of a tile as mma B fragments: column g of step x (rows 8 k + g) holds
// the elements that the lane's K bytes stand for.
template <typename T, int D, int R>
struct Query {
    uint32_t b[parts<T>()][R][Geo<D>::kSteps][2];
    float factor[R][2];  // of the scores of row 8 k + 2 c + e, to base 2
};
template <typename T, int D, int R>
__device__ __forceinline__ void load_query(const CacheFwdParams& p, const Tile& t, int hk, Query<T, D, R>& q) {
    using G = Geo<D>;
    const int lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
#pragma unroll
    for (int k = 0; k < R; ++k) {
        float x[D / 4];
        const int row = t.first_row + 8 * k + g;
        if (8 * k + g < t.rows) {
            const T* src = static_cast<const T*>(p.q) + t.b * p.q_sb + (hk * p.G + row % p.G) * p.q_sh +
                           (row / p.G) * p.q_sn;
            constexpr int V = 16 / sizeof(T);
#pragma unroll
            for (int i = 0; i < G::kKLoads; ++i)
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
        const float by = exp2f((float)up), factor = p.scale_log2 * exp2f((float)-up);
        q.factor[k][0] = __shfl_sync(0xffffffffu, factor, 8 * c);
        q.factor[k][1] = __shfl_sync(0xffffffffu, factor, 8 * c + 4);
#pragma unroll
        for (int s = 0; s < G::kSteps; ++s)
#pragma unroll
            for (int y = 0; y < 2; ++y) {
                const float v0 = x[4 * s + 2 * y] * by, v1 = x[4 * s + 2 * y + 1] * by;
                q.b[0][k][s][y] = half_pair(v0, v1);
                if constexpr (parts<T>() == 2) q.b[1][k][s][y] = half_rest(v0, v1, q.b[0][k][s][y], 1.f);
            }
    }
}

// The producer warp: lane x brings sub-block x of each stage.
template <int D, int R, int S>
__device__ __forceinline__ void produce(const CUtensorMap& k_map, const CUtensorMap& v_map, const CacheFwdParams& p,
                                        Shared<D, R, S>& sh, Part<Geo<D>::kGroup, 8 * R> part, int rts) {
    using G = Geo<D>;
    constexpr int kN = kWarps * G::kSub;  // sub-blocks of a stage
    const int lane = threadIdx.x & 31;
    const int page_mask = (1 << p.c.page_shift) - 1;
    const uint32_t ring_at = sm100::smem_u32(&sh.ring[0][0][0]), full_at = sm100::smem_u32(&sh.full[0]),
                   empty_at = sm100::smem_u32(&sh.empty[0]);
    // a step on its way: the table's entry (kUnread: none needed), then the page's scales
    struct Step {
        int raw, j, hk;
        bool more;
    };
    bool open = part.open(p, rts);
    Walk<Geo<D>::kGroup> w;
    if (open) w.begin(part.t, part.first);
    auto look_up = [&]() -> Step {
        Step s{kUnread, 0, 0, open};
        if (!open) return s;
        s.j = w.j + 16 * lane;
        s.hk = part.hk;
        if (lane < kN && s.j + 16 > w.lo(part.t) && s.j < w.hi(part.t))
            s.raw = __ldg(p.c.table + part.t.b * p.c.table_stride + (s.j >> p.c.page_shift));
        w.next(part.t);
        if (w.x >= part.last) {
            part.close(p);
            open = part.open(p, rts);
            if (open) w.begin(part.t, part.first);
        }
        return s;
    };
    auto scales_of = [&](Step& s, float& ks, float& vs) {
        ks = vs = kNoPage;
        if ((unsigned)s.raw >= (unsigned)p.c.num_pages) {
            if (s.raw != kUnread) atomicOr(p.c.err, kErrBadPage);
            s.raw = -1;
        } else {
            const int64_t at = (int64_t)s.raw * p.c.Hk + s.hk;
            ks = __ldg(p.c.k.scale + at);
            vs = __ldg(p.c.v.scale + at);
        }
    };
    Step now = look_up(), next = look_up();
    float ks, vs, ks_next = 0.f, vs_next = 0.f;
    scales_of(now, ks, vs);
    int stage = 0;
    uint32_t phase = 1;  // the first round's waits pass at once
    bool dead = false;
    int issued = 0;  // stages, up to S
    while (now.more) {
        dead = !__all_sync(0xffffffffu, sm100::mbar_wait_bounded(empty_at + 8 * stage, phase, kCacheWaitCycles));
        if (dead) break;
        const unsigned there = __ballot_sync(0xffffffffu, now.raw >= 0);
        const uint32_t bar = full_at + 8 * stage;
        if (now.raw >= 0) {
            const uint32_t dst = ring_at + ((stage * kWarps + lane / G::kSub) * 2 * G::kSub + lane % G::kSub) * G::kBox;
            sm100::tma_load_4d(dst, &k_map, bar, 0, now.j & page_mask, now.hk, now.raw);
            sm100::tma_load_4d(dst + G::kSide, &v_map, bar, 0, now.j & page_mask, now.hk, now.raw);
        }
        if (next.more) scales_of(next, ks_next, vs_next);
        const Step after = look_up();
        if (lane < kN) {
            sh.scales[stage][0][lane] = ks;
            sh.scales[stage][1][lane] = vs;
        }
        __syncwarp();
        // the copies above may have finished already: the barrier's phase waits for this arrival
        if (lane == 0) sm100::mbar_expect_tx(bar, 2 * G::kBox * __popc(there));
        stage = stage + 1 == S ? 0 : stage + 1;
        phase ^= stage == 0;
        issued = issued < S ? issued + 1 : S;
        now = next;
        next = after;
        ks = ks_next;
        vs = vs_next;
    }
    // No copy is on its way when the block's shared memory goes to another: the computing warps wait for
    // every stage, but not once one of their waits ran out. The last S stages, newest first (their full
    // barriers' phases are those of the round that filled them).
    for (int x = 0; x < issued; ++x) {
        if (stage == 0) phase ^= 1;
        stage = stage == 0 ? S - 1 : stage - 1;
        dead |= !sm100::mbar_wait_bounded(full_at + 8 * stage, phase ^ 1, kCacheWaitCycles);
    }
    if (__any_sync(0xffffffffu, dead) && lane == 0) atomicOr(p.c.err, kErrTimeout);
}

template <typename T, int CODE, int D, int R>
__global__ void __launch_bounds__(kThreads, blocks_per_sm<T, D, R>())
    k_fwd_cache(const __grid_constant__ CUtensorMap k_map, const __grid_constant__ CUtensorMap v_map, CacheFwdParams p,
                float* ws) {
    using G = Geo<D>;
    constexpr int kParts = parts<T>(), kStages = stages<T, D, R>();
    extern __shared__ __align__(16) uint8_t smem_raw[];
    using Sh = Shared<D, R, kStages>;
    Sh& sh = *reinterpret_cast<Sh*>(
        smem_raw + ((kRingAlign - (sm100::smem_u32(smem_raw) & (kRingAlign - 1))) & (kRingAlign - 1)));
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
    asm volatile("griddepcontrol.launch_dependents;");
    if (threadIdx.x == 0) {
        for (int x = 0; x < kStages; ++x) {
            sm100::mbar_init(sm100::smem_u32(&sh.full[x]), 1);
            sm100::mbar_init(sm100::smem_u32(&sh.empty[x]), kWarps);
        }
        sm100::fence_mbar_init();
        sm100::fence_proxy_async_smem();
        sm100::prefetch_tensormap(&k_map);
        sm100::prefetch_tensormap(&v_map);
    }

    Begun* const begun = reinterpret_cast<Begun*>(ws);
    float* const pieces = ws + (int64_t)gridDim.x * (sizeof(Begun) / 4);
    if (threadIdx.x == 0) begun[blockIdx.x].more = 0;
    const Line<G::kGroup, 8 * R> line(p);
    __syncthreads();  // the barriers are set up
    const Shares shares(line.total, (int)gridDim.x);
    if ((int)blockIdx.x >= shares.blocks) return;
    const int rts = line.rts;
    Part<Geo<D>::kGroup, 8 * R> part;
    part.at = shares.start(blockIdx.x);
    part.end = shares.start(blockIdx.x + 1);
    line.find(p, part.at, &part.entry, &part.place);
    if (warp == kWarps) {
        produce<D, R, kStages>(k_map, v_map, p, sh, part, rts);
        return;
    }

    const uint8_t* const ring = &sh.ring[0][warp][0];
    const uint32_t full_at = sm100::smem_u32(&sh.full[0]), empty_at = sm100::smem_u32(&sh.empty[0]);
    int k_at[G::kKLoads], v_at[2];  // this lane's bytes of a sub-block's first half
#pragma unroll
    for (int i = 0; i < G::kKLoads; ++i) k_at[i] = G::byte(G::token(g), (i * 4 + c) * G::kKBytes);
#pragma unroll
    for (int r = 0; r < 2; ++r) v_at[r] = G::byte(G::token(2 * c + r), g * G::kVBytes);
    int stage = 0;
    uint32_t phase = 0;
    bool dead = false;  // a wait ran out: no more waits

    while (part.open(p, rts)) {
        const Tile& t = part.t;
        Query<T, D, R> q;
        State<D, R> st;
        auto step = [&](const uint8_t* kd, const uint8_t* vd, const float* ksc, const float* vsc, int lo, int hi, int j0, auto all) {
            constexpr bool full = decltype(all)::value;  // every row attends to every token of the step
            // S^T = K Q^T: e[k][sb][2 x + y]: row 8 k + 2 c + y, token 16 sb + 8 x + token(g)
            float e[R][G::kSub][4];
            auto scores = [&]() {
#pragma unroll
                for (int sb = 0; sb < G::kSub; ++sb) {
#pragma unroll
                    for (int k = 0; k < R; ++k) e[k][sb][0] = e[k][sb][1] = e[k][sb][2] = e[k][sb][3] = 0.f;
                    [[maybe_unused]] float low[kParts == 2 ? R : 1][4] = {};  // of the second parts
#pragma unroll
                    for (int i = 0; i < G::kKLoads; ++i) {
                        uint32_t w[2][G::kKBytes / 4];
#pragma unroll
                        for (int nt = 0; nt < 2; ++nt)
                            load_words<G::kKBytes>(kd + sb * G::kBox + 8 * nt * D + k_at[i], w[nt]);
#pragma unroll
                        for (int y = 0; y < G::kKBytes / 4; ++y) {
                            uint32_t a[4];
                            codes_to_half<CODE>(w[0][y], a[0], a[2]);
                            codes_to_half<CODE>(w[1][y], a[1], a[3]);
#pragma unroll
                            for (int k = 0; k < R; ++k) {
                                const int at = i * (G::kKBytes / 4) + y;
                                mma_f16(e[k][sb], a, q.b[0][k][at][0], q.b[0][k][at][1]);
                                if constexpr (kParts == 2) mma_f16(low[k], a, q.b[1][k][at][0], q.b[1][k][at][1]);
                            }
                        }
                    }
                    if constexpr (kParts == 2) {
#pragma unroll
                        for (int k = 0; k < R; ++k)
#pragma unroll
                            for (int y = 0; y < 4; ++y) e[k][sb][y] += low[k][y];
                    }
                }
            };
            scores();
            // to exponents x + log2 vs - m, -inf where a row does not attend
            float ks[G::kSub], lv[G::kSub], inv_vs[G::kSub];
            [[maybe_unused]] float rest_vs[G::kSub];
#pragma unroll
            for (int sb = 0; sb < G::kSub; ++sb) {
                const float vs = vsc[sb];
                const bool none = !full && vs < kMinScale;
                ks[sb] = ksc[sb];
                if constexpr (kParts == 2) {  // vs = 2^lv * (1..2): the first exact in the exponent, the rest a factor
                    const uint32_t bits = __float_as_uint(vs), ex = min(bits >> 23, 253u);
                    lv[sb] = none ? kNoValues : (float)((int)ex - 127);
                    inv_vs[sb] = none ? kNoValuesInv : __uint_as_float((254u - ex) << 23);
                    rest_vs[sb] = __uint_as_float((bits & 0x007fffffu) | 0x3f800000u) * kLift<T>;
                } else {
                    lv[sb] = none ? kNoValues : sm100::lg2(vs);
                    inv_vs[sb] = none ? kNoValuesInv : __frcp_rn(vs);
                }
            }
            auto exponents = [&](bool from_zero) {
#pragma unroll
                for (int k = 0; k < R; ++k)
#pragma unroll
                    for (int sb = 0; sb < G::kSub; ++sb)
#pragma unroll
                        for (int y = 0; y < 2; ++y) {
                            const float f = ks[sb] * q.factor[k][y], a = from_zero ? lv[sb] : lv[sb] - st.m[k][y];
                            e[k][sb][y] = fmaf(e[k][sb][y], f, a);
                            e[k][sb][2 + y] = fmaf(e[k][sb][2 + y], f, a);
                        }
                if (!full) {
#pragma unroll
                    for (int k = 0; k < R; ++k)
#pragma unroll
                        for (int y = 0; y < 2; ++y) {
                            const int row = 8 * k + 2 * c + y;
                            const int pos = row < t.rows ? max(t.base + (t.first_row + row) / p.G, -1) : -1;
#pragma unroll
                            for (int sb = 0; sb < G::kSub; ++sb)
#pragma unroll
                                for (int x = 0; x < 2; ++x) {
                                    const int tok = j0 + 16 * sb + 8 * x + G::token(g);
                                    const bool sees = tok <= pos && tok >= lo && tok < hi && ks[sb] != kNoPage &&
                                                      (p.window < 0 || tok >= pos - p.window || tok < p.n_global);
                                    if (!sees) e[k][sb][2 * x + y] = -INFINITY;
                                }
                        }
                }
            };
            auto top_of = [&](int k, int y) {
                float top = -INFINITY;
#pragma unroll
                for (int sb = 0; sb < G::kSub; ++sb) top = sm100::fmax3(top, e[k][sb][y], e[k][sb][2 + y]);
                return top;
            };
            exponents(false);
            float most = -INFINITY;
#pragma unroll
            for (int k = 0; k < R; ++k) most = sm100::fmax3(most, top_of(k, 0), top_of(k, 1));
            if (__any_sync(0xffffffffu, most > kMoveAt<T>)) {
                scores();  // again: the exponents took their place
                exponents(true);
#pragma unroll
                for (int k = 0; k < R; ++k) {
                    float m[2];
#pragma unroll
                    for (int y = 0; y < 2; ++y) {
                        float top = top_of(k, y);
#pragma unroll
                        for (int z = 4; z < 32; z <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, z));
                        const float to = kParts == 2 ? floorf(top) : top - kHeadroom;
                        m[y] = top - st.m[k][y] > kMoveAt<T> ? to : st.m[k][y];
                    }
                    st.scale(k, ex2(st.m[k][0] - m[0]), ex2(st.m[k][1] - m[1]));
                    st.m[k][0] = m[0];
                    st.m[k][1] = m[1];
#pragma unroll
                    for (int sb = 0; sb < G::kSub; ++sb)
#pragma unroll
                        for (int y = 0; y < 4; ++y) e[k][sb][y] -= m[y & 1];
                }
            }
#pragma unroll
            for (int k = 0; k < R; ++k)
#pragma unroll
                for (int sb = 0; sb < G::kSub; ++sb) {
#pragma unroll
                    for (int y = 0; y < 4; ++y) e[k][sb][y] = ex2(e[k][sb][y]);
                    st.l[k][0] = fmaf(e[k][sb][0] + e[k][sb][2], inv_vs[sb], st.l[k][0]);
                    st.l[k][1] = fmaf(e[k][sb][1] + e[k][sb][3], inv_vs[sb], st.l[k][1]);
                }
            // O^T += V^T P^T
#pragma unroll
            for (int sb = 0; sb < G::kSub; ++sb) {
                if (!full && vsc[sb] < kMinScale) continue;
                uint32_t pb[kParts][R][2];
#pragma unroll
                for (int k = 0; k < R; ++k)
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        float p0 = e[k][sb][2 * x], p1 = e[k][sb][2 * x + 1];
                        if constexpr (kParts == 2) {
                            p0 *= rest_vs[sb];
                            p1 *= rest_vs[sb];
                        }
                        const uint32_t h = half_pair(p0, p1);
                        pb[0][k][x] = transpose8(h);
                        if constexpr (kParts == 2) pb[1][k][x] = transpose8(half_rest(p0, p1, h, kRestScale));
                    }
                uint32_t v[4][(G::kVBytes + 3) / 4];
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    load_words<G::kVBytes>(vd + sb * G::kBox + 8 * (r >> 1) * D + v_at[r & 1], v[r]);
                    if (!full) {  // tokens that no row may see: their codes may be anything
                        const int tok = j0 + 16 * sb + 8 * (r >> 1) + G::token(2 * c + (r & 1));
                        if (tok < lo || tok >= hi || ks[sb] == kNoPage) {
#pragma unroll
                            for (int y = 0; y < (G::kVBytes + 3) / 4; ++y) v[r][y] = 0;
                        }
                    }
                }
#pragma unroll
                for (int y = 0; y < G::kVBytes / 4; ++y)
#pragma unroll
                    for (int z = 0; z < 2; ++z) {  // byte columns 4 y + 2 z, + 1
                        const unsigned pick = z ? 0x7362 : 0x5140;
                        uint32_t a[4];
                        codes_to_half<CODE>(__byte_perm(v[0][y], v[1][y], pick), a[0], a[1]);
                        codes_to_half<CODE>(__byte_perm(v[2][y], v[3][y], pick), a[2], a[3]);
                        if constexpr (kParts == 1) {
#pragma unroll
                            for (int k = 0; k < R; ++k) mma_f16(st.o[k][2 * y + z], a, pb[0][k][0], pb[0][k][1]);
                        } else {  // on their own first: the products' accumulation truncates, these sums round
                            float t[R][4] = {};
                            uint32_t r[4];
#pragma unroll
                            for (int x = 0; x < 4; ++x) r[x] = rest_codes(a[x]);
#pragma unroll
                            for (int k = 0; k < R; ++k) mma_f16(t[k], r, pb[1][k][0], pb[1][k][1]);
#pragma unroll
                            for (int k = 0; k < R; ++k) mma_f16(t[k], a, pb[0][k][0], pb[0][k][1]);
#pragma unroll
                            for (int k = 0; k < R; ++k)
#pragma unroll
                                for (int x = 0; x < 4; ++x) st.o[k][2 * y + z][x] += t[k][x];
                        }
                    }
            }
        };
        load_query<T, D, R>(p, t, part.hk, q);
        st.clear();
        Walk<Geo<D>::kGroup> now;
        for (now.begin(t, part.first); now.x < part.last; now.next(t)) {
            if (!dead && !sm100::mbar_wait_bounded(full_at + 8 * stage, phase, kCacheWaitCycles)) dead = true;
            const int lo = now.lo(t), hi = now.hi(t), j0 = now.j + warp * G::kSub * 16;
            const uint8_t* kd = ring + stage * (kWarps * 2 * G::kSide);
            const uint8_t* vd = kd + G::kSide;
            const float *ksc = &sh.scales[stage][0][warp * G::kSub], *vsc = &sh.scales[stage][1][warp * G::kSub];
            if (j0 + 16 * G::kSub > lo && j0 < hi) {
                bool odd = false;  // a sub-block without a page or with a V scale of 0
#pragma unroll
                for (int sb = 0; sb < G::kSub; ++sb) odd |= vsc[sb] < kMinScale;
                const int j_end = j0 + 16 * G::kSub;
                const bool full = !odd && (now.x < t.na ? j_end <= t.full_a
                                                        : j_end <= t.full_hi && (j0 >= t.full_lo || j_end <= t.full_a));
                // two copies of the step, so that the common one carries no masks
                if (full)
                    step(kd, vd, ksc, vsc, lo, hi, j0, std::true_type{});
                else
                    step(kd, vd, ksc, vsc, lo, hi, j0, std::false_type{});
            }
            __syncwarp();
            if (lane == 0) sm100::mbar_arrive(empty_at + 8 * stage);
            stage = stage + 1 == kStages ? 0 : stage + 1;
            phase ^= stage == 0;
        }
#pragma unroll
        for (int k = 0; k < R; ++k)
#pragma unroll
            for (int e = 0; e < 2; ++e)
#pragma unroll
                for (int z = 4; z < 32; z <<= 1) st.l[k][e] += __shfl_xor_sync(0xffffffffu, st.l[k][e], z);
        join_warps<D, R>(st, sh.ml, sh.join);
        if (warp == 0) {
            if (part.first == 0 && part.last == t.groups)
                write_rows<T, D, R>(p, t, part.hk, st);
            else  // slot 0: a segment that an earlier block began; slot 1: one that later blocks go on with
                write_piece<D, R>(pieces + ((int64_t)blockIdx.x * 2 + (part.first == 0)) * piece_floats<D, R>(), st, t.rows);
            if (part.first == 0 && part.last < t.groups && lane == 0) {
                const int64_t end = part.place + (int64_t)(part.hk + 1) * t.groups - 1;
                begun[blockIdx.x] = Begun{shares.block_of(end) - (int)blockIdx.x, t.b, t.first_row, t.rows, part.hk, {}};
            }
        }
        part.close(p);
    }
    if (dead) atomicOr(p.c.err, kErrTimeout);  // any lane's: it went on with what the ring held before
}

// Block x: the segment that block x of the other kernel began and others went on
// with: out = sum_i 2^(m_i - m) O_i / sum_i 2^(m_i - m) l_i over its pieces.
template <typename T, int D, int R>
__global__ void __launch_bounds__(kJoinThreads) k_fwd_cache_join(CacheFwdParams p, const float* ws, int grid) {
    constexpr int N = Geo<D>::kSteps, kUnits = R * N * 32, kBatch = 16;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const Begun t = reinterpret_cast<const Begun*>(ws)[blockIdx.x];
    if (t.more <= 0) return;
    const int np = t.more + 1;
    const float* const pieces = ws + (int64_t)grid * (sizeof(Begun) / 4);
    // a thread: 2 rows x 2 elements; 16 pieces' values and their rows' m and l on the way at a time
    for (int u = threadIdx.x; u < kUnits; u += kJoinThreads) {
        const int i = u / 32 % N, g = (u & 31) >> 2, row = 8 * (u / (N * 32)) + 2 * (u & 3);
        if (t.first_row + row >= p.m * p.G) continue;
        float top0 = kNone, top1 = kNone, l0 = 0.f, l1 = 0.f;
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
        if (row < t.rows) {
            for (int x0 = 0; x0 < np; x0 += kBatch) {
                float4 v[kBatch];
                float2 m[kBatch], l[kBatch];
#pragma unroll
                for (int x = 0; x < kBatch; ++x) {
                    m[x] = make_float2(kNone, kNone);
                    l[x] = make_float2(0.f, 0.f);
                    v[x] = make_float4(0.f, 0.f, 0.f, 0.f);
                    if (x0 + x < np) {
                        const float* src = pieces + ((int64_t)(blockIdx.x + x0 + x) * 2 + (x0 + x == 0)) * piece_floats<D, R>();
                        m[x] = *reinterpret_cast<const float2*>(src + row);
                        l[x] = *reinterpret_cast<const float2*>(src + 8 * R + row);
                        v[x] = reinterpret_cast<const float4*>(src + 16 * R)[u];
                    }
                }
                float up0 = top0, up1 = top1;
#pragma unroll
                for (int x = 0; x < kBatch; ++x) {
                    up0 = fmaxf(up0, m[x].x);
                    up1 = fmaxf(up1, m[x].y);
                }
                const float a0 = ex2(top0 - up0), a1 = ex2(top1 - up1);
                top0 = up0;
                top1 = up1;
                l0 *= a0;
                l1 *= a1;
                o = make_float4(o.x * a0, o.y * a1, o.z * a0, o.w * a1);
#pragma unroll
                for (int x = 0; x < kBatch; ++x) {
                    const float w0 = ex2(m[x].x - up0), w1 = ex2(m[x].y - up1);
                    l0 = fmaf(w0, l[x].x, l0);
                    l1 = fmaf(w1, l[x].y, l1);
                    o.x = fmaf(w0, v[x].x, o.x);
                    o.y = fmaf(w1, v[x].y, o.y);
                    o.z = fmaf(w0, v[x].z, o.z);
                    o.w = fmaf(w1, v[x].w, o.w);
                }
            }
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int in_tile = row + e, r = t.first_row + in_tile;
            if (r >= p.m * p.G) continue;
            const int q = r / p.G, h = t.hk * p.G + r % p.G;
            const float l = e ? l1 : l0;
            const bool there = in_tile < t.rows && l != 0.f;
            const float inv = there ? 1.f / (kLift<T> * l) : 0.f;
            const float a = there ? (e ? o.y : o.x) * inv : 0.f, b = there ? (e ? o.w : o.z) * inv : 0.f;
            T* out = static_cast<T*>(p.out) + t.b * p.o_sb + h * p.o_sh + q * p.o_sn + Geo<D>::kVBytes * g + 2 * i;
            if constexpr (std::is_same<T, float>::value)
                *reinterpret_cast<float2*>(out) = make_float2(a, b);
            else
                *reinterpret_cast<__nv_bfloat162*>(out) = __floats2bfloat162_rn(a, b);
            if (p.lse && g == 0 && i == 0)
                p.lse[((int64_t)t.b * p.H + h) * p.m + q] = there ? ((e ? top1 : top0) + log2f(l)) * kLn2 : -INFINITY;
        }
    }
}

// {d, token, head, page} bytes, box {d, 16, 1, 1}.
typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                  const cuuint64_t*, const cuuint32_t*, const cuuint32_t*,
                                  CUtensorMapInterleave, CUtensorMapSwizzle, CUtensorMapL2promotion,
                                  CUtensorMapFloatOOBfill);
cudaError_t side_map(CUtensorMap* map, const CacheSide& side, const CacheView& c, int d) {
    static EncodeTiledFn fn = nullptr;
    static std::once_flag once;
    std::call_once(once, []() {
        void* f = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &f, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<EncodeTiledFn>(f);
    });
    if (!fn) return cudaErrorNotSupported;
    const uint64_t page = 1u << c.page_shift, st = side.s_t;
    const uint64_t sh = c.Hk > 1 ? side.s_h : st * page, sp = c.num_pages > 1 ? side.s_p : sh * c.Hk;
    const cuuint64_t dims[4] = {(cuuint64_t)d, page, (cuuint64_t)c.Hk, (cuuint64_t)c.num_pages};
    const cuuint64_t strides[3] = {st, sh, sp};
    const cuuint32_t box[4] = {(cuuint32_t)d, 16, 1, 1}, one[4] = {1, 1, 1, 1};
    const CUresult r = fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, side.codes, dims, strides, box, one,
                          CU_TENSOR_MAP_INTERLEAVE_NONE,
                          d == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : d == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_32B,
                          CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

template <typename T, int CODE, int D, int R>
cudaError_t fwd_r(const CacheFwdParams& p, int num_sms, float* ws, cudaStream_t s) {
    const int smem = (int)sizeof(Shared<D, R, stages<T, D, R>()>) + kRingAlign - 16;
    CUtensorMap k_map, v_map;
    cudaError_t e = side_map(&k_map, p.c.k, p.c, D);
    if (e == cudaSuccess) e = side_map(&v_map, p.c.v, p.c, D);
    if (e != cudaSuccess) return e;
    e = cudaFuncSetAttribute(k_fwd_cache<T, CODE, D, R>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    const int grid = num_sms * blocks_per_sm<T, D, R>();
    k_fwd_cache<T, CODE, D, R><<<grid, kThreads, smem, counted(s)>>>(k_map, v_map, p, ws);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(kJoinThreads);
    cfg.stream = counted(s);
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, k_fwd_cache_join<T, D, R>, p, (const float*)ws, grid);
}

// R as the rows need: each further 8 rows cost products but no bytes.
template <typename T, int CODE, int D>
cudaError_t fwd_d(const CacheFwdParams& p, int num_sms, float* ws, cudaStream_t s) {
    const int rows = p.m * p.G;
    if (rows <= 8) return fwd_r<T, CODE, D, 1>(p, num_sms, ws, s);
    if (rows <= 16 || parts<T>() == 2) return fwd_r<T, CODE, D, 2>(p, num_sms, ws, s);
    if constexpr (parts<T>() == 1) {
        if (rows <= 24) return fwd_r<T, CODE, D, 3>(p, num_sms, ws, s);
        return fwd_r<T, CODE, D, 4>(p, num_sms, ws, s);
    }
    return cudaErrorInvalidValue;
}

template <typename T, int CODE>
cudaError_t fwd_code(const CacheFwdParams& p, int d, int num_sms, float* ws, cudaStream_t s) {
    switch (d) {
        case 32: return fwd_d<T, CODE, 32>(p, num_sms, ws, s);
        case 64: return fwd_d<T, CODE, 64>(p, num_sms, ws, s);
        default: return fwd_d<T, CODE, 128>(p, num_sms, ws, s);
    }
}

template <typename T, int D, int R>
constexpr int64_t block_floats() {
    return blocks_per_sm<T, D, R>() * (2 * piece_floats<D, R>() + (int64_t)sizeof(Begun) / 4);
}
template <typename T, int D>
constexpr int64_t workspace_per_sm() {
    const int64_t a = block_floats<T, D, 1>(), b = block_floats<T, D, 2>(), c = block_floats<T, D, 3>(), d = block_floats<T, D, 4>();
    const int64_t ab = a > b ? a : b, cd = c > d ? c : d;
    return ab > cd ? ab : cd;
}

}  // namespace

int64_t fwd_cache_workspace(int real, int d, int num_sms) {
    if (real == 0)
        return num_sms * (d == 32 ? workspace_per_sm<__nv_bfloat16, 32>() : d == 64 ? workspace_per_sm<__nv_bfloat16, 64>()
                                                                                    : workspace_per_sm<__nv_bfloat16, 128>());
    return num_sms * (d == 32 ? workspace_per_sm<float, 32>() : d == 64 ? workspace_per_sm<float, 64>()
                                                                        : workspace_per_sm<float, 128>());
}

cudaError_t launch_fwd_cache(const CacheFwdParams& p, int real, int code, int d, int num_sms, float* ws,
                             cudaStream_t s) {
    if (real == 0)
        return code == kCodeI8 ? fwd_code<__nv_bfloat16, kCodeI8>(p, d, num_sms, ws, s)
                               : fwd_code<__nv_bfloat16, kCodeE4m3>(p, d, num_sms, ws, s);
    return code == kCodeI8 ? fwd_code<float, kCodeI8>(p, d, num_sms, ws, s)
                           : fwd_code<float, kCodeE4m3>(p, d, num_sms, ws, s);
}

}  // namespace spattn
