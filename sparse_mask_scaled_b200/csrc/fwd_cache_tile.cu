// Cache attention for many rows (chunks of a prompt, drafted tokens of wide
// groups): the same operation, line of steps and pieces as fwd_cache.cu, with
// tensor-core tiles (tcgen05) of 128 rows x 128 tokens. bf16 queries.
//
// One block an SM walks its part of the line in tiles of 256 rows of one K/V head:
// two halves of 128 rows share each group of 128 tokens, so that one half's
// softmax runs beside the other's products and every code is converted once for
// 256 rows. Roles:
//   warps 0-3, 4-7   softmax of half 0 and 1, a row a thread (its tensor-memory lane)
//   warps 8-11       codes from global memory to fp16 tiles in shared memory
//                    (K: rows of the B operand; V: the same layout read MN-major)
//   warp 12          issues the products
// Tensor memory: S of half t in columns [128 t, 128 t + 128), O in [256 + 128 t, + d).
// P (fp16) overwrites the front of S and is the A operand of O += P V.
//
// Numbers are held as in fwd_cache.cu: codes and scaled queries exact in fp16, fp32
// accumulators, exponents p' = 2^(x + log2 vs - m) with a reference m that moves
// only when a weight would pass 2^15; then O, l and the group's P so far are scaled.
//
// What bounds it: a 128 x 128 step of d = 128 is two 512-cycle products, 1024
// cycles of exponentials (16 a cycle) and about as many of the softmax's other
// work, shared by two halves. None of them is near its limit (a chunk of 2 x 2048
// tokens behind 8190: 390 us, 617 TFLOP/s; tensor pipe 30 %, exponentials 31 %,
// issue slots 41 % of the time): the halves wait for one another's hand-overs.
#include "cache_attn.cuh"

#include <type_traits>

namespace spattn {
namespace {

using namespace cache_attn;
using namespace sm100;

constexpr int kGroup = 128, kRows = 256;
constexpr int kTileThreads = 512;  // warps 13-15 only complete the last warpgroup
constexpr int kTmemCols = 512;
constexpr int kParamSlots = 4;  // scales of a group: read by the softmax after K's buffer is free again

template <int D>
struct TileGeo {
    static constexpr int kRowBytes = D >= 64 ? 128 : 64;     // of a swizzled row of fp16
    static constexpr int kChunkElems = kRowBytes / 2;
    static constexpr int kChunkBytes = 128 * kRowBytes;      // 128 rows of kChunkElems elements
    static constexpr int kTileBytes = 128 * D * 2;
    static constexpr int kStepsPerChunk = kChunkElems / 16;
    static constexpr int kPerToken = D / 16;                 // threads that load a token's codes, 16 each
    static constexpr int kPasses = kPerToken;                // of 128 / kPerToken tokens
    static constexpr cute::UMMA::LayoutType kLayout =
        D >= 64 ? cute::UMMA::LayoutType::SWIZZLE_128B : cute::UMMA::LayoutType::SWIZZLE_64B;
    // Byte of the 16-byte unit `u` (8 elements) of row r in a tile.
    static __device__ __forceinline__ int unit(int r, int u) {
        constexpr int kUnits = kRowBytes / 16;
        const int x = D >= 64 ? r & 7 : (r >> 1) & 3;
        return (u / kUnits) * kChunkBytes + r * kRowBytes + ((u % kUnits) ^ x) * 16;
    }
};

// fp16 x fp16 -> fp32, M x N, A K-major.
__device__ __forceinline__ uint32_t idesc_f16_f32(int M, int N, bool b_mn_major) {
    cute::UMMA::InstrDescriptor i;
    i.desc_ = 0;
    i.c_format_ = 1;  // F32 accumulator; A and B formats 0: F16
    i.b_major_ = b_mn_major ? 1 : 0;
    i.n_dim_ = static_cast<uint16_t>(N >> 3);
    i.m_dim_ = static_cast<uint16_t>(M >> 4);
    return i.desc_;
}

template <int D>
struct TileShared {
    uint8_t q[2][TileGeo<D>::kTileBytes];
    uint8_t k[2][TileGeo<D>::kTileBytes];
    uint8_t v[2][TileGeo<D>::kTileBytes];
    float ks[kParamSlots][8], lv[kParamSlots][8], inv[kParamSlots][8];  // of each 16 tokens
    uint64_t q_full[2], s_full[2], p_full[2], pv_done[2];               // of each half
    uint64_t k_full[2], k_empty[2], v_full[2], v_empty[2];              // of each buffer
    uint64_t drain;
    uint32_t tmem;
    volatile int abort;
};

template <int D>
constexpr int tile_piece_floats() {
    return kRows * (2 + D);
}

// Waits for phase `parity`, giving up when it or any other role's wait ran out.
// Whole warps call it and get one answer.
__device__ __forceinline__ bool tile_wait(uint32_t bar, uint32_t parity, volatile int* abort) {
    bool ok = mbar_try_wait(bar, parity);
    if (!ok) {
        const long long t0 = clock64();
        while (!(ok = mbar_try_wait(bar, parity)) && !*abort) {
            if (clock64() - t0 > kCacheWaitCycles) *abort = 1;
        }
    }
    return __all_sync(0xffffffffu, ok);
}

// ------------------------------------------------------------------ codes to tiles
template <int CODE, int D, typename Part>
__device__ __forceinline__ void convert_role(const CacheFwdParams& p, TileShared<D>& sh, Part part, int rts) {
    using G = TileGeo<D>;
    const int tid = threadIdx.x & 127, lane = tid & 31;
    const int page_mask = (1 << p.c.page_shift) - 1;
    struct Step {
        int raw;  // the table's entry for sub-block lane % 8, kUnread where none is needed
        int j, lo, hi, hk;
        bool more;
    };
    bool open = part.open(p, rts);
    Walk<kGroup> w;
    if (open) w.begin(part.t, part.first);
    auto look_up = [&]() -> Step {
        Step s{kUnread, 0, 0, 0, 0, open};
        if (!open) return s;
        s.j = w.j;
        s.lo = w.lo(part.t);
        s.hi = w.hi(part.t);
        s.hk = part.hk;
        const int j = w.j + 16 * (lane & 7);
        if (j + 16 > s.lo && j < s.hi) s.raw = __ldg(p.c.table + part.t.b * p.c.table_stride + (j >> p.c.page_shift));
        w.next(part.t);
        if (w.x >= part.last) {
            part.close(p);
            open = part.open(p, rts);
            if (open) w.begin(part.t, part.first);
        }
        return s;
    };
    const int sub_lane = tid % G::kPerToken, first_token = tid / G::kPerToken;
    constexpr int kTokens = 128 / G::kPerToken;  // of a pass, a multiple of 16
    const int in_sub = first_token & 15;
    // requests a step's codes of one side
    auto load = [&](uint4 (&x)[G::kPasses], const CacheSide& side, const Step& s) {
        int64_t at = -1;  // of this lane's sub-block
        if (s.raw >= 0) at = s.raw * side.s_p + s.hk * side.s_h + ((s.j + 16 * (lane & 7)) & page_mask) * side.s_t;
        const bool whole = s.j >= s.lo && s.j + kGroup <= s.hi;
        const uint8_t* const mine = side.codes + in_sub * side.s_t + 16 * sub_lane;
#pragma unroll
        for (int i = 0; i < G::kPasses; ++i) {
            const int o = i * kTokens + first_token;
            const int64_t from = __shfl_sync(0xffffffffu, at, o >> 4);
            x[i] = make_uint4(0, 0, 0, 0);  // tokens that no row may see: zeros, whatever their codes
            if (from >= 0 && (whole || (s.j + o >= s.lo && s.j + o < s.hi)))
                x[i] = __ldg(reinterpret_cast<const uint4*>(mine + from));
        }
    };
    auto check = [&](Step& s) {
        if ((unsigned)s.raw >= (unsigned)p.c.num_pages) {
            if (s.raw != kUnread) atomicOr(p.c.err, kErrBadPage);
            s.raw = -1;
        }
    };
    // sub-blocks whose bit in `zero` is set become zeros
    auto store = [&](const uint4 (&x)[G::kPasses], uint8_t* tile, unsigned zero) {
        const bool swap = (sub_lane >> 2) & 1;  // half the lanes of a token the other way round: no bank conflicts
        uint8_t* const first = tile + G::unit(first_token, 2 * sub_lane + swap);
        uint8_t* const second = tile + G::unit(first_token, 2 * sub_lane + !swap);
#pragma unroll
        for (int i = 0; i < G::kPasses; ++i) {  // rows a multiple of 16 apart are swizzled alike
            uint4 a, b;
            codes_to_half<CODE>(x[i].x, a.x, a.y);
            codes_to_half<CODE>(x[i].y, a.z, a.w);
            codes_to_half<CODE>(x[i].z, b.x, b.y);
            codes_to_half<CODE>(x[i].w, b.z, b.w);
            if (zero >> ((i * kTokens + first_token) >> 4) & 1) a = b = make_uint4(0, 0, 0, 0);
            *reinterpret_cast<uint4*>(first + i * kTokens * G::kRowBytes) = swap ? b : a;
            *reinterpret_cast<uint4*>(second + i * kTokens * G::kRowBytes) = swap ? a : b;
        }
    };
    const uint32_t k_full = smem_u32(&sh.k_full[0]), k_empty = smem_u32(&sh.k_empty[0]), v_full = smem_u32(&sh.v_full[0]),
                   v_empty = smem_u32(&sh.v_empty[0]);
    Step now = look_up(), next = look_up();
    uint4 kx[G::kPasses], vx[G::kPasses];
    check(now);
    load(kx, p.c.k, now);
    load(vx, p.c.v, now);
    float ks = kNoPage, vs = kNoPage;  // of sub-block lane % 8
    auto scales = [&](const Step& s) {
        ks = vs = kNoPage;
        if (s.raw >= 0) {
            const int64_t sc = (int64_t)s.raw * p.c.Hk + s.hk;
            ks = __ldg(p.c.k.scale + sc);
            vs = __ldg(p.c.v.scale + sc);
        }
    };
    scales(now);
    for (uint32_t n = 0; now.more; ++n) {
        check(next);
        const Step after = look_up();
        if (!tile_wait(k_empty + 8 * (n & 1), ((n >> 1) & 1) ^ 1, &sh.abort)) return;
        const bool none = vs < kMinScale;  // no page, or a scale that counts as 0: its values are zeros
        const unsigned zero = __ballot_sync(0xffffffffu, none) & 0xffu;
        if (tid < 8) {
            const int slot = n % kParamSlots;
            sh.ks[slot][tid] = ks;
            sh.lv[slot][tid] = none ? kNoValues : lg2(vs);
            sh.inv[slot][tid] = none ? kNoValuesInv : __frcp_rn(vs);
        }
        store(kx, sh.k[n & 1], 0u);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(k_full + 8 * (n & 1));
        if (next.more) {
            load(kx, p.c.k, next);
            scales(next);
        }
        if (!tile_wait(v_empty + 8 * (n & 1), ((n >> 1) & 1) ^ 1, &sh.abort)) return;
        store(vx, sh.v[n & 1], zero);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(v_full + 8 * (n & 1));
        if (next.more) load(vx, p.c.v, next);
        now = next;
        next = after;
    }
}

// ------------------------------------------------------------------ products
// a * b + c, two fp32 lanes.
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}

// Halves of a tile that have rows.
__device__ __forceinline__ int halves(const Tile& t) { return t.rows > 128 ? 2 : 1; }

template <int D, typename Part>
__device__ __forceinline__ void product_role(const CacheFwdParams& p, TileShared<D>& sh, Part part, int rts) {
    using G = TileGeo<D>;
    const uint32_t tmem = sh.tmem;
    const uint32_t id_s = idesc_f16_f32(128, 128, false), id_o = idesc_f16_f32(128, D, true);
    const uint32_t sbo = 8 * G::kRowBytes;
    const uint64_t dq = smem_desc(smem_u32(sh.q[0]), 16, sbo, G::kLayout), dk = smem_desc(smem_u32(sh.k[0]), 16, sbo, G::kLayout);
    const uint64_t dv = smem_desc(smem_u32(sh.v[0]), G::kChunkBytes, sbo, G::kLayout);
    auto bar = [&](uint64_t (&b)[2], int x) { return smem_u32(&b[x]); };
    auto scores = [&](int t, uint32_t n) {
        tc_fence_after();
#pragma unroll 1
        for (int k = 0; k < D / 16; ++k) {
            const uint64_t off = (uint64_t)(((k / G::kStepsPerChunk) * G::kChunkBytes + (k % G::kStepsPerChunk) * 32) >> 4);
            mma_bf16_ss_elect(tmem + 128 * t, dq + (uint64_t)((t * G::kTileBytes) >> 4) + off,
                              dk + (uint64_t)(((n & 1) * G::kTileBytes) >> 4) + off, id_s, k > 0);
        }
        mma_commit_elect(bar(sh.s_full, t));
    };
    auto values = [&](int t, uint32_t n, bool begin) {
        tc_fence_after();
#pragma unroll 1
        for (int k = 0; k < 8; ++k)
            mma_bf16_ts_elect(tmem + 256 + 128 * t, tmem + 128 * t + 8 * k,
                              dv + (uint64_t)(((n & 1) * G::kTileBytes + k * 16 * G::kRowBytes) >> 4), id_o, !(begin && k == 0));
        mma_commit_elect(bar(sh.pv_done, t));
    };
    volatile int* abort = &sh.abort;
    uint32_t n = 0;                        // groups so far
    uint32_t steps[2] = {0, 0}, segs[2] = {0, 0};  // of each half
    bool alive = true;
    for (; alive && part.open(p, rts); part.close(p)) {
        const int nt = halves(part.t), count = part.last - part.first;
        for (int t = 0; alive && t < nt; ++t) {
            alive = tile_wait(bar(sh.q_full, t), segs[t] & 1, abort) &&
                    (t > 0 || tile_wait(bar(sh.k_full, n & 1), (n >> 1) & 1, abort));
            if (!alive) break;
            ++segs[t];
            scores(t, n);
        }
        if (!alive) break;
        mma_commit_elect(bar(sh.k_empty, n & 1));
        for (int i = 0; alive && i < count; ++i, ++n) {
            for (int t = 0; t < nt; ++t) {
                alive = tile_wait(bar(sh.p_full, t), steps[t] & 1, abort) &&
                        (t > 0 || tile_wait(bar(sh.v_full, n & 1), (n >> 1) & 1, abort));
                if (!alive) break;
                values(t, n, i == 0);
                if (t == nt - 1) mma_commit_elect(bar(sh.v_empty, n & 1));
                if (i + 1 < count) {  // S takes the place of P
                    alive = tile_wait(bar(sh.pv_done, t), steps[t] & 1, abort) &&
                            (t > 0 || tile_wait(bar(sh.k_full, (n + 1) & 1), ((n + 1) >> 1) & 1, abort));
                    if (!alive) break;
                    scores(t, n + 1);
                    if (t == nt - 1) mma_commit_elect(bar(sh.k_empty, (n + 1) & 1));
                }
                ++steps[t];
            }
        }
    }
    // every product is done before tensor memory is given back
    mma_commit_elect(smem_u32(&sh.drain));
    mbar_wait_bounded(smem_u32(&sh.drain), 0, kCacheWaitCycles);
}

// Rows of a tile's second half that lie in it but whose half holds no query of the
// sequence (rows <= 128) are nobody's above: zeros.
__device__ __forceinline__ void clear_rows(const CacheFwdParams& p, const Tile& t, int hk, int d) {
    for (int x = threadIdx.x & 127; x < 128 * (d / 8); x += 128) {
        const int row = t.first_row + 128 + x / (d / 8);
        if (row >= p.m * p.G) continue;
        const int q = row / p.G, h = hk * p.G + row % p.G, at = x % (d / 8);
        __nv_bfloat16* out = static_cast<__nv_bfloat16*>(p.out) + t.b * p.o_sb + h * p.o_sh + q * p.o_sn;
        reinterpret_cast<uint4*>(out)[at] = make_uint4(0, 0, 0, 0);
        if (p.lse && at == 0) p.lse[((int64_t)t.b * p.H + h) * p.m + q] = -INFINITY;
    }
}

// ------------------------------------------------------------------ softmax
template <int D, typename Part>
__device__ __forceinline__ void softmax_role(const CacheFwdParams& p, TileShared<D>& sh, Part part, int rts,
                                             const Shares& shares, float* ws) {
    using G = TileGeo<D>;
    const int half = threadIdx.x >> 7, lane = threadIdx.x & 31, in_half = threadIdx.x & 127;
    const uint32_t lanes = (uint32_t)(in_half & 96) << 16;  // this warp's tensor-memory lanes
    const uint32_t s_at = sh.tmem + 128 * half + lanes, o_at = sh.tmem + 256 + 128 * half + lanes;
    const uint32_t q_full = smem_u32(&sh.q_full[half]), s_full = smem_u32(&sh.s_full[half]), p_full = smem_u32(&sh.p_full[half]),
                   pv_done = smem_u32(&sh.pv_done[half]);
    Begun* const begun = reinterpret_cast<Begun*>(ws);
    float* const pieces = ws + (int64_t)gridDim.x * (sizeof(Begun) / 4);
    uint32_t n = 0, steps = 0;  // groups so far, and those of this half
    for (; part.open(p, rts); part.close(p)) {
        const Tile& t = part.t;
        const int count = part.last - part.first;
        if (half >= halves(t)) {
            n += count;
            if (part.first == 0) clear_rows(p, t, part.hk, D);
            continue;
        }
        const int in_tile = 128 * half + in_half, row = t.first_row + in_tile;
        const bool valid = in_tile < t.rows;
        // the row's query, scaled by a power of two so that its largest element lies in [2^14, 2^15)
        float factor;
        {
            uint4 x[D / 8];
            const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(p.q);
            if (valid) src += t.b * p.q_sb + (part.hk * p.G + row % p.G) * p.q_sh + (row / p.G) * p.q_sn;
            uint32_t top2 = 0;
#pragma unroll
            for (int y = 0; y < D / 8; ++y) {
                x[y] = valid ? __ldg(reinterpret_cast<const uint4*>(src) + y) : make_uint4(0, 0, 0, 0);
                top2 = __vmaxu2(__vmaxu2(top2, x[y].x & 0x7fff7fffu), x[y].y & 0x7fff7fffu);
                top2 = __vmaxu2(__vmaxu2(top2, x[y].z & 0x7fff7fffu), x[y].w & 0x7fff7fffu);
            }
            const float top = __uint_as_float(max(top2 >> 16, top2 & 0xffffu) << 16);
            int up = 0;
            if (top > 0.f && top < INFINITY) up = 14 - ilogbf(top);
            up = up > 120 ? 120 : up;
            const float by = exp2f((float)up);
            factor = p.scale_log2 * exp2f((float)-up);
#pragma unroll
            for (int y = 0; y < D / 8; ++y) {
                const uint32_t u[4] = {x[y].x, x[y].y, x[y].z, x[y].w};
                uint32_t h[4];
#pragma unroll
                for (int z = 0; z < 4; ++z)
                    h[z] = half_pair(__uint_as_float(u[z] << 16) * by, __uint_as_float(u[z] & 0xffff0000u) * by);
                *reinterpret_cast<uint4*>(sh.q[half] + G::unit(in_half, y)) = make_uint4(h[0], h[1], h[2], h[3]);
            }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(q_full);
        const int pos = valid ? max(t.base + row / p.G, -1) : -1;  // (so that pos - window stays in range)
        // tokens that every row of this half attends to
        const int half_rows = t.rows - 128 * half < 128 ? t.rows - 128 * half : 128;
        const int lo_pos = t.base + (t.first_row + 128 * half) / p.G, hi_pos = t.base + (t.first_row + 128 * half + half_rows - 1) / p.G;
        const int full_hi = lo_pos + 1, full_lo = p.window >= 0 && hi_pos > p.window ? hi_pos - p.window : 0;
        const int full_a = p.n_global < full_hi ? p.n_global : full_hi;
        const bool idle = __all_sync(0xffffffffu, !valid);  // no row of this warp: nothing but the barriers
        float m = kNone, l = 0.f;
        Walk<kGroup> w;
        for (w.begin(t, part.first); w.x < part.last; w.next(t), ++n, ++steps) {
            if (!tile_wait(s_full, steps & 1, &sh.abort)) return;
            tc_fence_after();
            if (!idle) {
                const int slot = n % kParamSlots, lo = w.lo(t), hi = w.hi(t), j0 = w.j;
                bool pages = true;
#pragma unroll
                for (int x = 0; x < 8; ++x) pages &= sh.ks[slot][x] != kNoPage;
                const bool full = pages && (w.x < t.na ? j0 + kGroup <= full_a
                                                       : j0 + kGroup <= full_hi && (j0 >= full_lo || j0 + kGroup <= full_a));
                const bool begin = w.x == part.first;
                // 32 tokens: x holds their scores, then their exponents
                auto chunk = [&](float (&x)[32], int c, auto all) {
                    auto exponents = [&](float ref) {
#pragma unroll
                        for (int b = 0; b < 2; ++b) {
                            const float f = factor * sh.ks[slot][2 * c + b], a = sh.lv[slot][2 * c + b] - ref;
                            const uint64_t f2 = pack2(f, f), a2 = pack2(a, a);
#pragma unroll
                            for (int y = 16 * b; y < 16 * b + 16; y += 2)
                                unpack2(fma2(pack2(x[y], x[y + 1]), f2, a2), x[y], x[y + 1]);
                        }
                        if constexpr (!decltype(all)::value) {
#pragma unroll
                            for (int y = 0; y < 32; ++y) {
                                const int tok = j0 + 32 * c + y;
                                const bool sees = tok <= pos && tok >= lo && tok < hi && sh.ks[slot][2 * c + y / 16] != kNoPage &&
                                                  (p.window < 0 || tok >= pos - p.window || tok < p.n_global);
                                if (!sees) x[y] = -INFINITY;
                            }
                        }
                    };
                    auto top = [&]() {
                        float a = fmax3(x[0], x[1], x[2]), b = fmax3(x[3], x[4], x[5]);
#pragma unroll
                        for (int y = 6; y < 30; y += 4) {
                            a = fmax3(a, x[y], x[y + 1]);
                            b = fmax3(b, x[y + 2], x[y + 3]);
                        }
                        return fmax3(fmaxf(a, b), x[30], x[31]);
                    };
                    exponents(m);
                    if (__any_sync(0xffffffffu, top() > kRescaleAt)) {
                        tmem_ld32f(s_at + 32 * c, x);  // the scores again: no weight lies over them yet
                        tmem_wait_ld_depf(x);
                        exponents(0.f);
                        const float raw = top(), ref = raw - m > kRescaleAt ? raw - kHeadroom : m, by = ex2(m - ref);
                        l *= by;
                        if (!begin) {  // the products into O issued so far are done: S came after them
#pragma unroll 1
                            for (int y = 0; y < D; y += 32) {
                                uint32_t o[32];
                                tmem_ld32(o_at + y, o);
                                tmem_wait_ld_dep(o);
#pragma unroll
                                for (int z = 0; z < 32; ++z) o[z] = __float_as_uint(__uint_as_float(o[z]) * by);
                                tmem_st32(o_at + y, o);
                            }
                        }
                        tmem_wait_st();
#pragma unroll 1
                        for (int y = 0; y < c; ++y) {  // the group's weights so far
                            uint32_t h[16];
                            tmem_ld16(s_at + 16 * y, h);
                            tmem_wait_ld_dep16(h);
#pragma unroll
                            for (int z = 0; z < 16; ++z) {
                                const __half2 v = *reinterpret_cast<const __half2*>(&h[z]);
                                h[z] = half_pair(__low2float(v) * by, __high2float(v) * by);
                            }
                            tmem_st16(s_at + 16 * y, h);
                        }
                        m = ref;
#pragma unroll
                        for (int y = 0; y < 32; ++y) x[y] -= ref;
                    }
                    uint32_t h[16];
#pragma unroll
                    for (int b = 0; b < 2; ++b) {
                        uint64_t sum = pack2(0.f, 0.f);
#pragma unroll
                        for (int y = 0; y < 16; y += 2) {
                            const float p0 = ex2(x[16 * b + y]), p1 = ex2(x[16 * b + y + 1]);
                            sum = add2(sum, pack2(p0, p1));
                            h[8 * b + y / 2] = half_pair(p0, p1);
                        }
                        float s0, s1;
                        unpack2(sum, s0, s1);
                        l = fmaf(s0 + s1, sh.inv[slot][2 * c + b], l);
                    }
                    tmem_st16(s_at + 16 * c, h);
                };
                // one chunk's registers at a time: with a second one in flight far more spilled (483 us for 391;
                // this build spills 108 bytes a thread), and the other half's warps cover the load
#pragma unroll 1
                for (int c = 0; c < 4; ++c) {
                    float x[32];
                    tmem_ld32f(s_at + 32 * c, x);
                    tmem_wait_ld_depf(x);
                    if (full)
                        chunk(x, c, std::true_type{});
                    else
                        chunk(x, c, std::false_type{});
                }
                tmem_wait_st();
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(p_full);
        }
        if (!tile_wait(pv_done, (steps - 1) & 1, &sh.abort)) return;
        tc_fence_after();
        const bool whole = part.first == 0 && part.last == t.groups;
        // (warp-wide: tensor memory is read by whole warps)
        {
            const bool held = row < p.m * p.G;
            const int q = row / p.G, h = part.hk * p.G + row % p.G;
            const bool there = valid && l != 0.f;
            const float inv = there ? 1.f / l : 0.f;
            __nv_bfloat16* out = static_cast<__nv_bfloat16*>(p.out);
            if (held) out += t.b * p.o_sb + h * p.o_sh + q * p.o_sn;
            float* piece = pieces + ((int64_t)blockIdx.x * 2 + (part.first == 0)) * tile_piece_floats<D>();
            float* acc = piece + 2 * kRows + in_tile * D;
#pragma unroll 1
            for (int y = 0; y < D; y += 32) {
                float o[32];
                if (!idle) {
                    tmem_ld32f(o_at + y, o);
                    tmem_wait_ld_depf(o);
                }
                if (whole) {
                    if (held) {
#pragma unroll
                        for (int z = 0; z < 32; z += 8) {
                            uint32_t u[4];
#pragma unroll
                            for (int x = 0; x < 4; ++x) {
                                const __nv_bfloat162 v = __floats2bfloat162_rn(there ? o[z + 2 * x] * inv : 0.f,
                                                                               there ? o[z + 2 * x + 1] * inv : 0.f);
                                u[x] = *reinterpret_cast<const uint32_t*>(&v);
                            }
                            *reinterpret_cast<uint4*>(out + y + z) = make_uint4(u[0], u[1], u[2], u[3]);
                        }
                    }
                } else if (valid) {
#pragma unroll
                    for (int z = 0; z < 32; z += 4)
                        *reinterpret_cast<float4*>(acc + y + z) = make_float4(o[z], o[z + 1], o[z + 2], o[z + 3]);
                }
            }
            if (whole) {
                if (held && p.lse)
                    p.lse[((int64_t)t.b * p.H + h) * p.m + q] = there ? (m + log2f(l)) * kLn2 : -INFINITY;
            } else {
                if (valid) {
                    piece[in_tile] = m;
                    piece[kRows + in_tile] = l;
                }
                if (part.first == 0 && threadIdx.x == 0) {
                    const int64_t end = part.place + (int64_t)(part.hk + 1) * t.groups - 1;
                    begun[blockIdx.x] = Begun{shares.block_of(end) - (int)blockIdx.x, t.b, t.first_row, t.rows, part.hk, {}};
                }
            }
        }
        tc_fence_before();
    }
}

template <int CODE, int D>
__global__ void __launch_bounds__(kTileThreads, 1) k_fwd_cache_tile(CacheFwdParams p, float* ws) {
    extern __shared__ __align__(16) uint8_t smem_raw[];
    TileShared<D>& sh = *reinterpret_cast<TileShared<D>*>(smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023));
    const int warp = threadIdx.x >> 5;
    asm volatile("griddepcontrol.launch_dependents;");
    if (threadIdx.x == 0) {
        for (int x = 0; x < 2; ++x) {
            mbar_init(smem_u32(&sh.q_full[x]), 4);
            mbar_init(smem_u32(&sh.s_full[x]), 1);
            mbar_init(smem_u32(&sh.p_full[x]), 4);
            mbar_init(smem_u32(&sh.pv_done[x]), 1);
            mbar_init(smem_u32(&sh.k_full[x]), 4);
            mbar_init(smem_u32(&sh.k_empty[x]), 1);
            mbar_init(smem_u32(&sh.v_full[x]), 4);
            mbar_init(smem_u32(&sh.v_empty[x]), 1);
        }
        mbar_init(smem_u32(&sh.drain), 1);
        fence_mbar_init();
        sh.abort = 0;
        reinterpret_cast<Begun*>(ws)[blockIdx.x].more = 0;
    }
    if (warp == 12) tmem_alloc(smem_u32(&sh.tmem), kTmemCols);
    tc_fence_before();
    const Line<kGroup, kRows> line(p);
    __syncthreads();  // the barriers and the tensor memory's address are there
    tc_fence_after();
    const Shares shares(line.total, (int)gridDim.x);
    if ((int)blockIdx.x < shares.blocks) {
        const int rts = line.rts;
        Part<kGroup, kRows> part;
        part.at = shares.start(blockIdx.x);
        part.end = shares.start(blockIdx.x + 1);
        line.find(p, part.at, &part.entry, &part.place);
        // registers: 256 x 152 + 128 x 152 + 128 x 56 = the launch's 512 x 128
        if (warp < 8) {
            asm volatile("setmaxnreg.inc.sync.aligned.u32 152;");
            softmax_role<D>(p, sh, part, rts, shares, ws);
        } else if (warp < 12) {
            asm volatile("setmaxnreg.inc.sync.aligned.u32 152;");
            convert_role<CODE, D>(p, sh, part, rts);
        } else {
            asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
            if (warp == 12) product_role<D>(p, sh, part, rts);
        }
    }
    __syncthreads();
    if (threadIdx.x == 0 && sh.abort) atomicOr(p.c.err, kErrTimeout);
    if (warp == 12) {
        tc_fence_after();
        tmem_dealloc(sh.tmem, kTmemCols);
    }
}

// Blocks (x, y): rows 32 y .. of the segment that block x of the other kernel began
// and others went on with, a warp a row.
template <int D>
__global__ void __launch_bounds__(128) k_fwd_cache_tile_join(CacheFwdParams p, const float* ws) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const Begun t = reinterpret_cast<const Begun*>(ws)[blockIdx.x];
    if (t.more <= 0) return;
    const float* const pieces = ws + (int64_t)gridDim.x * (sizeof(Begun) / 4);
    const int lane = threadIdx.x & 31, np = t.more + 1;
    auto piece = [&](int i) { return pieces + ((int64_t)(blockIdx.x + i) * 2 + (i == 0)) * tile_piece_floats<D>(); };
    for (int x = threadIdx.x >> 5; x < 32; x += 4) {
        const int in_tile = 32 * blockIdx.y + x, row = t.first_row + in_tile;
        if (row >= p.m * p.G) break;
        const int q = row / p.G, h = t.hk * p.G + row % p.G;
        float top = kNone, l = 0.f;
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
        if (in_tile < t.rows) {
            for (int i = lane; i < np; i += 32) top = fmaxf(top, piece(i)[in_tile]);
#pragma unroll
            for (int z = 1; z < 32; z <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, z));
#pragma unroll 4
            for (int i = 0; i < np; ++i) {
                const float* src = piece(i);
                const float w = ex2(src[in_tile] - top);
                l = fmaf(w, src[kRows + in_tile], l);
                if (lane < D / 4) {
                    const float4 v = reinterpret_cast<const float4*>(src + 2 * kRows + in_tile * D)[lane];
                    o.x = fmaf(w, v.x, o.x);
                    o.y = fmaf(w, v.y, o.y);
                    o.z = fmaf(w, v.z, o.z);
                    o.w = fmaf(w, v.w, o.w);
                }
            }
        }
        const bool there = in_tile < t.rows && l != 0.f;
        const float inv = there ? 1.f / l : 0.f;
        if (lane < D / 4) {
            const __nv_bfloat162 a = __floats2bfloat162_rn(there ? o.x * inv : 0.f, there ? o.y * inv : 0.f),
                                 b = __floats2bfloat162_rn(there ? o.z * inv : 0.f, there ? o.w * inv : 0.f);
            __nv_bfloat16* out = static_cast<__nv_bfloat16*>(p.out) + t.b * p.o_sb + h * p.o_sh + q * p.o_sn;
            reinterpret_cast<uint2*>(out)[lane] =
                make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
        }
        if (p.lse && lane == 0) p.lse[((int64_t)t.b * p.H + h) * p.m + q] = there ? (top + log2f(l)) * kLn2 : -INFINITY;
    }
}

template <int CODE, int D>
cudaError_t tile_d(const CacheFwdParams& p, int num_sms, float* ws, cudaStream_t s) {
    const int smem = (int)sizeof(TileShared<D>) + 1024 - 16;
    cudaError_t e = cudaFuncSetAttribute(k_fwd_cache_tile<CODE, D>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    k_fwd_cache_tile<CODE, D><<<num_sms, kTileThreads, smem, counted(s)>>>(p, ws);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(num_sms, kRows / 32);
    cfg.blockDim = dim3(128);
    cfg.stream = counted(s);
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, k_fwd_cache_tile_join<D>, p, (const float*)ws);
}

}  // namespace

int64_t fwd_cache_tile_workspace(int d, int num_sms) {
    return num_sms * (2 * (int64_t)kRows * (2 + d) + (int64_t)sizeof(Begun) / 4);
}

cudaError_t launch_fwd_cache_tile(const CacheFwdParams& p, int code, int d, int num_sms, float* ws, cudaStream_t s) {
    if (code == kCodeI8)
        return d == 32 ? tile_d<kCodeI8, 32>(p, num_sms, ws, s)
               : d == 64 ? tile_d<kCodeI8, 64>(p, num_sms, ws, s) : tile_d<kCodeI8, 128>(p, num_sms, ws, s);
    return d == 32 ? tile_d<kCodeE4m3, 32>(p, num_sms, ws, s)
           : d == 64 ? tile_d<kCodeE4m3, 64>(p, num_sms, ws, s) : tile_d<kCodeE4m3, 128>(p, num_sms, ws, s);
}

}  // namespace spattn
