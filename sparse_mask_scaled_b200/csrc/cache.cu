// Writing the 8-bit key/value cache, and reading it back.
//
// Write. Token t of the call goes to place start[b] + t of sequence b. One
// thread block (one warp, for a few tokens) takes one page of one head, of K or
// of V, and reads that page's new tokens once; they stay in registers between
//     a = max |x| (finite x),  s = max(a / qmax, the page's scale if it already holds older tokens),
//     code = round(x / s), clipped to +-qmax,
// and where s grew the older tokens' codes become round((c * s_old) / s). Both
// quotients are IEEE fp32 quotients, so that the codes are a function of the
// inputs alone; a division is only made where the product with 1 / s lies so near
// a rounding border that it could round the other way. HBM (values in, codes
// out) would take 19 us of the 46 us that 8 prompts of up to 4096 tokens take
// (8 heads, d = 128, bf16 to e4m3): what bounds it is issue, 72 % of the time,
// about 25 instructions a value.
//
// Read. A thread turns 16 bytes' worth of values of several tokens, all loads
// before the first use. Bound: HBM (4 x up to 16384 tokens: 119 us on the device, 93 %
// of the measured copy rate).
#include "cache.cuh"

namespace spattn {
namespace {

template <typename T>
struct Real;
template <>
struct Real<__nv_bfloat16> {
    static constexpr int kVec = 8;  // values in 16 bytes
    static __device__ __forceinline__ void unpack(const uint4& w, float* x) {
        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[2 * i] = __uint_as_float(u[i] << 16);
            x[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
        }
    }
    // The largest magnitude (as bits, so that a NaN counts as more than infinity).
    template <int N>
    static __device__ __forceinline__ float top(const uint4 (&w)[N]) {
        uint32_t t = 0;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            t = __vmaxu2(t, w[i].x & 0x7fff7fffu);
            t = __vmaxu2(t, w[i].y & 0x7fff7fffu);
            t = __vmaxu2(t, w[i].z & 0x7fff7fffu);
            t = __vmaxu2(t, w[i].w & 0x7fff7fffu);
        }
        return __uint_as_float(max(t >> 16, t & 0xffffu) << 16);
    }
};
template <>
struct Real<float> {
    static constexpr int kVec = 4;
    static __device__ __forceinline__ void unpack(const uint4& w, float* x) {
        x[0] = __uint_as_float(w.x);
        x[1] = __uint_as_float(w.y);
        x[2] = __uint_as_float(w.z);
        x[3] = __uint_as_float(w.w);
    }
    template <int N>
    static __device__ __forceinline__ float top(const uint4 (&w)[N]) {
        uint32_t t = 0;
#pragma unroll
        for (int i = 0; i < N; ++i)
            t = max(max(t, max(w[i].x & 0x7fffffffu, w[i].y & 0x7fffffffu)), max(w[i].z & 0x7fffffffu, w[i].w & 0x7fffffffu));
        return __uint_as_float(t);
    }
};

// The code of x under scale s, by division. A NaN becomes 0, an infinity the
// largest code of its sign (the callers flag both).
template <int CODE>
__device__ __forceinline__ uint32_t exact_code(float x, float s) {
    if (!(s > 0.f) || x != x) return 0u;
    float q = __fdiv_rn(x, s);
    q = fminf(fmaxf(q, -code_max<CODE>()), code_max<CODE>());
    if constexpr (CODE == kCodeI8) return (uint32_t)(uint8_t)(int8_t)__float2int_rn(q);
    return (uint32_t)__nv_cvt_float_to_fp8(q, __NV_SATFINITE, __NV_E4M3);
}

// Four of them; kept out of line, since it is rare and long.
template <int CODE>
__device__ __noinline__ uint32_t exact_codes(float a, float b, float c, float d, float s) {
    return exact_code<CODE>(a, s) | exact_code<CODE>(b, s) << 8 | exact_code<CODE>(c, s) << 16 | exact_code<CODE>(d, s) << 24;
}

// The codes of finite x[0..V), |x| <= qmax s (1 + 2^-23), and inv = 1 / s rounded.
// x inv is off from the fp32 quotient by less than 4 units in the last place, so
// the two round to the same code unless a border lies that near: for int8 a half,
// at most 2^-14 away (|q| < 128 has units of 2^-17); for e4m3 the bits below the
// code's three, within 8 of a half. Quotients below e4m3's normal range are
// divided too, and so is everything where `divide` says so.
template <int CODE, int V>
__device__ __forceinline__ void make_codes(const float (&x)[V], float s, float inv, bool divide, uint32_t (&w)[V / 4]) {
    float q[V];
    if constexpr (CODE == kCodeI8) {
        float far = 0.f, r[V];
#pragma unroll
        for (int y = 0; y < V; ++y) {
            q[y] = __fmul_rn(x[y], inv);
            r[y] = __fadd_rn(q[y], 12582912.f);  // 1.5 * 2^23: q's integer, ties to even, in the low bits
            far = fmaxf(far, fabsf(q[y] - __fadd_rn(r[y], -12582912.f)));
        }
        divide |= far > 0.5f - 6.103515625e-5f;
#pragma unroll
        for (int y = 0; y < V / 4; ++y) {
            const uint32_t b[4] = {__float_as_uint(r[4 * y]), __float_as_uint(r[4 * y + 1]), __float_as_uint(r[4 * y + 2]),
                                   __float_as_uint(r[4 * y + 3])};
            w[y] = __byte_perm(__byte_perm(b[0], b[1], 0x0040), __byte_perm(b[2], b[3], 0x0040), 0x5410);
        }
    } else {
        uint32_t gap = ~0u;
        float low = INFINITY;
#pragma unroll
        for (int y = 0; y < V; ++y) {
            q[y] = __fmul_rn(x[y], inv);
            gap = min(gap, (__float_as_uint(q[y]) - 0x7fff8u) & 0xfffffu);
            low = fminf(low, fabsf(q[y]));
        }
        divide |= gap <= 16u || low < 0.015625f;
#pragma unroll
        for (int y = 0; y < V / 4; ++y) {
            const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(q[4 * y], q[4 * y + 1]), __NV_SATFINITE, __NV_E4M3);
            const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(q[4 * y + 2], q[4 * y + 3]), __NV_SATFINITE, __NV_E4M3);
            w[y] = lo | hi << 16;
        }
    }
    if (divide) {
#pragma unroll
        for (int y = 0; y < V / 4; ++y) w[y] = exact_codes<CODE>(x[4 * y], x[4 * y + 1], x[4 * y + 2], x[4 * y + 3], s);
    }
}

// V codes as the fp32 products c * s.
template <int CODE, int V>
__device__ __forceinline__ void code_values(const uint32_t (&w)[V / 4], float s, float (&x)[V]) {
#pragma unroll
    for (int y = 0; y < V / 4; ++y) {
        if constexpr (CODE == kCodeI8) {
            const uint32_t u = w[y] ^ 0x80808080u;  // 2^23 + (c + 128)
#pragma unroll
            for (int z = 0; z < 4; ++z)
                x[4 * y + z] = __fmul_rn(__uint_as_float(__byte_perm(u, 0x4b000000u, 0x7440 + z)) - 8388736.f, s);
        } else {
#pragma unroll
            for (int z = 0; z < 2; ++z) {
                const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w[y] >> (16 * z)), __NV_E4M3);
                const float2 f = __half22float2(__half2(h));
                x[4 * y + 2 * z] = __fmul_rn(f.x, s);
                x[4 * y + 2 * z + 1] = __fmul_rn(f.y, s);
            }
        }
    }
}

// V codes in one store or load.
template <int V>
__device__ __forceinline__ void store_codes(uint8_t* p, const uint32_t (&w)[V / 4]) {
    if constexpr (V == 8) {
        *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
    } else {
        *reinterpret_cast<uint32_t*>(p) = w[0];
    }
}
template <int V>
__device__ __forceinline__ void load_codes(const uint8_t* p, uint32_t (&w)[V / 4]) {
    if constexpr (V == 8) {
        const uint2 u = *reinterpret_cast<const uint2*>(p);
        w[0] = u.x;
        w[1] = u.y;
    } else {
        w[0] = *reinterpret_cast<const uint32_t*>(p);
    }
}

// W warps of a block share a page's D * page values as 16-byte vectors, NV a
// thread; vectors behind the first NV (the page's older codes to renew, in the
// one-warp form) are taken in further rounds. With W = 1 a block of four warps
// takes four pages.
template <typename T, int CODE, int D, int NV, bool kOneWarp>
__global__ void __launch_bounds__(kOneWarp ? 128 : 1024, kOneWarp ? 8 : 1)
    k_cache_write(CacheView c, CacheRows r, int slots, int64_t items) {
    constexpr int V = Real<T>::kVec;
    constexpr int kRow = D / V;  // vectors a token
    __shared__ float s_amax[32];
    const int me = kOneWarp ? threadIdx.x & 31 : threadIdx.x, count = kOneWarp ? 32 : blockDim.x;
    int64_t x = kOneWarp ? (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5) : blockIdx.x;
    if (x >= items) return;
    const int kv = (int)(x & 1);
    uint32_t u = (uint32_t)(x >> 1);
    const int h = (int)(u % (uint32_t)c.Hk);
    u /= (uint32_t)c.Hk;
    const int slot = (int)(u % (uint32_t)slots), b = (int)(u / (uint32_t)slots);
    const int64_t start = r.start ? r.start[b] : 0;
    int64_t end = r.length ? r.length[b] : r.m;
    end = start + (end < r.m ? end : r.m);
    const int64_t cap = cache_capacity(c);
    if (start < 0 || end > cap) {  // outside what the table can hold: the sequence is left out
        if (end > start && me == 0) atomicOr(c.err, kErrBadPage);
        return;
    }
    const int page = 1 << c.page_shift;
    const int64_t p0 = ((start >> c.page_shift) + slot) << c.page_shift;  // the page's first token
    if (end <= start || p0 >= end) return;
    const int64_t lo = p0 > start ? p0 : start;
    const int64_t hi = p0 + page < end ? p0 + page : end;
    const int pid = cache_page(c, b, p0);
    const int older = (int)(lo - p0), fresh = (int)(hi - lo);  // places [0, older), then `fresh` new ones
    const T* src = static_cast<const T*>(kv ? r.v : r.k) + b * (kv ? r.v_sb : r.k_sb) + h * (kv ? r.v_sh : r.k_sh) +
                   (lo - start) * (kv ? r.v_sn : r.k_sn);
    const int64_t s_n = kv ? r.v_sn : r.k_sn;
    const CacheSide& side = kv ? c.v : c.k;

    uint4 w[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int e = i * count + me;
        w[i] = make_uint4(0, 0, 0, 0);
        if (e < fresh * kRow) w[i] = __ldg(reinterpret_cast<const uint4*>(src + (e / kRow) * s_n + (e % kRow) * V));
    }
    if (pid < 0) return;
    uint8_t* const dst = side.codes + pid * side.s_p + h * side.s_h;
    float* const scale = side.scale + (int64_t)pid * c.Hk + h;
    const float before = older > 0 ? *scale : 0.f;
    float amax = Real<T>::template top<NV>(w);
    const bool odd = !(amax < INFINITY);
    if (odd) {  // the largest of the finite ones
        atomicOr(c.err, kErrNonFinite);
        amax = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            float f[V];
            Real<T>::unpack(w[i], f);
#pragma unroll
            for (int y = 0; y < V; ++y) amax = fmaxf(amax, fabsf(f[y]) < INFINITY ? fabsf(f[y]) : 0.f);
        }
    }
#pragma unroll
    for (int y = 16; y > 0; y >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, y));
    if constexpr (kOneWarp) {
        __syncwarp();  // every lane has read the scale (an exchange of values orders no memory)
    } else {
        if ((threadIdx.x & 31) == 0) s_amax[threadIdx.x >> 5] = amax;
        __syncthreads();  // and every thread has read the scale
        for (int y = 0; y < (int)(blockDim.x >> 5); ++y) amax = fmaxf(amax, s_amax[y]);
    }
    const float s_new = __fdiv_rn(amax, code_max<CODE>());
    const bool grown = s_new > before;
    const float s = grown ? s_new : before, inv = __frcp_rn(s);
    const bool divide = odd || !(s > 1e-30f);  // below, 1 / s or the products lose bits
    if (me == 0 && (grown || older == 0)) *scale = s;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int e = i * count + me;
        if (e >= fresh * kRow) continue;
        float f[V];
        uint32_t u8[V / 4];
        Real<T>::unpack(w[i], f);
        make_codes<CODE, V>(f, s, inv, divide, u8);
        store_codes<V>(dst + (older + e / kRow) * side.s_t + (e % kRow) * V, u8);
    }
    if (older > 0 && grown) {
        for (int e = me; e < older * kRow; e += count) {
            uint8_t* const at = dst + (e / kRow) * side.s_t + (e % kRow) * V;
            float f[V];
            uint32_t u8[V / 4];
            load_codes<V>(at, u8);
            code_values<CODE, V>(u8, before, f);
            make_codes<CODE, V>(f, s, inv, true, u8);
            store_codes<V>(at, u8);
        }
    }
}

// One 16-byte vector of V values.
template <typename T, int V>
__device__ __forceinline__ uint4 pack_values(const float (&f)[V]) {
    uint32_t u[4];
    if constexpr (V == 4) {
#pragma unroll
        for (int i = 0; i < 4; ++i) u[i] = __float_as_uint(f[i]);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
            u[i] = *reinterpret_cast<const uint32_t*>(&h);
        }
    }
    return make_uint4(u[0], u[1], u[2], u[3]);
}

// A block: kTokens tokens of one (b, h), of K (z = 0) or V (z = 1); a thread: one
// vector of kUnroll of them.
template <typename T, int CODE, int D>
struct ReadGeo {
    static constexpr int kThreads = 128, kUnroll = 8;
    static constexpr int kRow = D / Real<T>::kVec, kStep = kThreads / kRow, kTokens = kStep * kUnroll;
};
template <typename T, int CODE, int D>
__global__ void __launch_bounds__(128) k_cache_read(CacheView c, CacheRows r) {
    using G = ReadGeo<T, CODE, D>;
    constexpr int V = Real<T>::kVec, U = G::kUnroll;
    const int h = (int)(blockIdx.x % c.Hk), b = (int)(blockIdx.x / c.Hk);
    const bool kv = blockIdx.z != 0;
    const CacheSide& side = kv ? c.v : c.k;
    const int64_t start = r.start ? r.start[b] : 0;
    int64_t asked = r.length ? r.length[b] : r.m;
    const int64_t cap = cache_capacity(c);
    T* dst = static_cast<T*>(kv ? r.v : r.k) + b * (kv ? r.v_sb : r.k_sb) + h * (kv ? r.v_sh : r.k_sh);
    const int64_t s_n = kv ? r.v_sn : r.k_sn;
    const int at = (threadIdx.x % G::kRow) * V;
    const uint8_t* codes = side.codes + h * side.s_h + at;
    const int32_t* table = c.table + b * c.table_stride;
    for (int64_t t0 = (int64_t)blockIdx.y * G::kTokens + threadIdx.x / G::kRow; t0 < r.m;
         t0 += (int64_t)gridDim.y * G::kTokens) {
        int pid[U];
        float s[U];
        uint32_t w[U][V / 4];
#pragma unroll
        for (int i = 0; i < U; ++i) {
            const int64_t t = t0 + i * G::kStep, j = start + t;
            const bool in = t < asked && t < r.m, held = j >= 0 && j < cap;
            pid[i] = -1;
            if (in && held) pid[i] = __ldg(table + (j >> c.page_shift));
            if (in && (!held || (unsigned)pid[i] >= (unsigned)c.num_pages)) {
                atomicOr(c.err, kErrBadPage);
                pid[i] = -1;
            }
        }
#pragma unroll
        for (int i = 0; i < U; ++i) {
#pragma unroll
            for (int y = 0; y < V / 4; ++y) w[i][y] = 0;
            s[i] = 0.f;
            if (pid[i] >= 0) {
                const int o = (int)((start + t0 + i * G::kStep) & ((1 << c.page_shift) - 1));
                load_codes<V>(codes + pid[i] * side.s_p + o * side.s_t, w[i]);
                s[i] = __ldg(side.scale + (int64_t)pid[i] * c.Hk + h);
            }
        }
#pragma unroll
        for (int i = 0; i < U; ++i) {
            const int64_t t = t0 + i * G::kStep;
            if (t >= r.m) break;
            float f[V];
            code_values<CODE, V>(w[i], s[i], f);
            if (pid[i] < 0) {  // zeros, not 0 * 0 of some sign
#pragma unroll
                for (int y = 0; y < V; ++y) f[y] = 0.f;
            }
            *reinterpret_cast<uint4*>(dst + t * s_n + at) = pack_values<T, V>(f);
        }
    }
}

template <typename T, int CODE, int D>
cudaError_t write_d(const CacheView& c, const CacheRows& r, cudaStream_t s) {
    constexpr int V = Real<T>::kVec;
    const int page = 1 << c.page_shift;
    const int slots = (int)(((int64_t)r.m + page - 2) / page + 1);
    const int64_t items = (int64_t)c.B * slots * c.Hk * 2;
    // a warp holds four vectors a lane: enough for all new values of a page when the call brings few tokens
    if ((int64_t)(r.m < page ? r.m : page) * D / V <= 128) {
        k_cache_write<T, CODE, D, 4, true><<<(unsigned)((items + 3) / 4), 128, 0, counted(s)>>>(c, r, slots, items);
        return cudaGetLastError();
    }
    // eight vectors a thread share what is done once a thread (place, scale, reduction): 90 us with two,
    // 79 with eight, for 8 prompts written and read back; smaller pages fill a warp with four
    const int vecs = page * D / V;  // 256..8192 here
    if (vecs >= 512)
        k_cache_write<T, CODE, D, 8, false><<<(unsigned)items, vecs / 8, 0, counted(s)>>>(c, r, slots, items);
    else
        k_cache_write<T, CODE, D, 4, false><<<(unsigned)items, vecs / 4, 0, counted(s)>>>(c, r, slots, items);
    return cudaGetLastError();
}

template <typename T, int CODE, int D>
cudaError_t read_d(const CacheView& c, const CacheRows& r, cudaStream_t s) {
    using G = ReadGeo<T, CODE, D>;
    const int64_t y = ((int64_t)r.m + G::kTokens - 1) / G::kTokens;
    const dim3 grid((unsigned)(c.B * c.Hk), (unsigned)(y < 65535 ? y : 65535), 2);
    k_cache_read<T, CODE, D><<<grid, G::kThreads, 0, counted(s)>>>(c, r);
    return cudaGetLastError();
}

template <typename F>
cudaError_t by_kind(int real, int code, int d, F f) {
    auto by_code = [&](auto t) -> cudaError_t {
        auto by_d = [&](auto cc) -> cudaError_t {
            switch (d) {
                case 32: return f(t, cc, std::integral_constant<int, 32>{});
                case 64: return f(t, cc, std::integral_constant<int, 64>{});
                case 128: return f(t, cc, std::integral_constant<int, 128>{});
                default: return cudaErrorInvalidValue;
            }
        };
        return code == kCodeI8 ? by_d(std::integral_constant<int, kCodeI8>{})
                               : by_d(std::integral_constant<int, kCodeE4m3>{});
    };
    return real == 0 ? by_code(__nv_bfloat16{}) : by_code(float{});
}

}  // namespace

cudaError_t launch_cache_write(const CacheView& c, const CacheRows& r, int real, int code, int d, cudaStream_t s) {
    return by_kind(real, code, d, [&](auto t, auto cc, auto dd) {
        return write_d<decltype(t), decltype(cc)::value, decltype(dd)::value>(c, r, s);
    });
}

cudaError_t launch_cache_read(const CacheView& c, const CacheRows& r, int real, int code, int d, cudaStream_t s) {
    return by_kind(real, code, d, [&](auto t, auto cc, auto dd) {
        return read_d<decltype(t), decltype(cc)::value, decltype(dd)::value>(c, r, s);
    });
}

}  // namespace spattn
