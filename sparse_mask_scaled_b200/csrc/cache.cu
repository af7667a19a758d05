// Writing the 8-bit key/value cache, and reading it back.
//
// Write. Token t of the call goes to place start[b] + t of sequence b. One
// thread block takes one page of one head, of K or of V, and reads that page's
// new tokens once: they stay in registers between the two steps,
//     a = max |x| (finite x),  s = max(a / qmax, the page's scale if it already holds older tokens),
//     code = round(x / s), clipped to +-qmax,
// and where s grew the older tokens' codes become round((c * s_old) / s). Both
// quotients are IEEE fp32 quotients, so that the codes are a function of the
// inputs alone. Bound: HBM (values in, codes out).
//
// Read. One thread turns 16 codes (16 bytes) into 16 values. Bound: HBM.
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
};

// The code of x under scale s. A NaN becomes 0, an infinity the largest code of
// its sign (the callers flag both).
template <int CODE>
__device__ __forceinline__ uint32_t make_code(float x, float s) {
    if (!(s > 0.f) || x != x) return 0u;
    float q = __fdiv_rn(x, s);
    q = fminf(fmaxf(q, -code_max<CODE>()), code_max<CODE>());
    if constexpr (CODE == kCodeI8) return (uint32_t)(uint8_t)(int8_t)__float2int_rn(q);
    return (uint32_t)__nv_cvt_float_to_fp8(q, __NV_SATFINITE, __NV_E4M3);
}

// KV values of kVec codes in one store.
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

// Threads of a block that share one page: page * D / kVec 16-byte vectors, NV a
// thread.
template <typename T, int CODE, int D, int NV>
__global__ void __launch_bounds__(1024) k_cache_write(CacheView c, CacheRows r, int slots) {
    constexpr int V = Real<T>::kVec;
    constexpr int kRow = D / V;  // vectors a token
    __shared__ float s_amax[32];
    int64_t x = blockIdx.x;
    const int kv = (int)(x & 1);
    x >>= 1;
    const int h = (int)(x % c.Hk);
    x /= c.Hk;
    const int slot = (int)(x % slots);
    const int b = (int)(x / slots);
    const int64_t start = r.start ? r.start[b] : 0;
    int64_t end = r.length ? r.length[b] : r.m;
    end = start + (end < r.m ? end : r.m);
    const int64_t cap = cache_capacity(c);
    if (start < 0 || end > cap) {  // outside what the table can hold: the sequence is left out
        if (end > start && threadIdx.x == 0) atomicOr(c.err, kErrBadPage);
        return;
    }
    const int page = 1 << c.page_shift;
    const int64_t p0 = ((start >> c.page_shift) + slot) << c.page_shift;  // the page's first token
    if (end <= start || p0 >= end) return;
    const int64_t lo = p0 > start ? p0 : start;
    const int64_t hi = p0 + page < end ? p0 + page : end;
    const int pid = cache_page(c, b, p0);
    if (pid < 0) return;
    const CacheSide& side = kv ? c.v : c.k;
    const T* src = static_cast<const T*>(kv ? r.v : r.k) + b * (kv ? r.v_sb : r.k_sb) + h * (kv ? r.v_sh : r.k_sh);
    const int64_t s_n = kv ? r.v_sn : r.k_sn;
    uint8_t* dst = side.codes + pid * side.s_p + h * side.s_h;
    float* scale = side.scale + (int64_t)pid * c.Hk + h;
    const int older = (int)(lo - p0), fresh_end = (int)(hi - p0);  // places [older, fresh_end) are new

    uint4 w[NV];
    float amax = 0.f;
    bool odd = false;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int e = i * blockDim.x + threadIdx.x;
        const int o = e / kRow, at = (e % kRow) * V;
        w[i] = make_uint4(0, 0, 0, 0);
        if (o >= older && o < fresh_end)
            w[i] = *reinterpret_cast<const uint4*>(src + (p0 + o - start) * s_n + at);
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        float f[V];
        Real<T>::unpack(w[i], f);
#pragma unroll
        for (int y = 0; y < V; ++y) {
            const float a = fabsf(f[y]);
            const bool finite = a < INFINITY;
            odd |= !finite;
            amax = fmaxf(amax, finite ? a : 0.f);
        }
    }
    if (odd) atomicOr(c.err, kErrNonFinite);
#pragma unroll
    for (int y = 16; y > 0; y >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, y));
    if ((threadIdx.x & 31) == 0) s_amax[threadIdx.x >> 5] = amax;
    const float before = older > 0 ? *scale : 0.f;
    __syncthreads();
    for (int y = 0; y < (int)(blockDim.x >> 5); ++y) amax = fmaxf(amax, s_amax[y]);
    const float fresh = __fdiv_rn(amax, code_max<CODE>());
    const bool grown = fresh > before;
    const float s = grown ? fresh : before;
    if (threadIdx.x == 0 && (grown || older == 0)) *scale = s;  // every thread has read it before the barrier
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int e = i * blockDim.x + threadIdx.x;
        const int o = e / kRow, at = (e % kRow) * V;
        uint8_t* p = dst + o * side.s_t + at;
        float f[V];
        if (o >= older && o < fresh_end) {
            Real<T>::unpack(w[i], f);
        } else if (o < older && grown) {
            uint32_t u[V / 4];
            load_codes<V>(p, u);
#pragma unroll
            for (int y = 0; y < V; ++y)
                f[y] = __fmul_rn(code_value<CODE>((u[y / 4] >> (8 * (y % 4))) & 0xffu), before);
        } else {
            continue;
        }
        uint32_t u[V / 4];
#pragma unroll
        for (int y = 0; y < V / 4; ++y) u[y] = 0;
#pragma unroll
        for (int y = 0; y < V; ++y) u[y / 4] |= make_code<CODE>(f[y], s) << (8 * (y % 4));
        store_codes<V>(p, u);
    }
}

template <typename T>
__device__ __forceinline__ void store_values(T* p, const float (&f)[16]);
template <>
__device__ __forceinline__ void store_values<__nv_bfloat16>(__nv_bfloat16* p, const float (&f)[16]) {
    uint32_t u[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
        u[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    reinterpret_cast<uint4*>(p)[0] = make_uint4(u[0], u[1], u[2], u[3]);
    reinterpret_cast<uint4*>(p)[1] = make_uint4(u[4], u[5], u[6], u[7]);
}
template <>
__device__ __forceinline__ void store_values<float>(float* p, const float (&f)[16]) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
        reinterpret_cast<float4*>(p)[i] = make_float4(f[4 * i], f[4 * i + 1], f[4 * i + 2], f[4 * i + 3]);
}

// A block: 256 / (D / 16) tokens of one (b, h), of K (z = 0) or V (z = 1).
template <typename T, int CODE, int D>
__global__ void __launch_bounds__(256) k_cache_read(CacheView c, CacheRows r) {
    constexpr int kRow = D / 16, kTokens = 256 / kRow;
    const int h = (int)(blockIdx.x % c.Hk), b = (int)(blockIdx.x / c.Hk);
    const bool kv = blockIdx.z != 0;
    const CacheSide& side = kv ? c.v : c.k;
    const int64_t start = r.start ? r.start[b] : 0;
    const int64_t asked = r.length ? r.length[b] : r.m;
    const int64_t cap = cache_capacity(c);
    T* dst = static_cast<T*>(kv ? r.v : r.k) + b * (kv ? r.v_sb : r.k_sb) + h * (kv ? r.v_sh : r.k_sh);
    const int64_t s_n = kv ? r.v_sn : r.k_sn;
    const int at = (threadIdx.x % kRow) * 16;
    for (int64_t t = (int64_t)blockIdx.y * kTokens + threadIdx.x / kRow; t < r.m; t += (int64_t)gridDim.y * kTokens) {
        float f[16];
#pragma unroll
        for (int y = 0; y < 16; ++y) f[y] = 0.f;
        const int64_t j = start + t;
        if (t < asked) {
            int pid = -1;
            if (j >= 0 && j < cap)
                pid = cache_page(c, b, j);
            else
                atomicOr(c.err, kErrBadPage);
            if (pid >= 0) {
                const int o = (int)(j & ((1 << c.page_shift) - 1));
                const uint4 w = __ldg(reinterpret_cast<const uint4*>(side.codes + pid * side.s_p + h * side.s_h +
                                                                     o * side.s_t + at));
                const float s = __ldg(side.scale + (int64_t)pid * c.Hk + h);
                const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                for (int y = 0; y < 16; ++y)
                    f[y] = __fmul_rn(code_value<CODE>((u[y / 4] >> (8 * (y % 4))) & 0xffu), s);
            }
        }
        store_values<T>(dst + t * s_n + at, f);
    }
}

template <typename T, int CODE, int D>
cudaError_t write_d(const CacheView& c, const CacheRows& r, cudaStream_t s) {
    const int page = 1 << c.page_shift;
    const int slots = (int)(((int64_t)r.m + page - 2) / page + 1);
    const int vecs = page * D / Real<T>::kVec;
    const int threads = vecs / 4 < 32 ? 32 : vecs / 4 > 1024 ? 1024 : vecs / 4;
    const int64_t blocks = (int64_t)c.B * slots * c.Hk * 2;
    if (blocks > 0x7fffffff) return cudaErrorInvalidConfiguration;
    switch (vecs / threads) {
        case 2: k_cache_write<T, CODE, D, 2><<<(unsigned)blocks, threads, 0, counted(s)>>>(c, r, slots); break;
        case 4: k_cache_write<T, CODE, D, 4><<<(unsigned)blocks, threads, 0, counted(s)>>>(c, r, slots); break;
        case 8: k_cache_write<T, CODE, D, 8><<<(unsigned)blocks, threads, 0, counted(s)>>>(c, r, slots); break;
        default: return cudaErrorInvalidConfiguration;
    }
    return cudaGetLastError();
}

template <typename T, int CODE, int D>
cudaError_t read_d(const CacheView& c, const CacheRows& r, cudaStream_t s) {
    constexpr int kTokens = 256 / (D / 16);
    const int64_t y = ((int64_t)r.m + kTokens - 1) / kTokens;
    const dim3 grid((unsigned)(c.B * c.Hk), (unsigned)(y < 65535 ? y : 65535), 2);
    k_cache_read<T, CODE, D><<<grid, 256, 0, counted(s)>>>(c, r);
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
