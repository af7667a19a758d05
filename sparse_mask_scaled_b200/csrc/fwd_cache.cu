// Attention of a sequence's last tokens over its 8-bit key/value cache.
//
// Query t < qlen[b] of sequence b is token pos = seqlen[b] - qlen[b] + t. It
// attends to the tokens j <= pos, and with a window only to those with
// j >= pos - window or j < n_global:
//     s_j = scale <q, k_j>,  out = sum_j softmax_j(s) v_j,  lse = log sum_j exp(s_j)
// One warp a query row, with a running maximum and sum; a lane holds d / 32 of
// the row's elements.
#include "cache.cuh"
#include "sm100_ptx.cuh"

namespace spattn {
namespace {

template <typename T, int CODE, int D>
__global__ void __launch_bounds__(128) k_fwd_cache_row(CacheFwdParams p) {
    constexpr int E = D / 32;
    const int lane = threadIdx.x & 31;
    const int64_t row = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
    if (row >= (int64_t)p.B * p.H * p.m) return;
    const int t = (int)(row % p.m), h = (int)(row / p.m % p.H), b = (int)(row / p.m / p.H);
    const CacheView& c = p.c;
    const int hk = h / p.G;
    int64_t n = p.seqlen[b];
    const int64_t cap = cache_capacity(c);
    n = n < 0 ? 0 : n < cap ? n : cap;
    int64_t nq = p.qlen ? p.qlen[b] : p.m;
    nq = nq < 0 ? 0 : nq < p.m ? nq : p.m;
    const int64_t pos = t < nq ? n - nq + t : -1;
    float q[E], acc[E], m = -INFINITY, l = 0.f;
    const T* qp = static_cast<const T*>(p.q) + b * p.q_sb + h * p.q_sh + t * p.q_sn;
#pragma unroll
    for (int e = 0; e < E; ++e) {
        q[e] = (float)qp[lane + 32 * e] * p.scale_log2;
        acc[e] = 0.f;
    }
    const int64_t first = p.window < 0 || pos < p.window ? 0 : pos - p.window;
    for (int64_t j = 0; j <= pos; ++j) {
        if (j < first && j >= p.n_global) j = first;
        const int pid = cache_page(c, b, j);
        if (pid < 0) continue;
        const int64_t o = j & ((1 << c.page_shift) - 1);
        const uint8_t* kp = c.k.codes + pid * c.k.s_p + hk * c.k.s_h + o * c.k.s_t;
        const uint8_t* vp = c.v.codes + pid * c.v.s_p + hk * c.v.s_h + o * c.v.s_t;
        const float ks = c.k.scale[(int64_t)pid * c.Hk + hk], vs = c.v.scale[(int64_t)pid * c.Hk + hk];
        float s = 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e) s += q[e] * code_value<CODE>(kp[lane + 32 * e]);
#pragma unroll
        for (int y = 16; y > 0; y >>= 1) s += __shfl_xor_sync(0xffffffffu, s, y);
        s *= ks;
        const float m_new = fmaxf(m, s);
        const float a = exp2f(m - m_new), w = exp2f(s - m_new);
        l = l * a + w;
#pragma unroll
        for (int e = 0; e < E; ++e) acc[e] = acc[e] * a + w * (code_value<CODE>(vp[lane + 32 * e]) * vs);
        m = m_new;
    }
    T* op = static_cast<T*>(p.out) + b * p.o_sb + h * p.o_sh + t * p.o_sn;
#pragma unroll
    for (int e = 0; e < E; ++e) op[lane + 32 * e] = (T)(l != 0.f ? acc[e] / l : 0.f);
    if (p.lse && lane == 0) p.lse[row] = l != 0.f ? (m + log2f(l)) * kLn2 : -INFINITY;
}

template <typename T, int CODE>
cudaError_t fwd_d(const CacheFwdParams& p, int d, cudaStream_t s) {
    const unsigned grid = (unsigned)(((int64_t)p.B * p.H * p.m + 3) / 4);
    switch (d) {
        case 32: k_fwd_cache_row<T, CODE, 32><<<grid, 128, 0, counted(s)>>>(p); break;
        case 64: k_fwd_cache_row<T, CODE, 64><<<grid, 128, 0, counted(s)>>>(p); break;
        default: k_fwd_cache_row<T, CODE, 128><<<grid, 128, 0, counted(s)>>>(p); break;
    }
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_fwd_cache(const CacheFwdParams& p, int real, int code, int d, cudaStream_t s) {
    if (real == 0)
        return code == kCodeI8 ? fwd_d<__nv_bfloat16, kCodeI8>(p, d, s) : fwd_d<__nv_bfloat16, kCodeE4m3>(p, d, s);
    return code == kCodeI8 ? fwd_d<float, kCodeI8>(p, d, s) : fwd_d<float, kCodeE4m3>(p, d, s);
}

}  // namespace spattn
