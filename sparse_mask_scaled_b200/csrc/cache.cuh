// The 8-bit key/value cache: what its kernels (cache.cu, fwd_cache.cu) and the
// C ABI share.
//
// A cache is a pool of pages, each `page` tokens (a power of two) of every
// key/value head. The codes of page x, head h, token o are d consecutive bytes;
// a code c of page x and head h stands for the fp32 product c * scale[x, h]. Row
// b of the page table lists the pages of sequence b: token j lies in page
// table[b, j / page] at place j % page.
#pragma once

#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "spattn_internal.cuh"

namespace spattn {

constexpr int kCodeI8 = 0;
constexpr int kCodeE4m3 = 1;
constexpr int kMinPage = 16, kMaxPage = 256;
// Tokens of a sequence: the attention's token numbers are 32-bit and run on to the end of a step of
// up to 448 tokens, and to the one behind it.
constexpr int64_t kMaxCacheTokens = 0x7fffffff - 1023;

// Device error flag bits of the cache calls, beside those of spattn_internal.cuh. (That
// header is part of what the other kernels' profiles are hashed over: it stays as it is.)
constexpr unsigned kErrBadPage = 4u;    // a cache place without a page of the pool was left out
constexpr unsigned kErrNonFinite = 8u;  // a NaN or an infinity was written to a cache

struct CacheSide {  // K or V
    uint8_t* codes;
    float* scale;           // [num_pages, Hk]
    int64_t s_p, s_h, s_t;  // bytes between pages, heads, tokens
};

struct CacheView {
    CacheSide k, v;
    const int32_t* table;  // [B, max_pages], rows table_stride apart
    int64_t table_stride;
    int B, max_pages, num_pages, Hk, page_shift;
    unsigned* err;  // device error flags
};

// The page of sequence b that holds token j, or -1 (flagged) when the table
// names none of the pool's pages. Callers pass only tokens that have a place in
// the table.
__device__ __forceinline__ int cache_page(const CacheView& c, int b, int64_t j) {
    const int p = __ldg(c.table + b * c.table_stride + (j >> c.page_shift));
    if ((unsigned)p < (unsigned)c.num_pages) return p;
    atomicOr(c.err, kErrBadPage);
    return -1;
}

// Tokens sequence b can hold.
__device__ __forceinline__ int64_t cache_capacity(const CacheView& c) {
    return (int64_t)c.max_pages << c.page_shift;
}

template <int CODE>
constexpr float code_max() {
    return CODE == kCodeI8 ? 127.f : 448.f;
}

// Entry points of cache.cu. real: 0 bf16, 1 f32; code: kCodeI8 or kCodeE4m3.
struct CacheRows {  // K and V as [B, Hk, m, d]; strides in elements
    void* k;
    void* v;
    int64_t k_sb, k_sh, k_sn, v_sb, v_sh, v_sn;
    int m;
    const int32_t* start;   // nullable (all 0)
    const int32_t* length;  // nullable (all m)
};
cudaError_t launch_cache_write(const CacheView& c, const CacheRows& r, int real, int code, int d, cudaStream_t s);
cudaError_t launch_cache_read(const CacheView& c, const CacheRows& r, int real, int code, int d, cudaStream_t s);

// Entry point of fwd_cache.cu.
struct CacheFwdParams {
    CacheView c;
    const void* q;
    void* out;
    float* lse;  // nullable, [B * H * m]
    int64_t q_sb, q_sh, q_sn, o_sb, o_sh, o_sn;
    int B, H, G, m;         // G query heads share a key/value head
    const int32_t* seqlen;  // [B]
    const int32_t* qlen;    // nullable (all m)
    int window;             // < 0: none
    int n_global;
    float scale_log2;  // scale * log2(e)
};
// Floats of workspace a call needs.
int64_t fwd_cache_workspace(int real, int d, int num_sms);
cudaError_t launch_fwd_cache(const CacheFwdParams& p, int real, int code, int d, int num_sms, float* ws,
                             cudaStream_t s);


// Entry point of fwd_cache_tile.cu (bf16 queries).
int64_t fwd_cache_tile_workspace(int d, int num_sms);
cudaError_t launch_fwd_cache_tile(const CacheFwdParams& p, int code, int d, int num_sms, float* ws, cudaStream_t s);

}  // namespace spattn
