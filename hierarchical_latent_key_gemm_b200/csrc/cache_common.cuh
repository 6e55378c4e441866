// Shared by the paged KV cache calls: the cache as kernels see it, and the
// conversions between fp32 and the pages' 8-bit floats.
#pragma once

#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "lsa_internal.cuh"

namespace lsa {

struct CacheArgs {
    void* K;
    void* V;
    float* K_scale;
    float* V_scale;
    const int32_t* table;
    int64_t n_pages, ld_pages;
    int hkv, page, log2_page;
};

inline CacheArgs cache_args(const lsa_kv_cache& c) {
    int lg = 4;
    while ((1 << lg) < c.page) ++lg;
    return CacheArgs{c.K, c.V, c.K_scale, c.V_scale, c.page_table, c.n_pages, c.ld_pages, c.hkv, c.page, lg};
}

// Page id of token `tok` of sequence b, or -1 when the table does not cover it
// or names a page outside the pool.
__device__ __forceinline__ int cache_page(const CacheArgs& c, int64_t b, int64_t tok) {
    const int64_t col = tok >> c.log2_page;
    if (tok < 0 || col >= c.ld_pages) return -1;
    const int p = __ldg(c.table + b * c.ld_pages + col);
    return (p >= 0 && p < c.n_pages) ? p : -1;
}

// Row (of d values) of a token in the pools.
__device__ __forceinline__ int64_t cache_row(const CacheArgs& c, int page_id, int h, int64_t tok) {
    return (((int64_t)page_id * c.hkv + h) << c.log2_page) + (tok & (c.page - 1));
}

// Four e4m3 codes (low byte first) to two pairs of fp16 values; exact.
__device__ __forceinline__ void e4m3x4_to_f16x4(uint32_t v, uint32_t& lo, uint32_t& hi) {
    asm("{.reg .b16 l, h;\n"
        "mov.b32 {l, h}, %2;\n"
        "cvt.rn.f16x2.e4m3x2 %0, l;\n"
        "cvt.rn.f16x2.e4m3x2 %1, h;}"
        : "=r"(lo), "=r"(hi)
        : "r"(v));
}
__device__ __forceinline__ float4 e4m3x4_to_f32x4(uint32_t v) {
    uint32_t lo, hi;
    e4m3x4_to_f16x4(v, lo, hi);
    const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&lo));
    const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&hi));
    return make_float4(a.x, a.y, b.x, b.y);
}
// Round to nearest even, saturating; NaN stays NaN.  lo lands in the low byte.
__device__ __forceinline__ uint16_t f32x2_to_e4m3x2(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}

}  // namespace lsa
