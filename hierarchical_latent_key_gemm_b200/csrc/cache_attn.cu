// Exact softmax attention over selected tokens read from the paged cache.
//
// Per (query, query head): o = sum_j softmax_j(q . k_j / sqrt(d)) v_j over the
// row of tokens its KV head selected, k_j and v_j being the pages' values
// (8-bit codes times the scale of their page and head, or bf16).
//
// One warp per key, CUDA cores: lane l holds components l, l + 32, ...; the
// warps of a CTA take every kWarps-th key of the row, each with its own running
// maximum and sum, and are merged at the end.  The K scale multiplies the
// score, the V scale the weight.
#include "cache_common.cuh"

namespace lsa {
namespace {

constexpr int kWarps = 4;
constexpr int kHeads = 4;    // query heads of a CTA

struct AttnArgs {
    CacheArgs c;
    const void* Q;
    const int32_t* idx;
    const int32_t* cnt;
    void* O;
    float* lse;
    int64_t nq;
    int hq, G, max_sel, groups;
    float scale_log2;
    int32_t* err;
};

__device__ __forceinline__ float value(const __nv_bfloat16* p) { return __bfloat162float(*p); }
__device__ __forceinline__ float value(const uint8_t* p) { return e4m3x2_to_f32x2(*p).x; }
__device__ __forceinline__ float value(const float* p) { return *p; }
__device__ __forceinline__ void put(float* p, float x) { *p = x; }
__device__ __forceinline__ void put(__nv_bfloat16* p, float x) { *p = __float2bfloat16_rn(x); }

template <int D, typename T, typename CT>
__global__ __launch_bounds__(kWarps * 32) void cache_attn_kernel(const AttnArgs a) {
    constexpr bool kScaled = sizeof(CT) == 1;
    constexpr int PL = D / 32;
    __shared__ float Om[kWarps][kHeads][D];
    __shared__ float Mm[kWarps][kHeads], Lm[kWarps][kHeads];
    const CacheArgs& c = a.c;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int grp = blockIdx.x % a.groups;
    const int64_t row = blockIdx.x / a.groups;      // (b * nq + qi) * hkv + h
    const int h = (int)(row % c.hkv);
    const int64_t bq = row / c.hkv;
    const int64_t b = bq / a.nq;
    const int g0 = grp * kHeads, gn = min(kHeads, a.G - g0);
    const int64_t q0 = (bq * a.hq + (int64_t)h * a.G + g0) * D;
    int n = a.cnt[row];
    if (n < 0 || n > a.max_sel) {
        if (tid == 0) latch(a.err, kErrDevice);
        n = n < 0 ? 0 : a.max_sel;
    }
    const int32_t* ir = a.idx + row * a.max_sel;
    const T* Q = static_cast<const T*>(a.Q) + q0;
    float q[kHeads][PL], acc[kHeads][PL], m[kHeads], l[kHeads];
#pragma unroll
    for (int g = 0; g < kHeads; ++g) {
        m[g] = -INFINITY;
        l[g] = 0.f;
#pragma unroll
        for (int t = 0; t < PL; ++t) {
            acc[g][t] = 0.f;
            q[g][t] = g < gn ? value(Q + g * D + lane + 32 * t) : 0.f;
        }
    }
    for (int j = warp; j < n; j += kWarps) {
        const int64_t tok = ir[j];
        const int pid = cache_page(c, b, tok);
        if (pid < 0) {
            if (lane == 0) latch(a.err, kErrDevice);
            continue;
        }
        const int64_t o = cache_row(c, pid, h, tok) * D + lane;
        float ks = a.scale_log2, vs = 1.f;
        if (kScaled) {
            ks *= c.K_scale[(int64_t)pid * c.hkv + h];
            vs = c.V_scale[(int64_t)pid * c.hkv + h];
        }
        float k[PL], v[PL];
#pragma unroll
        for (int t = 0; t < PL; ++t) {
            k[t] = value(static_cast<const CT*>(c.K) + o + 32 * t);
            v[t] = value(static_cast<const CT*>(c.V) + o + 32 * t);
        }
#pragma unroll
        for (int g = 0; g < kHeads; ++g) {
            if (g >= gn) break;
            float s = 0.f;
#pragma unroll
            for (int t = 0; t < PL; ++t) s = fmaf(q[g][t], k[t], s);
#pragma unroll
            for (int i = 16; i >= 1; i >>= 1) s += __shfl_xor_sync(0xffffffffu, s, i);
            const float x = s * ks;
            const float mn = fmaxf(m[g], x);
            const float ref = mn == -INFINITY ? 0.f : mn;
            const float al = exp2f(m[g] - ref);
            const float p = exp2f(x - ref);
            l[g] = l[g] * al + p;
#pragma unroll
            for (int t = 0; t < PL; ++t) acc[g][t] = acc[g][t] * al + p * vs * v[t];
            m[g] = mn;
        }
    }
#pragma unroll
    for (int g = 0; g < kHeads; ++g) {
#pragma unroll
        for (int t = 0; t < PL; ++t) Om[warp][g][lane + 32 * t] = acc[g][t];
        if (lane == 0) { Mm[warp][g] = m[g]; Lm[warp][g] = l[g]; }
    }
    __syncthreads();
    for (int e = tid; e < gn * D; e += kWarps * 32) {
        const int g = e / D, col = e % D;
        float M = -INFINITY;
        for (int w = 0; w < kWarps; ++w) M = fmaxf(M, Mm[w][g]);
        const float ref = M == -INFINITY ? 0.f : M;
        float L = 0.f, o = 0.f;
        for (int w = 0; w < kWarps; ++w) {
            const float f = exp2f(Mm[w][g] - ref);
            L += f * Lm[w][g];
            o += f * Om[w][g][col];
        }
        put(static_cast<T*>(a.O) + q0 + e, L == 0.f ? 0.f : o / L);
        if (col == 0 && a.lse)
            a.lse[q0 / D + g] = L == 0.f ? -INFINITY : (M + log2f(L)) * 0.69314718055994531f;
    }
}

template <int D, typename T>
int launch(const AttnArgs& a, int cache_dtype, int64_t ctas, cudaStream_t s) {
    note_launch();
    if (cache_dtype == LSA_E4M3)
        cache_attn_kernel<D, T, uint8_t><<<(unsigned)ctas, kWarps * 32, 0, s>>>(a);
    else
        cache_attn_kernel<D, T, __nv_bfloat16><<<(unsigned)ctas, kWarps * 32, 0, s>>>(a);
    return cuda_status(cudaGetLastError());
}

}  // namespace

int launch_cache_attn(const lsa_kv_cache& cache, const void* Q, const int32_t* idx, const int32_t* cnt, int64_t nq,
                      int hq, int dtype, int max_sel, void* O, float* lse, int32_t* err, cudaStream_t s) {
    AttnArgs a{cache_args(cache), Q, idx, cnt, O, lse, nq, hq, hq / cache.hkv, max_sel};
    a.groups = (a.G + kHeads - 1) / kHeads;
    a.scale_log2 = 1.4426950408889634f / sqrtf((float)cache.d);
    a.err = err;
    const int64_t ctas = cache.batch * nq * cache.hkv * a.groups;
    if (cache.d == 128)
        return dtype == LSA_F32 ? launch<128, float>(a, cache.dtype, ctas, s)
                                : launch<128, __nv_bfloat16>(a, cache.dtype, ctas, s);
    return dtype == LSA_F32 ? launch<64, float>(a, cache.dtype, ctas, s)
                            : launch<64, __nv_bfloat16>(a, cache.dtype, ctas, s);
}

}  // namespace lsa
