// Exact softmax attention over selected tokens read from the paged cache.
//
// Per (query, query head): o = sum_j softmax_j(q . k_j / sqrt(d)) v_j over the
// row of tokens its KV head selected, k_j and v_j being the pages' values
// (8-bit codes times the scale of their page and head, or bf16).
//
// One pass with a running maximum.  With s_j the V scale of token j's page, the
// kernel keeps, per head and relative to a reference m,
//     w_j = 2^(x_j + log2 s_j - m),   acc = sum w_j code_j,   l = sum w_j / s_j,
// x_j being the score in base-2 units, so that o = acc / l: the V scale is part
// of the exponent, and weights of pages with very different scales meet the
// tensor cores at the size they contribute with.
//
// A warp takes 16 tokens at a time on the M side of mma.sync m16n8k16 (keys x
// heads, then components x heads), so 8 heads fill a tile without padding.
// The sums over d and over tokens do not depend on their order: a thread's
// fragments are therefore whole 16-byte pieces of the gathered rows, loaded
// from the pages straight into registers in the order the tensor cores want
// them, without shared memory.  8-bit codes become fp16 exactly; queries are
// scaled by a power of two per head so that bf16 values are fp16 values too.
//
// The warps of a CTA, and the CTAs of a cluster, take every n-th 16 tokens of
// one row; their (m, l, acc) are merged in shared and distributed shared
// memory in a fixed order.
#include <cooperative_groups.h>

#include <algorithm>

#include "cache_common.cuh"
#include "warp_mma.cuh"

namespace lsa {
namespace {

namespace cg = cooperative_groups;

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kTile = 16;                     // tokens of a warp's step
constexpr int kMaxCluster = 8;
constexpr uint32_t kNoRow = 0xffffffffu;
// Weights are at most 2^(kHeadroom + kLazy) and the largest at least 2^kHeadroom:
// the maximum is renewed only when a score passes it by 2^kLazy.  In fp16 a
// weight keeps 11 bits down to 2^-(14 + kHeadroom) of the largest, and what lies
// below 2^-(25 + kHeadroom) of it is lost.
constexpr float kLazy = 8.f, kHeadroom = 6.f;

struct AttnArgs {
    CacheArgs c;
    const void* Q;
    const int32_t* idx;
    const int32_t* cnt;
    void* O;
    float* lse;
    int64_t nq;
    int hq, G, max_sel, groups, cluster;
    float scale_log2;
    int32_t* err;
};

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float value(const __nv_bfloat16* p) { return __bfloat162float(*p); }
__device__ __forceinline__ float value(const float* p) { return *p; }
__device__ __forceinline__ void put(float* p, float x) { *p = x; }
__device__ __forceinline__ void put(__nv_bfloat16* p, float x) { *p = __float2bfloat16_rn(x); }

// Two floats as `N` pairs of 16-bit floats whose sums carry them: fp16 parts
// (11 bits each) next to 8-bit codes, bf16 parts (8 bits each) next to bf16.
template <bool F16, int N>
__device__ __forceinline__ void split(float a, float b, uint32_t* p) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
        if constexpr (F16) {
            const __half2 h = __floats2half2_rn(a, b);
            p[i] = *reinterpret_cast<const uint32_t*>(&h);
            const float2 f = __half22float2(h);
            a -= f.x;
            b -= f.y;
        } else {
            const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
            p[i] = *reinterpret_cast<const uint32_t*>(&h);
            const float2 f = __bfloat1622float2(h);
            a -= f.x;
            b -= f.y;
        }
    }
}

template <bool F16>
__device__ __forceinline__ void mma(float* c, const uint32_t* a, const uint32_t* b) {
    if constexpr (F16) mma_f16(c, a, b[0], b[1]);
    else mma_bf16(c, a, b[0], b[1]);
}

template <int D, typename CT, typename T, int NT>
__global__ __launch_bounds__(kThreads) void cache_attn_kernel(const AttnArgs a) {
    constexpr bool E4 = sizeof(CT) == 1;              // 8-bit codes, fp16 products; else bf16
    constexpr bool F32 = sizeof(T) == 4;
    constexpr int PQ = F32 ? (E4 ? 2 : 3) : 1;        // 16-bit parts of a query component
    constexpr int PP = F32 ? (E4 ? 2 : 3) : (E4 ? 1 : 2);   // and of a weight
    constexpr int KS = D / 16;                        // k steps of K Q^T, m tiles of V^T P^T
    constexpr int HG = 8 * NT;                        // heads of a warp
    constexpr int KW = D * (int)sizeof(CT) / 16;      // words of a K row in a thread (4 threads a row)
    constexpr int VW = D * (int)sizeof(CT) / 32;      // words of a V row in a thread (8 threads a row)
    constexpr int LD = D + 4;                         // row stride of the merge buffer: no bank conflicts
    __shared__ float acc_s[HG * LD];
    __shared__ float m_s[kWarps][HG], l_s[kWarps][HG];
    __shared__ float mc_s[HG], lc_s[HG];              // of the CTA
    __shared__ float f_s[kMaxCluster][HG], lt_s[HG], mt_s[HG];

    const CacheArgs& c = a.c;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int g = lane >> 2, t = lane & 3;
    const int rank = blockIdx.x % a.cluster;
    const int64_t unit = blockIdx.x / a.cluster;
    const int grp = (int)(unit % a.groups);
    const int64_t row = unit / a.groups;              // (b * nq + qi) * hkv + h
    const int h = (int)(row % c.hkv);
    const int64_t bq = row / c.hkv;
    const int64_t b = bq / a.nq;
    const int g0 = grp * HG, gn = min(HG, a.G - g0);
    const int64_t q0 = (bq * a.hq + (int64_t)h * a.G + g0) * D;
    int n = a.cnt[row];
    if (n < 0 || n > a.max_sel) {
        if (tid == 0) latch(a.err, kErrDevice);
        n = n < 0 ? 0 : a.max_sel;
    }
    const int32_t* ir = a.idx + row * a.max_sel;

    // ---- queries: B fragments, k slots in the order the K pieces come in
    uint32_t qf[PQ][KS][NT][2];
    float qs[NT][2];                                  // factor of the scores of heads 8 nt + 2 t, + 1
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        const T* q = static_cast<const T*>(a.Q) + q0 + (int64_t)(8 * nt + g) * D;
        const bool live = 8 * nt + g < gn;
        float v[KS][4];
        float top = 0.f;
#pragma unroll
        for (int s = 0; s < KS; ++s) {
            const int d0 = E4 ? 16 * (t + 4 * (s / 4)) + 4 * (s % 4) : 8 * (t + 4 * (s / 2)) + 4 * (s % 2);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                v[s][e] = live ? value(q + d0 + e) : 0.f;
                top = fmaxf(top, fabsf(v[s][e]));
            }
        }
        float up = 1.f, down = 1.f;
        if (E4) {
            // largest component to [2^14, 2^15): fp16's subnormals begin 2^-28 below it
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
            const int e = min(100, max(-100, 14 - ((__float_as_int(top) >> 23) - 127)));
            up = __int_as_float((127 + e) << 23);
            down = __int_as_float((127 - e) << 23);
        }
#pragma unroll
        for (int s = 0; s < KS; ++s) {
            uint32_t lo[PQ], hi[PQ];
            split<E4, PQ>(v[s][0] * up, v[s][1] * up, lo);
            split<E4, PQ>(v[s][2] * up, v[s][3] * up, hi);
#pragma unroll
            for (int p = 0; p < PQ; ++p) {
                qf[p][s][nt][0] = lo[p];
                qf[p][s][nt][1] = hi[p];
            }
        }
        qs[nt][0] = __shfl_sync(0xffffffffu, down, 8 * t) * a.scale_log2;
        qs[nt][1] = __shfl_sync(0xffffffffu, down, 8 * t + 4) * a.scale_log2;
    }

    float o[KS][NT][4];
    float m[NT][2], l[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int e = 0; e < 2; ++e) { m[nt][e] = -INFINITY; l[nt][e] = 0.f; }
#pragma unroll
        for (int i = 0; i < KS; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[i][nt][e] = 0.f;
    }

    // ---- tokens: lane j (and j + 16) looks up token j of the warp's step
    const int steps_all = (n + kTile - 1) / kTile;
    const int stride = kWarps * a.cluster;
    int step = rank * kWarps + warp;
    auto fetch_token = [&](int st) -> int64_t {
        const int j = st * kTile + (lane & 15);
        return j < n ? (int64_t)__ldg(ir + j) : (int64_t)-1 - INT32_MAX - 1;   // below every int32: no token
    };
    constexpr int64_t kNoToken = (int64_t)-1 - INT32_MAX - 1;
    struct Where { uint32_t row; float ks, vs; };
    auto look_up = [&](int64_t tok) -> Where {
        Where w{kNoRow, 1.f, 1.f};
        if (tok == kNoToken) return w;
        const int pid = cache_page(c, b, tok);
        if (pid < 0) {
            latch(a.err, kErrDevice);
            return w;
        }
        w.row = (uint32_t)cache_row(c, pid, h, tok);
        if (E4) {
            w.ks = __ldg(c.K_scale + (int64_t)pid * c.hkv + h);
            w.vs = __ldg(c.V_scale + (int64_t)pid * c.hkv + h);
        }
        return w;
    };
    const uint4* Kp = static_cast<const uint4*>(c.K);
    const uint32_t* Vp = static_cast<const uint32_t*>(c.V);

    int64_t tok = fetch_token(step);
    Where cur = look_up(tok);
    tok = fetch_token(step + stride);
    for (; step < steps_all; step += stride) {
        // K rows of tokens g and g + 8, V rows of tokens 2t, 2t + 1, 2t + 8, 2t + 9
        uint32_t kr[2][KW], vr[4][VW];
        bool valid[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const uint32_t r = __shfl_sync(0xffffffffu, cur.row, g + 8 * e);
            valid[e] = r != kNoRow;
#pragma unroll
            for (int i = 0; i < KW / 4; ++i) {
                uint4 v = make_uint4(0, 0, 0, 0);
                if (valid[e]) v = __ldg(Kp + (int64_t)r * (KW) + t + 4 * i);
                kr[e][4 * i] = v.x; kr[e][4 * i + 1] = v.y; kr[e][4 * i + 2] = v.z; kr[e][4 * i + 3] = v.w;
            }
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const uint32_t r = __shfl_sync(0xffffffffu, cur.row, 2 * t + (e & 1) + 8 * (e >> 1));
            const uint32_t* p = Vp + (int64_t)r * (8 * VW) + g * VW;
            if constexpr (VW == 2) {
                uint2 v = make_uint2(0, 0);
                if (r != kNoRow) v = __ldg(reinterpret_cast<const uint2*>(p));
                vr[e][0] = v.x; vr[e][1] = v.y;
            } else {
#pragma unroll
                for (int i = 0; i < VW / 4; ++i) {
                    uint4 v = make_uint4(0, 0, 0, 0);
                    if (r != kNoRow) v = __ldg(reinterpret_cast<const uint4*>(p) + i);
                    vr[e][4 * i] = v.x; vr[e][4 * i + 1] = v.y; vr[e][4 * i + 2] = v.z; vr[e][4 * i + 3] = v.w;
                }
            }
        }
        float ks[2] = {1.f, 1.f}, lv[2] = {0.f, 0.f}, iv[2] = {1.f, 1.f};
        if (E4) {
            const float lg = log2f(cur.vs), inv = __frcp_rn(cur.vs);   // both exact for powers of two
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                ks[e] = __shfl_sync(0xffffffffu, cur.ks, g + 8 * e);
                lv[e] = __shfl_sync(0xffffffffu, lg, g + 8 * e);
                iv[e] = __shfl_sync(0xffffffffu, inv, g + 8 * e);
            }
        }
        cur = look_up(tok);
        tok = fetch_token(step + 2 * stride);

        // ---- scores: 16 tokens x 8 NT heads
        float x[NT][4];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) x[nt][e] = 0.f;
#pragma unroll
        for (int s = 0; s < KS; ++s) {
            uint32_t ka[4];
            if constexpr (E4) {
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    ka[e] = e4m3x2_to_f16x2((uint16_t)kr[e][s]);
                    ka[2 + e] = e4m3x2_to_f16x2((uint16_t)(kr[e][s] >> 16));
                }
            } else {
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    ka[e] = kr[e][2 * s];
                    ka[2 + e] = kr[e][2 * s + 1];
                }
            }
#pragma unroll
            for (int p = 0; p < PQ; ++p)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) mma<E4>(x[nt], ka, qf[p][s][nt]);
        }
        bool higher = false;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float y = fmaf(x[nt][e], ks[e >> 1] * qs[nt][e & 1], lv[e >> 1]);
                x[nt][e] = valid[e >> 1] ? y : -INFINITY;
                higher |= x[nt][e] > m[nt][e & 1] + kLazy;
            }
        if (__any_sync(0xffffffffu, higher)) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float top = fmaxf(x[nt][e], x[nt][e + 2]);
                    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 4));
                    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 8));
                    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 16));
                    top = fmaxf(top, m[nt][e]);
                    const float f = top == -INFINITY ? 1.f : ex2(m[nt][e] - top);
                    m[nt][e] = top;
                    l[nt][e] *= f;
#pragma unroll
                    for (int i = 0; i < KS; ++i) {
                        o[i][nt][e] *= f;
                        o[i][nt][e + 2] *= f;
                    }
                }
        }
        // ---- weights: B fragments of P^T
        uint32_t pb[PP][NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            float w[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float ref = m[nt][e & 1];
                w[e] = ex2(x[nt][e] - (ref == -INFINITY ? 0.f : ref - kHeadroom));
                l[nt][e & 1] = fmaf(w[e], iv[e >> 1], l[nt][e & 1]);
            }
            uint32_t lo[PP], hi[PP];
            split<E4, PP>(w[0], w[1], lo);
            split<E4, PP>(w[2], w[3], hi);
#pragma unroll
            for (int p = 0; p < PP; ++p) {
                pb[p][nt][0] = movmatrix_t(lo[p]);
                pb[p][nt][1] = movmatrix_t(hi[p]);
            }
        }
        // ---- acc: rows g and g + 8 of m tile i are components (D/8) g + 2 i and the next
#pragma unroll
        for (int i = 0; i < KS; ++i) {
            uint32_t va[4];
#pragma unroll
            for (int e = 0; e < 2; ++e) {       // tokens 2t, 2t + 1, then 2t + 8, 2t + 9
                if constexpr (E4) {
                    const uint32_t two = __byte_perm(vr[2 * e][i / 2], vr[2 * e + 1][i / 2], i % 2 ? 0x7362 : 0x5140);
                    va[2 * e] = e4m3x2_to_f16x2((uint16_t)two);
                    va[2 * e + 1] = e4m3x2_to_f16x2((uint16_t)(two >> 16));
                } else {
                    va[2 * e] = __byte_perm(vr[2 * e][i], vr[2 * e + 1][i], 0x5410);
                    va[2 * e + 1] = __byte_perm(vr[2 * e][i], vr[2 * e + 1][i], 0x7632);
                }
            }
#pragma unroll
            for (int p = 0; p < PP; ++p)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) mma<E4>(o[i][nt], va, pb[p][nt]);
        }
    }

    // ---- merge the warps
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            float s = l[nt][e];
            s += __shfl_xor_sync(0xffffffffu, s, 4);
            s += __shfl_xor_sync(0xffffffffu, s, 8);
            s += __shfl_xor_sync(0xffffffffu, s, 16);
            if (g == 0) {
                m_s[warp][8 * nt + 2 * t + e] = m[nt][e];
                l_s[warp][8 * nt + 2 * t + e] = s;
            }
        }
    __syncthreads();
    for (int w = 0; w < kWarps; ++w) {
        if (warp == w) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int head = 8 * nt + 2 * t + e;
                    float M = m_s[0][head];
#pragma unroll
                    for (int i = 1; i < kWarps; ++i) M = fmaxf(M, m_s[i][head]);
                    const float f = M == -INFINITY ? 0.f : ex2(m[nt][e] - M);
#pragma unroll
                    for (int i = 0; i < KS; ++i) {
                        // components (D/8) g + 2 i and the next, at the places [i][g]
                        float2* p = reinterpret_cast<float2*>(acc_s + head * LD + 16 * i + 2 * g);
                        float2 s = make_float2(f * o[i][nt][e], f * o[i][nt][e + 2]);
                        if (w > 0) {
                            const float2 old = *p;
                            s.x += old.x;
                            s.y += old.y;
                        }
                        *p = s;
                    }
                }
        }
        __syncthreads();
    }
    if (tid < HG) {
        float M = m_s[0][tid], L = 0.f;
#pragma unroll
        for (int i = 1; i < kWarps; ++i) M = fmaxf(M, m_s[i][tid]);
#pragma unroll
        for (int i = 0; i < kWarps; ++i) L += (M == -INFINITY ? 0.f : ex2(m_s[i][tid] - M)) * l_s[i][tid];
        mc_s[tid] = M;
        lc_s[tid] = L;
    }
    // ---- merge the cluster: every CTA reads all of them and writes a share of the outputs
    cg::cluster_group cluster = cg::this_cluster();
    if (a.cluster > 1) cluster.sync();
    else __syncthreads();
    if (tid < HG) {
        float M = -INFINITY, L = 0.f;
        for (int i = 0; i < a.cluster; ++i) M = fmaxf(M, cluster.map_shared_rank(mc_s, i)[tid]);
        for (int i = 0; i < a.cluster; ++i) {
            const float f = M == -INFINITY ? 0.f : ex2(cluster.map_shared_rank(mc_s, i)[tid] - M);
            f_s[i][tid] = f;
            L += f * cluster.map_shared_rank(lc_s, i)[tid];
        }
        mt_s[tid] = M;
        lt_s[tid] = L;
    }
    __syncthreads();
    for (int e = rank * kThreads + tid; e < gn * D; e += a.cluster * kThreads) {
        const int head = e / D, d = e % D;
        const int at = head * LD + 16 * ((d % (D / 8)) / 2) + 2 * (d / (D / 8)) + (d & 1);
        float s = 0.f;
        for (int i = 0; i < a.cluster; ++i) s += f_s[i][head] * cluster.map_shared_rank(acc_s, i)[at];
        const float L = lt_s[head];
        put(static_cast<T*>(a.O) + q0 + e, L == 0.f ? 0.f : s / L);
    }
    if (a.lse && rank == 0 && tid < gn) {
        const float L = lt_s[tid];
        a.lse[q0 / D + tid] = L == 0.f ? -INFINITY : (mt_s[tid] - kHeadroom + log2f(L)) * 0.69314718055994531f;
    }
    if (a.cluster > 1) cluster.sync();
}

template <int D, typename CT, typename T, int NT>
int launch(AttnArgs a, int64_t rows, cudaStream_t s) {
    a.groups = (a.G + 8 * NT - 1) / (8 * NT);
    const int64_t units = rows * a.groups;
    // few rows: a cluster of CTAs shares each, as long as its warps have two steps
    const int steps = (a.max_sel + kTile - 1) / kTile;
    a.cluster = 1;
    while (a.cluster < kMaxCluster && units * a.cluster < 2 * 148 && a.cluster * 2 * kWarps * 2 <= steps) a.cluster *= 2;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(units * a.cluster));
    cfg.blockDim = dim3(kThreads);
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = a.cluster;
    at[0].val.clusterDim.y = 1;
    at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    note_launch();
    return cuda_status(cudaLaunchKernelEx(&cfg, cache_attn_kernel<D, CT, T, NT>, a));
}

template <int D, typename CT>
int launch_io(const AttnArgs& a, int dtype, int64_t rows, cudaStream_t s) {
    // fp32 queries take several parts of each fragment: 8 heads at a time keeps them in registers
    if (dtype == LSA_F32) return launch<D, CT, float, 1>(a, rows, s);
    return a.G <= 8 ? launch<D, CT, __nv_bfloat16, 1>(a, rows, s) : launch<D, CT, __nv_bfloat16, 2>(a, rows, s);
}

}  // namespace

int launch_cache_attn(const lsa_kv_cache& cache, const void* Q, const int32_t* idx, const int32_t* cnt, int64_t nq,
                      int hq, int dtype, int max_sel, void* O, float* lse, int32_t* err, cudaStream_t s) {
    AttnArgs a{cache_args(cache), Q, idx, cnt, O, lse, nq, hq, hq / cache.hkv, max_sel};
    a.scale_log2 = 1.4426950408889634f / sqrtf((float)cache.d);
    a.err = err;
    const int64_t rows = cache.batch * nq * cache.hkv;
    if (cache.d == 128)
        return cache.dtype == LSA_E4M3 ? launch_io<128, uint8_t>(a, dtype, rows, s)
                                       : launch_io<128, __nv_bfloat16>(a, dtype, rows, s);
    return cache.dtype == LSA_E4M3 ? launch_io<64, uint8_t>(a, dtype, rows, s)
                                   : launch_io<64, __nv_bfloat16>(a, dtype, rows, s);
}

}  // namespace lsa
