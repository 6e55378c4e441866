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
// What bounds it.  The rows are scattered (whole rows of 64 to 256 bytes, pages
// anywhere), each is used by the 4 to 16 heads of its group only, and a round of
// gathers takes 1 to 1.7 us on this GPU even from L2: the rate is what is in
// flight, so every warp keeps a step's rows (32 tokens, 8 KB) on their way to
// shared memory by cp.async while it works on the step before, and looks the
// rows of later steps up (token, page, scales) one load a step.  With that,
// decode is bound by HBM (96 sequences, 32 heads of 128 over 4 KV heads, 2,624
// rows of 8 bits: 47-54 us, 4.9-5.6 TB/s) and long chunks by instructions: the
// conversion of the codes, two a cvt, on half the lanes of the ALU (2,048
// queries x 16 heads, 3,136 rows: 379 us, 8.7 TB/s of rows, 139 TFLOP/s).
//
// A warp takes 16 tokens at a time on the M side of mma.sync m16n8k16 (keys x
// heads, then components x heads), so 8 heads fill a tile without padding; the
// 128 rows of a tcgen05 tile would have 8 heads to share them with.  The sums
// over d and over tokens do not depend on their order: a K fragment is whole
// 16-byte pieces of a row, with the queries laid out to match, a V fragment one
// transposed load, with the K rows' order to match.  8-bit codes become fp16
// exactly; queries are scaled by a power of two per head so that bf16 values are
// fp16 values too.  fp32 queries and weights go as two fp16 parts (three bf16
// parts next to bf16 pages), so fp32 results keep fp32's accuracy.
//
// The warps of a CTA, and the CTAs of a cluster, take every n-th step of one
// row; their (m, l, acc) are merged in shared and distributed shared memory in
// a fixed order.
#include <cooperative_groups.h>

#include <atomic>
#include <type_traits>

#include "ask_once.cuh"
#include "cache_common.cuh"
#include "warp_mma.cuh"

namespace lsa {
namespace {

namespace cg = cooperative_groups;

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kMaxCluster = 16;
// Weights are at most 2^(kHeadroom + kLazy) and the largest at least 2^kHeadroom:
// the maximum is renewed only when a score passes it by 2^kLazy.  Two fp16 parts
// keep 22 bits of a weight down to 2^-3 and nothing below 2^-25, 2^-32 of the largest.
constexpr float kLazy = 8.f, kHeadroom = 7.f;
// The weights hold the V scale, and a component of O may come from pages of small
// scales alone.  Steps with a scale 2^kScales below the largest so far take their
// weights by size, those within a factor of 2^kClass at a time, which keeps 22 bits of
// all that fp32 can hold; so a weight loses no more than 2^-(32 - kScales) of the largest
// softmax weight.  The look at the scales and the factors in two parts took the long
// chunk from 368 to 377 us, 4 sequences from 9.2 to 9.9.
constexpr int kScales = 4;
constexpr float kClass = 14.f;

struct AttnArgs {
    CacheArgs c;
    const void* Q;
    const int32_t* idx;
    const int32_t* cnt;
    void* O;
    float* lse;
    int64_t nq;
    int hq, G, max_sel, groups;
    uint32_t units;        // (row, group of heads)
    int warps, cluster;    // warps of a CTA that share a unit (1 or kWarps), CTAs that do
    float scale_log2;
    int32_t* err;
};

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// log2 of a positive normal number, exact for powers of two
__device__ __forceinline__ float log2_of(float x) {
    float y;
    const int bits = __float_as_int(x);
    asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(__int_as_float((bits & 0x7fffff) | 0x3f800000)));
    return (float)((bits >> 23) - 127) + y;
}
__device__ __forceinline__ float4 load4(const __nv_bfloat16* p) {
    const uint2 v = *reinterpret_cast<const uint2*>(p);
    return make_float4(__uint_as_float(v.x << 16), __uint_as_float(v.x & 0xffff0000u), __uint_as_float(v.y << 16),
                       __uint_as_float(v.y & 0xffff0000u));
}
__device__ __forceinline__ float4 load4(const float* p) { return *reinterpret_cast<const float4*>(p); }

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

// c = a b, the first product of a chain
template <bool F16>
__device__ __forceinline__ void mma_first(float* c, const uint32_t* a, const uint32_t* b) {
    if constexpr (F16)
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
            "{%10,%10,%10,%10};\n"
            : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]), "f"(0.f));
    else
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
            "{%10,%10,%10,%10};\n"
            : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]), "f"(0.f));
}

template <bool F16>
__device__ __forceinline__ void mma(float* c, const uint32_t* a, const uint32_t* b) {
    if constexpr (F16) mma_f16(c, a, b[0], b[1]);
    else mma_bf16(c, a, b[0], b[1]);
}

// Byte offset of 16-byte piece `i` of row r in a tile of rows of ROWB bytes:
// permuted so that neither a warp's K loads (8 rows, 4 neighbouring pieces) nor
// its V loads (one piece of 8 rows) meet in a bank.
template <int ROWB>
__device__ __forceinline__ int piece_at(int r, int i) {
    if constexpr (ROWB == 64) {
        const int line = r >> 1;
        return line * 128 + ((((r & 1) * 4 + i) ^ (line & 3)) << 4);
    } else {
        const int s = ((r & 1) << 2) | ((r >> 1) & 3);
        return r * ROWB + (((i & ~7) | ((i & 7) ^ s)) << 4);
    }
}

__device__ __forceinline__ void load_shared(uint32_t p, uint32_t* w) {
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                 : "r"(p)
                 : "memory");
}
// Two 16 x 16 byte matrices, transposed (lanes 0-15 and 16-31 hold the addresses
// of their rows): bytes 4t .. 4t + 3 of w[0] are rows 4t .. 4t + 3 of column g of
// the first, w[1] its column g + 8, w[2] and w[3] the second (lane = 4 g + t).
__device__ __forceinline__ void load_transposed(uint32_t p, uint32_t* w) {
    asm volatile("ldmatrix.sync.aligned.m16n16.x2.trans.shared.b8 {%0, %1, %2, %3}, [%4];"
                 : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                 : "r"(p)
                 : "memory");
}

// piece_at(i * 32 / PIECES + r, p) = (piece_at(r, p) ^ step_swizzle(i)) + i * (32 / PIECES) * ROWB
template <int ROWB>
__device__ __forceinline__ constexpr uint32_t step_swizzle(int i) {
    return ROWB == 64 ? 0u : ROWB == 128 ? (i & 1) << 5 : (i & 3) << 4;
}

__device__ __forceinline__ void put2(float* p, float x, float y) { *reinterpret_cast<float2*>(p) = make_float2(x, y); }
__device__ __forceinline__ void put2(__nv_bfloat16* p, float x, float y) {
    *reinterpret_cast<__nv_bfloat162*>(p) = __floats2bfloat162_rn(x, y);
}

// CTAs per SM that the registers are cut to
template <int D, typename CT, typename T, int NT>
constexpr int min_ctas() {
    if (sizeof(T) == 4) return 2;
    return NT == 2 ? (D == 64 ? 3 : 2) : (D * sizeof(CT) == 64 ? 4 : 3);
}

// Tiles of 16 tokens of a warp's step.  Two steps are in shared memory: 8 KB of
// rows each (4 KB of 64-byte rows).  For 128-byte rows one tile a step and the 16
// warps an SM that then fit were slower: the long chunk above, with weights of one
// part, 365 us with two steps in shared memory and 375 with three, against 311 (two
// tiles side by side hide each other's latencies); 96 sequences 48.7 and 47.5
// against 49.6.
template <int D, typename CT>
constexpr int tiles_per_step() { return D * sizeof(CT) <= 128 ? 2 : 1; }

// EXACT: acc is added up outside the tensor cores (always for fp32 results)
template <int D, typename CT, typename T, int NT, bool EXACT>
__global__ __launch_bounds__(kThreads, (min_ctas<D, CT, T, NT>())) void cache_attn_kernel(const AttnArgs a) {
    constexpr bool E4 = sizeof(CT) == 1;              // 8-bit codes, fp16 products; else bf16
    constexpr bool F32 = sizeof(T) == 4;
    static_assert(EXACT || !F32, "fp32 results");
    constexpr int PQ = F32 ? (E4 ? 2 : 3) : 1;        // 16-bit parts of a query component
    // And of a weight: two fp16 parts carry 22 bits (with one part, 11 bits, the long chunk above took 311 us against
    // 356, and its O was 4.8e-4 of its norm from that of fp32 weights, now 7e-5; bf16 rounds it by 1.6e-3), two bf16
    // parts 16, 2^-8 of what the rounding of bf16 results takes, three 24.
    constexpr int PP = F32 && !E4 ? 3 : 2;
    // The tensor cores cut a running sum off at 24 bits without rounding.  Sums over
    // d and, where EXACT, acc over the steps of a row are therefore kept outside, by
    // rounded additions (fp32: with sums in the tensor cores 7.7e-7 off the exact result on
    // the median, 4.9e-7 so; of rows of 2,000 to 3,000 up to 9e-6; bf16, the long chunk:
    // scores outside halve the error of lse to 6.6e-8, 368 us against 356; acc, too, 394).
    // Without EXACT acc is cut off four times a step (two of 16 tokens), each time by
    // less than 2^-23 of it: by 2^-15 at most over the steps that launch allows.
    constexpr int KS = D / 16;                        // k steps of K Q^T, m tiles of V^T P^T
    constexpr int MV = E4 ? 2 : 1;                    // m tiles of a V load
    constexpr int HG = 8 * NT;                        // heads of a warp
    constexpr int ROWB = D * (int)sizeof(CT);         // bytes of a row
    constexpr int KW = ROWB / 16;                     // words of a K row in a thread (4 threads a row)
    constexpr int PIECES = ROWB / 16;
    constexpr int TILE = 16 * ROWB;                   // bytes of 16 rows
    constexpr int TPS = tiles_per_step<D, CT>();
    constexpr int STEP = 16 * TPS;                    // tokens of a warp's step
    constexpr int BUFFER = TPS * 2 * TILE;            // bytes of a step: (K tile, V tile) TPS times
    constexpr int LD = D + 4;                         // row stride of the merge buffers
    static_assert(HG * LD * 4 <= 2 * BUFFER, "a warp's sums go where its rows were");
    extern __shared__ __align__(128) unsigned char ring_s[];   // [kWarps][2][BUFFER]; at the end [HG][LD] of a warp
    __shared__ float m_s[kWarps][HG], l_s[kWarps][HG];
    // what the CTAs of a cluster send: a share of the sums, and all maxima and sums of weights
    __shared__ float2 sum_r[HG * D / 2];
    __shared__ float m_r[kMaxCluster][HG], l_r[kMaxCluster][HG];

    const CacheArgs& c = a.c;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int g = lane >> 2, t = lane & 3;
    // Rows g and g + 8 of a K tile are tokens krow and krow + KROW of its 16: the order in which the transposed loads
    // of V rows bring the tokens (8-bit: 4t, 4t + 1, then 4t + 2, 4t + 3; bf16: 2t, 2t + 1, then 2t + 8, 2t + 9)
    constexpr int KROW = E4 ? 2 : 8;
    const int krow = E4 ? 4 * (g >> 1) + (g & 1) : g;
    const int rank = blockIdx.x % a.cluster;
    if (a.cluster > 1) asm volatile("barrier.cluster.arrive.relaxed.aligned;");   // all have started: waited for below
    const bool alone = a.warps == 1;                  // a warp takes a whole row
    const uint32_t unit = alone ? blockIdx.x * kWarps + warp : blockIdx.x / a.cluster;
    if (unit >= a.units) return;                      // only in the last CTA of whole-row warps
    const int grp = unit % a.groups;
    const uint32_t row = unit / a.groups;             // (b * nq + qi) * hkv + h
    const int h = row % c.hkv;
    const uint32_t bq = row / c.hkv;
    const uint32_t b = bq / (uint32_t)a.nq;
    const int g0 = grp * HG, gn = min(HG, a.G - g0);
    const int64_t q0 = ((int64_t)bq * a.hq + h * a.G + g0) * D;

    // ---- tokens: lane j looks up token j of the warp's step
    const int32_t* ir = a.idx + (int64_t)row * a.max_sel;
    const int32_t* table = c.table + (int64_t)b * c.ld_pages;
    const int stride = alone ? 1 : kWarps * a.cluster;
    int step = alone ? 0 : rank * kWarps + warp;
    // the first tokens are read with the row's length, not after it
    auto fetch_token = [&](int st, int end) -> int {  // -1 past the row's end
        const int j = st * STEP + lane;
        return (STEP == 32 || lane < STEP) && j < end ? __ldg(ir + j) : -1;
    };
    int n = __ldg(a.cnt + row);
    int tok = fetch_token(step, a.max_sel), tok1 = fetch_token(step + stride, a.max_sel);
    // and the queries before anything waits
    float4 qv[NT][KS];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        const T* q = static_cast<const T*>(a.Q) + q0 + (int64_t)(8 * nt + g) * D;
#pragma unroll
        for (int s = 0; s < KS; ++s) {
            // the 4 components of k step s in this thread: one word of codes, two of bf16
            const int w = E4 ? s : 2 * s;
            const int d0 = (64 * (w / 4) + 16 * t + 4 * (w % 4)) / (int)sizeof(CT);
            qv[nt][s] = 8 * nt + g < gn ? load4(q + d0) : make_float4(0.f, 0.f, 0.f, 0.f);
        }
    }
    if (n < 0 || n > a.max_sel) {
        if (lane == 0) latch(a.err, kErrDevice);      // every warp: it may have a row of its own
        n = n < 0 ? 0 : a.max_sel;
    }
    const int steps = (n + STEP - 1) / STEP;
    // Three loads follow one another for a row: the token, its page, the row and
    // its scales.  They are taken one step apart, so that none is waited for:
    // tokens are fetched three steps ahead, pages two, rows and scales one.
    struct Where {
        uint32_t row;       // of the pools; 0 where there is no token
        uint32_t ok;        // lanes that have one
        float ks, vs;
    };
    auto fetch_page = [&](int tok) -> int {
        const int col = tok >> c.log2_page;           // negative for a negative token
        return (uint32_t)col < (uint32_t)c.ld_pages ? __ldg(table + col) : -1;
    };
    auto locate = [&](int st, int tok, int pid) -> Where {
        Where w{0u, 0u, 1.f, 1.f};
        const bool is = (STEP == 32 || lane < STEP) && st * STEP + lane < n;
        const bool ok = is && (uint32_t)pid < (uint32_t)c.n_pages;
        w.ok = __ballot_sync(0xffffffffu, ok);
        if (ok) {
            const uint32_t ph = (uint32_t)pid * c.hkv + h;
            w.row = (ph << c.log2_page) + (tok & (c.page - 1));
            if (E4) {
                w.ks = __ldg(c.K_scale + ph);
                w.vs = __ldg(c.V_scale + ph);
            }
        } else if (is) {
            latch(a.err, kErrDevice);
        }
        return w;
    };

    // ---- gathered rows: a step's K and V rows to the warp's shared memory, 16
    // bytes a lane and copy; zeros where there is no token
    const uint32_t ring = smem_u32(ring_s) + warp * 2 * BUFFER;
    const unsigned char* Kc = static_cast<const unsigned char*>(c.K) + 16 * (lane % PIECES);
    const unsigned char* Vc = static_cast<const unsigned char*>(c.V) + 16 * (lane % PIECES);
    const uint32_t lane_at = piece_at<ROWB>(lane / PIECES, lane % PIECES);
    auto gather = [&](const Where& w, int half, uint32_t buffer) {
        constexpr int RP = 32 / PIECES;               // rows of a copy
        if ((w.ok >> (16 * half) & 0xffffu) == 0xffffu) {
#pragma unroll
            for (int i = 0; i < 16 / RP; ++i) {
                const uint32_t at = __shfl_sync(0xffffffffu, w.row, 16 * half + i * RP + lane / PIECES);
                const uint32_t dst = buffer + (lane_at ^ step_swizzle<ROWB>(i)) + (half * 2 * TILE + i * RP * ROWB);
                cp_async16(dst, Kc + (uint64_t)at * ROWB);
                cp_async16(dst + TILE, Vc + (uint64_t)at * ROWB);
            }
        } else {
#pragma unroll
            for (int i = 0; i < 16 / RP; ++i) {
                const int j = 16 * half + i * RP + lane / PIECES;
                const uint32_t at = __shfl_sync(0xffffffffu, w.row, j);
                const uint32_t dst = buffer + (lane_at ^ step_swizzle<ROWB>(i)) + (half * 2 * TILE + i * RP * ROWB);
                const int bytes = w.ok >> j & 1u ? 16 : 0;
                cp_async16(dst, Kc + (uint64_t)at * ROWB, bytes);
                cp_async16(dst + TILE, Vc + (uint64_t)at * ROWB, bytes);
            }
        }
    };
    int pid = fetch_page(tok1);
    Where cur = locate(step, tok, fetch_page(tok));
#pragma unroll
    for (int half = 0; half < TPS; ++half) {
        if (step < steps) gather(cur, half, ring);
        cp_async_commit();
    }
    int tok2 = fetch_token(step + 2 * stride, n);

    // ---- queries: B fragments, k slots in the order the K pieces come in
    uint32_t qf[PQ][KS][NT][2];
    float qs[NT][2];                                  // factor of the scores of heads 8 nt + 2 t, + 1
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        const float4* v = qv[nt];
        float top = 0.f;
#pragma unroll
        for (int s = 0; s < KS; ++s)
            top = fmaxf(top, fmaxf(fmaxf(fabsf(v[s].x), fabsf(v[s].y)), fmaxf(fabsf(v[s].z), fabsf(v[s].w))));
        float up = 1.f, down = 1.f;
        if (E4) {
            // largest component to [2^14, 2^15): fp16's subnormals begin 2^-28 below it
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
            const int e = min(100, 14 - ((__float_as_int(top) >> 23) - 127));    // -114 for an infinity
            up = __int_as_float((127 + e) << 23);
            down = __int_as_float((127 - e) << 23);
        }
#pragma unroll
        for (int s = 0; s < KS; ++s) {
            uint32_t lo[PQ], hi[PQ];
            split<E4, PQ>(v[s].x * up, v[s].y * up, lo);
            split<E4, PQ>(v[s].z * up, v[s].w * up, hi);
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
    // m: reference of a head's exponents, its largest so far less kHeadroom; unset: no score yet above -inf
    float m[NT][2], l[NT][2];
    int most = 0;                                     // largest V scale so far, its exponent field
    bool unset[NT][2], any_unset = true;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int e = 0; e < 2; ++e) { m[nt][e] = 0.f; l[nt][e] = 0.f; unset[nt][e] = true; }
#pragma unroll
        for (int i = 0; i < KS; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[i][nt][e] = 0.f;
    }

    // shared addresses: K pieces t and t + 4 of rows krow and krow + KROW (they differ in bits that the permutation
    // of piece_at changes), and this lane's rows of the V tile's transposed loads
    uint32_t kp[2][2], vp[ROWB / 32 > 4 ? 4 : ROWB / 32];
#pragma unroll
    for (int e = 0; e < 2; ++e)
#pragma unroll
        for (int i = 0; i < 2; ++i)
            kp[e][i] = ring + piece_at<ROWB>(krow + KROW * e, t + (PIECES < 8 ? 0 : 4 * i));
    const int vrow = E4 ? lane & 15 : (lane & 7) + 8 * (lane >> 4);
#pragma unroll
    for (int i = 0; i < (int)(sizeof(vp) / 4); ++i)
        vp[i] = ring + TILE + piece_at<ROWB>(vrow, 2 * i + (E4 ? lane >> 4 : lane >> 3 & 1));
    uint32_t ahead = ring + BUFFER;
    int32_t flip = BUFFER;
    for (; step < steps; step += stride) {
        // the next step's rows into the buffer that the last one left
        const Where next = locate(step + stride, tok1, pid);
        tok1 = tok2;
        pid = fetch_page(tok1);
        tok2 = fetch_token(step + 3 * stride, n);
#pragma unroll
        for (int half = 0; half < TPS; ++half) {
            if (step + stride < steps) gather(next, half, ahead);
            cp_async_commit();
        }
        const float lg = E4 ? log2_of(cur.vs) : 0.f, inv = E4 ? ex2(-lg) : 1.f;
        cp_async_wait<TPS>();
        __syncwarp();
        // ---- scores: STEP tokens x 8 NT heads, even and odd k steps apart for shorter chains
        float y[TPS][NT][4];
#pragma unroll
        for (int half = 0; half < TPS; ++half) {
            uint32_t kr[2][KW];
#pragma unroll
            for (int e = 0; e < 2; ++e)
#pragma unroll
                for (int i = 0; i < KW / 4; ++i)
                    load_shared(kp[e][i & 1] + (half * 2 * TILE + 128 * (i / 2)), kr[e] + 4 * i);
            float z[NT][4];
#pragma unroll
            for (int s = 0; s < KS; ++s) {
                uint32_t ka[4];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    if constexpr (E4) {
                        e4m3x4_to_f16x4(kr[e][s], ka[e], ka[2 + e]);
                    } else {
                        ka[e] = kr[e][2 * s];
                        ka[2 + e] = kr[e][2 * s + 1];
                    }
                }
#pragma unroll
                for (int p = 0; p < PQ; ++p)
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        float* acc = (s & 1) ? z[nt] : y[half][nt];
                        if (s < 2 && p == 0) mma_first<E4>(acc, ka, qf[p][s][nt]);
                        else {
                            float sum[4];
                            mma_first<E4>(sum, ka, qf[p][s][nt]);
#pragma unroll
                            for (int e = 0; e < 4; ++e) acc[e] += sum[e];
                        }
                    }
            }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 4; ++e) y[half][nt][e] += z[nt][e];
        }

        // ---- base-2 exponents of the weights
        float iv[TPS][2];
        float top = -INFINITY;
#pragma unroll
        for (int half = 0; half < TPS; ++half)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float ks = 1.f, lv = 0.f;
                iv[half][e] = 1.f;
                if (E4) {
                    ks = __shfl_sync(0xffffffffu, cur.ks, 16 * half + krow + KROW * e);
                    lv = __shfl_sync(0xffffffffu, lg, 16 * half + krow + KROW * e);
                    iv[half][e] = __shfl_sync(0xffffffffu, inv, 16 * half + krow + KROW * e);
                }
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        float& v = y[half][nt][2 * e + i];
                        // ks first: v * ks stays in range, ks * qs may not
                        v = fmaf(v * ks, qs[nt][i], lv - m[nt][i]);
                        top = fmaxf(top, v);
                    }
            }
        constexpr uint32_t kFull = STEP == 32 ? 0xffffffffu : 0xffffu;
        if (cur.ok != kFull) {         // past the row's end, or a token that was refused
#pragma unroll
            for (int half = 0; half < TPS; ++half)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (!(cur.ok >> (16 * half + krow + KROW * (e >> 1)) & 1u)) y[half][nt][e] = -INFINITY;
            top = INFINITY;            // maxima of what is left
        }
        if (__any_sync(0xffffffffu, top > kHeadroom + kLazy || any_unset)) {
            // new references: 2^kHeadroom for the largest weight so far
            any_unset = false;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float up = -INFINITY;
#pragma unroll
                    for (int half = 0; half < TPS; ++half) up = fmaxf(up, fmaxf(y[half][nt][e], y[half][nt][e + 2]));
                    up = fmaxf(up, __shfl_xor_sync(0xffffffffu, up, 4));
                    up = fmaxf(up, __shfl_xor_sync(0xffffffffu, up, 8));
                    up = fmaxf(up, __shfl_xor_sync(0xffffffffu, up, 16)) - kHeadroom;
                    const bool first = unset[nt][e];
                    unset[nt][e] = first && up == -INFINITY;
                    any_unset |= unset[nt][e];
                    if (first ? up == -INFINITY : !(up > 0.f)) up = 0.f;
                    // the root of the factor, for two products: it may be below what fp32 can hold when l and o are not
                    const float f = first ? 1.f : ex2(-0.5f * up);
                    m[nt][e] += up;
                    l[nt][e] = l[nt][e] * f * f;
#pragma unroll
                    for (int half = 0; half < TPS; ++half) {
                        y[half][nt][e] -= up;
                        y[half][nt][e + 2] -= up;
                    }
#pragma unroll
                    for (int i = 0; i < KS; ++i) {
                        o[i][nt][e] = o[i][nt][e] * f * f;
                        o[i][nt][e + 2] = o[i][nt][e + 2] * f * f;
                    }
                }
        }
        // ---- weights: B fragments of P^T
        uint32_t pb[TPS][PP][NT][2];
        auto put_weights = [&](int half, int nt, const float* w) {
            uint32_t lo[PP], hi[PP];
            split<E4, PP>(w[0], w[1], lo);
            split<E4, PP>(w[2], w[3], hi);
#pragma unroll
            for (int p = 0; p < PP; ++p) {
                pb[half][p][nt][0] = movmatrix_t(lo[p]);
                pb[half][p][nt][1] = movmatrix_t(hi[p]);
            }
        };
        // ---- acc: rows g and g + 8 of m tile i are components 16 i + g and 16 i + g + 8; OUTSIDE: the step's products
        // are summed first and added `times` over
        auto add_products = [&](auto outside, float times) {
            constexpr bool OUTSIDE = decltype(outside)::value;
#pragma unroll
            for (int i = 0; i < KS; i += MV) {
                float sum[MV][NT][4];
#pragma unroll
                for (int half = 0; half < TPS; ++half) {
                    uint32_t va[MV][4];
                    // 32 bytes of every row: of 256-byte rows the second 128 are a fixed distance on
                    constexpr int NV = (int)(sizeof(vp) / 4);
                    const int j = i / MV;
                    const uint32_t p = vp[j % NV] + (half * 2 * TILE + 128 * (j / NV));
                    if constexpr (E4) {
                        uint32_t w[4];
                        load_transposed(p, w);
#pragma unroll
                        for (int x = 0; x < MV; ++x) {
                            e4m3x4_to_f16x4(w[2 * x], va[x][0], va[x][2]);
                            e4m3x4_to_f16x4(w[2 * x + 1], va[x][1], va[x][3]);
                        }
                    } else {
                        ldsm_x4_t(p, va[0][0], va[0][1], va[0][2], va[0][3]);
                    }
#pragma unroll
                    for (int x = 0; x < MV; ++x)
#pragma unroll
                        for (int q = 0; q < PP; ++q)
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt) {
                                if constexpr (!OUTSIDE) mma<E4>(o[i + x][nt], va[x], pb[half][q][nt]);
                                else if (half == 0 && q == 0) mma_first<E4>(sum[x][nt], va[x], pb[half][q][nt]);
                                else mma<E4>(sum[x][nt], va[x], pb[half][q][nt]);
                            }
                }
                if constexpr (OUTSIDE)
#pragma unroll
                    for (int x = 0; x < MV; ++x)
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                            for (int e = 0; e < 4; ++e) o[i + x][nt][e] = fmaf(sum[x][nt][e], times, o[i + x][nt][e]);
            }
        };
        bool apart = false;
        if constexpr (E4) {
            const int field = cur.ok >> lane & 1u ? __float_as_int(cur.vs) >> 23 : most;
            if (__any_sync(0xffffffffu, (uint32_t)(most - field) > (uint32_t)kScales)) {
                most = max(most, __reduce_max_sync(0xffffffffu, field));
                apart = __any_sync(0xffffffffu, (cur.ok >> lane & 1u) && field < most - kScales);
            }
        }
        if (!apart) {
#pragma unroll
            for (int half = 0; half < TPS; ++half)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    float w[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        w[e] = ex2(y[half][nt][e]);
                        l[nt][e & 1] = fmaf(w[e], iv[half][e >> 1], l[nt][e & 1]);
                    }
                    put_weights(half, nt, w);
                }
            add_products(std::integral_constant<bool, EXACT>{}, 1.f);
        } else {
            float low = INFINITY;      // smallest exponent whose weight fp32 can hold
#pragma unroll
            for (int half = 0; half < TPS; ++half)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float lv = __shfl_sync(0xffffffffu, lg, 16 * half + krow + KROW * (e >> 1));
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        const float v = y[half][nt][e];
                        l[nt][e & 1] += ex2(v - lv);
                        if (v > -125.f) low = fminf(low, v);
                    }
                }
            // from `up` down to `up - kClass`, times 2^down; NaN with the first
            float up = kHeadroom + kLazy, down = 0.f;
            for (bool more = true; more; up -= kClass, down += kClass) {
#pragma unroll
                for (int half = 0; half < TPS; ++half)
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        float w[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const float v = y[half][nt][e];
                            const bool mine = down == 0.f ? !(v <= up - kClass) : v <= up && v > up - kClass;
                            w[e] = mine ? ex2(v + down) : 0.f;
                        }
                        put_weights(half, nt, w);
                    }
                add_products(std::true_type{}, ex2(-down));
                more = __any_sync(0xffffffffu, low <= up - kClass);
            }
        }
        __syncwarp();          // the buffer is free
        cur = next;
        ahead -= flip;
#pragma unroll
        for (int i = 0; i < 4; ++i) kp[i / 2][i % 2] += flip;
#pragma unroll
        for (int i = 0; i < (int)(sizeof(vp) / 4); ++i) vp[i] += flip;
        flip = -flip;
    }
    cp_async_wait<0>();

    // ---- every warp puts its sums where its rows were
    __syncwarp();
    float* mine = reinterpret_cast<float*>(ring_s + warp * 2 * BUFFER);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int head = 8 * nt + 2 * t + e;
            float s = l[nt][e];
            s += __shfl_xor_sync(0xffffffffu, s, 4);
            s += __shfl_xor_sync(0xffffffffu, s, 8);
            s += __shfl_xor_sync(0xffffffffu, s, 16);
            if (g == 0) {
                // a head whose every score is NaN stays unset: its l is NaN and reaches the output, unlike that of no token
                m_s[warp][head] = unset[nt][e] && s == 0.f ? -INFINITY : m[nt][e];
                l_s[warp][head] = s;
            }
#pragma unroll
            for (int i = 0; i < KS; ++i) {
                mine[head * LD + 16 * i + g] = o[i][nt][e];
                mine[head * LD + 16 * i + 8 + g] = o[i][nt][e + 2];
            }
        }
    if (alone) __syncwarp();
    else __syncthreads();
    // ---- merge the warps: a head's pairs are taken by as many threads as there are for it
    const int w0 = alone ? warp : 0, w1 = alone ? warp + 1 : kWarps;
    const int per_head = (alone ? 32 : kThreads) / HG, id = alone ? lane : tid;
    const int head = id / per_head;
    float M = -INFINITY, L = 0.f, f[kWarps];
    for (int w = w0; w < w1; ++w) M = fmaxf(M, m_s[w][head]);
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        f[w] = 0.f;
        if (w >= w0 && w < w1 && M != -INFINITY) {
            f[w] = ex2(0.5f * (m_s[w][head] - M));    // the root, as above
            L += f[w] * l_s[w][head] * f[w];
        }
    }
    const float* part = reinterpret_cast<const float*>(ring_s) + head * LD;
    T* out = static_cast<T*>(a.O) + q0;
    auto pair_sum = [&](int q) {
        float2 s = make_float2(0.f, 0.f);
#pragma unroll
        for (int w = 0; w < kWarps; ++w)
            if (w >= w0 && w < w1) {
                const float2 v = *reinterpret_cast<const float2*>(part + w * (2 * BUFFER / 4) + 2 * q);
                s.x += f[w] * v.x * f[w];
                s.y += f[w] * v.y * f[w];
            }
        return s;
    };
    if (a.cluster == 1) {
        if (head >= gn) return;
        for (int q = id % per_head; q < D / 2; q += per_head) {
            const float2 s = pair_sum(q);
            put2(out + head * D + 2 * q, L == 0.f ? 0.f : s.x / L, L == 0.f ? 0.f : s.y / L);
        }
        if (a.lse && id % per_head == 0)
            a.lse[q0 / D + head] = L == 0.f ? -INFINITY : (M + log2f(L)) * 0.69314718055994531f;
        return;
    }
    // ---- merge the cluster: CTA r writes share r of the outputs, the others send it theirs
    cg::cluster_group cluster = cg::this_cluster();
    const int share = HG * D / 2 / a.cluster;
    asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
    for (int q = id % per_head; q < D / 2; q += per_head) {
        const int e = head * (D / 2) + q;
        cluster.map_shared_rank(sum_r, e / share)[rank * share + e % share] = pair_sum(q);
    }
    if (id % per_head == 0)
        for (int r = 0; r < a.cluster; ++r) {
            cluster.map_shared_rank(&m_r[0][0], r)[rank * HG + head] = M;
            cluster.map_shared_rank(&l_r[0][0], r)[rank * HG + head] = L;
        }
    cluster.sync();
    for (int j = tid; j < share; j += kThreads) {
        const int e = rank * share + j, hd = e / (D / 2), q = e % (D / 2);
        if (hd >= gn) break;
        float top = -INFINITY, sum = 0.f;
        for (int r = 0; r < a.cluster; ++r) top = fmaxf(top, m_r[r][hd]);
        float2 s = make_float2(0.f, 0.f);
        for (int r = 0; r < a.cluster; ++r) {
            const float fr = top == -INFINITY ? 0.f : ex2(0.5f * (m_r[r][hd] - top));
            const float2 v = sum_r[r * share + j];
            sum += fr * l_r[r][hd] * fr;
            s.x += fr * v.x * fr;
            s.y += fr * v.y * fr;
        }
        put2(out + hd * D + 2 * q, sum == 0.f ? 0.f : s.x / sum, sum == 0.f ? 0.f : s.y / sum);
        if (a.lse && q == 0) a.lse[q0 / D + hd] = sum == 0.f ? -INFINITY : (top + log2f(sum)) * 0.69314718055994531f;
    }
}

template <int D, typename CT>
constexpr size_t ring_bytes() { return (size_t)kWarps * 2 * tiles_per_step<D, CT>() * 32 * D * sizeof(CT); }

// How many clusters of `size` CTAs the current device runs at once (a property of
// the kernel and the device, asked for once); 0 where it cannot.
template <int D, typename CT, typename T, int NT, bool EXACT>
int resident(int size) {
    static std::atomic<int> known[128][5];
    int dev = 0, lg = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 128) return 0;
    while ((1 << lg) < size) ++lg;
    return ask_once(known[dev][lg], [size] {
        const auto kernel = cache_attn_kernel<D, CT, T, NT, EXACT>;
        int n = 0;
        cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)ring_bytes<D, CT>());
        if (e == cudaSuccess && size > 8)
            e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
        if (e == cudaSuccess) {
            cudaLaunchConfig_t cfg = {};
            cfg.gridDim = dim3(size);
            cfg.blockDim = dim3(kThreads);
            cfg.dynamicSmemBytes = ring_bytes<D, CT>();
            cudaLaunchAttribute at[1];
            at[0].id = cudaLaunchAttributeClusterDimension;
            at[0].val.clusterDim.x = size;
            at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
            cfg.attrs = at;
            cfg.numAttrs = 1;
            e = cudaOccupancyMaxActiveClusters(&n, kernel, &cfg);
        }
        if (e == cudaSuccess) return n;
        cudaGetLastError();
        return e == cudaErrorInvalidClusterSize ? 0 : -1;
    });
}

template <int D, typename CT, typename T, int NT, bool EXACT>
int launch_split(const AttnArgs& a, cudaStream_t s) {
    if (resident<D, CT, T, NT, EXACT>(a.cluster) < 1) return LSA_ERR_CUDA;      // sets the kernel's attributes, too
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(a.warps == 1 ? (a.units + kWarps - 1) / kWarps : a.units * a.cluster);
    cfg.blockDim = dim3(kThreads);
    cfg.stream = s;
    cfg.dynamicSmemBytes = ring_bytes<D, CT>();
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = a.cluster;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    note_launch();
    return cuda_status(cudaLaunchKernelEx(&cfg, cache_attn_kernel<D, CT, T, NT, EXACT>, a));
}

// Steps of a warp up to which bf16 results are added up inside the tensor cores
// (EXACT: 8 % longer for the long chunk above, whose warps take 25 steps).
constexpr int64_t kCutSteps = 64;

template <int D, typename CT, typename T, int NT>
int launch(AttnArgs a, int64_t rows, cudaStream_t s) {
    constexpr bool F32 = sizeof(T) == 4;
    a.groups = (a.G + 8 * NT - 1) / (8 * NT);
    const int64_t units = rows * a.groups;
    a.units = (uint32_t)units;
    const int step = 16 * tiles_per_step<D, CT>();
    const int64_t steps = (a.max_sel + step - 1) / step;
    const int64_t ctas = resident<D, CT, T, NT, F32>(1);
    if (ctas < 1) return LSA_ERR_CUDA;
    // Few rows: a cluster of CTAs shares each, while all of them run at once and
    // every warp has a step (4 rows of 4,160 tokens, 16 heads of 128, 8-bit pages:
    // 9.9 us with 16 CTAs a row, 12.0 with 8, 16.7 with 4, 43 with one; 128 rows of up
    // to 1,599, 4 heads of 64, bf16: 10.4 with 2, 12.2 with one, 12.1 with 4).
    a.cluster = 1;
    while (a.cluster < kMaxCluster && a.cluster * 2 * kWarps <= steps &&
           units <= resident<D, CT, T, NT, F32>(a.cluster * 2))
        a.cluster *= 2;
    // Many rows: a warp takes a whole one, which needs no merge, unless the last
    // round of warps would then run long.  In microseconds a CTA that shares a row
    // takes about 4 + steps / 4, four whole rows side by side 6 + steps (8 heads of
    // 128, 8-bit pages; 4,096 rows of 64 tokens: 42 us shared, 23 whole; 16,384 of
    // 512: 346 and 272; 1,024 of 2,048: 70 and 81).
    const int64_t shared = (units + ctas - 1) / ctas * (4 + (steps + kWarps - 1) / kWarps);
    const int64_t whole = (units + kWarps * ctas - 1) / (kWarps * ctas) * (6 + steps);
    a.warps = a.cluster == 1 && whole < shared ? 1 : kWarps;
    if constexpr (!F32)
        if (steps <= kCutSteps * (a.warps == 1 ? 1 : kWarps * a.cluster))
            return launch_split<D, CT, T, NT, false>(a, s);
    return launch_split<D, CT, T, NT, true>(a, s);
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
