// New tokens' keys and values into the paged cache, the position rotation
// applied to keys and queries on the way.
//
// Per token at position t: every pair (x, y) of the first `rot` components of
// K and Q is turned by t * inv_freq; K and V are then rounded to the pages'
// type.  8-bit pages have one power-of-two scale per (page, head), so all new
// tokens of a page are handled by one CTA per head.  The scale comes from the
// unrotated magnitudes (a rotation grows a component by at most sqrt(2)): it
// needs no angle, and it is an exact function of the inputs.  A power of two
// loses nothing against a free scale (the codes are floats) and makes the
// change to a larger scale exact down to the codes' subnormals.
//
// The angle t * inv_freq reaches 1e7 radians: it is formed and reduced to one
// turn in fp64, and its sine and cosine are taken in fp32 with the rest of the
// reduction added to first order.
//
// Work: one CTA per (page that a sequence writes, range of heads).  A row
// (token, head) is taken by d/16 threads, each holding two 8-element pieces
// whose elements are each other's partners, so a pair never leaves a thread;
// the sines of a token are kept in registers for all its heads.
#include "cache_common.cuh"

namespace lsa {
namespace {

constexpr int kWriteThreads = 256;

struct WriteArgs {
    CacheArgs c;
    const void* K;
    const void* V;
    const void* Q;
    void* K_out;
    void* Q_out;
    const int64_t* cu;
    const int64_t* pos0;
    const double* inv_freq;
    int64_t n;
    int batch, hq, rot, interleaved;
    int by_token;          // units are tokens (few of them) instead of page slots
    int tokens_per_pass;   // tokens of a page that a CTA takes at a time (a power of two)
    int kv_per, q_per;     // heads of a CTA (blockIdx.y)
    int32_t* err;
};

// ---- 8 elements at a time
__device__ __forceinline__ void load8(const float* p, float* x) {
    const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
    x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
    x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
}
__device__ __forceinline__ void load8(const __nv_bfloat16* p, float* x) {
    const uint4 v = *reinterpret_cast<const uint4*>(p);
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}
__device__ __forceinline__ void store8(float* p, const float* x) {
    *reinterpret_cast<float4*>(p) = make_float4(x[0], x[1], x[2], x[3]);
    *reinterpret_cast<float4*>(p + 4) = make_float4(x[4], x[5], x[6], x[7]);
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float* x) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}
// 8-bit pages: x times the inverse scale, values that are not finite as NaN
__device__ __forceinline__ void store8(uint8_t* p, const float* x, float inv) {
    uint32_t w[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        float y[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float v = x[4 * i + j];
            y[j] = fabsf(v) < INFINITY ? v * inv : NAN;
        }
        w[i] = (uint32_t)f32x2_to_e4m3x2(y[0], y[1]) | ((uint32_t)f32x2_to_e4m3x2(y[2], y[3]) << 16);
    }
    *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
}

// largest finite magnitude of 8 elements, at least m
__device__ __forceinline__ float amax8(const float* x, float m) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float a = fabsf(x[i]);
        m = fmaxf(m, a < INFINITY ? a : 0.f);
    }
    return m;
}

// Smallest e in [-64, 64] with amax <= lim 2^e, lim = lim_m 2^8 with 1 <= lim_m < 2.
__device__ __forceinline__ int scale_exp(float amax, float lim_m) {
    if (amax <= 0.f) return -64;
    const int bits = __float_as_int(amax);
    const int E = (bits >> 23) - 127;                       // a subnormal reads -127: clamped below
    const float m = __int_as_float((bits & 0x7fffff) | 0x3f800000);
    return min(64, max(-64, E - 8 + (m > lim_m ? 1 : 0)));
}
__device__ __forceinline__ float pow2i(int e) { return __int_as_float((e + 127) << 23); }

// cos and sin of 8 pairs at position t
__device__ __forceinline__ void turn8(const double* inv_freq, int64_t t, float* cs, float* sn) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const double th = (double)t * inv_freq[i];
        // r = th - 2 pi k, |r| <= pi, with 2 pi in two parts
        const double k = rint(th * 0.15915494309189535);
        const double r = fma(-k, 2.4492935982947064e-16, fma(-k, 6.283185307179586, th));
        const float hi = (float)r;
        const float lo = (float)(r - (double)hi);
        float s, c;
        sincosf(hi, &s, &c);
        cs[i] = fmaf(-lo, s, c);
        sn[i] = fmaf(lo, c, s);
    }
}

// Turn the pairs of pieces a and b (see piece_a, piece_b).
__device__ __forceinline__ void rotate16(float* a, float* b, const float* cs, const float* sn, bool interleaved) {
    if (interleaved) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float x = a[2 * i], y = a[2 * i + 1], u = b[2 * i], v = b[2 * i + 1];
            a[2 * i] = x * cs[i] - y * sn[i];
            a[2 * i + 1] = x * sn[i] + y * cs[i];
            b[2 * i] = u * cs[4 + i] - v * sn[4 + i];
            b[2 * i + 1] = u * sn[4 + i] + v * cs[4 + i];
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float x = a[i], y = b[i];
            a[i] = x * cs[i] - y * sn[i];
            b[i] = x * sn[i] + y * cs[i];
        }
    }
}

template <int D, typename T, typename CT>
__global__ __launch_bounds__(kWriteThreads) void cache_write_kernel(const WriteArgs a) {
    constexpr bool kScaled = sizeof(CT) == 1;
    constexpr int TPR = D / 16;                     // threads per row
    constexpr int ROWS = kWriteThreads / TPR;
    extern __shared__ uint32_t sm[];                // [2][kv_per] largest magnitudes, then scales
    __shared__ int found_b, broken;
    const int tid = threadIdx.x;
    const CacheArgs& c = a.c;

    // the sequence of this unit, all sequences checked on the way
    if (tid == 0) { found_b = -1; broken = 0; }
    __syncthreads();
    const int64_t x = blockIdx.x;
    for (int b = tid; b < a.batch; b += kWriteThreads) {
        const int64_t c0 = a.cu[b], c1 = a.cu[b + 1];
        if (c0 < 0 || c1 < c0 || c1 > a.n) broken = 1;
        const int64_t u0 = a.by_token ? c0 : (c0 >> c.log2_page) + 2 * (int64_t)b;
        const int64_t u1 = a.by_token ? c1 : (c1 >> c.log2_page) + 2 * (int64_t)(b + 1);
        if (x >= u0 && x < u1) found_b = b;
    }
    __syncthreads();
    if (broken) {
        if (tid == 0) latch(a.err, kErrDevice);
        return;
    }
    const int b = found_b;
    if (b < 0) return;
    const int64_t c0 = a.cu[b], c1 = a.cu[b + 1], p0 = a.pos0[b];
    if (p0 < 0) {
        if (tid == 0) latch(a.err, kErrDevice);
        return;
    }
    // the unit's rows [r0, r0 + m) and their first slot
    int64_t r0;
    if (a.by_token) {
        r0 = x;
        if (r0 > c0 && ((p0 + r0 - c0) & (c.page - 1)) != 0) return;   // not the first new token of its page
    } else {
        const int64_t pg = (p0 >> c.log2_page) + (x - ((c0 >> c.log2_page) + 2 * (int64_t)b));
        r0 = max(c0, c0 + (pg << c.log2_page) - p0);
    }
    if (r0 >= c1) return;
    const int64_t pos = p0 + r0 - c0;
    const int slot0 = (int)(pos & (c.page - 1));
    const int m = (int)min((int64_t)(c.page - slot0), c1 - r0);
    const int pid = cache_page(c, b, pos);
    if (pid < 0) {
        if (tid == 0) latch(a.err, kErrDevice);
        return;
    }

    const int piece = tid % TPR, row = tid / TPR;
    const int TT = a.tokens_per_pass, HT = ROWS / TT;
    const int hh = row % HT, tt = row / HT;
    const int kv0 = blockIdx.y * a.kv_per, kv1 = min(c.hkv, kv0 + a.kv_per);
    const int q0 = blockIdx.y * a.q_per, q1 = min(a.hq, q0 + a.q_per);
    // this thread's two 8-element pieces of a K or Q row: partners of each other
    const bool turned = piece < a.rot / 16;
    const int pa = turned && !a.interleaved ? 8 * piece : 16 * piece;
    const int pb = turned && !a.interleaved ? 8 * piece + a.rot / 2 : 16 * piece + 8;

    const T* K = static_cast<const T*>(a.K);
    const T* V = static_cast<const T*>(a.V);
    float* scales = reinterpret_cast<float*>(sm);
    if (kScaled) {
        for (int i = tid; i < 2 * a.kv_per; i += kWriteThreads) sm[i] = 0;
        __syncthreads();
        for (int h = kv0 + hh; h < kv1; h += HT) {
            float mk = 0.f, mv = 0.f;
            for (int t = tt; t < m; t += TT) {
                const int64_t o = ((r0 + t) * c.hkv + h) * D + 16 * piece;
                float v[8];
                load8(K + o, v);
                mk = amax8(v, mk);
                load8(K + o + 8, v);
                mk = amax8(v, mk);
                load8(V + o, v);
                mv = amax8(v, mv);
                load8(V + o + 8, v);
                mv = amax8(v, mv);
            }
            // magnitudes are >= 0: their bit patterns order like the values
            atomicMax(&sm[h - kv0], __float_as_uint(mk));
            atomicMax(&sm[a.kv_per + h - kv0], __float_as_uint(mv));
        }
        __syncthreads();
        for (int i = tid; i < 2 * (kv1 - kv0); i += kWriteThreads) {
            const bool is_v = i >= kv1 - kv0;
            const int h = is_v ? i - (kv1 - kv0) : i;
            const int j = (is_v ? a.kv_per : 0) + h;
            float* gs = (is_v ? c.V_scale : c.K_scale) + (int64_t)pid * c.hkv + kv0 + h;
            float s = pow2i(scale_exp(__uint_as_float(sm[j]), is_v ? 1.75f : 1.234375f));   // 448, 316 = that * 2^8
            if (slot0 > 0) {
                const float old = *gs;
                if (s > old) {
                    // what the page holds, under the larger scale
                    uint8_t* p = static_cast<uint8_t*>(is_v ? c.V : c.K) + cache_row(c, pid, kv0 + h, 0) * D;
                    const float ratio = old / s;
                    for (int e = 0; e < slot0 * D; e += 8) {
                        const uint2 w = *reinterpret_cast<const uint2*>(p + e);
                        const float4 f0 = e4m3x4_to_f32x4(w.x), f1 = e4m3x4_to_f32x4(w.y);
                        const float v[8] = {f0.x, f0.y, f0.z, f0.w, f1.x, f1.y, f1.z, f1.w};
                        store8(p + e, v, ratio);
                    }
                } else {
                    s = old;
                }
            }
            *gs = s;
            scales[j] = 1.f / s;
        }
        __syncthreads();
    }

    for (int t = tt; t < m; t += TT) {
        float cs[8], sn[8];
        if (turned) turn8(a.inv_freq + 8 * piece, pos + t, cs, sn);
        for (int h = kv0 + hh; h < kv1; h += HT) {
            const int64_t o = ((r0 + t) * c.hkv + h) * D;
            CT* kp = static_cast<CT*>(c.K) + cache_row(c, pid, h, slot0 + t) * D;
            CT* vp = static_cast<CT*>(c.V) + cache_row(c, pid, h, slot0 + t) * D;
            float u[8], v[8];
            load8(K + o + pa, u);
            load8(K + o + pb, v);
            if (turned) rotate16(u, v, cs, sn, a.interleaved);
            if (a.K_out) {
                store8(static_cast<T*>(a.K_out) + o + pa, u);
                store8(static_cast<T*>(a.K_out) + o + pb, v);
            }
            if constexpr (kScaled) {
                store8(kp + pa, u, scales[h - kv0]);
                store8(kp + pb, v, scales[h - kv0]);
            } else {
                store8(kp + pa, u);
                store8(kp + pb, v);
            }
            load8(V + o + 16 * piece, u);
            load8(V + o + 16 * piece + 8, v);
            if constexpr (kScaled) {
                store8(vp + 16 * piece, u, scales[a.kv_per + h - kv0]);
                store8(vp + 16 * piece + 8, v, scales[a.kv_per + h - kv0]);
            } else {
                store8(vp + 16 * piece, u);
                store8(vp + 16 * piece + 8, v);
            }
        }
        for (int h = q0 + hh; h < q1; h += HT) {
            const int64_t o = ((r0 + t) * a.hq + h) * D;
            float u[8], v[8];
            load8(static_cast<const T*>(a.Q) + o + pa, u);
            load8(static_cast<const T*>(a.Q) + o + pb, v);
            if (turned) rotate16(u, v, cs, sn, a.interleaved);
            store8(static_cast<T*>(a.Q_out) + o + pa, u);
            store8(static_cast<T*>(a.Q_out) + o + pb, v);
        }
    }
}

template <int D, typename T, typename CT>
int launch(const WriteArgs& a, dim3 grid, cudaStream_t s) {
    note_launch();
    cache_write_kernel<D, T, CT><<<grid, kWriteThreads, 2 * (size_t)a.kv_per * sizeof(float), s>>>(a);
    return cuda_status(cudaGetLastError());
}

template <int D, typename T>
int launch_ct(const WriteArgs& a, int cache_dtype, dim3 grid, cudaStream_t s) {
    return cache_dtype == LSA_E4M3 ? launch<D, T, uint8_t>(a, grid, s) : launch<D, T, __nv_bfloat16>(a, grid, s);
}

}  // namespace

int launch_cache_write(const lsa_kv_cache& cache, const void* K, const void* V, const void* Q, int64_t n,
                       const int64_t* cu, const int64_t* pos0, int hq, int dtype, const double* inv_freq, int rot,
                       int interleaved, void* K_out, void* Q_out, int32_t* err, cudaStream_t s) {
    WriteArgs a{cache_args(cache), K, V, Q, K_out, Q_out, cu, pos0, inv_freq, n, (int)cache.batch, hq, rot, interleaved};
    a.err = err;
    // A sequence of m tokens touches at most m / page + 2 pages; units are page
    // slots in that numbering, or tokens (each page taken by its first) when
    // those are fewer.
    const int64_t slots = n / cache.page + 2 * cache.batch;
    a.by_token = n < slots;
    const int64_t units = a.by_token ? n : slots;
    const int rows = kWriteThreads / (cache.d / 16);
    a.tokens_per_pass = 1;
    while (a.tokens_per_pass < rows && a.tokens_per_pass < cache.page && a.tokens_per_pass * 2 * cache.batch <= n)
        a.tokens_per_pass *= 2;
    a.kv_per = cache.hkv;
    a.q_per = hq;
    const dim3 grid((unsigned)units, 1);
    if (cache.d == 128)
        return dtype == LSA_F32 ? launch_ct<128, float>(a, cache.dtype, grid, s)
                                : launch_ct<128, __nv_bfloat16>(a, cache.dtype, grid, s);
    return dtype == LSA_F32 ? launch_ct<64, float>(a, cache.dtype, grid, s)
                            : launch_ct<64, __nv_bfloat16>(a, cache.dtype, grid, s);
}

}  // namespace lsa
