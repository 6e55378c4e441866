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
// Work: one CTA per (page that a sequence writes, range of its lists).  A row
// (token, head) is taken by d/16 threads, each holding two 8-element pieces
// whose elements are each other's partners, so a pair never leaves a thread.
//
// What bounds it.  A prompt is bound by HBM: 131,072 tokens of 32 query and 4 KV
// heads of 128 into 8-bit pages take 462-476 us for 2.68 GB (5.6-5.8 TB/s, 0.86-0.89
// of the measured copy rate), every row read once: K and V rows stay in registers
// while their page's scales are settled (reading them again took 495-510 us).  A
// token a sequence is bound by latency (offsets, page, scale and rows follow one
// another): 4.5 us for 4 sequences, 4.7 for 96.  8,191 fp32 tokens of 8 query and 2
// KV heads into pages of 128 are one wave of 130 CTAs: 19 us.
#include <algorithm>
#include <atomic>

#include "cache_common.cuh"

namespace lsa {
namespace {

constexpr int kWriteThreads = 256;
constexpr int kMaxPageThreads = 512;

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
    int most_tokens;       // of a unit
    int lists;             // rows of a token: its K heads, its V heads, its query heads
    // blockIdx.y, few tokens: per_cta lists each; many: kv_ctas CTAs
    // with kv_per KV heads each, then others with the query heads of q_per tokens
    // each, q_side heads side by side
    int per_cta, kv_ctas, kv_per, q_per, q_side;
    int32_t* err;
};

// ---- a piece: 8 elements of a row, two runs of 4 that are `gap` elements apart.
// Loaded as they are, unpacked where they are used.  bf16 pieces are 16 bytes in
// one run (gap 4); of fp32 rows the 16 bytes of a run are neighbours of the next
// thread's.
template <typename T>
struct Piece {
    uint4 w[sizeof(T) / 2];
    __device__ __forceinline__ void load(const T* p, int gap) {
        w[0] = *reinterpret_cast<const uint4*>(p);
        if constexpr (sizeof(T) == 4) w[1] = *reinterpret_cast<const uint4*>(p + gap);
    }
    __device__ __forceinline__ void unpack(float* x) const {
        if constexpr (sizeof(T) == 4) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                x[4 * i] = __uint_as_float(w[i].x);
                x[4 * i + 1] = __uint_as_float(w[i].y);
                x[4 * i + 2] = __uint_as_float(w[i].z);
                x[4 * i + 3] = __uint_as_float(w[i].w);
            }
        } else {
            const uint32_t v[4] = {w[0].x, w[0].y, w[0].z, w[0].w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                x[2 * i] = __uint_as_float(v[i] << 16);
                x[2 * i + 1] = __uint_as_float(v[i] & 0xffff0000u);
            }
        }
    }
};
__device__ __forceinline__ uint32_t bf16x2(float a, float b) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
}
// 8 elements to a row of the activations' type or of bf16 pages
__device__ __forceinline__ void store8(float* p, const float* x, int gap) {
    *reinterpret_cast<float4*>(p) = make_float4(x[0], x[1], x[2], x[3]);
    *reinterpret_cast<float4*>(p + gap) = make_float4(x[4], x[5], x[6], x[7]);
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float* x, int gap) {
    const uint2 u = make_uint2(bf16x2(x[0], x[1]), bf16x2(x[2], x[3]));
    const uint2 v = make_uint2(bf16x2(x[4], x[5]), bf16x2(x[6], x[7]));
    if (gap == 4) {
        *reinterpret_cast<uint4*>(p) = make_uint4(u.x, u.y, v.x, v.y);
    } else {
        *reinterpret_cast<uint2*>(p) = u;
        *reinterpret_cast<uint2*>(p + gap) = v;
    }
}
// 8-bit pages: x times the inverse scale, values that are not finite as NaN
__device__ __forceinline__ void store8(uint8_t* p, const float* x, int gap, float inv) {
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
    if (gap == 4) {
        *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
    } else {
        *reinterpret_cast<uint32_t*>(p) = w[0];
        *reinterpret_cast<uint32_t*>(p + gap) = w[1];
    }
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

// cos and sin of 8 pairs at position t: pairs p, p + 1, .. up to the next multiple
// of `run`, then those `hop` pairs on, and so forth
__device__ __forceinline__ void turn8(const double* inv_freq, int p, int run, int hop, int64_t t, float* cs, float* sn) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        // half turns, less whole turns: r in [-1, 1], exact but for the two products
        const double th = (double)t * inv_freq[p + i % run + i / run * hop] * 0.31830988618379067;
        const double r = fma(-2.0, rint(0.5 * th), th);
        const float hi = (float)r;
        const float lo = (float)(r - (double)hi) * 3.14159274f;
        float s, c;
        sincospif(hi, &s, &c);
        cs[i] = fmaf(-lo, s, c);
        sn[i] = fmaf(lo, c, s);
    }
}

// Turn the pairs of pieces a and b.
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

// What a CTA writes: rows [r0, r0 + m) of one sequence, the first of them token
// `pos`, all in one page from slot `slot0` on.
struct Unit {
    int64_t r0, pos;
    int m, slot0, pid;
};

// The unit of this CTA (blockIdx.x); false where there is none.  Up to kScanned
// sequences every CTA looks all of them over, so that a broken cu stops all CTAs, as
// the call promises; of more, where that takes long, it looks for its own in two
// steps, and all CTAs together look all over (a token each, 8 query and 1 KV heads,
// pages of 16, 1,024 sequences: 8.9 us with all looked over by every CTA, 7.7 in two
// steps; 4,096: 43 and 22.5; 65,535: 7.5 and 0.38 ms).
constexpr int kScanned = 1024;
__device__ __forceinline__ bool find_unit(const WriteArgs& a, Unit& u) {
    __shared__ int found_b, broken, part;
    const CacheArgs& c = a.c;
    const int tid = threadIdx.x;
    if (tid == 0) { found_b = -1; broken = 0; part = 0; }
    __syncthreads();
    const int64_t x = blockIdx.x;
    // first unit of sequence b, whose first row is c0
    auto unit0 = [&](int64_t c0, int64_t b) { return a.by_token ? c0 : (c0 >> c.log2_page) + 2 * b; };
    auto look = [&](int b) {
        const int64_t c0 = a.cu[b], c1 = a.cu[b + 1];
        if (c0 < 0 || c1 < c0 || c1 > a.n) broken = 1;
        if (x >= unit0(c0, b) && x < unit0(c1, b + 1)) found_b = b;
    };
    if (a.batch <= kScanned) {
#pragma unroll 4
        for (int b = tid; b < a.batch; b += blockDim.x) look(b);
    } else {
        const int len = (a.batch + blockDim.x - 1) / blockDim.x;
        if (tid * len < a.batch && x >= unit0(a.cu[tid * len], tid * len)) atomicMax(&part, tid);
        const int share = (a.batch + gridDim.x - 1) / gridDim.x;
        const int64_t s1 = min((int64_t)a.batch, (x + 1) * share);
        for (int64_t b = x * share + tid; b < s1; b += blockDim.x) look((int)b);
        __syncthreads();
        const int b1 = min(a.batch, (part + 1) * len);
        for (int b = part * len + tid; b < b1; b += blockDim.x) look(b);
    }
    __syncthreads();
    const int b = found_b;
    if (broken) {
        if (tid == 0) latch(a.err, kErrDevice);
        return false;
    }
    if (b < 0) return false;
    const int64_t c0 = a.cu[b], c1 = a.cu[b + 1], p0 = a.pos0[b];
    if (c0 == c1) return false;        // has page slots, but no token whose position would matter
    if (p0 < 0) {
        if (tid == 0) latch(a.err, kErrDevice);
        return false;
    }
    if (a.by_token) {
        u.r0 = x;
        if (u.r0 > c0 && ((p0 + u.r0 - c0) & (c.page - 1)) != 0) return false;   // not its page's first new token
    } else {
        const int64_t pg = (p0 >> c.log2_page) + (x - ((c0 >> c.log2_page) + 2 * (int64_t)b));
        u.r0 = max(c0, c0 + (pg << c.log2_page) - p0);
    }
    if (u.r0 >= c1) return false;
    u.pos = p0 + u.r0 - c0;
    u.slot0 = (int)(u.pos & (c.page - 1));
    u.m = (int)min((int64_t)(c.page - u.slot0), c1 - u.r0);
    u.pid = cache_page(c, b, u.pos);
    if (u.pid < 0) {
        if (tid == 0) latch(a.err, kErrDevice);
        return false;
    }
    return true;
}

// A list: one head's rows of K, V or Q.  A token's lists are its K heads [0, hkv),
// its V heads [hkv, 2 hkv), its query heads from 2 hkv on.
template <typename T>
struct List {
    const T* src;          // row r0
    T* out;                // where the (rotated) row r0 goes, or null
    int64_t step;          // elements from one token to the next
    int h;                 // head
    bool is_k, is_v;
};
template <int D, typename T>
__device__ __forceinline__ List<T> list_of(const WriteArgs& a, int64_t r0, int l) {
    const int hkv = a.c.hkv;
    List<T> s;
    s.is_k = l < hkv;
    s.is_v = !s.is_k && l < 2 * hkv;
    const bool q = l >= 2 * hkv;
    const int heads = q ? a.hq : hkv;
    s.h = q ? l - 2 * hkv : s.is_v ? l - hkv : l;
    s.step = (int64_t)heads * D;
    const int64_t off = (r0 * heads + s.h) * D;
    s.src = static_cast<const T*>(q ? a.Q : s.is_v ? a.V : a.K) + off;
    T* out = static_cast<T*>(q ? a.Q_out : s.is_v ? nullptr : a.K_out);
    s.out = out ? out + off : nullptr;
    return s;
}

// Where the scale of K or V list s of the unit's page is.
template <typename T>
__device__ __forceinline__ float* scale_at(const WriteArgs& a, const Unit& u, const List<T>& s) {
    return (s.is_v ? a.c.V_scale : a.c.K_scale) + (int64_t)u.pid * a.c.hkv + s.h;
}
// The scale that the largest finite magnitude written asks for; 448 = 1.75 * 2^8, 316 = 1.234375 * 2^8.
__device__ __forceinline__ float new_scale(float top, bool is_v) {
    return pow2i(scale_exp(top, is_v ? 1.75f : 1.234375f));
}

// What the page holds below slot0, under the larger scale.  All threads of the CTA.
template <int D, typename T>
__device__ __forceinline__ void shrink_held(const WriteArgs& a, const Unit& u, const List<T>& s, float shrink) {
    uint8_t* p = static_cast<uint8_t*>(s.is_v ? a.c.V : a.c.K) + cache_row(a.c, u.pid, s.h, 0) * D;
    for (int e = 8 * threadIdx.x; e < u.slot0 * D; e += 8 * blockDim.x) {
        const uint2 w = *reinterpret_cast<const uint2*>(p + e);
        const float4 f0 = e4m3x4_to_f32x4(w.x), f1 = e4m3x4_to_f32x4(w.y);
        const float v[8] = {f0.x, f0.y, f0.z, f0.w, f1.x, f1.y, f1.z, f1.w};
        store8(p + e, v, 4, shrink);
    }
}

// Where this thread's two pieces of a row are: the same pairs' components in K
// and Q, anything in V.
struct Pieces {
    int a, b, gap;         // of K and Q rows
    int va, vb, vgap;      // of V rows
    int piece;
    bool turned;
    __device__ __forceinline__ int first(bool is_v) const { return is_v ? va : a; }
    __device__ __forceinline__ int second(bool is_v) const { return is_v ? vb : b; }
    __device__ __forceinline__ int step(bool is_v) const { return is_v ? vgap : gap; }
};
template <int D, typename T>
__device__ __forceinline__ Pieces pieces_of(const WriteArgs& a, int piece) {
    constexpr int TPR = D / 16;
    const int n8 = a.rot / 16;                     // threads of a row that turn something
    Pieces p;
    p.piece = piece;
    p.turned = piece < n8;
    if constexpr (sizeof(T) == 4) {
        const int n = p.turned ? n8 : TPR - n8;    // threads that share the turned or the other components
        p.gap = 4 * n;
        p.a = p.turned ? 4 * piece : a.rot + 4 * (piece - n8);
        p.b = p.a + 8 * n;                         // turned halves: rot / 2 = 8 n8 apart, too
        p.va = 4 * piece;
        p.vb = p.va + 8 * TPR;
        p.vgap = 4 * TPR;
    } else {
        p.gap = p.vgap = 4;
        p.a = p.turned && !a.interleaved ? 8 * piece : 16 * piece;
        p.b = p.turned && !a.interleaved ? p.a + a.rot / 2 : p.a + 8;
        p.va = 16 * piece;
        p.vb = p.va + 8;
    }
    return p;
}

// Store one row's pieces (token r0 + t of the unit), turned already.
template <int D, typename T, typename CT>
__device__ __forceinline__ void store_row(const WriteArgs& a, const Unit& u, const List<T>& s, const Pieces& pc, int t,
                                          const float* x, const float* y, float inv) {
    const int oa = pc.first(s.is_v), ob = pc.second(s.is_v), gap = sizeof(T) == 4 ? pc.step(s.is_v) : 4;
    if (s.out) {
        store8(s.out + t * s.step + oa, x, gap);
        store8(s.out + t * s.step + ob, y, gap);
    }
    if (s.is_k || s.is_v) {
        CT* p = static_cast<CT*>(s.is_v ? a.c.V : a.c.K) + cache_row(a.c, u.pid, s.h, u.slot0 + t) * D;
        if constexpr (sizeof(CT) == 1) {
            store8(p + oa, x, gap, inv);
            store8(p + ob, y, gap, inv);
        } else {
            store8(p + oa, x, gap);
            store8(p + ob, y, gap);
        }
    }
}

// Sines and cosines of the unit's tokens [t0, t1), for all their heads: [token][4]
// [rot / 16] float4, cos 0-3, cos 4-7, sin 0-3, sin 4-7 of 8 pairs.
template <typename T>
__device__ __forceinline__ void fill_turns(const WriteArgs& a, const Unit& u, int t0, int t1, float4* turns) {
    const int n8 = a.rot / 16;
    for (int i = t0 * n8 + threadIdx.x; i < t1 * n8; i += blockDim.x) {
        const int t = i / n8, p = i % n8;
        float cs[8], sn[8];
        // the pairs of pieces a and b (see pieces_of)
        if (sizeof(T) == 2) turn8(a.inv_freq, 8 * p, 8, 0, u.pos + t, cs, sn);
        else if (a.interleaved) turn8(a.inv_freq, 2 * p, 2, 2 * n8, u.pos + t, cs, sn);
        else turn8(a.inv_freq, 4 * p, 4, 4 * n8, u.pos + t, cs, sn);
        float4* at = turns + (t - t0) * 4 * n8 + p;
        at[0] = make_float4(cs[0], cs[1], cs[2], cs[3]);
        at[n8] = make_float4(cs[4], cs[5], cs[6], cs[7]);
        at[2 * n8] = make_float4(sn[0], sn[1], sn[2], sn[3]);
        at[3 * n8] = make_float4(sn[4], sn[5], sn[6], sn[7]);
    }
}
// Turn the pieces x, y of a row of the t-th of these tokens.
__device__ __forceinline__ void turn_row(const WriteArgs& a, const float4* turns, const Pieces& pc, int t, float* x,
                                         float* y) {
    const int n8 = a.rot / 16;
    const float4* at = turns + t * 4 * n8 + pc.piece;
    float cs[8], sn[8];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const float4 c4 = at[k * n8], s4 = at[(2 + k) * n8];
        cs[4 * k] = c4.x; cs[4 * k + 1] = c4.y; cs[4 * k + 2] = c4.z; cs[4 * k + 3] = c4.w;
        sn[4 * k] = s4.x; sn[4 * k + 1] = s4.y; sn[4 * k + 2] = s4.z; sn[4 * k + 3] = s4.w;
    }
    rotate16(x, y, cs, sn, a.interleaved);
}

// Few tokens, or little: the unit's rows (token, list) in order, ROWS side by side.
// The largest magnitudes of 8-bit pages take a pass of their own.
template <int D, typename T, typename CT>
__global__ __launch_bounds__(kWriteThreads) void cache_write_few_kernel(const WriteArgs a) {
    constexpr bool kScaled = sizeof(CT) == 1;
    constexpr int TPR = D / 16;                     // threads per row
    const int ROWS = blockDim.x / TPR;
    extern __shared__ float4 turn_s[];              // then [per_cta] largest magnitudes or inverse scales, [per_cta] shrinks
    uint32_t* top_s = reinterpret_cast<uint32_t*>(turn_s + a.most_tokens * (a.rot / 4));
    float *inv_s = reinterpret_cast<float*>(top_s), *shrink_s = inv_s + a.per_cta;
    Unit u;
    if (!find_unit(a, u)) return;
    const int tid = threadIdx.x, row = tid / TPR;
    const Pieces pc = pieces_of<D, T>(a, tid % TPR);
    const int l0 = blockIdx.y * a.per_cta, l1 = min(a.lists, l0 + a.per_cta);
    const int le = kScaled ? max(l0, min(l1, 2 * a.c.hkv)) : l0;    // lists with a scale
    fill_turns<T>(a, u, 0, u.m, turn_s);
    for (int i = tid; i < le - l0; i += blockDim.x) top_s[i] = 0;
    __syncthreads();
    if (l0 < le) {
        const int lists = le - l0;
        for (int r = row; r < u.m * lists; r += ROWS) {
            const int t = r / lists, l = l0 + r % lists;
            const List<T> s = list_of<D, T>(a, u.r0, l);
            Piece<T> x, y;
            x.load(s.src + t * s.step + pc.va, pc.vgap);
            y.load(s.src + t * s.step + pc.vb, pc.vgap);
            float v[8];
            x.unpack(v);
            float top = amax8(v, 0.f);
            y.unpack(v);
            top = amax8(v, top);
            // only the threads of one row run the same trips of this loop
            const uint32_t row_mask = ((1u << TPR) - 1u) << ((tid & 31) / TPR * TPR);
#pragma unroll
            for (int i = 1; i < TPR; i *= 2) top = fmaxf(top, __shfl_xor_sync(row_mask, top, i));
            // magnitudes are >= 0: their bit patterns order like the values
            if (pc.piece == 0) atomicMax(&top_s[l - l0], __float_as_uint(top));
        }
        __syncthreads();
        for (int l = l0 + tid; l < le; l += blockDim.x) {
            const List<T> s = list_of<D, T>(a, u.r0, l);
            const float old = u.slot0 > 0 ? *scale_at(a, u, s) : 0.f;
            const float scale = fmaxf(new_scale(__uint_as_float(top_s[l - l0]), s.is_v), old);
            *scale_at(a, u, s) = scale;
            inv_s[l - l0] = 1.f / scale;
            shrink_s[l - l0] = old / scale;
        }
        __syncthreads();
        if (u.slot0 > 0)
            for (int l = l0; l < le; ++l)
                if (shrink_s[l - l0] != 1.f) shrink_held<D, T>(a, u, list_of<D, T>(a, u.r0, l), shrink_s[l - l0]);
    }
    const int lists = l1 - l0;
    for (int r = row; r < u.m * lists; r += ROWS) {
        const int t = r / lists, l = l0 + r % lists;
        const List<T> s = list_of<D, T>(a, u.r0, l);
        Piece<T> x, y;
        x.load(s.src + t * s.step + pc.first(s.is_v), pc.step(s.is_v));
        y.load(s.src + t * s.step + pc.second(s.is_v), pc.step(s.is_v));
        float v[8], w[8];
        x.unpack(v);
        y.unpack(w);
        if (pc.turned && !s.is_v) turn_row(a, turn_s, pc, t, v, w);
        store_row<D, T, CT>(a, u, s, pc, t, v, w, l < le ? inv_s[l - l0] : 1.f);
    }
}

// Many tokens a page.  blockIdx.y: CTAs for KV heads, then CTAs for query heads.  A KV
// head's K and V rows of the page are in registers while their scales are
// settled, two tokens a thread, so they are read once; queries stream through,
// several rows on their way in every thread.
template <typename T>
constexpr int rows_ahead() { return sizeof(T) == 4 ? 4 : 8; }
template <int D, typename T, typename CT>
__global__ __launch_bounds__(kMaxPageThreads) void cache_write_page_kernel(const WriteArgs a) {
    constexpr bool kScaled = sizeof(CT) == 1;
    constexpr int TPR = D / 16, kAhead = rows_ahead<T>();
    const int ROWS = blockDim.x / TPR;              // a page has at most 2 ROWS tokens
    extern __shared__ float4 turn_s[];              // then [kv_per][2] largest magnitudes
    uint32_t* top_s = reinterpret_cast<uint32_t*>(turn_s + a.most_tokens * (a.rot / 4));
    Unit u;
    if (!find_unit(a, u)) return;
    const int tid = threadIdx.x, row = tid / TPR;
    const Pieces pc = pieces_of<D, T>(a, tid % TPR);
    const int y = blockIdx.y;
    if (y < a.kv_ctas) {
        fill_turns<T>(a, u, 0, u.m, turn_s);
        const int h0 = y * a.kv_per, h1 = min(a.c.hkv, h0 + a.kv_per);
        for (int i = tid; i < 2 * (h1 - h0); i += blockDim.x) top_s[i] = 0;
        __syncthreads();
        for (int h = h0; h < h1; ++h) {
            const List<T> ks = list_of<D, T>(a, u.r0, h), vs = list_of<D, T>(a, u.r0, a.c.hkv + h);
            Piece<T> k[2][2], v[2][2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int t = row + i * ROWS;
                if (t < u.m) {
                    k[i][0].load(ks.src + t * ks.step + pc.a, pc.gap);
                    k[i][1].load(ks.src + t * ks.step + pc.b, pc.gap);
                    v[i][0].load(vs.src + t * vs.step + pc.va, pc.vgap);
                    v[i][1].load(vs.src + t * vs.step + pc.vb, pc.vgap);
                }
            }
            float ki = 1.f, vi = 1.f;
            if constexpr (kScaled) {
                const float k_old = u.slot0 > 0 ? *scale_at(a, u, ks) : 0.f;
                const float v_old = u.slot0 > 0 ? *scale_at(a, u, vs) : 0.f;
                float kt = 0.f, vt = 0.f;
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    if (row + i * ROWS < u.m) {
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            float x[8];
                            k[i][j].unpack(x);
                            kt = amax8(x, kt);
                            v[i][j].unpack(x);
                            vt = amax8(x, vt);
                        }
                    }
                // magnitudes are >= 0: their bit patterns order like the values
                const uint32_t kb = __reduce_max_sync(0xffffffffu, __float_as_uint(kt));
                const uint32_t vb = __reduce_max_sync(0xffffffffu, __float_as_uint(vt));
                uint32_t* top = top_s + 2 * (h - h0);
                if (tid % 32 == 0) {
                    atomicMax(&top[0], kb);
                    atomicMax(&top[1], vb);
                }
                __syncthreads();                    // the old scales are read, too
                const float k_new = fmaxf(new_scale(__uint_as_float(top[0]), false), k_old);
                const float v_new = fmaxf(new_scale(__uint_as_float(top[1]), true), v_old);
                if (tid == 0) {
                    *scale_at(a, u, ks) = k_new;
                    *scale_at(a, u, vs) = v_new;
                }
                if (u.slot0 > 0 && k_new > k_old) shrink_held<D, T>(a, u, ks, k_old / k_new);
                if (u.slot0 > 0 && v_new > v_old) shrink_held<D, T>(a, u, vs, v_old / v_new);
                ki = 1.f / k_new;
                vi = 1.f / v_new;
            }
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int t = row + i * ROWS;
                if (t < u.m) {
                    float x[8], w[8];
                    k[i][0].unpack(x);
                    k[i][1].unpack(w);
                    if (pc.turned) turn_row(a, turn_s, pc, t, x, w);
                    store_row<D, T, CT>(a, u, ks, pc, t, x, w, ki);
                    v[i][0].unpack(x);
                    v[i][1].unpack(w);
                    store_row<D, T, CT>(a, u, vs, pc, t, x, w, vi);
                }
            }
        }
        return;
    }
    // all query heads of a share of the tokens, LT of a token's side by side, so that a warp's loads and stores are runs
    const int t0 = (y - a.kv_ctas) * a.q_per, t1 = min(u.m, t0 + a.q_per);
    fill_turns<T>(a, u, t0, t1, turn_s);
    __syncthreads();
    const int LT = a.q_side, TT = ROWS / LT;
    const int hh = row % LT, h1 = a.hq;
    for (int t = t0 + row / LT; t < t1; t += TT) {
        const int64_t at = ((u.r0 + t) * a.hq + hh) * D;
        const T* src = static_cast<const T*>(a.Q) + at;
        T* out = static_cast<T*>(a.Q_out) + at;
        // Q_out may be Q: a row's pieces are loaded before they are stored, and no two rows share elements
        for (int h = hh; h < h1; h += kAhead * LT) {
            Piece<T> x[kAhead], w[kAhead];
#pragma unroll
            for (int i = 0; i < kAhead; ++i)
                if (h + i * LT < h1) {
                    x[i].load(src + i * LT * D + pc.a, pc.gap);
                    w[i].load(src + i * LT * D + pc.b, pc.gap);
                }
#pragma unroll
            for (int i = 0; i < kAhead; ++i)
                if (h + i * LT < h1) {
                    float p[8], q[8];
                    x[i].unpack(p);
                    w[i].unpack(q);
                    if (pc.turned) turn_row(a, turn_s, pc, t - t0, p, q);
                    store8(out + i * LT * D + pc.a, p, pc.gap);
                    store8(out + i * LT * D + pc.b, q, pc.gap);
                }
            src += kAhead * LT * D;
            out += kAhead * LT * D;
        }
    }
}

// What a launch may ask for: the sines of a page's tokens and two words a list of a token.
constexpr int kMaxShared = 128 * (128 / 4) * (int)sizeof(float4) + 2 * (2 * 1024 + 4096) * (int)sizeof(float);

// The limit of a kernel's shared memory is set once a device, to the same for all
// calls: two threads that set what their calls need would lower each other's.
template <auto Kernel>
int launch_with(const WriteArgs& a, dim3 grid, int threads, size_t smem, cudaStream_t s) {
    static std::atomic<bool> set[128];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 128) return LSA_ERR_CUDA;
    if (!set[dev].load(std::memory_order_relaxed)) {
        const cudaError_t e = cudaFuncSetAttribute(Kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxShared);
        if (e != cudaSuccess) return cuda_status(e);
        set[dev].store(true, std::memory_order_relaxed);
    }
    note_launch();
    Kernel<<<grid, threads, smem, s>>>(a);
    return cuda_status(cudaGetLastError());
}

template <int D, typename T, typename CT>
int launch(WriteArgs a, int64_t units, bool pages, cudaStream_t s) {
    const size_t turns = (size_t)a.most_tokens * (a.rot / 4) * sizeof(float4);
    if (!pages) {
        const int64_t want = 148 * 3;
        // 148 SMs.  Few units: their lists are split over CTAs, down to the rows that a CTA takes side by side
        // (8,191 fp32 tokens, 8 query and 2 KV heads, pages of 128, on this kernel: one CTA an SM
        // 27.8 us, two 23.1, three 22.9, eight 26.5)
        constexpr int ROWS = kWriteThreads / (D / 16);
        const int64_t per_unit = std::max<int64_t>(1, std::min<int64_t>(a.c.page, a.n / a.batch));   // tokens, on average
        const int64_t most = std::min<int64_t>((a.lists * per_unit + ROWS - 1) / ROWS, (want + units - 1) / units);
        a.per_cta = (int)((a.lists + most - 1) / most);
        const dim3 grid((unsigned)units, (unsigned)((a.lists + a.per_cta - 1) / a.per_cta));
        // More CTAs than run at once (4 an SM): half the threads each, which have more to do (a token each
        // for 4,096 sequences of 8 query and 1 KV heads 20.9 us against 35.2, 32 and 4 heads 31.2 and 46.7; of 96
        // sequences, 32 and 4 heads, 5.3 and 5.0).
        const int threads = (int64_t)grid.x * grid.y > 148 * 4 ? kWriteThreads / 2 : kWriteThreads;
        return launch_with<cache_write_few_kernel<D, T, CT>>(a, grid, threads,
                                                             turns + 2 * (size_t)a.per_cta * sizeof(float), s);
    }
    const int threads = std::min(kMaxPageThreads, std::max(64, a.c.page * (D / 16) / 2));
    // few units: their KV heads and their queries' tokens are split over CTAs; a KV head is about three query
    // heads' work (8,191 fp32 tokens, 8 query and 2 KV heads, pages of 128: one wave 24.7 us a call, more CTAs 27-31)
    const int64_t want = (int64_t)148 * kMaxPageThreads / threads;
    const int64_t most = std::max<int64_t>(1, (want + units / 2) / units), work = 3 * a.c.hkv + a.hq;
    const int64_t kv_ctas = std::min<int64_t>(a.c.hkv, std::max<int64_t>(1, (3 * a.c.hkv * most + work / 2) / work));
    const int64_t q_ctas = a.hq > 0 ? std::min<int64_t>(8, std::max<int64_t>(1, (a.hq * most + work / 2) / work)) : 0;
    a.kv_per = (int)((a.c.hkv + kv_ctas - 1) / kv_ctas);
    a.kv_ctas = (a.c.hkv + a.kv_per - 1) / a.kv_per;
    a.q_per = (int)(q_ctas > 0 ? (a.c.page + q_ctas - 1) / q_ctas : 1);
    a.q_side = 1;
    while (a.q_side * 2 <= std::min(a.hq / rows_ahead<T>(), threads / (D / 16))) a.q_side *= 2;
    const dim3 grid((unsigned)units, (unsigned)(a.kv_ctas + q_ctas));
    return launch_with<cache_write_page_kernel<D, T, CT>>(a, grid, threads, turns + 2 * (size_t)a.kv_per * sizeof(float),
                                                          s);
}

template <int D, typename T>
int launch_ct(const WriteArgs& a, int cache_dtype, int64_t units, bool pages, cudaStream_t s) {
    return cache_dtype == LSA_E4M3 ? launch<D, T, uint8_t>(a, units, pages, s)
                                   : launch<D, T, __nv_bfloat16>(a, units, pages, s);
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
    a.most_tokens = (int)std::min<int64_t>(cache.page, n);
    a.lists = 2 * cache.hkv + hq;
    // Tokens of a page are worth a kernel that reads them once when a sequence brings
    // ten or more, and when there is enough of it: bytes of a unit's rows times bytes
    // of all rows.  Few-token kernel and page kernel in microseconds, 32 query and 4 KV
    // heads of 128, 8-bit pages, sequences x tokens: pages of 16, 16 x 16 (4.3e11) 6.3
    // and 7.7, 16 x 32 (8.6e11) 8.6 and 7.2, 512 x 4 (8.6e11) 16.1 and 20.0; of 32, 300 x
    // 10 (3.1e12) 29.8 and 19.8; of 64, 8 x 32 (8.6e11) 7.3 and 6.8, 64 x 256 127 and 71;
    // of 128, 128 x 16 (3.4e12) 17.5 and 16.1, 512 x 8 (3.4e12) 39.8 and 56.5.  12 and 4 heads of
    // 64, bf16 pages of 16: 64 x 64 (4.3e11) 8.0 and 11.1; of 64, 300 x 50 (4.9e12) 33.2 and 25.9.
    const double token_bytes = (double)a.lists * cache.d * (dtype == LSA_F32 ? 4 : 2);
    const double unit_bytes = token_bytes * std::min<int64_t>(cache.page, n / cache.batch);
    const bool pages = n >= 10 * cache.batch && unit_bytes * (token_bytes * n) >= 5e11;
    if (cache.d == 128)
        return dtype == LSA_F32 ? launch_ct<128, float>(a, cache.dtype, units, pages, s)
                                : launch_ct<128, __nv_bfloat16>(a, cache.dtype, units, pages, s);
    return dtype == LSA_F32 ? launch_ct<64, float>(a, cache.dtype, units, pages, s)
                            : launch_ct<64, __nv_bfloat16>(a, cache.dtype, units, pages, s);
}

}  // namespace lsa
