// Norm and rotation of the heads of queries and keys. With r = (mean(x^2) + eps)^-1/2,
// n = r x, z = n w (z = x without a weight) and c, s the cosine and sine of a
// pair's angle times the magnitude:
//   forward    y1 = c z1 - s z2, y2 = c z2 + s z1 for the pairs, y = z behind them
//   backward   g1 = c dy1 + s dy2, g2 = c dy2 - s dy1 (the transpose), g = dy behind;
//              dw = sum over rows of g n, u = g w, dx = r (u - n mean(u n)); dx = g
// The angle of position p is p f turns, f < 1 in units of 2^-64: one 64-bit integer
// product, whose wrap is the reduction mod a turn, so a far position costs no accuracy.
//
// A lane holds 16 elements of a row, eight pairs: two wide loads of 8 elements
// (the lanes of a row read adjacent ones), no exchange for the rotation, and a
// shuffle over the row's lanes for the norm's sum. A warp takes a few heads of a token
// (of several where a token has few), UN rows for each of its groups of lanes: it asks for
// all of them first and works out the angles, the same for all, while they come. One
// pass: every element is read once and written once.
#include "blocks.cuh"

namespace spmm {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kSms = 152;

struct HeadTensor {                  // one [B, T, heads, D] tensor and what becomes of it
    const void *x, *g;               // inputs; gradients of the results (backward)
    int64_t sb, st, sh, g_sb, g_st, g_sh;
    const void *w;
    void *out;                       // results, or gradients of the inputs
    int64_t o_sb, o_st, o_sh;
    int heads, at_once, tokens;      // heads of a token, and tokens, that a warp's rows are of
    unsigned chunks, items;          // warps' items per (group of tokens), in all
};

struct HeadArgs {
    HeadTensor t[2];                 // queries, keys
    const void *v;                   // append: the values, copied by the keys' warps
    void *v_out;
    int64_t v_sb, v_st, v_sh, vo_sb, vo_st, vo_sh;
    unsigned q_ctas;                 // the first CTAs are the queries'
    int all, T, D, R, lanes;         // B T; lanes of a row
    int w32;                         // weights are fp32
    float eps, magnitude, inv_D;
    const uint64_t *turns;
    const int32_t *positions, *lengths;
    int64_t p_sb, p_st;
    int Tk;                          // rows of the caches that k and v go to, or -1
    float *parts;                    // backward: [CTAs][D] parts of the weights' gradients
};

// Two floats to an instruction: the arithmetic of a row would else take longer to issue
// than the row takes to come.
using F2 = unsigned long long;
__device__ __forceinline__ F2 two(float lo, float hi) {
    F2 x;
    asm("mov.b64 %0, {%1, %2};" : "=l"(x) : "f"(lo), "f"(hi));
    return x;
}
__device__ __forceinline__ float2 both(F2 x) {
    float2 y;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(y.x), "=f"(y.y) : "l"(x));
    return y;
}
__device__ __forceinline__ F2 swap(F2 x) {
    const float2 y = both(x);
    return two(y.y, y.x);
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
    F2 x;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(x) : "l"(a), "l"(b), "l"(c));
    return x;
}
__device__ __forceinline__ F2 mul2(F2 a, F2 b) {
    F2 x;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(x) : "l"(a), "l"(b));
    return x;
}

// 16 elements as they lie in memory: 8 from one place and 8 from another. As floats,
// number i holds elements 2 i and 2 i + 1.
template <typename T> struct Raw {
    static constexpr int N = sizeof(T) / 2;        // 16-byte words of 8 elements
    uint4 w[2 * N];
    __device__ __forceinline__ void load(const T *lo, const T *hi) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            w[i] = __ldg((const uint4 *)lo + i);
            w[N + i] = __ldg((const uint4 *)hi + i);
        }
    }
    __device__ __forceinline__ void store(T *lo, T *hi) const {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            ((uint4 *)lo)[i] = w[i];
            ((uint4 *)hi)[i] = w[N + i];
        }
    }
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int i = 0; i < 2 * N; ++i) w[i] = make_uint4(0, 0, 0, 0);
    }
    __device__ __forceinline__ void get(F2 (&x)[8]) const {
        const T *e = reinterpret_cast<const T *>(w);
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = two(to_f32(e[2 * i]), to_f32(e[2 * i + 1]));
    }
    __device__ __forceinline__ void set(const F2 (&x)[8]) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float2 y = both(x[i]);
            if constexpr (sizeof(T) == 4)
                reinterpret_cast<float2 *>(w)[i] = y;
            else
                reinterpret_cast<uint32_t *>(w)[i] = pack2<T>(y.x, y.y);
        }
    }
};

// A lane's place: row `row` of the warp's rows at a time, and in it the 8 elements
// from `lo` and the 8 from `hi`. D and R are multiples of 16, so a lane's elements
// are all turned (its eight pairs) or none is.
struct HeadLane {
    int row, lo, hi;
    bool live, turned;
    __device__ __forceinline__ HeadLane(const HeadArgs &a, bool interleaved) {
        const int lane = threadIdx.x & 31, u = lane & (a.lanes - 1);
        row = lane / a.lanes;
        live = u * 16 < a.D;
        turned = u * 16 < a.R;
        lo = turned && !interleaved ? 8 * u : 16 * u;
        hi = turned && !interleaved ? a.R / 2 + 8 * u : 16 * u + 8;
    }
};

// Which token and first head the lane's rows are of; its u-th is at_once heads further.
struct HeadPlace {
    int64_t b;
    int t, head;
    bool live;
    __device__ __forceinline__ HeadPlace(const HeadArgs &a, const HeadTensor &h, const HeadLane &l,
                                         unsigned item, int un) {
        const unsigned group = item / h.chunks, chunk = item % h.chunks;
        const int64_t token = (int64_t)group * h.tokens + l.row / h.at_once;
        live = l.live && l.row < h.tokens * h.at_once && token < a.all;
        b = live ? (unsigned)token / (unsigned)a.T : 0;
        t = live ? (int)((unsigned)token % (unsigned)a.T) : 0;
        head = (int)chunk * un * h.at_once + l.row % h.at_once;
    }
    __device__ __forceinline__ int64_t position(const HeadArgs &a) const {
        if (!live) return 0;
        if (a.positions) return a.positions[b * a.p_sb + t * a.p_st];
        return (a.lengths ? (int64_t)a.lengths[b] - a.T : 0) + t;
    }
};

// Sines and cosines of the lane's pairs, times the magnitude (of pairs 2 i and 2 i + 1 in
// number i). The turn is cut to the nearest half (exactly, in integers) before it
// becomes a float. What is left, x of at most pi / 2, is off by 2^-24 of itself and goes
// into the two functions' power series, whose first terms left out, x^13 / 13! and
// x^14 / 14!, are below 2^-24.
__device__ __forceinline__ void angles(const HeadArgs &a, const HeadLane &l, bool interleaved,
                                       int64_t pos, F2 (&c)[4], F2 (&s)[4]) {
    const ulonglong2 *f = (const ulonglong2 *)(a.turns + (interleaved ? l.lo / 2 : l.lo));
    auto all = [](float x) { return two(x, x); };
    const F2 unit = all(1.46291807926716e-9f), size = all(a.magnitude);      // 2 pi / 2^32
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const ulonglong2 t2 = __ldg(f + i);
        const uint32_t t0 = (uint32_t)(((uint64_t)pos * t2.x) >> 32);
        const uint32_t t1 = (uint32_t)(((uint64_t)pos * t2.y) >> 32);
        // the sign of both functions: whether the nearest half turn is an odd one
        const uint32_t odd0 = (t0 + (1u << 30)) & (1u << 31), odd1 = (t1 + (1u << 30)) & (1u << 31);
        const F2 x = mul2(two((float)(int32_t)(t0 ^ odd0), (float)(int32_t)(t1 ^ odd1)), unit);
        const F2 y = mul2(x, x);
        F2 sx = fma2(y, all(-1.0f / 39916800), all(1.0f / 362880));
        sx = fma2(y, sx, all(-1.0f / 5040));
        sx = fma2(y, sx, all(1.0f / 120));
        sx = fma2(y, sx, all(-1.0f / 6));
        sx = fma2(mul2(x, y), sx, x);
        F2 cx = fma2(y, all(1.0f / 479001600), all(-1.0f / 3628800));
        cx = fma2(y, cx, all(1.0f / 40320));
        cx = fma2(y, cx, all(-1.0f / 720));
        cx = fma2(y, cx, all(1.0f / 24));
        cx = fma2(y, cx, all(-0.5f));
        cx = fma2(y, cx, all(1.0f));
        const F2 odd = (F2)odd1 << 32 | odd0;
        s[i] = mul2(sx, size) ^ odd;
        c[i] = mul2(cx, size) ^ odd;
    }
}

// z by its matrix: element i of a pair times a, and its partner times b.
template <bool INTER>
__device__ __forceinline__ void by_matrix(F2 (&z)[8], const F2 (&a)[8], const F2 (&b)[8]) {
    if constexpr (INTER) {
#pragma unroll
        for (int i = 0; i < 8; ++i) z[i] = fma2(swap(z[i]), b[i], mul2(z[i], a[i]));
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const F2 x = z[i], y = z[4 + i];
            z[i] = fma2(y, b[i], mul2(x, a[i]));
            z[4 + i] = fma2(x, b[4 + i], mul2(y, a[4 + i]));
        }
    }
}

// That matrix for w, then the turn by the angles; w of 1 and back: the transposed turn.
template <bool INTER>
__device__ __forceinline__ void matrix(const F2 (&c)[4], const F2 (&s)[4], const F2 (&w)[8],
                                       bool back, F2 (&a)[8], F2 (&b)[8]) {
    const float minus = back ? 1.0f : -1.0f;
    if constexpr (INTER) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float2 cc = both(c[i / 2]), ss = both(s[i / 2]), ww = both(w[i]);
            const float ci = i & 1 ? cc.y : cc.x, si = i & 1 ? ss.y : ss.x;
            a[i] = two(ww.x * ci, ww.y * ci);
            b[i] = two(minus * ww.y * si, -minus * ww.x * si);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            a[i] = mul2(w[i], c[i]);
            a[4 + i] = mul2(w[4 + i], c[i]);
            b[i] = mul2(mul2(w[4 + i], s[i]), two(minus, minus));
            b[4 + i] = mul2(mul2(w[i], s[i]), two(-minus, -minus));
        }
    }
}

__device__ __forceinline__ float row_sum(float x, int lanes) {
    for (int o = 1; o < lanes; o <<= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

// The lane's part of a weight; 1 without one.
template <typename T>
__device__ __forceinline__ void load_weight(const HeadArgs &a, const HeadLane &l, const void *w,
                                            F2 (&x)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = two(1.0f, 1.0f);
    if (!l.live || !w) return;
    if (a.w32) {
        Raw<float> r;
        r.load((const float *)w + l.lo, (const float *)w + l.hi);
        r.get(x);
    } else {
        Raw<T> r;
        r.load((const T *)w + l.lo, (const T *)w + l.hi);
        r.get(x);
    }
}

template <typename T, bool INTER, int UN>
__global__ void __launch_bounds__(kThreads, 2) k_heads_rotate(const __grid_constant__ HeadArgs a) {
    const HeadLane l(a, INTER);
    const bool keys = blockIdx.x >= a.q_ctas;
    const HeadTensor &h = a.t[keys];
    const unsigned item = (blockIdx.x - (keys ? a.q_ctas : 0)) * kWarps + threadIdx.x / 32;
    if (item >= h.items) return;
    const HeadPlace at(a, h, l, item, UN);
    Raw<T> x[UN];
    bool live[UN];
    const T *from = (const T *)h.x + at.b * h.sb + at.t * h.st + at.head * h.sh;
#pragma unroll
    for (int u = 0; u < UN; ++u) {
        live[u] = at.live && at.head + u * h.at_once < h.heads;
        const T *p = from + u * h.at_once * h.sh;
        if (live[u]) x[u].load(p + l.lo, p + l.hi);
        else x[u].zero();
    }
    const int64_t pos = at.position(a);
    const bool cached = keys && a.Tk >= 0, put = !cached || (pos >= 0 && pos < a.Tk);
    const int64_t row = cached ? pos : at.t;
    F2 w[8], ma[8], mb[8];
    load_weight<T>(a, l, h.w, w);
    if (l.turned) {
        F2 c[4], s[4];
        angles(a, l, INTER, pos, c, s);
        matrix<INTER>(c, s, w, false, ma, mb);
    }
    T *to = (T *)h.out + at.b * h.o_sb + row * h.o_st + at.head * h.o_sh;
#pragma unroll
    for (int u = 0; u < UN; ++u) {
        if (u * h.at_once >= h.heads) break;     // no lane has one more
        F2 z[8];
        x[u].get(z);
        if (h.w) {
            F2 sum = mul2(z[0], z[0]);
#pragma unroll
            for (int i = 1; i < 8; ++i) sum = fma2(z[i], z[i], sum);
            const float2 t = both(sum);
            const float r = rsqrtf(fmaf(row_sum(t.x + t.y, a.lanes), a.inv_D, a.eps));
#pragma unroll
            for (int i = 0; i < 8; ++i) z[i] = mul2(z[i], two(r, r));
        }
        if (l.turned) {
            by_matrix<INTER>(z, ma, mb);
        } else if (h.w) {
#pragma unroll
            for (int i = 0; i < 8; ++i) z[i] = mul2(z[i], w[i]);
        }
        x[u].set(z);
        T *p = to + u * h.at_once * h.o_sh;
        if (live[u] && put) x[u].store(p + l.lo, p + l.hi);
    }
    if (!cached || !put) return;
    const T *v = (const T *)a.v + at.b * a.v_sb + at.t * a.v_st + at.head * a.v_sh;
    T *v_to = (T *)a.v_out + at.b * a.vo_sb + pos * a.vo_st + at.head * a.vo_sh;
#pragma unroll
    for (int u = 0; u < UN; ++u) {
        const T *p = v + u * h.at_once * a.v_sh;
        if (live[u]) x[u].load(p + l.lo, p + l.hi);
    }
#pragma unroll
    for (int u = 0; u < UN; ++u) {
        T *p = v_to + u * h.at_once * a.vo_sh;
        if (live[u]) x[u].store(p + l.lo, p + l.hi);
    }
}

// The weights' gradients: a lane's sums over its rows, then over the rows of the
// warp, the warps of the CTA and, by a second kernel, the CTAs, each in a fixed order.
template <typename T, bool INTER, int UN>
__global__ void __launch_bounds__(kThreads, 2) k_heads_backward(const __grid_constant__ HeadArgs a) {
    __shared__ float sums[kWarps][256];
    const HeadLane l(a, INTER);
    const int warp = threadIdx.x / 32, lane = threadIdx.x & 31;
    const bool keys = blockIdx.x >= a.q_ctas;
    const HeadTensor &h = a.t[keys];
    const unsigned ctas = keys ? gridDim.x - a.q_ctas : a.q_ctas;
    F2 w[8], dw[8];
    load_weight<T>(a, l, h.w, w);
#pragma unroll
    for (int i = 0; i < 8; ++i) dw[i] = two(0.0f, 0.0f);
    for (uint64_t item = (uint64_t)(blockIdx.x - (keys ? a.q_ctas : 0)) * kWarps + warp;
         item < h.items; item += (uint64_t)ctas * kWarps) {
        const HeadPlace at(a, h, l, (unsigned)item, UN);
        Raw<T> g[UN], x[UN];
        bool live[UN];
        const T *gs = (const T *)h.g + at.b * h.g_sb + at.t * h.g_st + at.head * h.g_sh;
        const T *xs = (const T *)h.x + at.b * h.sb + at.t * h.st + at.head * h.sh;
#pragma unroll
        for (int u = 0; u < UN; ++u) {
            live[u] = at.live && at.head + u * h.at_once < h.heads;
            g[u].zero();
            x[u].zero();
            if (!live[u]) continue;
            const T *p = gs + u * h.at_once * h.g_sh;
            g[u].load(p + l.lo, p + l.hi);
            p = xs + u * h.at_once * h.sh;
            if (h.w) x[u].load(p + l.lo, p + l.hi);
        }
        F2 ma[8], mb[8];
        if (l.turned) {
            F2 c[4], s[4], ones[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) ones[i] = two(1.0f, 1.0f);
            angles(a, l, INTER, at.position(a), c, s);
            matrix<INTER>(c, s, ones, true, ma, mb);
        }
        T *to = (T *)h.out + at.b * h.o_sb + at.t * h.o_st + at.head * h.o_sh;
#pragma unroll
        for (int u = 0; u < UN; ++u) {
            if (u * h.at_once >= h.heads) break;
            F2 y[8];
            g[u].get(y);
            if (l.turned) by_matrix<INTER>(y, ma, mb);
            if (h.w) {
                F2 z[8], sums = two(0.0f, 0.0f), dots = sums;
                x[u].get(z);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    sums = fma2(z[i], z[i], sums);
                    dots = fma2(mul2(y[i], w[i]), z[i], dots);
                }
                float2 t = both(sums);
                float sum = t.x + t.y;
                t = both(dots);
                float dot = t.x + t.y;
                for (int o = 1; o < a.lanes; o <<= 1) {
                    sum += __shfl_xor_sync(0xffffffffu, sum, o);
                    dot += __shfl_xor_sync(0xffffffffu, dot, o);
                }
                const float r = rsqrtf(fmaf(sum, a.inv_D, a.eps));
                const float m = -dot * r * a.inv_D;        // -mean(u n)
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const F2 n = mul2(z[i], two(r, r));
                    dw[i] = fma2(y[i], n, dw[i]);
                    y[i] = mul2(two(r, r), fma2(n, two(m, m), mul2(y[i], w[i])));
                }
            }
            g[u].set(y);
            T *p = to + u * h.at_once * h.o_sh;
            if (live[u]) g[u].store(p + l.lo, p + l.hi);
        }
    }
    if (!h.w) return;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        float2 t = both(dw[i]);
        for (int o = a.lanes; o < 32; o <<= 1) {
            t.x += __shfl_xor_sync(0xffffffffu, t.x, o);
            t.y += __shfl_xor_sync(0xffffffffu, t.y, o);
        }
        if (lane < a.lanes && l.live) {
            const int at = (i < 4 ? l.lo : l.hi) + 2 * (i & 3);
            sums[warp][at] = t.x;
            sums[warp][at + 1] = t.y;
        }
    }
    __syncthreads();
    if ((int)threadIdx.x < a.D) {
        float x = 0.0f;
        for (int i = 0; i < kWarps; ++i) x += sums[i][threadIdx.x];
        a.parts[(int64_t)blockIdx.x * a.D + threadIdx.x] = x;
    }
}

// A weight's gradient is the sum of its tensor's CTAs' parts: 32 columns a CTA, its warps
// in turn over the parts; CTAs y = 0 for the queries', 1 for the keys'.
__global__ void __launch_bounds__(1024) k_heads_weights(const float *parts, int q_ctas, int ctas,
                                                        int D, int w32, int half, void *dwq,
                                                        void *dwk) {
    __shared__ float sums[32][33];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int j = blockIdx.x * 32 + lane;
    void *out = blockIdx.y ? dwk : dwq;
    if (!out) return;
    const int end = blockIdx.y ? ctas : q_ctas;
    float x = 0.0f;
    if (j < D)
        for (int i = (blockIdx.y ? q_ctas : 0) + warp; i < end; i += 32) x += parts[(int64_t)i * D + j];
    sums[warp][lane] = x;
    __syncthreads();
    if (warp || j >= D) return;
    x = 0.0f;
#pragma unroll
    for (int i = 0; i < 32; ++i) x += sums[i][lane];
    if (w32) ((float *)out)[j] = x;
    else if (half) ((__half *)out)[j] = from_f32<__half>(x);
    else ((__nv_bfloat16 *)out)[j] = from_f32<__nv_bfloat16>(x);
}

// ------------------------------------------------------------------- host
spmm_status heads_check(const spmm_heads_shape *s) {
    if (!s || s->B < 0 || s->T < 0 || s->Hq < 0 || s->Hk < 0 || s->D < 1 || s->R < 0 || s->R > s->D)
        return SPMM_ERR_INVALID_ARG;
    if (!dtype_ok(s->dtype) || (s->weight_dtype != SPMM_F32 && s->weight_dtype != s->dtype))
        return SPMM_ERR_INVALID_ARG;
    if (s->positions && s->lengths) return SPMM_ERR_INVALID_ARG;
    if ((uintptr_t)s->wq % 16 || (uintptr_t)s->wk % 16) return SPMM_ERR_INVALID_ARG;
    if (s->D % 16 || s->R % 16 || s->D > 256) return SPMM_ERR_UNSUPPORTED;
    if (s->T > (1 << 26) || s->Hq > 65535 || s->Hk > 65535 || s->B > INT32_MAX)
        return SPMM_ERR_UNSUPPORTED;
    if (s->B && (s->Hq + s->Hk) * std::max<int64_t>(s->T, 1) > (int64_t)INT32_MAX / s->B)
        return SPMM_ERR_UNSUPPORTED;
    if (s->R && (!s->turns || (uintptr_t)s->turns % 16)) return SPMM_ERR_INVALID_ARG;
    return SPMM_OK;
}

bool heads_empty(const spmm_heads_shape *s) { return !s->B || !s->T || !(s->Hq + s->Hk); }

void contiguous_out(HeadTensor &h, void *out, const spmm_heads_shape *s) {
    h.out = out;
    h.o_sh = s->D;
    h.o_st = h.heads * s->D;
    h.o_sb = s->T * h.o_st;
}

// Rows of 16-byte words that a lane asks for at a time: 128 bytes of them.
constexpr int kForwardRows = 8, kBackwardRows = 4;   // over the element's bytes

HeadArgs heads_args(const spmm_heads_shape *s, int rows) {
    HeadArgs a{};
    a.all = (int)(s->B * s->T);
    a.T = (int)s->T;
    a.D = (int)s->D;
    a.R = (int)s->R;
    a.lanes = 1;
    while (a.lanes * 16 < a.D) a.lanes *= 2;
    a.w32 = s->weight_dtype == SPMM_F32;
    a.eps = s->eps;
    a.magnitude = s->magnitude;
    a.inv_D = 1.0f / (float)s->D;
    a.turns = s->turns;
    a.positions = s->positions;
    a.p_sb = s->p_sb;
    a.p_st = s->p_st;
    a.lengths = s->lengths;
    a.Tk = -1;
    const int groups = 32 / a.lanes, un = rows / dtype_bytes(s->dtype);
    for (int i = 0; i < 2; ++i) {
        HeadTensor &h = a.t[i];
        h.heads = (int)(i ? s->Hk : s->Hq);
        h.w = i ? s->wk : s->wq;
        h.at_once = std::max(1, std::min(h.heads, groups));
        h.tokens = groups / h.at_once;
        h.chunks = (unsigned)((h.heads + un * h.at_once - 1) / (un * h.at_once));
        h.items = (unsigned)(((int64_t)a.all + h.tokens - 1) / h.tokens) * h.chunks;
    }
    return a;
}

unsigned warps_ctas(unsigned items) { return items / kWarps + (items % kWarps > 0); }

// Two CTAs to an SM stay (their sums do), in proportion to the tensors' elements.
void backward_grid(HeadArgs &a, unsigned &grid) {
    const double q = (double)a.t[0].heads, k = (double)a.t[1].heads;
    const unsigned most = 2 * kSms;
    unsigned n[2] = {(unsigned)(most * q / (q + k) + 0.5), 0};
    if (k > 0) n[0] = std::min(n[0], most - 1);
    if (q > 0) n[0] = std::max(n[0], 1u);
    n[1] = most - n[0];
    for (int i = 0; i < 2; ++i) n[i] = std::min(n[i], warps_ctas(a.t[i].items));
    a.q_ctas = n[0];
    grid = n[0] + n[1];
}

template <template <typename, bool> class K>
cudaError_t launch_heads(const spmm_heads_shape *s, const HeadArgs &a, unsigned grid,
                         cudaStream_t cs) {
    if (s->dtype == SPMM_F32)
        s->interleaved ? K<float, true>::go(a, grid, cs) : K<float, false>::go(a, grid, cs);
    else if (s->dtype == SPMM_BF16)
        s->interleaved ? K<__nv_bfloat16, true>::go(a, grid, cs)
                       : K<__nv_bfloat16, false>::go(a, grid, cs);
    else
        s->interleaved ? K<__half, true>::go(a, grid, cs) : K<__half, false>::go(a, grid, cs);
    count_launch();
    return cudaGetLastError();
}
template <typename T, bool INTER> struct Rotate {
    static void go(const HeadArgs &a, unsigned grid, cudaStream_t cs) {
        k_heads_rotate<T, INTER, kForwardRows / (int)sizeof(T)><<<grid, kThreads, 0, cs>>>(a);
    }
};
template <typename T, bool INTER> struct Backward {
    static void go(const HeadArgs &a, unsigned grid, cudaStream_t cs) {
        k_heads_backward<T, INTER, kBackwardRows / (int)sizeof(T)><<<grid, kThreads, 0, cs>>>(a);
    }
};

cudaError_t rotate(const spmm_heads_shape *s, HeadArgs &a, void *stream) {
    a.q_ctas = warps_ctas(a.t[0].items);
    return launch_heads<Rotate>(s, a, a.q_ctas + warps_ctas(a.t[1].items), (cudaStream_t)stream);
}

bool written_ok(const spmm_rows &r, int64_t e, const spmm_heads_shape *s, int64_t Tk) {
    // rows that two tokens share (stride 0) would be written twice
    return rows_ok(r, e) && (s->B == 1 || r.sb > 0) && (Tk <= 1 || r.st > 0) &&
           (s->Hk == 1 || r.sh > 0);
}

}  // namespace
}  // namespace spmm

extern "C" {

spmm_status spmm_heads_rotate(const spmm_heads_shape *s, spmm_rows q, spmm_rows k, void *q_out,
                              void *k_out, void *stream) {
    using namespace spmm;
    const spmm_status st = heads_check(s);
    if (st != SPMM_OK) return st;
    if (heads_empty(s)) return SPMM_OK;
    const int e = dtype_bytes(s->dtype);
    if (s->Hq && (!rows_ok(q, e) || !q_out || (uintptr_t)q_out % 16)) return SPMM_ERR_INVALID_ARG;
    if (s->Hk && (!rows_ok(k, e) || !k_out || (uintptr_t)k_out % 16)) return SPMM_ERR_INVALID_ARG;
    HeadArgs a = heads_args(s, kForwardRows);
    set_rows(a.t[0].x, a.t[0].sb, a.t[0].st, a.t[0].sh, q);
    set_rows(a.t[1].x, a.t[1].sb, a.t[1].st, a.t[1].sh, k);
    contiguous_out(a.t[0], q_out, s);
    contiguous_out(a.t[1], k_out, s);
    return cuda_status(rotate(s, a, stream));
}

spmm_status spmm_heads_append(const spmm_heads_shape *s, spmm_rows q, spmm_rows k, spmm_rows v,
                              void *q_out, spmm_rows cache_k, spmm_rows cache_v, int64_t Tk,
                              void *stream) {
    using namespace spmm;
    const spmm_status st = heads_check(s);
    if (st != SPMM_OK) return st;
    if (!s->lengths || s->positions || Tk < 0 || s->Hk < 1) return SPMM_ERR_INVALID_ARG;
    if (Tk > (1 << 26)) return SPMM_ERR_UNSUPPORTED;
    if (heads_empty(s)) return SPMM_OK;
    const int e = dtype_bytes(s->dtype);
    if (s->Hq && (!rows_ok(q, e) || !q_out || (uintptr_t)q_out % 16)) return SPMM_ERR_INVALID_ARG;
    if (!rows_ok(k, e) || !rows_ok(v, e)) return SPMM_ERR_INVALID_ARG;
    if (Tk && (!written_ok(cache_k, e, s, Tk) || !written_ok(cache_v, e, s, Tk)))
        return SPMM_ERR_INVALID_ARG;
    HeadArgs a = heads_args(s, kForwardRows);
    set_rows(a.t[0].x, a.t[0].sb, a.t[0].st, a.t[0].sh, q);
    set_rows(a.t[1].x, a.t[1].sb, a.t[1].st, a.t[1].sh, k);
    contiguous_out(a.t[0], q_out, s);
    set_rows(a.v, a.v_sb, a.v_st, a.v_sh, v);
    a.Tk = (int)Tk;
    a.t[1].out = const_cast<void *>(cache_k.data);
    a.t[1].o_sb = cache_k.sb, a.t[1].o_st = cache_k.st, a.t[1].o_sh = cache_k.sh;
    a.v_out = const_cast<void *>(cache_v.data);
    a.vo_sb = cache_v.sb, a.vo_st = cache_v.st, a.vo_sh = cache_v.sh;
    return cuda_status(rotate(s, a, stream));
}

int64_t spmm_heads_backward_workspace(const spmm_heads_shape *s) {
    using namespace spmm;
    if (heads_check(s) != SPMM_OK || heads_empty(s) || (!s->wq && !s->wk)) return 0;
    HeadArgs a = heads_args(s, kBackwardRows);
    unsigned grid;
    backward_grid(a, grid);
    return grid * s->D * (int64_t)sizeof(float);
}

spmm_status spmm_heads_rotate_backward(const spmm_heads_shape *s, spmm_rows grad_q,
                                       spmm_rows grad_k, spmm_rows q, spmm_rows k, void *dq,
                                       void *dk, void *dwq, void *dwk, void *work,
                                       int64_t work_bytes, void *stream) {
    using namespace spmm;
    const spmm_status st = heads_check(s);
    if (st != SPMM_OK) return st;
    if ((s->wq && !dwq) || (s->wk && !dwk)) return SPMM_ERR_INVALID_ARG;
    const int e = dtype_bytes(s->dtype);
    cudaStream_t cs = (cudaStream_t)stream;
    if (heads_empty(s)) {
        const size_t n = s->D * (size_t)dtype_bytes(s->weight_dtype);
        cudaError_t err = cudaSuccess;
        if (s->wq) err = cudaMemsetAsync(dwq, 0, n, cs);
        if (err == cudaSuccess && s->wk) err = cudaMemsetAsync(dwk, 0, n, cs);
        return cuda_status(err);
    }
    if (s->Hq && (!rows_ok(grad_q, e) || !dq || (uintptr_t)dq % 16 || (s->wq && !rows_ok(q, e))))
        return SPMM_ERR_INVALID_ARG;
    if (s->Hk && (!rows_ok(grad_k, e) || !dk || (uintptr_t)dk % 16 || (s->wk && !rows_ok(k, e))))
        return SPMM_ERR_INVALID_ARG;
    const int64_t need = spmm_heads_backward_workspace(s);
    if (need && (!work || work_bytes < need || (uintptr_t)work % 16)) return SPMM_ERR_INVALID_ARG;
    HeadArgs a = heads_args(s, kBackwardRows);
    set_rows(a.t[0].x, a.t[0].sb, a.t[0].st, a.t[0].sh, q);
    set_rows(a.t[1].x, a.t[1].sb, a.t[1].st, a.t[1].sh, k);
    set_rows(a.t[0].g, a.t[0].g_sb, a.t[0].g_st, a.t[0].g_sh, grad_q);
    set_rows(a.t[1].g, a.t[1].g_sb, a.t[1].g_st, a.t[1].g_sh, grad_k);
    contiguous_out(a.t[0], dq, s);
    contiguous_out(a.t[1], dk, s);
    a.parts = need ? (float *)work : nullptr;
    unsigned grid;
    backward_grid(a, grid);
    cudaError_t err = launch_heads<Backward>(s, a, grid, cs);
    if (err == cudaSuccess && need) {
        k_heads_weights<<<dim3((unsigned)((s->D + 31) / 32), 2), 1024, 0, cs>>>(
            a.parts, (int)a.q_ctas, (int)grid, a.D, a.w32, s->dtype == SPMM_F16, s->wq ? dwq : nullptr,
            s->wk ? dwk : nullptr);
        count_launch();
        err = cudaGetLastError();
    }
    return cuda_status(err);
}

}  // extern "C"
