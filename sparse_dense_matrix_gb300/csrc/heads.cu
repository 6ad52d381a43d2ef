// Norm and rotation of the heads of queries and keys. With r = (mean(x^2) + eps)^-1/2,
// n = r x, z = n w (z = x without a weight) and c, s the cosine and sine of a
// pair's angle times the magnitude:
//   forward    y1 = c z1 - s z2, y2 = c z2 + s z1 for the pairs, y = z behind them
//   backward   g1 = c dy1 + s dy2, g2 = c dy2 - s dy1 (the transpose), g = dy behind;
//              dw = sum over rows of g n, u = g w, dx = r (u - n mean(u n)); dx = g
// The angle of position p is p f turns, f < 1 in units of 2^-64: one 64-bit integer
// product, whose wrap is the reduction mod a turn, so a far position costs no accuracy.
//
// A lane holds 16 elements of a row, eight pairs: two wide loads each 8 elements
// (the lanes of a row read adjacent ones), no exchange for the rotation, and a
// shuffle over the row's lanes for the norm's sum. A warp takes a token: the eight
// sines and cosines of a lane are formed once for all of the token's heads of
// queries and keys. One pass: every element is read once and written once.
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
    int heads;
};

struct HeadArgs {
    HeadTensor q, k, v;              // v: copied (append)
    int64_t tokens;                  // B T
    int T, D, R, lanes, splits;      // lanes of a row; warps per token
    int w32;                         // weights are fp32
    float eps, magnitude;
    const uint64_t *turns;
    const int32_t *positions, *lengths;
    int64_t p_sb, p_st;
    int Tk;                          // rows of the caches that k and v go to, or -1
    float *parts;                    // backward: [CTAs][2][D] parts of the weights' gradients
};

template <typename T> __device__ __forceinline__ void load8(const T *p, float *x) {
    if constexpr (sizeof(T) == 4) {
        const float4 a = *(const float4 *)p, b = *(const float4 *)(p + 4);
        x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w;
        x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
    } else {
        float y[8];
        ld_pack<T, 8>(p, y);
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = y[i];
    }
}

template <typename T> __device__ __forceinline__ void store8(T *p, const float *x) {
    if constexpr (sizeof(T) == 4) {
        *(float4 *)p = make_float4(x[0], x[1], x[2], x[3]);
        *(float4 *)(p + 4) = make_float4(x[4], x[5], x[6], x[7]);
    } else {
        float y[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = x[i];
        st_pack<T, 8>(p, y);
    }
}

// A lane's place: row `row` of the warp's rows at a time, and in it the 8 elements
// from `lo` and the 8 from `hi`. D and R are multiples of 16, so a lane's elements
// are all turned (its eight pairs) or none is.
struct HeadLane {
    int row, rows, lo, hi;
    bool live, turned;
    __device__ __forceinline__ HeadLane(const HeadArgs &a, bool interleaved) {
        const int lane = threadIdx.x & 31, u = lane & (a.lanes - 1);
        rows = 32 / a.lanes;
        row = lane / a.lanes;
        live = u * 16 < a.D;
        turned = u * 16 < a.R;
        lo = turned && !interleaved ? 8 * u : 16 * u;
        hi = turned && !interleaved ? a.R / 2 + 8 * u : 16 * u + 8;
    }
};

// Sines and cosines of the lane's pairs. The turn is cut to the nearest quarter
// (exactly, in integers) before it becomes a float: the rest, at most an eighth of a
// turn, is off by 2^-27 of pi at most.
__device__ __forceinline__ void angles(const HeadArgs &a, const HeadLane &l, bool interleaved,
                                       int64_t pos, float (&c)[8], float (&s)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        c[i] = 1.0f;
        s[i] = 0.0f;
    }
    if (!l.turned) return;
    const uint64_t *f = a.turns + (interleaved ? l.lo / 2 : l.lo);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const uint32_t t = (uint32_t)(((uint64_t)pos * __ldg(f + i)) >> 32);
        const uint32_t quarter = (t + (1u << 29)) >> 30;
        float x, y;
        sincospif((float)(int32_t)(t - (quarter << 30)) * 0x1p-31f, &y, &x);
        const float cc = quarter & 1 ? y : x, ss = quarter & 1 ? x : y;
        c[i] = ((quarter + 1) & 2 ? -cc : cc) * a.magnitude;
        s[i] = (quarter & 2 ? -ss : ss) * a.magnitude;
    }
}

// Turned by the angles (back: by their negatives).
template <bool INTER>
__device__ __forceinline__ void turn(float (&z)[16], const float (&c)[8], const float (&s)[8],
                                     bool back) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        float &p = z[INTER ? 2 * i : i], &q = z[INTER ? 2 * i + 1 : 8 + i];
        const float sn = back ? -s[i] : s[i], x = p, y = q;
        p = x * c[i] - y * sn;
        q = y * c[i] + x * sn;
    }
}

__device__ __forceinline__ float row_sum(float x, int lanes) {
    for (int o = 1; o < lanes; o <<= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

template <typename T>
__device__ __forceinline__ void load_weight(const HeadArgs &a, const HeadLane &l, const void *w,
                                            float (&x)[16]) {
#pragma unroll
    for (int i = 0; i < 16; ++i) x[i] = 0.0f;
    if (!l.live || !w) return;
    if (a.w32) {
        load8((const float *)w + l.lo, x);
        load8((const float *)w + l.hi, x + 8);
    } else {
        load8((const T *)w + l.lo, x);
        load8((const T *)w + l.hi, x + 8);
    }
}

// Heads of one token: rows split * rows + row, then splits * rows further.
template <typename T, bool INTER, bool NORM>
__device__ __forceinline__ void forward_heads(const HeadArgs &a, const HeadTensor &h,
                                              const HeadLane &l, int split, const T *x, T *out,
                                              const float (&c)[8], const float (&s)[8]) {
    float w[16];
    if (NORM) load_weight<T>(a, l, h.w, w);
    const int step = a.splits * l.rows;
    for (int base = split * l.rows; base < h.heads; base += step) {
        const int at = base + l.row;
        const bool live = l.live && at < h.heads;
        float z[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) z[i] = 0.0f;
        if (live) {
            load8(x + at * h.sh + l.lo, z);
            load8(x + at * h.sh + l.hi, z + 8);
        }
        if (NORM) {
            float sum = 0.0f;
#pragma unroll
            for (int i = 0; i < 16; ++i) sum = fmaf(z[i], z[i], sum);
            const float r = rsqrtf(row_sum(sum, a.lanes) / (float)a.D + a.eps);
#pragma unroll
            for (int i = 0; i < 16; ++i) z[i] = z[i] * r * w[i];
        }
        if (l.turned) turn<INTER>(z, c, s, false);
        if (live) {
            store8(out + at * h.o_sh + l.lo, z);
            store8(out + at * h.o_sh + l.hi, z + 8);
        }
    }
}

__device__ __forceinline__ int64_t position(const HeadArgs &a, int64_t b, int t) {
    if (a.positions) return a.positions[b * a.p_sb + t * a.p_st];
    return (a.lengths ? (int64_t)a.lengths[b] - a.T : 0) + t;
}

template <typename T, bool INTER>
__global__ void __launch_bounds__(kThreads) k_heads_rotate(const HeadArgs a) {
    const HeadLane l(a, INTER);
    const int64_t items = a.tokens * a.splits;
    for (int64_t i = (int64_t)blockIdx.x * kWarps + threadIdx.x / 32; i < items;
         i += (int64_t)gridDim.x * kWarps) {
        const int64_t token = i / a.splits, b = token / a.T;
        const int split = (int)(i % a.splits), t = (int)(token % a.T);
        const int64_t pos = position(a, b, t);
        float c[8], s[8];
        angles(a, l, INTER, pos, c, s);
        auto heads = [&](const HeadTensor &h, int64_t row) {
            const T *x = (const T *)h.x + b * h.sb + t * h.st;
            T *out = (T *)h.out + b * h.o_sb + row * h.o_st;
            if (h.w) forward_heads<T, INTER, true>(a, h, l, split, x, out, c, s);
            else forward_heads<T, INTER, false>(a, h, l, split, x, out, c, s);
        };
        heads(a.q, t);
        if (a.Tk < 0) {
            heads(a.k, t);
        } else if (pos >= 0 && pos < a.Tk) {
            heads(a.k, pos);
            const T *x = (const T *)a.v.x + b * a.v.sb + t * a.v.st;
            T *out = (T *)a.v.out + b * a.v.o_sb + pos * a.v.o_st;
            constexpr int V = 16 / sizeof(T);
            const int n = a.D / V;
            for (int j = split * 32 + (threadIdx.x & 31); j < a.v.heads * n; j += a.splits * 32)
                *(uint4 *)(out + j / n * a.v.o_sh + j % n * V) =
                    *(const uint4 *)(x + j / n * a.v.sh + j % n * V);
        }
    }
}

template <typename T, bool INTER, bool NORM>
__device__ __forceinline__ void backward_heads(const HeadArgs &a, const HeadTensor &h,
                                               const HeadLane &l, int split, const T *g, const T *x,
                                               T *out, const float (&c)[8], const float (&s)[8],
                                               float (&dw)[16]) {
    float w[16];
    if (NORM) load_weight<T>(a, l, h.w, w);
    const int step = a.splits * l.rows;
    for (int base = split * l.rows; base < h.heads; base += step) {
        const int at = base + l.row;
        const bool live = l.live && at < h.heads;
        float u[16], z[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) u[i] = z[i] = 0.0f;
        if (live) {
            load8(g + at * h.g_sh + l.lo, u);
            load8(g + at * h.g_sh + l.hi, u + 8);
            if (NORM) {
                load8(x + at * h.sh + l.lo, z);
                load8(x + at * h.sh + l.hi, z + 8);
            }
        }
        if (l.turned) turn<INTER>(u, c, s, true);
        if (NORM) {
            float sum = 0.0f, dot = 0.0f;
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                sum = fmaf(z[i], z[i], sum);
                dot = fmaf(u[i] * w[i], z[i], dot);
            }
            const float r = rsqrtf(row_sum(sum, a.lanes) / (float)a.D + a.eps);
            const float m = row_sum(dot, a.lanes) * r / (float)a.D;    // mean(u n)
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const float n = z[i] * r;
                dw[i] = fmaf(u[i], n, dw[i]);
                u[i] = r * (u[i] * w[i] - n * m);
            }
        }
        if (live) {
            store8(out + at * h.o_sh + l.lo, u);
            store8(out + at * h.o_sh + l.hi, u + 8);
        }
    }
}

// The weights' gradients: a lane's sums over its rows, then over the rows of the
// warp, the warps of the CTA and, by a second kernel, the CTAs, each in a fixed order.
template <typename T, bool INTER>
__global__ void __launch_bounds__(kThreads) k_heads_backward(const HeadArgs a) {
    __shared__ float sums[kWarps][256];
    const HeadLane l(a, INTER);
    const int warp = threadIdx.x / 32, lane = threadIdx.x & 31;
    float dwq[16], dwk[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) dwq[i] = dwk[i] = 0.0f;
    const int64_t items = a.tokens * a.splits;
    for (int64_t i = (int64_t)blockIdx.x * kWarps + warp; i < items;
         i += (int64_t)gridDim.x * kWarps) {
        const int64_t token = i / a.splits, b = token / a.T;
        const int split = (int)(i % a.splits), t = (int)(token % a.T);
        float c[8], s[8];
        angles(a, l, INTER, position(a, b, t), c, s);
        auto heads = [&](const HeadTensor &h, float (&dw)[16]) {
            const T *g = (const T *)h.g + b * h.g_sb + t * h.g_st;
            const T *x = (const T *)h.x + b * h.sb + t * h.st;
            T *out = (T *)h.out + b * h.o_sb + t * h.o_st;
            if (h.w) backward_heads<T, INTER, true>(a, h, l, split, g, x, out, c, s, dw);
            else backward_heads<T, INTER, false>(a, h, l, split, g, x, out, c, s, dw);
        };
        heads(a.q, dwq);
        heads(a.k, dwk);
    }
    if (!a.parts) return;
    auto total = [&](float (&dw)[16], float *out) {
#pragma unroll
        for (int i = 0; i < 16; ++i)
            for (int o = a.lanes; o < 32; o <<= 1)
                dw[i] += __shfl_xor_sync(0xffffffffu, dw[i], o);
        __syncthreads();
        if (lane < a.lanes && l.live) {
#pragma unroll
            for (int i = 0; i < 16; ++i) sums[warp][i < 8 ? l.lo + i : l.hi + i - 8] = dw[i];
        }
        __syncthreads();
        if ((int)threadIdx.x < a.D) {
            float x = 0.0f;
            for (int w = 0; w < kWarps; ++w) x += sums[w][threadIdx.x];
            out[threadIdx.x] = x;
        }
    };
    float *out = a.parts + (int64_t)blockIdx.x * 2 * a.D;
    total(dwq, out);
    total(dwk, out + a.D);
}

// dw[j] = the sum of n parts `pitch` apart: 32 columns a CTA, its warps in turn over the parts.
__global__ void __launch_bounds__(1024) k_heads_weights(const float *parts, int n, int D, int w32,
                                                        int half, void *dwq, void *dwk) {
    __shared__ float sums[32][33];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int j = blockIdx.x * 32 + lane;
    float x = 0.0f;
    if (j < 2 * D)
        for (int i = warp; i < n; i += 32) x += parts[(int64_t)i * 2 * D + j];
    sums[warp][lane] = x;
    __syncthreads();
    if (warp || j >= 2 * D) return;
    x = 0.0f;
#pragma unroll
    for (int i = 0; i < 32; ++i) x += sums[i][lane];
    void *out = j < D ? dwq : dwk;
    const int at = j < D ? j : j - D;
    if (!out) return;
    if (w32) ((float *)out)[at] = x;
    else if (half) ((__half *)out)[at] = from_f32<__half>(x);
    else ((__nv_bfloat16 *)out)[at] = from_f32<__nv_bfloat16>(x);
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
    if (s->R && !s->turns) return SPMM_ERR_INVALID_ARG;
    return SPMM_OK;
}

bool heads_empty(const spmm_heads_shape *s) { return !s->B || !s->T || !(s->Hq + s->Hk); }

HeadTensor tensor(int64_t heads, const void *w) {
    HeadTensor h{};
    h.heads = (int)heads;
    h.w = w;
    return h;
}

void contiguous_out(HeadTensor &h, void *out, const spmm_heads_shape *s) {
    h.out = out;
    h.o_sh = s->D;
    h.o_st = h.heads * s->D;
    h.o_sb = s->T * h.o_st;
}

HeadArgs heads_args(const spmm_heads_shape *s) {
    HeadArgs a{};
    a.q = tensor(s->Hq, s->wq);
    a.k = tensor(s->Hk, s->wk);
    a.v = tensor(0, nullptr);
    a.tokens = s->B * s->T;
    a.T = (int)s->T;
    a.D = (int)s->D;
    a.R = (int)s->R;
    a.lanes = 1;
    while (a.lanes * 16 < a.D) a.lanes *= 2;
    a.w32 = s->weight_dtype == SPMM_F32;
    a.eps = s->eps;
    a.magnitude = s->magnitude;
    a.turns = s->turns;
    a.positions = s->positions;
    a.p_sb = s->p_sb;
    a.p_st = s->p_st;
    a.lengths = s->lengths;
    a.Tk = -1;
    // few tokens: a warp takes a part of a token's heads only
    const int64_t rows = 32 / a.lanes, most = (std::max(s->Hq, s->Hk) + rows - 1) / rows;
    const int64_t want = (kSms * 16 + a.tokens - 1) / std::max<int64_t>(a.tokens, 1);
    a.splits = (int)std::max<int64_t>(1, std::min(most, want));
    return a;
}

unsigned heads_grid(const HeadArgs &a, int per_sm) {
    const int64_t ctas = (a.tokens * a.splits + kWarps - 1) / kWarps;
    return (unsigned)std::min<int64_t>(ctas, kSms * per_sm);
}

constexpr int kForwardCtas = 8, kBackwardCtas = 4;     // per SM

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
        k_heads_rotate<T, INTER><<<grid, kThreads, 0, cs>>>(a);
    }
};
template <typename T, bool INTER> struct Backward {
    static void go(const HeadArgs &a, unsigned grid, cudaStream_t cs) {
        k_heads_backward<T, INTER><<<grid, kThreads, 0, cs>>>(a);
    }
};

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
    HeadArgs a = heads_args(s);
    set_rows(a.q.x, a.q.sb, a.q.st, a.q.sh, q);
    set_rows(a.k.x, a.k.sb, a.k.st, a.k.sh, k);
    contiguous_out(a.q, q_out, s);
    contiguous_out(a.k, k_out, s);
    return cuda_status(launch_heads<Rotate>(s, a, heads_grid(a, kForwardCtas), (cudaStream_t)stream));
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
    HeadArgs a = heads_args(s);
    set_rows(a.q.x, a.q.sb, a.q.st, a.q.sh, q);
    set_rows(a.k.x, a.k.sb, a.k.st, a.k.sh, k);
    contiguous_out(a.q, q_out, s);
    a.v = tensor(s->Hk, nullptr);
    set_rows(a.v.x, a.v.sb, a.v.st, a.v.sh, v);
    a.Tk = (int)Tk;
    a.k.out = const_cast<void *>(cache_k.data);
    a.k.o_sb = cache_k.sb, a.k.o_st = cache_k.st, a.k.o_sh = cache_k.sh;
    a.v.out = const_cast<void *>(cache_v.data);
    a.v.o_sb = cache_v.sb, a.v.o_st = cache_v.st, a.v.o_sh = cache_v.sh;
    return cuda_status(launch_heads<Rotate>(s, a, heads_grid(a, kForwardCtas), (cudaStream_t)stream));
}

int64_t spmm_heads_backward_workspace(const spmm_heads_shape *s) {
    using namespace spmm;
    if (heads_check(s) != SPMM_OK || heads_empty(s) || (!s->wq && !s->wk)) return 0;
    return heads_grid(heads_args(s), kBackwardCtas) * 2 * s->D * (int64_t)sizeof(float);
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
    HeadArgs a = heads_args(s);
    set_rows(a.q.x, a.q.sb, a.q.st, a.q.sh, q);
    set_rows(a.k.x, a.k.sb, a.k.st, a.k.sh, k);
    set_rows(a.q.g, a.q.g_sb, a.q.g_st, a.q.g_sh, grad_q);
    set_rows(a.k.g, a.k.g_sb, a.k.g_st, a.k.g_sh, grad_k);
    contiguous_out(a.q, dq, s);
    contiguous_out(a.k, dk, s);
    a.parts = need ? (float *)work : nullptr;
    const unsigned grid = heads_grid(a, kBackwardCtas);
    cudaError_t err = launch_heads<Backward>(s, a, grid, cs);
    if (err == cudaSuccess && need) {
        k_heads_weights<<<(unsigned)((2 * s->D + 31) / 32), 1024, 0, cs>>>(
            a.parts, (int)grid, a.D, a.w32, s->dtype == SPMM_F16, s->wq ? dwq : nullptr,
            s->wk ? dwk : nullptr);
        count_launch();
        err = cudaGetLastError();
    }
    return cuda_status(err);
}

}  // extern "C"
