// Norm and rotation of the heads of queries and keys. With r = (mean(x^2) + eps)^-1/2,
// n = r x, z = n w (z = x without a weight) and c, s the cosine and sine of a
// pair's angle times the magnitude:
//   forward    y1 = c z1 - s z2, y2 = c z2 + s z1 for the pairs, y = z behind them
//   backward   g1 = c dy1 + s dy2, g2 = c dy2 - s dy1 (the transpose), g = dy behind;
//              dw = sum over rows of g n, u = g w, dx = r (u - n mean(u n)); dx = g
// The angle of position p is p f turns, f < 1 in units of 2^-64: one 64-bit integer
// product, whose wrap is the reduction mod a turn, so a far position costs no accuracy.
//
// A lane holds 8 elements of a row, four pairs: two loads of 4 elements
// (the lanes of a row read adjacent ones), no exchange for the rotation, and a
// shuffle over the row's lanes for the norm's sum. A warp takes a token (several where
// they have few heads) and walks its heads of queries and keys: the angles are the same
// for all of them. One pass: every element is read once and written once.
// A warp works the angles out once, a pair to a lane, and hands them round in shared memory.
// Two rows are worked on side by side, as one row's chain (its sum over the lanes, the
// root, the products) leaves the pipes idle, and four more are on their way meanwhile.
//
// Measured (replayed graphs): 8192 tokens of 32 + 4 heads of 128 in bf16 (151 MB) 33 to 35 us, 4.4
// TB/s, heads of 64 18.5, 96 33, 256 (half as many) 36; in fp32 (302 MB) 54 us, 5.6 TB/s. A
// training step of 2 x 4096 tokens of 16 + 2 heads 18.5 us forward and 43 backward (113 MB, 2.7
// TB/s), in fp32 33 and 53. The walk without the arithmetic took 24 of 31 us, a norm 2 and the
// angles 2 of the rest. Bound by latency: instructions issue in 56% and 46% of the cycles (forward,
// backward), and the 20 and 12 warps that fit an SM's registers (27% and 17% of its places)
// wait, for each that issues, 2.1 and 1.5 for memory, 1.5 and 1.5 for the instruction before and
// 0.9 and 0.6 for the shuffles and shared memory.
#include "blocks.cuh"

namespace spmm {
namespace {

constexpr int kThreads = 128, kWarps = kThreads / 32;
constexpr int kForwardCtas = 5, kBackwardCtas = 3;      // that share an SM
constexpr int kSms = 152, kCtas = kForwardCtas * kSms;

// Strided [B, T, heads, D] tensors: what is read, with its weight, and what is written.
struct HeadFrom {
    const void *x, *w;
    int64_t sb, st, sh;
    int heads;
};
struct HeadTo {
    void *out;
    int64_t sb, st, sh;
};

// How warps share the tokens: their rows at a time are of at_once heads of `tokens` tokens;
// `splits` warps share a token's heads; `items` shares in all.
struct HeadWalk {
    int at_once, tokens;
    unsigned splits, items;
};

struct HeadArgs {
    int all, T, D, R, lanes;         // B T; lanes of a row
    int w32;                         // weights are fp32
    float eps, magnitude, inv_D;
    const uint64_t *turns;
    const int32_t *positions, *lengths;
    int64_t p_sb, p_st;
    HeadFrom from[3];                // queries, keys, values (append); backward: the gradients
    HeadTo to[3];
    HeadFrom x[2];                   // backward: queries, keys
    HeadWalk walk;
    int Tk;                          // rows of the caches that k and v go to, or -1
    float *parts;                    // backward: [CTAs][2][D] parts of the weights' gradients
};

// Two floats to an instruction: the arithmetic of a row would else take longer to issue
// than the row takes to come.
using F2 = unsigned long long;
constexpr F2 kMinus2 = 0x8000000080000000ull;
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

// 8 elements as they lie in memory: 4 from one place and 4 from another. As floats,
// number i holds elements 2 i and 2 i + 1.
template <typename T> struct Raw {
    using V = typename std::conditional<sizeof(T) == 4, uint4, uint2>::type;
    V w[2];
    __device__ __forceinline__ void load(const T *lo, const T *hi) {
        w[0] = __ldg((const V *)lo);
        w[1] = __ldg((const V *)hi);
    }
    __device__ __forceinline__ void store(T *lo, T *hi) const {
        *(V *)lo = w[0];
        *(V *)hi = w[1];
    }
    __device__ __forceinline__ void zero() { w[0] = w[1] = V{}; }
    __device__ __forceinline__ void get(F2 (&x)[4]) const {
        const T *e = reinterpret_cast<const T *>(w);
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = two(to_f32(e[2 * i]), to_f32(e[2 * i + 1]));
    }
    __device__ __forceinline__ void set(const F2 (&x)[4]) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 y = both(x[i]);
            if constexpr (sizeof(T) == 4)
                reinterpret_cast<float2 *>(w)[i] = y;
            else
                reinterpret_cast<uint32_t *>(w)[i] = pack2<T>(y.x, y.y);
        }
    }
};

// A lane's place: row `row` of the warp's rows at a time, and in it the 4 elements
// from `lo` and the 4 from `hi`. D and R are multiples of 16, so a lane's elements
// are all turned (its four pairs) or none is.
struct HeadLane {
    int row, lo, hi;
    bool live, turned;
    __device__ __forceinline__ HeadLane(const HeadArgs &a, bool interleaved) {
        const int lane = threadIdx.x & 31, u = lane & (a.lanes - 1);
        row = lane / a.lanes;
        live = u * 8 < a.D;
        turned = u * 8 < a.R;
        lo = turned && !interleaved ? 4 * u : 8 * u;
        hi = turned && !interleaved ? a.R / 2 + 4 * u : 8 * u + 4;
    }
};

// One token of each of the warp's groups of lanes, and where among its heads the lane begins.
struct HeadPlace {
    int64_t b, pos;
    int t, first;
    bool live;
    __device__ __forceinline__ HeadPlace(const HeadArgs &a, const HeadWalk &w, const HeadLane &l,
                                         unsigned item) {
        const int which = w.tokens == 1 ? 0 : l.row / w.at_once;
        const int64_t token = (int64_t)(item / w.splits) * w.tokens + which;
        live = l.live && which < w.tokens && token < a.all;
        b = live ? (unsigned)token / (unsigned)a.T : 0;
        t = live ? (int)((unsigned)token - (unsigned)b * (unsigned)a.T) : 0;
        first = l.row - which * w.at_once;
        pos = t;
        if (a.positions) pos = live ? a.positions[b * a.p_sb + t * a.p_st] : 0;
        else if (a.lengths) pos = live ? (int64_t)a.lengths[b] - a.T + t : 0;
    }
};

// Sines and cosines of the warp's tokens' pairs, times the magnitude. The turn is cut to the
// nearest half (exactly, in integers) before it becomes a float: with all of its 64 bits, as the
// slowest pair's angles near position 0 are a few millionths of a radian, and its sine is
// as exact as any. What is left, x of at most pi / 2, is off by at most 3 x 2^-24 of itself (its
// conversion, the constant, their product) and goes into the two functions' power
// series, whose first terms left out, x^13 / 13! and x^14 / 14!, are below 2^-24.
struct HeadAngles {
    float c[128], s[128];            // of a warp: tokens x R / 2, at most 32 / lanes x 4 lanes
};
__device__ __forceinline__ void angles(const HeadArgs &a, const HeadWalk &w, int64_t pos,
                                       HeadAngles &to) {
    const int pairs = a.R / 2, lane = threadIdx.x & 31;
#pragma unroll 1
    for (int i0 = 0; i0 < pairs * w.tokens; i0 += 32) {
        const int i = i0 + lane, token = w.tokens == 1 ? 0 : i / pairs;
        const int64_t p =
            __shfl_sync(0xffffffffu, pos, (w.tokens == 1 ? 0 : token * w.at_once * a.lanes) & 31);
        if (i >= pairs * w.tokens) continue;
        const uint64_t t = (uint64_t)p * __ldg(a.turns + (i - token * pairs));
        // the sign of both functions: whether the nearest half turn is an odd one
        const uint32_t odd = ((uint32_t)(t >> 32) + (1u << 30)) & (1u << 31);
        const float x = (float)(int64_t)(t ^ (uint64_t)odd << 32) * 3.40612158008655e-19f;  // 2 pi / 2^64
        const float y = x * x;
        float sx = fmaf(y, -1.0f / 39916800, 1.0f / 362880);
        sx = fmaf(y, sx, -1.0f / 5040);
        sx = fmaf(y, sx, 1.0f / 120);
        sx = fmaf(y, sx, -1.0f / 6);
        sx = fmaf(x * y, sx, x);
        float cx = fmaf(y, 1.0f / 479001600, -1.0f / 3628800);
        cx = fmaf(y, cx, 1.0f / 40320);
        cx = fmaf(y, cx, -1.0f / 720);
        cx = fmaf(y, cx, 1.0f / 24);
        cx = fmaf(y, cx, -0.5f);
        cx = fmaf(y, cx, 1.0f);
        to.c[i] = __uint_as_float(__float_as_uint(cx * a.magnitude) ^ odd);
        to.s[i] = __uint_as_float(__float_as_uint(sx * a.magnitude) ^ odd);
    }
    __syncwarp();
}
// The lane's: of pairs 2 i and 2 i + 1 in number i.
__device__ __forceinline__ void take_angles(const HeadArgs &a, const HeadWalk &w, const HeadLane &l,
                                            const HeadAngles &from, F2 (&c)[2], F2 (&s)[2]) {
    if (!l.turned) return;
    const int which = w.tokens == 1 ? 0 : min(l.row / w.at_once, w.tokens - 1);
    const int at = which * (a.R / 2) + ((threadIdx.x & 31) & (a.lanes - 1)) * 4;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        c[i] = two(from.c[at + 2 * i], from.c[at + 2 * i + 1]);
        s[i] = two(from.s[at + 2 * i], from.s[at + 2 * i + 1]);
    }
}

// z by its matrix: element i of a pair times a, and its partner times b.
template <bool INTER>
__device__ __forceinline__ void by_matrix(F2 (&z)[4], const F2 (&a)[4], const F2 (&b)[4]) {
    if constexpr (INTER) {
#pragma unroll
        for (int i = 0; i < 4; ++i) z[i] = fma2(swap(z[i]), b[i], mul2(z[i], a[i]));
    } else {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const F2 x = z[i], y = z[2 + i];
            z[i] = fma2(y, b[i], mul2(x, a[i]));
            z[2 + i] = fma2(x, b[2 + i], mul2(y, a[2 + i]));
        }
    }
}

// That matrix for the product with w and then the turn by the angles.
template <bool INTER>
__device__ __forceinline__ void matrix(const F2 (&c)[2], const F2 (&s)[2], const F2 (&w)[4],
                                       F2 (&a)[4], F2 (&b)[4]) {
    if constexpr (INTER) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 cc = both(c[i / 2]), ss = both(s[i / 2]), ww = both(w[i]);
            const float ci = i & 1 ? cc.y : cc.x, si = i & 1 ? ss.y : ss.x;
            a[i] = two(ww.x * ci, ww.y * ci);
            b[i] = two(-ww.y * si, ww.x * si);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            a[i] = mul2(w[i], c[i]);
            a[2 + i] = mul2(w[2 + i], c[i]);
            b[i] = mul2(w[2 + i], s[i]) ^ kMinus2;
            b[2 + i] = mul2(w[i], s[i]);
        }
    }
}

// Turned by the negatives of the angles.
template <bool INTER>
__device__ __forceinline__ void turn_back(F2 (&z)[4], const F2 (&c)[2], const F2 (&s)[2]) {
    if constexpr (INTER) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 cc = both(c[i / 2]), ss = both(s[i / 2]), x = both(z[i]);
            const float ci = i & 1 ? cc.y : cc.x, si = i & 1 ? ss.y : ss.x;
            z[i] = two(fmaf(x.y, si, x.x * ci), fmaf(-x.x, si, x.y * ci));
        }
    } else {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const F2 x = z[i], y = z[2 + i];
            z[i] = fma2(y, s[i], mul2(x, c[i]));
            z[2 + i] = fma2(x, s[i] ^ kMinus2, mul2(y, c[i]));
        }
    }
}

// Two sums over the lanes of a row (LANES: their number, where it is a constant).
template <int LANES> __device__ __forceinline__ void row_sums(float &x, float &y, int lanes) {
    const int n = LANES ? LANES : lanes;
#pragma unroll
    for (int d = 1; d < (LANES ? LANES : 32); d <<= 1) {
        if (!LANES && d >= n) break;
        const float u = __shfl_xor_sync(0xffffffffu, x, d), v = __shfl_xor_sync(0xffffffffu, y, d);
        x += u;
        y += v;
    }
}

// The lane's part of a weight; 1 without one.
template <typename T>
__device__ __forceinline__ void load_weight(const HeadArgs &a, const HeadLane &l, const void *w,
                                            F2 (&x)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = two(1.0f, 1.0f);
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

// Rows asked for ahead of the work, of a lane.
template <typename T> constexpr int kForwardRows = 8 / (int)sizeof(T);

// Heads split * at_once + first of a token, then splits * at_once further. COPY: as they are.
template <typename T, bool INTER, int LANES, bool COPY>
__device__ __forceinline__ void forward_heads(const HeadArgs &a, const HeadWalk &w,
                                              const HeadLane &l, const HeadPlace &at, int split,
                                              const HeadFrom &h, const HeadTo &o, int64_t row,
                                              bool put, const HeadAngles *told) {
    constexpr int AHEAD = kForwardRows<T>;
    static_assert(AHEAD % 2 == 0, "rows come in twos");
    const int step = (int)w.splits * w.at_once;
    const int left = h.heads - split * w.at_once, n = left > 0 ? (left + step - 1) / step : 0;
    if (n == 0) return;
    const int off = l.hi - l.lo;
    const int64_t from_step = step * h.sh, to_step = step * o.sh;
    int head = split * w.at_once + at.first;
    const T *from = (const T *)h.x + at.b * h.sb + at.t * h.st + head * h.sh + l.lo;
    T *to = (T *)o.out + at.b * o.sb + row * o.st + head * o.sh + l.lo;
    Raw<T> x[AHEAD];
#pragma unroll
    for (int u = 0; u < AHEAD; ++u) {
        x[u].zero();                             // (lanes without a part of a row add 0 to it)
        if (at.live && head + u * step < h.heads) x[u].load(from, from + off);
        from += from_step;
    }
    const bool norm = !COPY && h.w;
    F2 ma[4], mb[4];                             // (ma: of lanes that are not turned, the weight)
    if (!COPY) {
        load_weight<T>(a, l, h.w, ma);
        if (l.turned) {
            F2 c[2], s[2], weight[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) weight[j] = ma[j];
            take_angles(a, w, l, *told, c, s);
            matrix<INTER>(c, s, weight, ma, mb);
        }
    }
#pragma unroll 1
    for (int i = 0; i < n; i += AHEAD) {
#pragma unroll
        for (int u = 0; u < AHEAD; u += 2) {
            if (i + u >= n) break;
            Raw<T> y[2];
            if (COPY) {
                y[0] = x[u];
                y[1] = x[u + 1];
            } else {
                F2 z[2][4];
                x[u].get(z[0]);
                x[u + 1].get(z[1]);
                if (norm) {
                    float sum[2];
#pragma unroll
                    for (int v = 0; v < 2; ++v) {
                        F2 sq = mul2(z[v][0], z[v][0]);
#pragma unroll
                        for (int j = 1; j < 4; ++j) sq = fma2(z[v][j], z[v][j], sq);
                        const float2 t = both(sq);
                        sum[v] = t.x + t.y;
                    }
                    row_sums<LANES>(sum[0], sum[1], a.lanes);
#pragma unroll
                    for (int v = 0; v < 2; ++v) {
                        const float r = rsqrtf(fmaf(sum[v], a.inv_D, a.eps));
#pragma unroll
                        for (int j = 0; j < 4; ++j) z[v][j] = mul2(z[v][j], two(r, r));
                    }
                }
                if (l.turned) {
                    by_matrix<INTER>(z[0], ma, mb);
                    by_matrix<INTER>(z[1], ma, mb);
                } else if (norm) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        z[0][j] = mul2(z[0][j], ma[j]);
                        z[1][j] = mul2(z[1][j], ma[j]);
                    }
                }
                y[0].set(z[0]);
                y[1].set(z[1]);
            }
#pragma unroll
            for (int v = 0; v < 2; ++v) {
                if (at.live && put && head < h.heads) y[v].store(to, to + off);
                to += to_step;
                if (at.live && head + AHEAD * step < h.heads) x[u + v].load(from, from + off);
                from += from_step;
                head += step;
            }
        }
    }
}

// A warp takes a token's queries, keys and (append) values, or every splits-th of their rows.
template <typename T, bool INTER, int LANES>
__global__ void __launch_bounds__(kThreads, kForwardCtas) k_heads_rotate(const __grid_constant__ HeadArgs a) {
    __shared__ HeadAngles told[kWarps];
    const HeadLane l(a, INTER);
    const HeadWalk &w = a.walk;
    const int warp = threadIdx.x / 32;
    const unsigned item = blockIdx.x * kWarps + warp;
    if (item >= w.items) return;
    const int split = w.splits == 1 ? 0 : (int)(item % w.splits);
    const HeadPlace at(a, w, l, item);
    angles(a, w, at.pos, told[warp]);
    const bool cached = a.Tk >= 0, put = !cached || (at.pos >= 0 && at.pos < a.Tk);
    const int64_t row = cached ? at.pos : at.t;
    forward_heads<T, INTER, LANES, false>(a, w, l, at, split, a.from[0], a.to[0], at.t, true, &told[warp]);
    forward_heads<T, INTER, LANES, false>(a, w, l, at, split, a.from[1], a.to[1], row, put, &told[warp]);
    if (cached)
        forward_heads<T, INTER, LANES, true>(a, w, l, at, split, a.from[2], a.to[2], row, put, nullptr);
}

// The same heads' gradients; dw: the lane's part of the weight's, added to.
template <typename T, bool INTER, int LANES>
__device__ __forceinline__ void backward_heads(const HeadArgs &a, const HeadWalk &w,
                                               const HeadLane &l, const HeadPlace &at, int split,
                                               const HeadFrom &g, const HeadFrom &x,
                                               const HeadTo &o, const HeadAngles &told,
                                               F2 (&dw)[4]) {
    const int step = (int)w.splits * w.at_once;
    const int left = g.heads - split * w.at_once, n = left > 0 ? (left + step - 1) / step : 0;
    if (n == 0) return;
    const bool norm = x.w != nullptr;
    const int off = l.hi - l.lo;
    const int64_t g_step = step * g.sh, x_step = step * x.sh, o_step = step * o.sh;
    int head = split * w.at_once + at.first;
    const T *gs = (const T *)g.x + at.b * g.sb + at.t * g.st + head * g.sh + l.lo;
    const T *xs = (const T *)x.x + at.b * x.sb + at.t * x.st + head * x.sh + l.lo;
    T *to = (T *)o.out + at.b * o.sb + at.t * o.st + head * o.sh + l.lo;
    Raw<T> rg[2], rx[2];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
        rg[u].zero();
        rx[u].zero();
        const bool live = at.live && head + u * step < g.heads;
        if (live) rg[u].load(gs, gs + off);
        if (live && norm) rx[u].load(xs, xs + off);
        gs += g_step;
        xs += x_step;
    }
    F2 c[2], s[2], weight[4];
    load_weight<T>(a, l, x.w, weight);
    take_angles(a, w, l, told, c, s);
#pragma unroll 1
    for (int i = 0; i < n; i += 2) {
        F2 y[2][4], z[2][4];
        bool live[2];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            live[u] = at.live && head + u * step < g.heads;
            rg[u].get(y[u]);
            rx[u].get(z[u]);
            if (at.live && head + (u + 2) * step < g.heads) {
                rg[u].load(gs, gs + off);
                if (norm) rx[u].load(xs, xs + off);
            }
            gs += g_step;
            xs += x_step;
        }
        if (l.turned) {
            turn_back<INTER>(y[0], c, s);
            turn_back<INTER>(y[1], c, s);
        }
        if (norm) {
            float sum[2], dot[2];
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                F2 sq = mul2(z[u][0], z[u][0]);
                F2 dots = mul2(mul2(y[u][0], weight[0]), z[u][0]);
#pragma unroll
                for (int j = 1; j < 4; ++j) {
                    sq = fma2(z[u][j], z[u][j], sq);
                    dots = fma2(mul2(y[u][j], weight[j]), z[u][j], dots);
                }
                float2 v = both(sq);
                sum[u] = v.x + v.y;
                v = both(dots);
                dot[u] = v.x + v.y;
            }
            row_sums<LANES>(sum[0], sum[1], a.lanes);
            row_sums<LANES>(dot[0], dot[1], a.lanes);
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const float q = rsqrtf(fmaf(sum[u], a.inv_D, a.eps));
                const float m = -dot[u] * q * a.inv_D;     // -mean(u n)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const F2 nj = mul2(z[u][j], two(q, q));
                    if (live[u]) dw[j] = fma2(y[u][j], nj, dw[j]);
                    y[u][j] = mul2(two(q, q), fma2(nj, two(m, m), mul2(y[u][j], weight[j])));
                }
            }
        }
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            Raw<T> r;
            r.set(y[u]);
            if (live[u]) r.store(to, to + off);
            to += o_step;
        }
        head += 2 * step;
    }
}

// The weights' gradients: a lane's sums over its rows, then over the rows of the
// warp, the warps of the CTA and, by a second kernel, the CTAs, each in a fixed order.
template <typename T, bool INTER, int LANES>
__global__ void __launch_bounds__(kThreads, kBackwardCtas)
    k_heads_backward(const __grid_constant__ HeadArgs a) {
    __shared__ HeadAngles told[kWarps];
    const HeadLane l(a, INTER);
    const HeadWalk &w = a.walk;
    const int warp = threadIdx.x / 32, lane = threadIdx.x & 31;
    F2 dwq[4], dwk[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) dwq[i] = dwk[i] = two(0.0f, 0.0f);
    for (unsigned item = blockIdx.x * kWarps + warp; item < w.items; item += gridDim.x * kWarps) {
        const int split = w.splits == 1 ? 0 : (int)(item % w.splits);
        const HeadPlace at(a, w, l, item);
        __syncwarp();                            // (the angles before are read)
        angles(a, w, at.pos, told[warp]);
        backward_heads<T, INTER, LANES>(a, w, l, at, split, a.from[0], a.x[0], a.to[0], told[warp],
                                        dwq);
        backward_heads<T, INTER, LANES>(a, w, l, at, split, a.from[1], a.x[1], a.to[1], told[warp],
                                        dwk);
    }
    if (!a.parts) return;
    float *sums = reinterpret_cast<float *>(told);         // [kWarps][256]
    auto total = [&](const F2 (&dw)[4], float *out) {
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float2 v = both(dw[i]);
            for (int j = a.lanes; j < 32; j <<= 1) {
                v.x += __shfl_xor_sync(0xffffffffu, v.x, j);
                v.y += __shfl_xor_sync(0xffffffffu, v.y, j);
            }
            if (lane < a.lanes && l.live) {
                const int j = warp * 256 + (i < 2 ? l.lo : l.hi) + 2 * (i & 1);
                sums[j] = v.x;
                sums[j + 1] = v.y;
            }
        }
        __syncthreads();
        for (int j = threadIdx.x; j < a.D; j += kThreads) {
            float v = 0.0f;
            for (int i = 0; i < kWarps; ++i) v += sums[i * 256 + j];
            out[j] = v;
        }
    };
    float *out = a.parts + (int64_t)blockIdx.x * 2 * a.D;
    if (a.x[0].w) total(dwq, out);
    if (a.x[1].w) total(dwk, out + a.D);
}

// A weight's gradient is the sum of the CTAs' parts: 8 columns a CTA, 128 parts at a time, then
// over the lanes and warps; CTAs y = 0 for the queries', 1 for the keys'. (A row of 8 parts is
// a sector; with 32 columns a CTA the eight CTAs took 6 us for 2048 parts of heads of 128.)
__global__ void __launch_bounds__(1024) k_heads_weights(const float *parts, int n, int D, int w32,
                                                        int half, void *dwq, void *dwk) {
    __shared__ float sums[32][9];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int j = blockIdx.x * 8 + (lane & 7);             // (D is a multiple of 16)
    void *out = blockIdx.y ? dwk : dwq;
    if (!out) return;
    parts += blockIdx.y * D + j;
    float x = 0.0f;
#pragma unroll 8
    for (int i = warp * 4 + (lane >> 3); i < n; i += 128) x += parts[(int64_t)i * 2 * D];
    x += __shfl_xor_sync(0xffffffffu, x, 8);
    x += __shfl_xor_sync(0xffffffffu, x, 16);
    if (lane < 8) sums[warp][lane] = x;
    __syncthreads();
    if (threadIdx.x >= 8) return;
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

HeadFrom from(const spmm_rows &r, int64_t heads, const void *w) {
    HeadFrom h{};
    set_rows(h.x, h.sb, h.st, h.sh, r);
    h.w = w;
    h.heads = (int)heads;
    return h;
}
HeadTo to(const spmm_rows &r) {
    return HeadTo{const_cast<void *>(r.data), r.sb, r.st, r.sh};
}
HeadTo contiguous(void *out, int64_t heads, const spmm_heads_shape *s) {
    return HeadTo{out, s->T * heads * s->D, heads * s->D, s->D};
}

unsigned warps_ctas(unsigned items) { return items / kWarps + (items % kWarps > 0); }

HeadArgs shared_args(const spmm_heads_shape *s) {
    HeadArgs a{};
    a.all = (int)(s->B * s->T);
    a.T = (int)s->T;
    a.D = (int)s->D;
    a.R = (int)s->R;
    a.lanes = 1;
    while (a.lanes * 8 < a.D) a.lanes *= 2;
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
    return a;
}

constexpr int64_t kWaves = 2;
// For tokens of up to `heads` heads. Few tokens: a warp takes a part of a token's heads only.
HeadWalk walk(const HeadArgs &a, int64_t heads) {
    HeadWalk w{};
    const int groups = 32 / a.lanes;
    w.at_once = (int)std::max<int64_t>(1, std::min<int64_t>(heads, groups));
    w.tokens = groups / w.at_once;
    w.splits = 1;
    const int64_t warps = heads ? ((int64_t)a.all + w.tokens - 1) / w.tokens : 0;
    if (warps)
        w.splits = (unsigned)std::max<int64_t>(
            1, std::min<int64_t>((heads + w.at_once - 1) / w.at_once, kWaves * kCtas * kWarps / warps));
    w.items = (unsigned)(warps * w.splits);
    return w;
}

HeadArgs forward_args(const spmm_heads_shape *s, const spmm_rows &q, const spmm_rows &k, void *q_out,
                      void *k_out) {
    HeadArgs a = shared_args(s);
    a.from[0] = from(q, s->Hq, s->wq);
    a.from[1] = from(k, s->Hk, s->wk);
    a.to[0] = contiguous(q_out, s->Hq, s);
    a.to[1] = contiguous(k_out, s->Hk, s);
    a.walk = walk(a, std::max(s->Hq, s->Hk));
    return a;
}

// Backward: CTAs that each add up a part of the weights' gradients, three times as many as the
// SMs hold. A training step of 2 x 4096 tokens, 16 + 2 heads of 128, took 57 us with 9 or 6 for
// each SM, 61 with 14 (a token a warp: more parts to add up), 85 with 2 (the last ones' tokens
// alone on the GPU).
constexpr unsigned kParts = 9 * kSms;
HeadArgs backward_args(const spmm_heads_shape *s, unsigned &grid) {
    HeadArgs a = shared_args(s);
    a.walk = walk(a, std::max(s->Hq, s->Hk));
    grid = std::min(kParts, warps_ctas(a.walk.items));
    return a;
}

// f(element, interleaved, lanes) for the call's: lanes of heads of 64 and 128, the widths that
// the attention takes, are constants (two sums over 16 lanes then take 16 instructions,
// with a loop 40, of some 110 that a row takes in all); those of other widths 0.
template <typename F> cudaError_t by_kind(const spmm_heads_shape *s, F f) {
    auto lanes = [&](auto t, auto inter) {
        if (s->D == 64) return f(t, inter, std::integral_constant<int, 8>{});
        if (s->D == 128) return f(t, inter, std::integral_constant<int, 16>{});
        return f(t, inter, std::integral_constant<int, 0>{});
    };
    auto type = [&](auto inter) {
        if (s->dtype == SPMM_F32) return lanes(float{}, inter);
        if (s->dtype == SPMM_BF16) return lanes(__nv_bfloat16{}, inter);
        return lanes(__half{}, inter);
    };
    return s->interleaved ? type(std::true_type{}) : type(std::false_type{});
}

template <typename K>
cudaError_t launch(K kernel, const HeadArgs &a, unsigned grid, cudaStream_t cs) {
    kernel<<<grid, kThreads, 0, cs>>>(a);
    count_launch();
    return cudaGetLastError();
}

cudaError_t rotate(const spmm_heads_shape *s, const HeadArgs &a, cudaStream_t cs) {
    return by_kind(s, [&](auto t, auto inter, auto lanes) {
        using T = decltype(t);
        return launch(k_heads_rotate<T, decltype(inter)::value, decltype(lanes)::value>, a, warps_ctas(a.walk.items), cs);
    });
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
    return cuda_status(rotate(s, forward_args(s, q, k, q_out, k_out), (cudaStream_t)stream));
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
    if (Tk && (!written_ok(cache_k, e, s, Tk) || !written_ok(cache_v, e, s, Tk) ||
               cache_k.data == cache_v.data))    // keys and values in one place
        return SPMM_ERR_INVALID_ARG;
    HeadArgs a = forward_args(s, q, k, q_out, nullptr);
    a.from[2] = from(v, s->Hk, nullptr);
    a.to[1] = to(cache_k);
    a.to[2] = to(cache_v);
    a.Tk = (int)Tk;
    return cuda_status(rotate(s, a, (cudaStream_t)stream));
}

int64_t spmm_heads_backward_workspace(const spmm_heads_shape *s) {
    using namespace spmm;
    if (heads_check(s) != SPMM_OK || heads_empty(s) || (!s->wq && !s->wk)) return 0;
    unsigned grid;
    backward_args(s, grid);
    return grid * 2 * s->D * (int64_t)sizeof(float);
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
    unsigned grid;
    HeadArgs a = backward_args(s, grid);
    const bool sums = s->wq || s->wk;
    if (sums && (!work || work_bytes < grid * 2 * s->D * (int64_t)sizeof(float) || (uintptr_t)work % 16))
        return SPMM_ERR_INVALID_ARG;
    a.from[0] = from(grad_q, s->Hq, nullptr);
    a.from[1] = from(grad_k, s->Hk, nullptr);
    a.x[0] = from(q, s->Hq, s->wq);
    a.x[1] = from(k, s->Hk, s->wk);
    a.to[0] = contiguous(dq, s->Hq, s);
    a.to[1] = contiguous(dk, s->Hk, s);
    a.parts = sums ? (float *)work : nullptr;
    cudaError_t err = by_kind(s, [&](auto t, auto inter, auto lanes) {
        using T = decltype(t);
        return launch(k_heads_backward<T, decltype(inter)::value, decltype(lanes)::value>, a, grid,
                      cs);
    });
    if (err == cudaSuccess && sums) {
        k_heads_weights<<<dim3((unsigned)(s->D / 8), 2), 1024, 0, cs>>>(
            a.parts, (int)grid, a.D, a.w32, s->dtype == SPMM_F16, s->wq ? dwq : nullptr,
            s->wk ? dwk : nullptr);
        count_launch();
        err = cudaGetLastError();
    }
    return cuda_status(err);
}

}  // extern "C"
