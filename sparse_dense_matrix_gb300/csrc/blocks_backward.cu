// Selected-block attention, backward. With P = exp(scale Q K^T - lse),
// dP = dO V^T, delta = <dO, O> and dS = scale P (dP - delta):
//   dQ = dS K       by query, like the forward;
//   dV = P^T dO, dK = dS^T Q       by key block, over the queries that chose it:
// the transpose of the selection, as one bit per query in a row of words per
// (sequence, kv head, block), set with integer atomics (order-independent).
#include "blocks_keys.cuh"

namespace spmm {
namespace {

// delta, and the bits cleared for k_set_bits. Bound by memory: 14 us for 2 x 4096 x
// 16 rows of 128 (67 MB). It is summed in fp32 from the rounded output, the only one that
// a caller has (an fp32 copy would be twice its bytes to write and read): it is off by
// what that rounding left out, which dQ shows.
template <typename T, int D>
__global__ void __launch_bounds__(128) k_delta(BwdArgs p, int64_t rows, int64_t words) {
    constexpr int U = D / 8;
    for (int64_t w = (int64_t)blockIdx.x * 128 + threadIdx.x; w < words; w += (int64_t)gridDim.x * 128)
        p.bits[w] = 0u;
    const int64_t i = (int64_t)blockIdx.x * (128 / U) + threadIdx.x / U;
    const int u = threadIdx.x % U;
    float s = 0.0f;
    if (i < rows) {
        const int head = (int)(i % p.a.Hq);
        const int64_t bt = i / p.a.Hq;
        const int64_t t = bt % p.a.Tq, b = bt / p.a.Tq;
        float x[8], y[8];
        ld_pack<T, 8>((const T *)p.out + i * D + u * 8, x);
        ld_pack<T, 8>((const T *)p.dout + b * p.do_sb + t * p.do_st + head * p.do_sh + u * 8, y);
#pragma unroll
        for (int e = 0; e < 8; ++e) s = fmaf(x[e], y[e], s);
    }
#pragma unroll
    for (int o = U / 2; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if (i < rows && u == 0) p.delta[i] = s;
}

__global__ void k_set_bits(BwdArgs p, int64_t entries) {
    const BlkArgs &a = p.a;
    const int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
    if (i >= entries) return;
    const int64_t row = i / a.n;
    const int j = (int)(i % a.n);
    const int32_t *list = a.blocks + row * a.n;
    if (!blk_entry_ok(list, j, a.NB)) return;
    const int h = (int)(row % a.Hk);
    const int64_t bt = row / a.Hk;
    const int t = (int)(bt % a.Tq);
    const int64_t b = bt / a.Tq;
    // a query that sees none of the block's keys adds nothing, whatever its rows hold
    if (list[j] * a.block >= blk_limit(a, blk_len(a, (int)b), t)) return;
    atomicOr(p.bits + ((b * a.Hk + h) * a.NB + list[j]) * p.words + (t >> 5), 1u << (t & 31));
}

// dS is used twice over, as its rounded value plus what that left out. The rows of
// dS sum to 0, so dQ = dS K (and, to a degree, dK) is what remains after the keys'
// common part cancels, and a single rounding of dS shows in it: the error was 1.7
// times that of rounding dQ alone, and is 1.27 times with both parts (the rest is
// delta's, from the rounded output: given that output it is 1.00 times, where one part
// alone gives 8 on keys whose common part is 8 times the rest).

// fp16 has 5 bits of exponent: weights and gradients well below 2^-14 would lose
// their digits in it. So P is held as P 2^14 (at most 2^14, up to its rounding),
// and dS as dS 2^e, where a warp lowers its e (and rescales what it has summed)
// whenever a tile's largest |dS| would reach 2^15; both are exact powers of two,
// taken out of the sums at the end. bf16 has fp32's exponent and needs neither.
template <typename T> constexpr bool kNarrow = std::is_same<T, __half>::value;
template <typename T> constexpr float kPShift = kNarrow<T> ? 14.0f : 0.0f;
template <typename T> constexpr float kPUnit = kNarrow<T> ? 1.0f / 16384.0f : 1.0f;

__device__ __forceinline__ float pow2i(int e) { return __int_as_float((127 + e) << 23); }

struct DsScale {
    int e = 100;
    // Folds in one tile's largest finite |dS| (per lane); returns the factor for
    // what is summed already (1 mostly; the same in the whole warp).
    __device__ __forceinline__ float lower(float lane_max) {
        const uint32_t m = __reduce_max_sync(0xffffffffu, __float_as_uint(lane_max));
        const int want = 14 - ((int)(m >> 23) - 127);
        if (want >= e) return 1.0f;
        const float f = pow2i(max(want - e, -126));
        e = want;
        return f;
    }
};

__device__ __forceinline__ float finite_max(float m, float x) {
    x = fabsf(x);
    return x < INFINITY ? fmaxf(m, x) : m;       // false for NaN
}

// ----------------------------------------------------------------- dQ
constexpr int kRowWarps = 4;
constexpr int kRowThreads = 32 * kRowWarps;

// By query: as the forward by query, for the few queries that do not go by tile.
// Two keys' rows (r, r + 8) of a slice as the A operand over D.
template <typename T, int D>
__device__ __forceinline__ void load_keys(uint4 (&x)[D / 32][2], const T *p, int64_t st, int key0,
                                          int limit, int r, int c) {
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        const int key = key0 + r + 8 * e;
#pragma unroll
        for (int i = 0; i < D / 32; ++i)
            x[i][e] = key < limit ? __ldg((const uint4 *)(p + key * st + 32 * i + 8 * c))
                                  : make_uint4(0, 0, 0, 0);
    }
}

template <typename T, int D, int NT>
__global__ void __launch_bounds__(kRowThreads) k_dq_rows(BwdArgs p) {
    constexpr int R = 8 * NT;
    __shared__ float sm[kRowWarps][R][D + 4];
    const BlkArgs &a = p.a;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, r = lane >> 2, c = lane & 3;
    const int gt = blockIdx.x % p.gt;
    const int64_t list_id = blockIdx.x / p.gt;
    const int h = (int)(list_id % a.Hk);
    const int64_t bt = list_id / a.Hk;
    const int t = (int)(bt % a.Tq), b = (int)(bt / a.Tq);
    const int g0 = gt * R, ng = min(a.G - g0, R);
    const int limit = blk_limit(a, blk_len(a, b), t);
    const int32_t *list = a.blocks + list_id * a.n;
    const float scale2 = a.scale * kLog2e;
    const int head0 = h * a.G + g0;
    const int64_t row0 = bt * a.Hq + head0;

    uint4 q[NT][D / 32], g[NT][D / 32];
    const T *qp = (const T *)a.q + b * a.q_sb + t * a.q_st + head0 * a.q_sh;
    const T *gp = (const T *)p.dout + b * p.do_sb + t * p.do_st + head0 * p.do_sh;
    float lse2[NT][2], delta[NT][2];
#pragma unroll
    for (int i = 0; i < NT; ++i) {
        const int row = 8 * i + r;
#pragma unroll
        for (int d = 0; d < D / 32; ++d) {
            const uint4 zero = make_uint4(0, 0, 0, 0);
            q[i][d] = row < ng ? __ldg((const uint4 *)(qp + row * a.q_sh + 32 * d + 8 * c)) : zero;
            g[i][d] = row < ng ? __ldg((const uint4 *)(gp + row * p.do_sh + 32 * d + 8 * c)) : zero;
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int w = 8 * i + 2 * c + e;
            const float x = w < ng ? p.lse[row0 + w] * kLog2e : -INFINITY;
            lse2[i][e] = x == -INFINITY ? INFINITY : x;     // a row without keys: P = 0
            delta[i][e] = w < ng ? p.delta[row0 + w] : 0.0f;
        }
    }
    float o[D / 16][NT][4] = {};
    DsScale ds_scale;
    const T *kp = (const T *)a.k + b * a.k_sb + h * a.k_sh;
    const T *vp = (const T *)a.v + b * a.v_sb + h * a.v_sh;
    const int per = a.block / 16, all = a.n * per;
    for (int s = warp; s < all; s += kRowWarps) {
        const int j = s / per;
        if (!blk_entry_ok(list, j, a.NB)) continue;
        const int key0 = list[j] * a.block + (s % per) * 16;
        if (key0 >= limit) continue;
        uint4 x[D / 32][2];
        float st[NT][4] = {}, dp[NT][4] = {};
        load_keys<T, D>(x, kp, a.k_st, key0, limit, r, c);
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
            for (int d = 0; d < D / 32; ++d) {
                mma16816<T>(st[i], x[d][0].x, x[d][1].x, x[d][0].y, x[d][1].y, q[i][d].x, q[i][d].y);
                mma16816<T>(st[i], x[d][0].z, x[d][1].z, x[d][0].w, x[d][1].w, q[i][d].z, q[i][d].w);
            }
        load_keys<T, D>(x, vp, a.v_st, key0, limit, r, c);
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
            for (int d = 0; d < D / 32; ++d) {
                mma16816<T>(dp[i], x[d][0].x, x[d][1].x, x[d][0].y, x[d][1].y, g[i][d].x, g[i][d].y);
                mma16816<T>(dp[i], x[d][0].z, x[d][1].z, x[d][0].w, x[d][1].w, g[i][d].z, g[i][d].w);
            }
        uint4 kt[D / 64][4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int key = key0 + 2 * c + (e & 1) + (e >> 1) * 8;
#pragma unroll
            for (int i = 0; i < D / 64; ++i)
                kt[i][e] = key < limit ? __ldg((const uint4 *)(kp + key * a.k_st + 64 * i + 8 * r))
                                       : make_uint4(0, 0, 0, 0);
        }
        float ds_max = 0.0f;
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const bool seen = key0 + r + (e >> 1) * 8 < limit;
                const float pr = ex2(fmaf(st[i][e], scale2, -lse2[i][e & 1]));
                st[i][e] = seen ? pr * (dp[i][e] - delta[i][e & 1]) * a.scale : 0.0f;
                if constexpr (kNarrow<T>) ds_max = finite_max(ds_max, st[i][e]);
            }
        if constexpr (kNarrow<T>) {
            const float f = ds_scale.lower(ds_max);
            if (f != 1.0f)
#pragma unroll
                for (int d = 0; d < D / 16; ++d)
#pragma unroll
                    for (int i = 0; i < NT; ++i)
#pragma unroll
                        for (int e = 0; e < 4; ++e) o[d][i][e] *= f;
            const float u = pow2i(ds_scale.e);
#pragma unroll
            for (int i = 0; i < NT; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) st[i][e] *= u;
        }
#pragma unroll
        for (int i = 0; i < NT; ++i) {
            uint32_t h0, l0, h1, l1;
            split2<T>(st[i][0], st[i][1], h0, l0);
            split2<T>(st[i][2], st[i][3], h1, l1);
            h0 = movmatrix(h0);
            l0 = movmatrix(l0);
            h1 = movmatrix(h1);
            l1 = movmatrix(l1);
#pragma unroll
            for (int d = 0; d < D / 16; ++d) {
                const int u = d / 4, w = d % 4;
                const uint32_t k0 = (&kt[u][0].x)[w], k1 = (&kt[u][1].x)[w];
                const uint32_t k8 = (&kt[u][2].x)[w], k9 = (&kt[u][3].x)[w];
                const uint32_t a0 = __byte_perm(k0, k1, 0x5410), a1 = __byte_perm(k0, k1, 0x7632);
                const uint32_t a2 = __byte_perm(k8, k9, 0x5410), a3 = __byte_perm(k8, k9, 0x7632);
                mma16816<T>(o[d][i], a0, a1, a2, a3, h0, h1);
                mma16816<T>(o[d][i], a0, a1, a2, a3, l0, l1);
            }
        }
    }
    const float unit = kNarrow<T> ? pow2i(-ds_scale.e) : 1.0f;
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int e = 0; e < 2; ++e)
#pragma unroll
            for (int d = 0; d < D / 16; ++d) {
                float *x = &sm[warp][8 * i + 2 * c + e][64 * (d / 4) + 8 * r + 2 * (d % 4)];
                x[0] = o[d][i][e] * unit;
                x[1] = o[d][i][e + 2] * unit;
            }
    __syncthreads();
    constexpr int U = D / 8;
    for (int i = threadIdx.x; i < R * U; i += kRowThreads) {
        const int row = i / U, d = i % U * 8;
        if (row >= ng) continue;
        float x[8] = {};
#pragma unroll
        for (int w = 0; w < kRowWarps; ++w)
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] += sm[w][row][d + e];
        st_pack<T, 8>((T *)p.dq + (row0 + row) * D + d, x);
    }
}

// ---------------------------------------------------------- dQ by tile of rows
struct DqTileArgs {
    TileArgs t;
    const void *dout;
    int64_t do_sb, do_st, do_sh;
    const float *lse, *delta;
    void *dq;
};

// One row, key by key, for rows whose tile gave a result that is not finite (an
// infinite or NaN key times the weight 0 of a row that does not see it), until all
// of it is NaN.
template <typename T, int D>
__device__ __noinline__ void dq_row_alone(const DqTileArgs &p, int b, int h, int t, int head) {
    const BlkArgs &a = p.t.a;
    constexpr int E = D / 32;
    const int lane = threadIdx.x & 31;
    const int limit = blk_limit(a, blk_len(a, b), t);
    const int64_t row = ((int64_t)b * a.Tq + t) * a.Hq + head;
    const float lse2 = p.lse[row] * kLog2e, delta = p.delta[row];
    float q[E], g[E], o[E] = {};
    ld_pack<T, E>((const T *)a.q + b * a.q_sb + t * a.q_st + head * a.q_sh + lane * E, q);
    ld_pack<T, E>((const T *)p.dout + b * p.do_sb + t * p.do_st + head * p.do_sh + lane * E, g);
    const int32_t *list = a.blocks + (((int64_t)b * a.Tq + t) * a.Hk + h) * a.n;
    bool more = lse2 != -INFINITY;
    for (int j = 0; j < a.n && more; ++j) {
        if (!blk_entry_ok(list, j, a.NB)) continue;
        const int k0 = list[j] * a.block, k1 = min(k0 + a.block, limit);
        for (int key = k0; key < k1 && more; ++key) {
            float k[E], v[E], sk = 0.0f, sv = 0.0f;
            ld_pack<T, E>((const T *)a.k + b * a.k_sb + key * a.k_st + h * a.k_sh + lane * E, k);
            ld_pack<T, E>((const T *)a.v + b * a.v_sb + key * a.v_st + h * a.v_sh + lane * E, v);
#pragma unroll
            for (int e = 0; e < E; ++e) {
                sk = fmaf(q[e], k[e], sk);
                sv = fmaf(g[e], v[e], sv);
            }
#pragma unroll
            for (int w = 16; w; w >>= 1) {
                sk += __shfl_xor_sync(0xffffffffu, sk, w);
                sv += __shfl_xor_sync(0xffffffffu, sv, w);
            }
            const float ds = ex2(fmaf(sk, a.scale * kLog2e, -lse2)) * (sv - delta) * a.scale;
#pragma unroll
            for (int e = 0; e < E; ++e) o[e] = fmaf(ds, k[e], o[e]);
            more = !all_nan(o);
        }
    }
    st_pack<T, E>((T *)p.dq + row * D + lane * E, o);
}

constexpr int kDqWarps = 4;          // consumers; two CTAs to an SM
template <int D, int KB> using DqSmem = TileSmem<D, KB, kDqWarps, 2, 113 * 1024>;

template <typename T, int D, int KB>
__global__ void __launch_bounds__(32 * (kDqWarps + 1), 2)
    k_dq_tile(const __grid_constant__ DqTileArgs p) {
    constexpr int W = kDqWarps;
    using S = DqSmem<D, KB>;
    extern __shared__ unsigned char smem_raw[];
    __shared__ uint64_t full[S::stages], empty[S::stages];
    __shared__ TileStage<W> info[S::stages];
    const uint32_t smem = (smem_addr(smem_raw) + 1023u) & ~1023u;
    const BlkArgs &a = p.t.a;
    const TilePlace at(p.t, 16 * W);
    if (threadIdx.x == 0) {
        for (int i = 0; i < S::stages; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], W);
        }
        mbar_init_fence();
    }
    __syncthreads();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, r = lane >> 2, c = lane & 3;
    if (warp == W) {
        tile_produce<S, D, KB, W>(
            p.t, at, smem, full, empty, info,
            (int32_t *)(smem_raw + (smem - smem_addr(smem_raw)) + S::at_lists));
        return;
    }
    const int len = blk_len(a, at.b);
    const float scale2 = a.scale * kLog2e;
    const uint32_t sq = smem + S::at_rows + warp * 16 * D * 2, sg = sq + S::rows;
    {
        int64_t row;
        const bool live = at.row_of(p.t, len, warp * 16 + (lane & 15), row);
        fetch_rows<T, D>(sq, (const T *)a.q, live, at.offset(p.t, row, a.q_sb, a.q_st, a.q_sh));
        fetch_rows<T, D>(sg, (const T *)p.dout, live,
                         at.offset(p.t, row, p.do_sb, p.do_st, p.do_sh));
    }
    int limit[2], qi[2];
    float lse2[2], delta[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        const int64_t f = at.f0 + warp * 16 + r + 8 * e;
        const bool live = f < p.t.rows;
        const int t = live ? (int)(f / a.G) : at.t_first;
        qi[e] = t - at.t_first;
        limit[e] = live ? blk_limit(a, len, t) : 0;
        const float x = live ? p.lse[at.out_row(p.t, f)] * kLog2e : -INFINITY;
        lse2[e] = x == -INFINITY ? INFINITY : x;            // a row without keys: P = 0
        delta[e] = live ? p.delta[at.out_row(p.t, f)] : 0.0f;
    }
    cp_wait<0>();
    __syncwarp();
    const int least_limit = __reduce_min_sync(0xffffffffu, min(limit[0], limit[1]));

    float o[D / 8][4] = {};
    DsScale ds_scale;
    int stage = 0;
    uint32_t parity = 0;
    while (mbar_wait(&full[stage], parity, p.t.err)) {
        const int key0 = info[stage].key0;
        if (key0 < 0) break;
        bool mine[2];
#pragma unroll
        for (int e = 0; e < 2; ++e)
            mine[e] = (info[stage].mask[qi[e] >> 5] >> (qi[e] & 31) & 1u) && key0 < limit[e];
        if (__any_sync(0xffffffffu, mine[0] || mine[1])) {
            const uint32_t sk = smem + stage * S::stage, sv = sk + S::operand;
            if (key0 + KB > len) zero_tail<D, KB>(sk, len - key0);
            float s[KB / 8][4] = {}, dp[KB / 8][4] = {};
#pragma unroll
            for (int i = 0; i < D / 16; ++i) {
                uint32_t q[4], g[4];
                ldsm4(sq + rows_at<D>(lane & 15, 2 * i + (lane >> 4)), q);
                ldsm4(sg + rows_at<D>(lane & 15, 2 * i + (lane >> 4)), g);
#pragma unroll
                for (int n = 0; n < KB / 16; ++n) {
                    uint32_t x[4], y[4];
                    const uint32_t at_ = panel_at<KB>(16 * n + (lane >> 4) * 8 + (lane & 7),
                                                      2 * i + ((lane >> 3) & 1));
                    ldsm4(sk + at_, x);
                    ldsm4(sv + at_, y);
                    mma16816<T>(s[2 * n], q[0], q[1], q[2], q[3], x[0], x[1]);
                    mma16816<T>(s[2 * n + 1], q[0], q[1], q[2], q[3], x[2], x[3]);
                    mma16816<T>(dp[2 * n], g[0], g[1], g[2], g[3], y[0], y[1]);
                    mma16816<T>(dp[2 * n + 1], g[0], g[1], g[2], g[3], y[2], y[3]);
                }
            }
            const bool whole = key0 + KB <= least_limit;
            float ds_max = 0.0f;
#pragma unroll
            for (int n = 0; n < KB / 8; ++n)
#pragma unroll
                for (int w = 0; w < 4; ++w) {
                    const int e = w >> 1;
                    float x = ex2(fmaf(s[n][w], scale2, -lse2[e])) * (dp[n][w] - delta[e]) * a.scale;
                    if (!mine[e] || (!whole && key0 + 8 * n + 2 * c + (w & 1) >= limit[e])) x = 0.0f;
                    s[n][w] = x;
                    if constexpr (kNarrow<T>) ds_max = finite_max(ds_max, x);
                }
            if constexpr (kNarrow<T>) {
                const float f = ds_scale.lower(ds_max);
                if (f != 1.0f)
#pragma unroll
                    for (int n = 0; n < D / 8; ++n)
#pragma unroll
                        for (int w = 0; w < 4; ++w) o[n][w] *= f;
                const float u = pow2i(ds_scale.e);
#pragma unroll
                for (int n = 0; n < KB / 8; ++n)
#pragma unroll
                    for (int w = 0; w < 4; ++w) s[n][w] *= u;
            }
#pragma unroll
            for (int i = 0; i < KB / 16; ++i) {
                uint32_t hi[4], lo[4];
#pragma unroll
                for (int w = 0; w < 4; ++w) {
                    const float x = s[2 * i + (w >> 1)][2 * (w & 1)];
                    const float y = s[2 * i + (w >> 1)][2 * (w & 1) + 1];
                    split2<T>(x, y, hi[w], lo[w]);
                }
#pragma unroll
                for (int n = 0; n < D / 16; ++n) {
                    uint32_t x[4];
                    ldsm4_t(sk + panel_at<KB>(16 * i + (lane & 15), 2 * n + (lane >> 4)), x);
                    mma16816<T>(o[2 * n], hi[0], hi[1], hi[2], hi[3], x[0], x[1]);
                    mma16816<T>(o[2 * n + 1], hi[0], hi[1], hi[2], hi[3], x[2], x[3]);
                    mma16816<T>(o[2 * n], lo[0], lo[1], lo[2], lo[3], x[0], x[1]);
                    mma16816<T>(o[2 * n + 1], lo[0], lo[1], lo[2], lo[3], x[2], x[3]);
                }
            }
            if (key0 + KB > len) fence_proxy_async_shared();   // zeros, then the next copy
            __syncwarp();
        }
        if (lane == 0) mbar_arrive(&empty[stage]);
        if (++stage == S::stages) {
            stage = 0;
            parity ^= 1;
        }
    }
    const float unit = kNarrow<T> ? pow2i(-ds_scale.e) : 1.0f;
    unsigned redo = 0;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        float odd = 0.0f;                          // NaN if anything is not finite
#pragma unroll
        for (int n = 0; n < D / 8; ++n) {
            odd = fmaf(o[n][2 * e], 0.0f, odd);
            odd = fmaf(o[n][2 * e + 1], 0.0f, odd);
        }
        const unsigned bad = __ballot_sync(0xffffffffu, odd != 0.0f);
        const int64_t f = at.f0 + warp * 16 + r + 8 * e;
        const bool live = f < p.t.rows;
        redo |= __ballot_sync(0xffffffffu, c == 0 && live && (bad >> (4 * r) & 15u)) << e;
        if (!live) continue;
        T *out = (T *)p.dq + at.out_row(p.t, f) * D + 2 * c;
#pragma unroll
        for (int n = 0; n < D / 8; ++n)
            *(uint32_t *)(out + 8 * n) = pack2<T>(o[n][2 * e] * unit, o[n][2 * e + 1] * unit);
    }
    __syncwarp();
    while (redo) {                                  // bit 4 r + e: row r + 8 e
        const int bit = __ffs(redo) - 1;
        redo &= redo - 1;
        const int64_t f = at.f0 + warp * 16 + (bit >> 2) + 8 * (bit & 1);
        const int t = (int)(f / a.G);
        dq_row_alone<T, D>(p, at.b, at.h, t, at.h * a.G + (int)(f - (int64_t)t * a.G));
    }
}

// ------------------------------------------- dQ by tile of rows, on tensor memory
// As the forward on tensor memory, for bf16 (fp16's dS needs its scale): 128 rows
// against each block of their union, S = Q K^T and dP = dO V^T, dS by eight warps
// (half a row's keys a thread), dQ += dS K with dS in tensor memory, twice over
// as above. One CTA fills an SM: S and dP of a step run under the dS of the one
// before. 242 us for 2 x 4096 queries x 16 heads of 128 over 2, 16 of 64-key blocks;
// bound like the forward by the chain of a step (the tensor pipe computes 31% of
// the time). By mma.sync it took 333 us.
constexpr int kDqRows = 128, kDqKeys = 64, kDqThreads = 320;   // 8 + producer + issuer
template <int D> using DqMmaSmem = TileSmem<D, kDqKeys, 8, 2, 227 * 1024>;

template <typename T, int D>
__global__ void __launch_bounds__(kDqThreads, 1) k_dq_mma(const __grid_constant__ DqTileArgs p) {
    using S = DqMmaSmem<D>;
    constexpr int KB = kDqKeys, C = D / 8, panel = kDqRows * 128, N = S::stages;
    // tensor memory: two steps' S and dP, their dS (rounded, remainder), dQ
    constexpr int kTmDp = 64, kTmStep = 128, kTmDs = 256, kTmDq = 384, columns = 512;
    extern __shared__ unsigned char smem_raw[];
    __shared__ uint64_t full[N], ready[2], made[2], done[N];   // done: dQ, and the stage is free
    __shared__ uint64_t drained;
    __shared__ TileStage<8> info[N];
    __shared__ uint32_t tmem_slot, odd_rows[4];
    const uint32_t smem = (smem_addr(smem_raw) + 1023u) & ~1023u;
    const uint32_t sq = smem + S::at_rows, sg = sq + S::rows;
    const BlkArgs &a = p.t.a;
    const TilePlace at(p.t, kDqRows);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int len = blk_len(a, at.b);
    if (threadIdx.x == 0) {
        for (int i = 0; i < N; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&done[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&ready[i], 2);
            mbar_init(&made[i], 256);
        }
        mbar_init(&drained, 1);
        mbar_init_fence();
    }
    if (threadIdx.x < 4) odd_rows[threadIdx.x] = 0;
    if (warp == 9) {
        tmem_alloc(&tmem_slot, columns);
        mma_fence_before();
    }
    const int half = warp >> 2, row = (warp & 3) * 32 + lane;     // of warps 0 to 7
    if (warp < 8) {                                 // warps 0-3 fetch Q, 4-7 dO
        int64_t f;
        const bool live = at.row_of(p.t, len, row, f);
        const int64_t mine = !live ? -1
                             : half ? at.offset(p.t, f, p.do_sb, p.do_st, p.do_sh)
                                    : at.offset(p.t, f, a.q_sb, a.q_st, a.q_sh);
        const T *src = (const T *)(half ? p.dout : a.q);
#pragma unroll
        for (int i = 0; i < C; ++i) {
            const int r = i * (32 / C) + lane / C, ch = lane % C;
            const int64_t x = __shfl_sync(0xffffffffu, mine, r);
            cp16((half ? sg : sq) + (ch >> 3) * panel + chunk_at((warp & 3) * 32 + r, ch & 7),
                 src + (x < 0 ? 0 : x + ch * 8), x >= 0);
        }
        cp_commit();
        cp_wait<0>();
        fence_proxy_async_shared();
    }
    __syncthreads();
    mma_fence_after();
    const uint32_t tmem = tmem_slot;

    if (warp == 8) {
        tile_produce<S, D, KB, 8>(
            p.t, at, smem, full, done, info,
            (int32_t *)(smem_raw + (smem - smem_addr(smem_raw)) + S::at_lists));
    } else if (warp == 9) {
        if (lane == 0) {
            constexpr uint32_t qk = instr_f16<T>(kDqRows, KB, false, false);
            constexpr uint32_t sk = instr_f16<T>(kDqRows, D, false, true);
            bool more = true, ok = true;
            for (int j = 0; ok && more; ++j) {
                const int st = j % N, before = (j + N - 1) % N;
                bool a_left = true, b_left = j > 0;
                const uint64_t t0 = global_ns();
                for (uint32_t spin = 1; a_left || b_left; ++spin) {
                    // S and dP take the columns that step j - 2's dS was made from,
                    // and its dS those that step j's will: its product comes first
                    if (a_left && mbar_test(&full[st], (j / N) & 1) &&
                        (j < 2 || mbar_test(&done[(j - 2) % N], ((j - 2) / N) & 1))) {
                        a_left = false;
                        const int key0 = info[st].key0;
                        more = key0 >= 0;
                        mbar_arrive(&ready[j & 1]);  // of what the producer said
                        if (more) {
                            const uint32_t k = smem + st * S::stage, v = k + S::operand;
                            if (key0 + KB > len) {   // keys past the length may be anything
                                zero_tail_one<D, KB>(k, len - key0);
                                fence_proxy_async_shared();
                            }
                            const uint32_t tm = tmem + (j & 1) * kTmStep;
                            mma_fence_after();
#pragma unroll
                            for (int i = 0; i < D / 16; ++i) {
                                const uint32_t r = (i >> 2) * panel + (i & 3) * 32;
                                const uint32_t c = (i >> 2) * KB * 128 + (i & 3) * 32;
                                mma_f16(tm, desc_k(sq + r), desc_k(k + c), qk, i > 0);
                                mma_f16(tm + kTmDp, desc_k(sg + r), desc_k(v + c), qk, i > 0);
                            }
                            mma_commit(&ready[j & 1]);
                        } else {
                            mbar_arrive(&ready[j & 1]);
                        }
                    }
                    if (b_left && mbar_test(&made[(j - 1) & 1], ((j - 1) >> 1) & 1)) {
                        b_left = false;
                        const uint32_t k = smem + before * S::stage;
                        const uint32_t ds = tmem + kTmDs + ((j - 1) & 1) * KB;
                        mma_fence_after();
#pragma unroll
                        for (int w = 0; w < 2; ++w)  // the rounded dS, then the remainder
#pragma unroll
                            for (int i = 0; i < KB / 16; ++i)
                                mma_f16_ta(tmem + kTmDq, ds + w * 32 + i * 8,
                                           desc_mn(k + i * 2048, KB * 128), sk,
                                           j > 1 || w > 0 || i > 0);
                        mma_commit(&done[before]);
                    }
                    if (spin >= kSpinLimit || ((spin & 255) == 0 && global_ns() - t0 > kWaitLimitNs)) {
                        ok = !a_left && !b_left;
                        if (!ok) atomicOr(p.t.err + kErrTimeout, 1);
                        break;
                    }
                }
            }
            if (!ok) mma_drain(&drained, p.t.err);
        }
        __syncwarp();
    } else {
        const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
        const int64_t f = at.f0 + row;
        const bool live = f < p.t.rows;
        const int t = live ? (int)(f / a.G) : at.t_first;
        const int limit = live ? blk_limit(a, len, t) : 0;
        const int qi = t - at.t_first;
        const int64_t o_row = at.out_row(p.t, live ? f : at.f0);
        const float scale2 = a.scale * kLog2e;
        float lse2 = live ? p.lse[o_row] * kLog2e : -INFINITY;
        if (lse2 == -INFINITY) lse2 = INFINITY;      // a row without keys: P = 0
        const float ds_off = live ? -p.delta[o_row] * a.scale : 0.0f;
        int j = 0;
        bool ok = true;
        for (;; ++j) {
            ok = mbar_wait_poll(&ready[j & 1], (j >> 1) & 1, p.t.err);
            if (!ok) break;
            mma_fence_after();
            const TileStage<8> &step = info[j % N];
            const int key0 = step.key0;
            if (key0 < 0) break;
            const bool mine = (step.mask[qi >> 5] >> (qi & 31) & 1u) && key0 < limit;
            uint32_t hi[16], lo[16];
            if (__any_sync(0xffffffffu, mine)) {
                uint32_t s[32], dp[32];
                tmem_ld32(tmem + lanes + (j & 1) * kTmStep + half * 32, s);
                tmem_ld32(tmem + lanes + (j & 1) * kTmStep + kTmDp + half * 32, dp);
                tmem_wait_ld();
                const int seen = mine ? limit - key0 - half * 32 : 0;
                const bool whole = __all_sync(0xffffffffu, seen >= 32);
#pragma unroll
                for (int i = 0; i < 32; i += 2) {
                    float ds[2];
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        ds[e] = ex2(fmaf(__uint_as_float(s[i + e]), scale2, -lse2)) *
                                fmaf(__uint_as_float(dp[i + e]), a.scale, ds_off);
                        if (!whole && i + e >= seen) ds[e] = 0.0f;
                    }
                    split2<T>(ds[0], ds[1], hi[i / 2], lo[i / 2]);
                }
            } else {
#pragma unroll
                for (int i = 0; i < 16; ++i) hi[i] = lo[i] = 0u;
            }
            const uint32_t to = tmem + lanes + kTmDs + (j & 1) * KB + half * 16;
            tmem_st16(to, hi);
            tmem_st16(to + 32, lo);
            tmem_wait_st();
            mma_fence_before();
            mbar_arrive(&made[j & 1]);   // two: a warp may be a step ahead of another
        }
        if (ok && j > 0) mbar_wait_poll(&done[(j - 1) % N], ((j - 1) / N) & 1, p.t.err);
        mma_fence_after();
        float odd = 0.0f;                            // NaN if anything is not finite
#pragma unroll
        for (int i = 0; i < D / 64; ++i) {           // half of the row's elements
            const int d = half * (D / 2) + 32 * i;
            uint32_t o[32];
            if (j > 0) {
                tmem_ld32(tmem + lanes + kTmDq + d, o);
                tmem_wait_ld();
            } else {
#pragma unroll
                for (int e = 0; e < 32; ++e) o[e] = 0u;
            }
#pragma unroll
            for (int e = 0; e < 32; ++e) odd = fmaf(__uint_as_float(o[e]), 0.0f, odd);
            if (live) {
#pragma unroll
                for (int e = 0; e < 32; e += 8) {
                    float x[8];
#pragma unroll
                    for (int w = 0; w < 8; ++w) x[w] = __uint_as_float(o[e + w]);
                    st_pack<T, 8>((T *)p.dq + o_row * D + d + e, x);
                }
            }
        }
        const unsigned bad = __ballot_sync(0xffffffffu, live && odd != 0.0f);
        if (lane == 0 && bad) atomicOr(&odd_rows[warp & 3], bad);
        asm volatile("bar.sync 1, 256;" ::: "memory");
        for (int r = warp; r < kDqRows; r += 8) {
            if (!(odd_rows[r >> 5] >> (r & 31) & 1u)) continue;
            const int64_t g = at.f0 + r;
            const int tt = (int)(g / a.G);
            dq_row_alone<T, D>(p, at.b, at.h, tt, at.h * a.G + (int)(g - (int64_t)tt * a.G));
        }
        mma_fence_before();
    }
    __syncthreads();
    if (warp == 9) {
        mma_fence_after();
        tmem_free(tmem, columns);
    }
}

// ------------------------------------------------------------- dK and dV
// A CTA per (64 keys, kv head, sequence, range of queries), a warp per 16 keys.
// The range's words are expanded to a list of queries, whose (query, head) rows are
// taken 32 at a time: Q and dO rows are gathered into shared memory by asynchronous
// copies, two tiles in flight. 64 keys are NS blocks of 16 or 32: the list is then
// the union of theirs, a row counts for the warps of the blocks that it chose, and
// is gathered once for all of them (with a CTA per block of 16 a training step of 5
// x 784 queries x 6 heads of 128 over 2, 19 of 16-key blocks, took 306 us for 186).
// For fp16, heads of 64, blocks of 16 and 32 keys and few rows; 23 us for 4 x 777
// queries x 4 heads of 64 in fp16, bound by the latency of its gathers and barriers.
constexpr int kRt = 32;             // rows per tile
constexpr int kSegWords = 32;       // words expanded at a time (1024 queries)

// 16-byte chunk `i` of row `row` of a [rows][D] tile: the chunks of eight
// consecutive rows at the same i fall in different banks.
template <int D> __device__ __forceinline__ uint32_t tile_at(int row, int i) {
    return (uint32_t)(row * D * 2 + ((i ^ (row & 7)) << 4));
}

template <typename T, int D, int NS>
__global__ void __launch_bounds__(128) k_dkdv(BwdArgs p) {
    constexpr int KT = 64, C = D / 8, threads = 128, kPer = kRt / 4;   // rows a warp gathers
    extern __shared__ __align__(128) unsigned char smem[];
    // K, V [KT][D]; two stages of Q, dO [kRt][D]; then per stage lse, delta, limit and
    // chosen blocks [kRt]
    const uint32_t sK = smem_addr(smem), sV = sK + KT * D * 2, sQ = sV + KT * D * 2;
    constexpr int stage_bytes = 2 * kRt * D * 2;
    float *row_f = (float *)(smem + 2 * KT * D * 2 + 2 * stage_bytes);   // [2][4][kRt]
    int *list = (int *)(row_f + 2 * 4 * kRt);         // [1024] query, chosen blocks << 27
    __shared__ int word_base[kSegWords + 1];

    const BlkArgs &a = p.a;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, r = lane >> 2, c = lane & 3;
    const int pair = p.pair0 + blockIdx.y, b = pair / a.Hk, h = pair % a.Hk;
    const int chunk = blockIdx.z;
    const int key0 = blockIdx.x * KT, blk = key0 / a.block;
    if (key0 >= a.Tk) return;
    const int len = blk_len(a, b);
    const uint32_t *bits = p.bits + ((int64_t)pair * a.NB + blk) * p.words;
    const int subs = min(NS, a.NB - blk), my_sub = warp * NS / 4;    // of the CTA, of the warp
    const int w_end = min(p.words, (chunk + 1) * p.chunk_words);
    const float scale2 = a.scale * kLog2e, ds_unit = a.scale * kPUnit<T>;

    const T *kp = (const T *)a.k + b * a.k_sb + h * a.k_sh;
    const T *vp = (const T *)a.v + b * a.v_sb + h * a.v_sh;
    for (int i = threadIdx.x; i < KT * C; i += threads) {
        const int row = i / C, d = i % C;
        const int key = key0 + row;
        const bool live = key < len;
        cp16(sK + tile_at<D>(row, d), kp + (live ? key : 0) * a.k_st + d * 8, live);
        cp16(sV + tile_at<D>(row, d), vp + (live ? key : 0) * a.v_st + d * 8, live);
    }
    cp_commit();

    const T *qp = (const T *)a.q + b * a.q_sb + (int64_t)h * a.G * a.q_sh;
    const T *gp = (const T *)p.dout + b * p.do_sb + (int64_t)h * a.G * p.do_sh;
    float dk[D / 8][4] = {}, dv[D / 8][4] = {};
    DsScale ds_scale;
    for (int w0 = chunk * p.chunk_words; w0 < w_end; w0 += kSegWords) {
        __syncthreads();
        if (warp == 0) {                         // counts of the words, then the list
            uint32_t sub[NS], x = 0;
#pragma unroll
            for (int i = 0; i < NS; ++i) {
                sub[i] = i < subs && w0 + lane < w_end ? bits[i * (int64_t)p.words + w0 + lane] : 0u;
                x |= sub[i];
            }
            int n = __popc(x), incl = n;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, incl, o);
                if (lane >= o) incl += y;
            }
            word_base[lane] = incl - n;
            if (lane == 31) word_base[32] = incl;
            int at = incl - n;
            for (uint32_t m = x; m; m &= m - 1) {
                const int bit = __ffs(m) - 1;
                int chosen = 0;
#pragma unroll
                for (int i = 0; i < NS; ++i) chosen |= (int)(sub[i] >> bit & 1u) << i;
                list[at++] = ((w0 + lane) * 32 + bit) | chosen << 27;
            }
        }
        __syncthreads();
        const int rows = word_base[32] * a.G;
        const int steps = (rows + kRt - 1) / kRt;
        auto fetch = [&](int step) {
            const uint32_t base = sQ + (step & 1) * stage_bytes;
            // a warp gathers kPer rows; its first lanes know where they are
            const int row0 = warp * kPer, f = step * kRt + row0 + lane;
            int64_t q_at = -1, g_at = 0;
            float lse2 = INFINITY, delta = 0.0f;
            int limit = 0, chosen = 0;
            if (lane < kPer && f < rows) {
                const int q = f / a.G, g = f - q * a.G;
                const int t = list[q] & ((1 << 27) - 1);
                chosen = (unsigned)list[q] >> 27;
                q_at = t * a.q_st + g * a.q_sh;
                g_at = t * p.do_st + g * p.do_sh;
                const int64_t i = ((int64_t)b * a.Tq + t) * a.Hq + h * a.G + g;
                lse2 = p.lse[i] * kLog2e;
                delta = p.delta[i];
                limit = blk_limit(a, len, t);
            }
#pragma unroll
            for (int i = 0; i < kPer * C / 32; ++i) {
                const int row = i * (32 / C) + lane / C, ch = lane % C;
                const int64_t x = __shfl_sync(0xffffffffu, q_at, row);
                const int64_t y = __shfl_sync(0xffffffffu, g_at, row);
                const uint32_t at = base + tile_at<D>(row0 + row, ch);
                cp16(at, qp + (x < 0 ? 0 : x + ch * 8), x >= 0);
                cp16(at + kRt * D * 2, gp + (x < 0 ? 0 : y + ch * 8), x >= 0);
            }
            cp_commit();
            if (lane < kPer) {
                float *m = row_f + (step & 1) * 4 * kRt + row0 + lane;
                m[0] = lse2 == -INFINITY ? INFINITY : lse2;  // a row without keys: P = 0
                m[kRt] = delta;
                m[2 * kRt] = __int_as_float(limit);
                m[3 * kRt] = __int_as_float(chosen);
            }
        };
        if (steps) fetch(0);
        for (int step = 0; step < steps; ++step) {
            if (step + 1 < steps) {
                fetch(step + 1);
                cp_wait<1>();
            } else {
                cp_wait<0>();
            }
            __syncthreads();
            const uint32_t tq = sQ + (step & 1) * stage_bytes, tg = tq + kRt * D * 2;
            const float *m = row_f + (step & 1) * 4 * kRt;
            // a warp whose block none of the rows chose goes without
            if (NS > 1 && !__any_sync(0xffffffffu,
                                      __float_as_int(m[3 * kRt + lane]) >> my_sub & 1)) {
                __syncthreads();
                continue;
            }
            float st[4][4] = {}, dp[4][4] = {};
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
                uint32_t ka[4], va[4];
                // A: rows (keys) lane % 16 of the warp's 16, chunk 2 kk + lane / 16
                const uint32_t at = tile_at<D>(warp * 16 + (lane & 15), 2 * kk + (lane >> 4));
                ldsm4(sK + at, ka);
                ldsm4(sV + at, va);
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    // B: rows 16 i + (lane / 16) 8 + lane % 8, chunk 2 kk + (lane / 8) % 2
                    uint32_t x[4];
                    const uint32_t bt = tile_at<D>(16 * i + (lane >> 4) * 8 + (lane & 7),
                                                   2 * kk + ((lane >> 3) & 1));
                    ldsm4(tq + bt, x);
                    mma16816<T>(st[2 * i], ka[0], ka[1], ka[2], ka[3], x[0], x[1]);
                    mma16816<T>(st[2 * i + 1], ka[0], ka[1], ka[2], ka[3], x[2], x[3]);
                    ldsm4(tg + bt, x);
                    mma16816<T>(dp[2 * i], va[0], va[1], va[2], va[3], x[0], x[1]);
                    mma16816<T>(dp[2 * i + 1], va[0], va[1], va[2], va[3], x[2], x[3]);
                }
            }
            uint32_t pa[4][2], da[4][2], dl[4][2];   // P^T, dS^T, its rest: keys r and r + 8
            float ds_max = 0.0f;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int row = 8 * i + 2 * c;
                const float2 l = *(const float2 *)(m + row), d = *(const float2 *)(m + kRt + row);
                int2 lim = *(const int2 *)(m + 2 * kRt + row);
                if (NS > 1) {
                    const int2 in = *(const int2 *)(m + 3 * kRt + row);
                    if (!(in.x >> my_sub & 1)) lim.x = 0;
                    if (!(in.y >> my_sub & 1)) lim.y = 0;
                }
                float pr[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int key = key0 + warp * 16 + r + (e >> 1) * 8;
                    const bool seen = key < (e & 1 ? lim.y : lim.x);
                    pr[e] = seen ? ex2(fmaf(st[i][e], scale2, kPShift<T> - (e & 1 ? l.y : l.x))) : 0.0f;
                    st[i][e] = seen ? pr[e] * (dp[i][e] - (e & 1 ? d.y : d.x)) * ds_unit : 0.0f;
                    if constexpr (kNarrow<T>) ds_max = finite_max(ds_max, st[i][e]);
                }
                // one part: dV = P^T dO does not cancel as dQ does, and is off by no more
                // than the output is by its P
                pa[i][0] = pack2<T>(pr[0], pr[1]);
                pa[i][1] = pack2<T>(pr[2], pr[3]);
            }
            float u = 1.0f;
            if constexpr (kNarrow<T>) {
                const float f = ds_scale.lower(ds_max);
                if (f != 1.0f)
#pragma unroll
                    for (int n = 0; n < D / 8; ++n)
#pragma unroll
                        for (int e = 0; e < 4; ++e) dk[n][e] *= f;
                u = pow2i(ds_scale.e);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                split2<T>(st[i][0] * u, st[i][1] * u, da[i][0], dl[i][0]);
                split2<T>(st[i][2] * u, st[i][3] * u, da[i][1], dl[i][1]);
            }
#pragma unroll
            for (int i = 0; i < 2; ++i)          // 16 rows at a time
#pragma unroll
                for (int n = 0; n < D / 16; ++n) {
                    uint32_t x[4];
                    // B: row 16 i + lane % 16, chunk 2 n + lane / 16, transposed
                    const uint32_t bt = tile_at<D>(16 * i + (lane & 15), 2 * n + (lane >> 4));
                    ldsm4_t(tg + bt, x);
                    mma16816<T>(dv[2 * n], pa[2 * i][0], pa[2 * i][1], pa[2 * i + 1][0],
                                pa[2 * i + 1][1], x[0], x[1]);
                    mma16816<T>(dv[2 * n + 1], pa[2 * i][0], pa[2 * i][1], pa[2 * i + 1][0],
                                pa[2 * i + 1][1], x[2], x[3]);
                    ldsm4_t(tq + bt, x);
                    mma16816<T>(dk[2 * n], da[2 * i][0], da[2 * i][1], da[2 * i + 1][0],
                                da[2 * i + 1][1], x[0], x[1]);
                    mma16816<T>(dk[2 * n + 1], da[2 * i][0], da[2 * i][1], da[2 * i + 1][0],
                                da[2 * i + 1][1], x[2], x[3]);
                    mma16816<T>(dk[2 * n], dl[2 * i][0], dl[2 * i][1], dl[2 * i + 1][0],
                                dl[2 * i + 1][1], x[0], x[1]);
                    mma16816<T>(dk[2 * n + 1], dl[2 * i][0], dl[2 * i][1], dl[2 * i + 1][0],
                                dl[2 * i + 1][1], x[2], x[3]);
                }
            __syncthreads();
        }
    }
    cp_wait<0>();
    const float k_unit = kNarrow<T> ? pow2i(-ds_scale.e) : 1.0f, v_unit = kPUnit<T>;
#pragma unroll
    for (int n = 0; n < D / 8; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            dk[n][e] *= k_unit;
            dv[n][e] *= v_unit;
        }
    unsigned redo_k = 0, redo_v = 0;             // bit 4 r + e: key r + 8 e is not finite
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        float odd_k = 0.0f, odd_v = 0.0f;
#pragma unroll
        for (int n = 0; n < D / 8; ++n) {
            odd_k += (dk[n][2 * e] + dk[n][2 * e + 1]) * 0.0f;
            odd_v += (dv[n][2 * e] + dv[n][2 * e + 1]) * 0.0f;
        }
        const unsigned bad_k = __ballot_sync(0xffffffffu, odd_k != 0.0f);
        const unsigned bad_v = __ballot_sync(0xffffffffu, odd_v != 0.0f);
        const bool live = key0 + warp * 16 + r + 8 * e < a.Tk && c == 0;
        redo_k |= __ballot_sync(0xffffffffu, live && (bad_k >> (4 * r) & 15u)) << e;
        redo_v |= __ballot_sync(0xffffffffu, live && (bad_v >> (4 * r) & 15u)) << e;
    }
    // keys r and r + 8 of the warp's 16, elements 8 n + 2 c and the next
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        const int key = key0 + warp * 16 + r + 8 * e;
        if (key >= a.Tk) continue;
        const int64_t at = (((int64_t)b * a.Tk + key) * a.Hk + h) * D + 2 * c;
#pragma unroll
        for (int n = 0; n < D / 8; ++n) {
            if (p.chunks == 1) {
                *(uint32_t *)((T *)p.dk + at + 8 * n) = pack2<T>(dk[n][2 * e], dk[n][2 * e + 1]);
                *(uint32_t *)((T *)p.dv + at + 8 * n) = pack2<T>(dv[n][2 * e], dv[n][2 * e + 1]);
            } else {
                float *x = p.part + (int64_t)(2 * chunk) * p.part_stride + at + 8 * n;
                *(float2 *)x = make_float2(dk[n][2 * e], dk[n][2 * e + 1]);
                *(float2 *)(x + p.part_stride) = make_float2(dv[n][2 * e], dv[n][2 * e + 1]);
            }
        }
    }
    __syncwarp();
    for (unsigned redo = redo_k | redo_v; redo; redo &= redo - 1) {
        const int bit = __ffs(redo) - 1;
        const bool want_k = redo_k >> bit & 1u, want_v = redo_v >> bit & 1u;
        constexpr int E = D / 32;
        const int key = key0 + warp * 16 + (bit >> 2) + 8 * (bit & 1);
        float x[E], y[E];
        dkdv_key_alone<T, D>(
            p, b, h, key, want_k, want_v,
            [&](auto body) {
                const uint32_t *mine = bits + my_sub * (int64_t)p.words;
                for (int w = chunk * p.chunk_words; w < w_end; ++w)
                    for (uint32_t m = mine[w]; m; m &= m - 1)
                        if (!body(w * 32 + __ffs(m) - 1)) return;
            },
            x, y);
        const int64_t at = (((int64_t)b * a.Tk + key) * a.Hk + h) * D + lane * E;
        float *part = p.part + (int64_t)(2 * chunk) * p.part_stride + at;
        if (p.chunks == 1) {
            if (want_k) st_pack<T, E>((T *)p.dk + at, x);
            if (want_v) st_pack<T, E>((T *)p.dv + at, y);
        } else {
            if (want_k) st_pack<float, E>(part, x);
            if (want_v) st_pack<float, E>(part + p.part_stride, y);
        }
    }
}

// The ranges' parts, added in order.
template <typename T> __global__ void __launch_bounds__(256) k_dkdv_join(BwdArgs p) {
    const int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 8;
    if (i >= p.part_stride) return;
#pragma unroll
    for (int w = 0; w < 2; ++w) {
        float s[8];
        ld_pack<float, 8>(p.part + w * p.part_stride + i, s);
        for (int ch = 1; ch < p.chunks; ++ch) {
            float x[8];
            ld_pack<float, 8>(p.part + (2 * ch + w) * p.part_stride + i, x);
#pragma unroll
            for (int e = 0; e < 8; ++e) s[e] += x[e];
        }
        st_pack<T, 8>((T *)(w ? p.dv : p.dk) + i, s);
    }
}

// ------------------------------------------------------------------- host
struct BwdPlan {
    int64_t words, chunk_words, chunks;
    int64_t bits_bytes, delta_bytes, part_bytes;
    bool keys;               // k_dkdv_keys, over at most so many tiles and items
    int64_t tiles = 0, items = 0;
};

// The tensor-core kernel: bf16 (fp16 needs dS scaled as it goes, which sums in
// tensor memory do not allow), heads of 128 (its second products' M), blocks of
// whole 64-key tiles, and enough rows that its 128-row steps fill.
bool by_keys(const spmm_blocks_shape *s) {
    return s->dtype == SPMM_BF16 && s->D == kKeysD && s->block % kKeysN == 0 &&
           s->Tq * (s->Hq / s->Hk) >= 2 * kKeysRows;
}

// Ranges of queries per key block: enough CTAs to fill the SMs several times
// over (and to cut up a block that every query chose), each of 256 queries or more.
BwdPlan bwd_plan(const spmm_blocks_shape *s) {
    BwdPlan p;
    const int64_t NB = (s->Tk + s->block - 1) / s->block;
    p.words = (s->Tq + 31) / 32;
    const int64_t ctas = std::max<int64_t>(1, s->B * s->Hk * ((s->Tk + 63) / 64));
    int64_t chunks = std::min<int64_t>((152 * 8 + ctas - 1) / ctas, (p.words + 7) / 8);
    chunks = std::max<int64_t>(1, std::min<int64_t>(chunks, 64));
    p.chunk_words = std::max<int64_t>(1, (p.words + chunks - 1) / chunks);
    p.chunks = std::max<int64_t>(1, (p.words + p.chunk_words - 1) / p.chunk_words);
    p.bits_bytes = round_up(s->B * s->Hk * NB * p.words * 4, 256);
    p.delta_bytes = round_up(s->B * s->Tq * s->Hq * 4, 256);
    p.part_bytes = p.chunks > 1 ? p.chunks * 2 * s->B * s->Tk * s->Hk * s->D * 4 : 0;
    p.keys = by_keys(s);
    if (p.keys) {
        const int64_t parts = s->block / kKeysN;
        p.tiles = s->B * s->Hk * NB * parts;
        p.items = p.tiles + s->B * s->Tq * s->Hk * s->n * parts / kKeysSegment;   // at most
        p.chunks = 1;
        p.part_bytes = round_up((p.tiles + 1) * 4, 256) + round_up(p.items * 8, 256) +
                       p.items * 2 * kKeysN * kKeysD * 4;
    }
    return p;
}

template <typename T, int D, int NS>
cudaError_t launch_dkdv(BwdArgs &p, int64_t B, cudaStream_t s) {
    const size_t smem = 2 * 64 * D * 2 + 4 * kRt * D * 2 + 2 * 4 * kRt * 4 + kSegWords * 32 * 4;
    const cudaError_t e = cudaFuncSetAttribute(
        k_dkdv<T, D, NS>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    const int64_t pairs = B * p.a.Hk;
    for (int64_t i = 0; i < pairs; i += kPairs) {
        p.pair0 = (int)i;
        k_dkdv<T, D, NS><<<dim3((unsigned)((p.a.Tk + 63) / 64), (unsigned)std::min(kPairs, pairs - i),
                                (unsigned)p.chunks),
                           128, smem, s>>>(p);
        count_launch();
    }
    return cudaGetLastError();
}

template <typename T> cudaError_t launch_keys(BwdArgs &p, const BwdPlan &bp, cudaStream_t s) {
    char *w = (char *)p.part;
    p.keys.tiles = bp.tiles;
    p.keys.first = (int32_t *)w;
    p.keys.item = (int2 *)(w + round_up((bp.tiles + 1) * 4, 256));
    p.keys.part = (float *)((char *)p.keys.item + round_up(bp.items * 8, 256));
    cudaError_t e = dynamic_err(s, &p.err);
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute(k_dkdv_keys<T>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 kKeysSmem);
    if (e != cudaSuccess) return e;
    const int64_t blocks = bp.tiles / (p.a.block / kKeysN);
    k_key_counts<<<(unsigned)((blocks + 7) / 8), 256, 0, s>>>(p);
    k_key_items<<<1, 1024, 0, s>>>(p);
    k_dkdv_keys<T><<<(unsigned)bp.items, kKeysThreads, kKeysSmem, s>>>(p);
    k_keys_join<T><<<dim3((unsigned)bp.tiles, 8), 256, 0, s>>>(p);
    count_launch(4);
    return cudaGetLastError();
}

template <typename T, int D, int KB>
cudaError_t launch_dq_tile(DqTileArgs &p, int64_t B, cudaStream_t s) {
    constexpr int bytes = DqSmem<D, KB>::bytes;
    const cudaError_t e = cudaFuncSetAttribute(
        k_dq_tile<T, D, KB>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != cudaSuccess) return e;
    p.t.tiles = (int)((p.t.rows + 16 * kDqWarps - 1) / (16 * kDqWarps));
    k_dq_tile<T, D, KB><<<dim3((unsigned)p.t.tiles, (unsigned)(B * p.t.a.Hk)), 32 * (kDqWarps + 1),
                          bytes, s>>>(p);
    count_launch();
    return cudaGetLastError();
}

template <typename T, int D> cudaError_t launch_dq_mma(DqTileArgs &p, int64_t B, cudaStream_t s) {
    constexpr int bytes = DqMmaSmem<D>::bytes;
    const cudaError_t e = cudaFuncSetAttribute(
        k_dq_mma<T, D>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != cudaSuccess) return e;
    p.t.tiles = (int)((p.t.rows + kDqRows - 1) / kDqRows);
    k_dq_mma<T, D><<<dim3((unsigned)p.t.tiles, (unsigned)(B * p.t.a.Hk)), kDqThreads, bytes, s>>>(p);
    count_launch();
    return cudaGetLastError();
}

template <typename T, int D>
cudaError_t launch_dq_by_tile(DqTileArgs &p, int64_t B, cudaStream_t s) {
    if (p.t.a.block == 16) return launch_dq_tile<T, D, 16>(p, B, s);
    if (p.t.a.block == 32) return launch_dq_tile<T, D, 32>(p, B, s);
    if constexpr (kNarrow<T>) return launch_dq_tile<T, D, 64>(p, B, s);
    else return launch_dq_mma<T, D>(p, B, s);
}

template <typename T, int D>
cudaError_t launch_bwd(BwdArgs &p, const BwdPlan &bp, const spmm_blocks_shape *s, spmm_rows k,
                       spmm_rows v, cudaStream_t cs) {
    const int64_t rows = s->B * s->Tq * s->Hq, lists = s->B * s->Tq * s->Hk;
    cudaError_t e = cudaSuccess;
    constexpr int per = 128 / (D / 8);
    k_delta<T, D><<<(unsigned)((rows + per - 1) / per), 128, 0, cs>>>(p, rows, bp.bits_bytes / 4);
    count_launch();
    if (blocks_by_tile(s, k, v)) {
        DqTileArgs t{};
        t.t.a = p.a;
        t.t.rows = s->Tq * p.a.G;
        t.dout = p.dout;
        t.do_sb = p.do_sb;
        t.do_st = p.do_st;
        t.do_sh = p.do_sh;
        t.lse = p.lse;
        t.delta = p.delta;
        t.dq = p.dq;
        const int box = (int)std::min<int64_t>(s->block, 64);
        e = dynamic_err(cs, &t.t.err);
        if (e == cudaSuccess) e = encode_rows(k, s, box, &t.t.k_map);
        if (e == cudaSuccess) e = encode_rows(v, s, box, &t.t.v_map);
        if (e == cudaSuccess)
            e = launch_dq_by_tile<T, D>(t, s->B, cs);
    } else {
        if (p.a.G <= 8) {
            p.gt = 1;
            k_dq_rows<T, D, 1><<<(unsigned)lists, kRowThreads, 0, cs>>>(p);
        } else {
            p.gt = (p.a.G + 15) / 16;
            k_dq_rows<T, D, 2><<<(unsigned)(lists * p.gt), kRowThreads, 0, cs>>>(p);
        }
        count_launch();
        e = cudaGetLastError();
    }
    if (e != cudaSuccess || s->Tk == 0) return e;
    const int64_t entries = lists * s->n;
    k_set_bits<<<(unsigned)((entries + 255) / 256), 256, 0, cs>>>(p, entries);
    count_launch();
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    if (bp.keys) {
        if constexpr (D == kKeysD && !kNarrow<T>) e = launch_keys<T>(p, bp, cs);
        return e;
    }
    if (s->block == 16) e = launch_dkdv<T, D, 4>(p, s->B, cs);
    else if (s->block == 32) e = launch_dkdv<T, D, 2>(p, s->B, cs);
    else e = launch_dkdv<T, D, 1>(p, s->B, cs);
    if (e != cudaSuccess || p.chunks == 1) return e;
    k_dkdv_join<T><<<(unsigned)((p.part_stride / 8 + 255) / 256), 256, 0, cs>>>(p);
    count_launch();
    return cudaGetLastError();
}

}  // namespace
}  // namespace spmm

extern "C" {

int64_t spmm_blocks_backward_workspace(const spmm_blocks_shape *s) {
    using namespace spmm;
    if (blk_check(s, true) != SPMM_OK) return 0;
    const BwdPlan p = bwd_plan(s);
    return p.bits_bytes + p.delta_bytes + p.part_bytes;
}

spmm_status spmm_blocks_backward(const spmm_blocks_shape *s, spmm_rows q, spmm_rows k,
                                 spmm_rows v, const int32_t *blocks, const void *out,
                                 const float *lse, spmm_rows dout, void *dq, void *dk, void *dv,
                                 void *work, int64_t work_bytes, void *stream) {
    using namespace spmm;
    const spmm_status st = blk_check(s, true);
    if (st != SPMM_OK) return st;
    if (s->B == 0 || (s->Tq == 0 && s->Tk == 0)) return SPMM_OK;
    cudaStream_t cs = (cudaStream_t)stream;
    if (s->Tk > 0 && (!dk || !dv || (uintptr_t)dk % 16 || (uintptr_t)dv % 16))
        return SPMM_ERR_INVALID_ARG;
    if (s->Tq == 0) {
        const size_t bytes = (size_t)(s->B * s->Tk * s->Hk * s->D * 2);
        cudaError_t e = cudaMemsetAsync(dk, 0, bytes, cs);
        if (e == cudaSuccess) e = cudaMemsetAsync(dv, 0, bytes, cs);
        return cuda_status(e);
    }
    if (!blocks || !lse || !out || (uintptr_t)out % 16 || !dq || (uintptr_t)dq % 16)
        return SPMM_ERR_INVALID_ARG;
    if (!rows_ok(q, 2) || !rows_ok(dout, 2) ||
        (s->Tk > 0 && (!rows_ok(k, 2) || !rows_ok(v, 2))))
        return SPMM_ERR_INVALID_ARG;
    const BwdPlan bp = bwd_plan(s);
    if (!work || (uintptr_t)work % 16 || work_bytes < bp.bits_bytes + bp.delta_bytes + bp.part_bytes)
        return SPMM_ERR_INVALID_ARG;
    // launches of 2^31 CTAs: more lists, keys or items than memory holds
    if ((s->B * s->Tq * s->Hk * s->n + 255) / 256 > INT32_MAX || bp.items > INT32_MAX ||
        s->B * s->Tk * s->Hk * s->D / 2048 >= INT32_MAX)
        return SPMM_ERR_UNSUPPORTED;
    BwdArgs p{};
    p.a = blk_args(s, blocks);
    set_rows(p.a.q, p.a.q_sb, p.a.q_st, p.a.q_sh, q);
    set_rows(p.a.k, p.a.k_sb, p.a.k_st, p.a.k_sh, k);
    set_rows(p.a.v, p.a.v_sb, p.a.v_st, p.a.v_sh, v);
    set_rows(p.dout, p.do_sb, p.do_st, p.do_sh, dout);
    p.out = out;
    p.lse = lse;
    p.dq = dq;
    p.dk = dk;
    p.dv = dv;
    char *w = (char *)work;
    p.bits = (uint32_t *)w;
    p.delta = (float *)(w + bp.bits_bytes);
    p.part = (float *)(w + bp.bits_bytes + bp.delta_bytes);
    p.part_stride = s->B * s->Tk * s->Hk * s->D;
    p.words = (int)bp.words;
    p.chunks = (int)bp.chunks;
    p.chunk_words = (int)bp.chunk_words;
    cudaError_t e;
    if (s->dtype == SPMM_BF16)
        e = s->D == 64 ? launch_bwd<__nv_bfloat16, 64>(p, bp, s, k, v, cs)
                       : launch_bwd<__nv_bfloat16, 128>(p, bp, s, k, v, cs);
    else
        e = s->D == 64 ? launch_bwd<__half, 64>(p, bp, s, k, v, cs) : launch_bwd<__half, 128>(p, bp, s, k, v, cs);
    return cuda_status(e);
}

}  // extern "C"
