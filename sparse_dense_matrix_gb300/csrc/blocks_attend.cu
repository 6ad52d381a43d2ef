// Selected-block attention, forward. By query: a CTA takes the G query rows that
// share one list (a query and its group of heads) and walks the list's keys, 16
// at a time per warp, with the running maximum m and sum l of a softmax:
//   S^T = K Q^T (keys x rows), P^T = exp(scale S^T - m), O^T += V^T P^T.
// The keys are the M dimension of the 16x8x16 matrix instruction and the rows
// its N = 8, so a group of up to 8 heads wastes nothing, and K and V go from
// memory straight into fragments: a lane reads 16 adjacent bytes of a key's row
// and the order of the summed index is permuted to suit (Q is read the same
// way; for V^T two keys' words are interleaved).
#include "blocks.cuh"

namespace spmm {
namespace {

constexpr int kRowWarps = 4;
constexpr int kRowThreads = 32 * kRowWarps;

struct RowArgs {
    BlkArgs a;
    int gt;                  // tiles of 8 NT rows per group
    int splits;              // CTAs per list
    void *out;               // [B, Tq, Hq, D]
    float *lse;              // [B, Tq, Hq]
    float *part_o;           // [item][splits][8 NT][D]: O / l of a split's keys
    float *part_lse;         // [item][splits][8 NT], in powers of 2
};

// Registers of 16 keys: rows r and r + 8 of the slice for K, keys 2c, 2c+1,
// 2c+8, 2c+9 for V (r = lane / 4, c = lane % 4).
template <int D> struct Slice {
    uint4 k[D / 32][2];
    uint4 v[D / 64][4];
};

template <typename T, int D>
__device__ __forceinline__ void load_slice(Slice<D> &x, const T *k, const T *v, int64_t k_st,
                                           int64_t v_st, int key0, int limit, int r, int c) {
    const uint4 zero = make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        const int key = key0 + r + 8 * e;
        const bool live = key < limit;
#pragma unroll
        for (int i = 0; i < D / 32; ++i)
            x.k[i][e] = live ? __ldg((const uint4 *)(k + key * k_st + 32 * i + 8 * c)) : zero;
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const int key = key0 + 2 * c + (e & 1) + (e >> 1) * 8;
        // past the limit a value is 0, whatever the memory holds: its weight is
        // 0, and 0 times what lies there might be NaN
        const bool live = key < limit;
#pragma unroll
        for (int i = 0; i < D / 64; ++i)
            x.v[i][e] = live ? __ldg((const uint4 *)(v + key * v_st + 64 * i + 8 * r)) : zero;
    }
}

template <typename T, int D, int NT>
__global__ void __launch_bounds__(kRowThreads) k_attend_rows(RowArgs p) {
    constexpr int R = 8 * NT;                       // rows of the CTA
    __shared__ float sm_o[kRowWarps][R][D + 4];
    __shared__ float sm_m[kRowWarps][R], sm_l[kRowWarps][R];
    const BlkArgs &a = p.a;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, r = lane >> 2, c = lane & 3;
    const int64_t item = blockIdx.x / p.splits;
    const int split = blockIdx.x % p.splits;
    const int gt = (int)(item % p.gt);
    const int64_t list_id = item / p.gt;            // (b, t, h)
    const int h = (int)(list_id % a.Hk);
    const int64_t bt = list_id / a.Hk;
    const int t = (int)(bt % a.Tq), b = (int)(bt / a.Tq);
    const int g0 = gt * R, ng = min(a.G - g0, R);
    const int limit = blk_limit(a, blk_len(a, b), t);
    const int32_t *list = a.blocks + list_id * a.n;
    const float scale2 = a.scale * kLog2e;

    // Q^T fragments: column r of n-tile i is row g0 + 8 i + r
    uint4 q[NT][D / 32];
    const T *qp = (const T *)a.q + b * a.q_sb + t * a.q_st + (int64_t)(h * a.G + g0) * a.q_sh;
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int d = 0; d < D / 32; ++d)
            q[i][d] = 8 * i + r < ng
                          ? __ldg((const uint4 *)(qp + (8 * i + r) * a.q_sh + 32 * d + 8 * c))
                          : make_uint4(0, 0, 0, 0);

    float o[D / 16][NT][4];
    float m[NT][2], l[NT][2];                       // of rows 8 i + 2 c + (0, 1); m in powers of 2
#pragma unroll
    for (int i = 0; i < NT; ++i) {
        m[i][0] = m[i][1] = -INFINITY;
        l[i][0] = l[i][1] = 0.0f;
#pragma unroll
        for (int d = 0; d < D / 16; ++d)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[d][i][e] = 0.0f;
    }

    const T *kp = (const T *)a.k + b * a.k_sb + h * a.k_sh;
    const T *vp = (const T *)a.v + b * a.v_sb + h * a.v_sh;
    const int per = a.block / 16;                   // slices per block
    const int all = a.n * per;
    const int s0 = (int)((int64_t)all * split / p.splits);
    const int s1 = (int)((int64_t)all * (split + 1) / p.splits);
    for (int s = s0 + warp; s < s1; s += kRowWarps) {
        const int j = s / per;
        if (!blk_entry_ok(list, j, a.NB)) continue;
        const int key0 = list[j] * a.block + (s % per) * 16;
        if (key0 >= limit) continue;
        Slice<D> x;
        load_slice<T, D>(x, kp, vp, a.k_st, a.v_st, key0, limit, r, c);
#pragma unroll
        for (int i = 0; i < NT; ++i) {
            float st[4] = {};
#pragma unroll
            for (int d = 0; d < D / 32; ++d) {
                mma16816<T>(st, x.k[d][0].x, x.k[d][1].x, x.k[d][0].y, x.k[d][1].y, q[i][d].x, q[i][d].y);
                mma16816<T>(st, x.k[d][0].z, x.k[d][1].z, x.k[d][0].w, x.k[d][1].w, q[i][d].z, q[i][d].w);
            }
            // lane: keys r (st[0], st[1]) and r + 8 (st[2], st[3]), rows 2c and 2c + 1
            float pr[4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
                pr[e] = key0 + r + (e >> 1) * 8 < limit ? st[e] * scale2 : -INFINITY;
            float corr[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float mx = fmaxf(pr[e], pr[e + 2]);
#pragma unroll
                for (int w = 4; w < 32; w <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, w));
                mx = fmaxf(mx, m[i][e]);
                const float base = mx == -INFINITY ? 0.0f : mx;
                corr[e] = ex2(m[i][e] - base);
                m[i][e] = mx;
                pr[e] = ex2(pr[e] - base);
                pr[e + 2] = ex2(pr[e + 2] - base);
                l[i][e] = l[i][e] * corr[e] + pr[e] + pr[e + 2];
            }
            // P is rounded to the inputs' type for the matrix instruction; l sums
            // the unrounded weights
            const uint32_t b0 = movmatrix(pack2<T>(pr[0], pr[1]));
            const uint32_t b1 = movmatrix(pack2<T>(pr[2], pr[3]));
#pragma unroll
            for (int d = 0; d < D / 16; ++d) {
                const int u = d / 4, w = d % 4;
                const uint32_t k0 = (&x.v[u][0].x)[w], k1 = (&x.v[u][1].x)[w];
                const uint32_t k8 = (&x.v[u][2].x)[w], k9 = (&x.v[u][3].x)[w];
                o[d][i][0] *= corr[0];
                o[d][i][1] *= corr[1];
                o[d][i][2] *= corr[0];
                o[d][i][3] *= corr[1];
                // row r of the tile is element 64 u + 8 r + 2 w, row r + 8 the next
                mma16816<T>(o[d][i], __byte_perm(k0, k1, 0x5410), __byte_perm(k0, k1, 0x7632),
                            __byte_perm(k8, k9, 0x5410), __byte_perm(k8, k9, 0x7632), b0, b1);
            }
        }
    }
    // the warps' parts
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
#pragma unroll
            for (int w = 4; w < 32; w <<= 1) l[i][e] += __shfl_xor_sync(0xffffffffu, l[i][e], w);
            const int row = 8 * i + 2 * c + e;
            if (r == 0) {
                sm_m[warp][row] = m[i][e];
                sm_l[warp][row] = l[i][e];
            }
#pragma unroll
            for (int u = 0; u < D / 64; ++u) {
                float4 lo, hi;
                lo.x = o[4 * u][i][e];     lo.y = o[4 * u][i][e + 2];
                lo.z = o[4 * u + 1][i][e]; lo.w = o[4 * u + 1][i][e + 2];
                hi.x = o[4 * u + 2][i][e]; hi.y = o[4 * u + 2][i][e + 2];
                hi.z = o[4 * u + 3][i][e]; hi.w = o[4 * u + 3][i][e + 2];
                *(float4 *)&sm_o[warp][row][64 * u + 8 * r] = lo;
                *(float4 *)&sm_o[warp][row][64 * u + 8 * r + 4] = hi;
            }
        }
    __syncthreads();
    constexpr int U = D / 8;
    for (int i = threadIdx.x; i < R * U; i += kRowThreads) {
        const int row = i / U, d = i % U * 8;
        if (row >= ng) continue;
        float mx = -INFINITY;
#pragma unroll
        for (int w = 0; w < kRowWarps; ++w) mx = fmaxf(mx, sm_m[w][row]);
        const float base = mx == -INFINITY ? 0.0f : mx;
        float sum = 0.0f, x[8] = {};
#pragma unroll
        for (int w = 0; w < kRowWarps; ++w) {
            const float f = ex2(sm_m[w][row] - base);
            sum = fmaf(sm_l[w][row], f, sum);
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] = fmaf(sm_o[w][row][d + e], f, x[e]);
        }
        const float inv = sum != 0.0f ? __fdiv_rn(1.0f, sum) : 0.0f;   // NaN stays NaN
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] *= inv;
        const float lse2 = sum != 0.0f ? base + log2f(sum) : -INFINITY;
        if (p.splits == 1) {
            const int64_t o_row = (int64_t)bt * a.Hq + h * a.G + g0 + row;
            st_pack<T, 8>((T *)p.out + o_row * D + d, x);
            if (d == 0) p.lse[o_row] = lse2 * kLn2;
        } else {
            const int64_t o_row = ((int64_t)item * p.splits + split) * R + row;
            st_pack<float, 8>(p.part_o + o_row * D + d, x);
            if (d == 0) p.part_lse[o_row] = lse2;
        }
    }
}

// The splits' parts of a row: out = sum_s 2^(lse_s - lse) O_s.
template <typename T, int D>
__global__ void __launch_bounds__(128) k_attend_join(RowArgs p, int R, int64_t rows) {
    constexpr int U = D / 8;
    const int64_t i = (int64_t)blockIdx.x * (128 / U) + threadIdx.x / U;   // (b, t, head)
    if (i >= rows) return;
    const int d = threadIdx.x % U * 8;
    const BlkArgs &a = p.a;
    const int head = (int)(i % a.Hq);
    const int64_t bt = i / a.Hq;
    const int h = head / a.G, g = head % a.G;
    const int64_t first = ((bt * a.Hk + h) * p.gt + g / R) * p.splits * R + g % R;
    float mx = -INFINITY;
    for (int s = 0; s < p.splits; ++s) mx = fmaxf(mx, p.part_lse[first + (int64_t)s * R]);
    const float base = mx == -INFINITY ? 0.0f : mx;
    float sum = 0.0f, x[8] = {};
    for (int s = 0; s < p.splits; ++s) {
        const float f = ex2(p.part_lse[first + (int64_t)s * R] - base);
        float y[8];
        ld_pack<float, 8>(p.part_o + (first + (int64_t)s * R) * D + d, y);
        sum += f;
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = fmaf(y[e], f, x[e]);
    }
    const float inv = sum != 0.0f ? __fdiv_rn(1.0f, sum) : 0.0f;
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] *= inv;
    st_pack<T, 8>((T *)p.out + i * D + d, x);
    if (d == 0) p.lse[i] = (sum != 0.0f ? base + log2f(sum) : -INFINITY) * kLn2;
}

// ------------------------------------------------------------------- host
struct RowPlan {
    int nt, gt, splits;
    int64_t items;
};

// Splits of a list: enough CTAs for a few per SM, while each warp of a split
// keeps at least one slice of 16 keys.
RowPlan row_plan(const spmm_blocks_shape *s) {
    RowPlan p;
    const int64_t G = s->Hq / s->Hk;
    p.nt = G > 8 ? 2 : 1;
    p.gt = (int)((G + 8 * p.nt - 1) / (8 * p.nt));
    p.items = s->B * s->Tq * s->Hk * p.gt;
    const int64_t slices = s->n * (s->block / 16);
    int64_t most = std::max<int64_t>(1, slices / kRowWarps);
    most = std::min<int64_t>(most, 64);
    const int64_t want = p.items > 0 ? (152 * 4 + p.items - 1) / p.items : 1;
    p.splits = (int)std::max<int64_t>(1, std::min(most, want));
    return p;
}

template <typename T, int D>
cudaError_t launch_rows(const RowArgs &p, const RowPlan &rp, int64_t rows, cudaStream_t s) {
    const unsigned grid = (unsigned)(rp.items * rp.splits);
    if (rp.nt == 1) k_attend_rows<T, D, 1><<<grid, kRowThreads, 0, s>>>(p);
    else k_attend_rows<T, D, 2><<<grid, kRowThreads, 0, s>>>(p);
    count_launch();
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || rp.splits == 1) return e;
    constexpr int per = 128 / (D / 8);
    k_attend_join<T, D><<<(unsigned)((rows + per - 1) / per), 128, 0, s>>>(p, 8 * rp.nt, rows);
    count_launch();
    return cudaGetLastError();
}

}  // namespace
}  // namespace spmm

extern "C" {

int64_t spmm_blocks_attend_workspace(const spmm_blocks_shape *s) {
    using namespace spmm;
    if (blk_check(s, true) != SPMM_OK) return 0;
    const RowPlan p = row_plan(s);
    if (p.splits == 1) return 0;
    return p.items * p.splits * 8 * p.nt * (s->D + 1) * 4;
}

spmm_status spmm_blocks_attend(const spmm_blocks_shape *s, spmm_rows q, spmm_rows k, spmm_rows v,
                               const int32_t *blocks, void *out, float *lse, void *work,
                               int64_t work_bytes, void *stream) {
    using namespace spmm;
    const spmm_status st = blk_check(s, true);
    if (st != SPMM_OK) return st;
    if (s->B == 0 || s->Tq == 0) return SPMM_OK;
    if (!blocks || !lse || !out || (uintptr_t)out % 16) return SPMM_ERR_INVALID_ARG;
    if (!rows_ok(q, 2) || (s->Tk > 0 && (!rows_ok(k, 2) || !rows_ok(v, 2))))
        return SPMM_ERR_INVALID_ARG;
    const int64_t need = spmm_blocks_attend_workspace(s);
    if (need && (!work || (uintptr_t)work % 16 || work_bytes < need)) return SPMM_ERR_INVALID_ARG;
    RowArgs p{};
    p.a = blk_args(s, blocks);
    set_rows(p.a.q, p.a.q_sb, p.a.q_st, p.a.q_sh, q);
    set_rows(p.a.k, p.a.k_sb, p.a.k_st, p.a.k_sh, k);
    set_rows(p.a.v, p.a.v_sb, p.a.v_st, p.a.v_sh, v);
    const RowPlan rp = row_plan(s);
    if (rp.items * rp.splits > INT32_MAX) return SPMM_ERR_UNSUPPORTED;
    p.gt = rp.gt;
    p.splits = rp.splits;
    p.out = out;
    p.lse = lse;
    p.part_o = (float *)work;
    p.part_lse = p.part_o + rp.items * rp.splits * 8 * rp.nt * s->D;
    cudaStream_t cs = (cudaStream_t)stream;
    const int64_t rows = s->B * s->Tq * s->Hq;
    cudaError_t e;
    if (s->dtype == SPMM_BF16)
        e = s->D == 64 ? launch_rows<__nv_bfloat16, 64>(p, rp, rows, cs)
                       : launch_rows<__nv_bfloat16, 128>(p, rp, rows, cs);
    else
        e = s->D == 64 ? launch_rows<__half, 64>(p, rp, rows, cs)
                       : launch_rows<__half, 128>(p, rp, rows, cs);
    return cuda_status(e);
}

}  // extern "C"
