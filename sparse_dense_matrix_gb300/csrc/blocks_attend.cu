// Selected-block attention, forward. By query: a CTA takes the G query rows that
// share one list (a query and its group of heads) and walks the list's keys, 16
// at a time per warp, with the running maximum m and sum l of a softmax:
//   S^T = K Q^T (keys x rows), P^T = exp(scale S^T - m), O^T += V^T P^T.
// The keys are the M dimension of the 16x8x16 matrix instruction and the rows
// its N = 8, so a group of up to 8 heads wastes nothing, and K and V go from
// memory straight into fragments: a lane reads 16 adjacent bytes of a key's row
// and the order of the summed index is permuted to suit (Q is read the same
// way; for V^T two keys' words are interleaved). Bound by memory, and short of its
// rate by the latency of a few rounds of loads: 33 us for 64 caches of up to 32768
// keys, 16 of 64-key blocks of each of 4 heads of 128 (123 MB, 3.7 TB/s).
#include <cudaTypedefs.h>

#include <cstring>

#include "blocks_tile.cuh"
#include "umma.cuh"

namespace spmm {
namespace {

PFN_cuTensorMapEncodeTiled_v12000 g_encode = nullptr;

// Warps of a CTA: eight for one n-tile (two CTAs per SM, 128 registers), four for two.
template <int NT> constexpr int kRowWarps = NT == 1 ? 8 : 4;

struct RowArgs {
    BlkArgs a;
    int gt;                  // tiles of 8 NT rows per group
    int splits;              // CTAs per list: the CTAs of a cluster
    void *out;               // [B, Tq, Hq, D]
    float *lse;              // [B, Tq, Hq]
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

__device__ __forceinline__ void cluster_barrier() {
    asm volatile("barrier.cluster.arrive.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
}

// The same shared variable of CTA `rank` of the cluster (this one is `mine`).
__device__ __forceinline__ const float *peer(const float *x, int rank, int mine) {
    if (rank == mine) return x;
    uint64_t y;
    asm("mapa.u64 %0, %1, %2;" : "=l"(y) : "l"(x), "r"(rank));
    return (const float *)y;
}

template <typename T, int D, int NT>
__global__ void __launch_bounds__(32 * kRowWarps<NT>, 2) k_attend_rows(RowArgs p) {
    constexpr int R = 8 * NT;                       // rows of the CTA
    constexpr int W = kRowWarps<NT>, threads = 32 * W;
    __shared__ __align__(16) float sm_o[W][R][D + 4];
    __shared__ float sm_m[W][R], sm_l[W][R];
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
    const int s1 = (int)((int64_t)all * (split + 1) / p.splits);
    int s = (int)((int64_t)all * split / p.splits) + warp;
    // first key of the warp's next slice that counts, or -1
    auto next = [&]() {
        for (; s < s1; s += W) {
            const int j = s / per;
            if (!blk_entry_ok(list, j, a.NB)) continue;
            const int key0 = list[j] * a.block + (s % per) * 16;
            if (key0 >= limit) continue;
            s += W;
            return key0;
        }
        return -1;
    };
    auto add = [&](const Slice<D> &x, int key0) {
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
            // P is rounded to the inputs' type, as the matrix instruction takes nothing
            // wider next to V (two parts of it would double that product): each weight
            // is off by up to 2^-8 (bf16) or 2^-11 (fp16) of itself, independently, and
            // the output's error is 1.1 to 1.4 times that of rounding it alone. l sums the
            // unrounded weights
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
    };
    // One slice at a time: the other warps of the SM cover its loads (a second
    // slice in registers would halve their number)
    Slice<D> x;
    for (int key0 = next(); key0 >= 0; key0 = next()) {
        load_slice<T, D>(x, kp, vp, a.k_st, a.v_st, key0, limit, r, c);
        add(x, key0);
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
    // the CTA's parts join in its first warp's buffers, an element per thread
    __shared__ float cta_m[R], cta_l[R];
    for (int i = threadIdx.x; i < R * D; i += threads) {
        const int row = i / D, d = i % D;
        float mx = -INFINITY;
#pragma unroll
        for (int w = 0; w < W; ++w) mx = fmaxf(mx, sm_m[w][row]);
        const float base = mx == -INFINITY ? 0.0f : mx;
        float sum = 0.0f, x = 0.0f;
#pragma unroll
        for (int w = 0; w < W; ++w) {
            const float f = ex2(sm_m[w][row] - base);
            sum = fmaf(sm_l[w][row], f, sum);
            x = fmaf(sm_o[w][row][d], f, x);
        }
        sm_o[0][row][d] = x;
        if (d == 0) {
            cta_m[row] = mx;
            cta_l[row] = sum;
        }
    }
    // Then the cluster's CTAs, each finishing a share of the elements from
    // everybody's shared memory: no second launch, no scratch.
    if (p.splits > 1) cluster_barrier();
    else __syncthreads();
    for (int i = split * threads + threadIdx.x; i < ng * D; i += p.splits * threads) {
        const int row = i / D, d = i % D;
        float mx = -INFINITY, sum = 0.0f, x = 0.0f;
        for (int v = 0; v < p.splits; ++v) mx = fmaxf(mx, *peer(&cta_m[row], v, split));
        const float base = mx == -INFINITY ? 0.0f : mx;
        for (int v = 0; v < p.splits; ++v) {
            const float f = ex2(*peer(&cta_m[row], v, split) - base);
            sum = fmaf(*peer(&cta_l[row], v, split), f, sum);
            x = fmaf(*peer(&sm_o[0][row][d], v, split), f, x);
        }
        x *= sum != 0.0f ? __fdiv_rn(1.0f, sum) : 0.0f;                // NaN stays NaN
        const int64_t o_row = (int64_t)bt * a.Hq + h * a.G + g0 + row;
        ((T *)p.out)[o_row * D + d] = from_f32<T>(x);
        if (d == 0) p.lse[o_row] = sum != 0.0f ? (base + log2f(sum)) * kLn2 : -INFINITY;
    }
    if (p.splits > 1) cluster_barrier();            // nobody leaves while it is read
}

// ------------------------------------------------------------- by tile of rows
struct AttendTileArgs {
    TileArgs t;
    void *out;
    float *lse;
};

// One row, key by key, for rows whose tile gave a result that is not finite: in
// the tile a value that is infinite or NaN times the weight 0 of a row that does
// not see it spoils that row's sums too (not its lse); here each row meets the
// keys it sees only, until all of it is NaN. (A row whose sum of weights is NaN is NaN
// throughout as it stands.)
template <typename T, int D>
__device__ __noinline__ void attend_row_alone(const AttendTileArgs &p, int b, int h, int t, int head) {
    const BlkArgs &a = p.t.a;
    constexpr int E = D / 32;
    const int lane = threadIdx.x & 31;
    const int limit = blk_limit(a, blk_len(a, b), t);
    const float scale2 = a.scale * kLog2e;
    float q[E], o[E] = {}, m = -INFINITY, l = 0.0f;
    ld_pack<T, E>((const T *)a.q + b * a.q_sb + t * a.q_st + head * a.q_sh + lane * E, q);
    const int32_t *list = a.blocks + (((int64_t)b * a.Tq + t) * a.Hk + h) * a.n;
    bool more = true;
    for (int j = 0; j < a.n && more; ++j) {
        if (!blk_entry_ok(list, j, a.NB)) continue;
        const int k0 = list[j] * a.block, k1 = min(k0 + a.block, limit);
        for (int key = k0; key < k1 && more; ++key) {
            float x[E], dot = 0.0f;
            ld_pack<T, E>((const T *)a.k + b * a.k_sb + key * a.k_st + h * a.k_sh + lane * E, x);
#pragma unroll
            for (int e = 0; e < E; ++e) dot = fmaf(q[e], x[e], dot);
#pragma unroll
            for (int w = 16; w; w >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, w);
            const float s = dot * scale2, mx = fmaxf(m, s);
            const float base = mx == -INFINITY ? 0.0f : mx;
            const float corr = ex2(m - base), pr = ex2(s - base);
            m = mx;
            l = fmaf(l, corr, pr);
            ld_pack<T, E>((const T *)a.v + b * a.v_sb + key * a.v_st + h * a.v_sh + lane * E, x);
            const float pt = to_f32(from_f32<T>(pr));
#pragma unroll
            for (int e = 0; e < E; ++e) o[e] = fmaf(pt, x[e], o[e] * corr);
            more = !all_nan(o);
        }
    }
    const float inv = l != 0.0f ? __fdiv_rn(1.0f, l) : 0.0f;
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] *= inv;
    const int64_t row = ((int64_t)b * a.Tq + t) * a.Hq + head;
    st_pack<T, E>((T *)p.out + row * D + lane * E, o);
}

// For blocks of 16 and 32 keys; the longer ones go to k_attend_mma. Four consumer
// warps a CTA, two CTAs to an SM: the consumers wait for one another over the
// ring, and the other CTA's work while they do (one CTA of 11 warps took 300 us for
// 277 at 2 x 4096 queries x 4 heads of 64 x 4, and 39 for 28 at 4 x 777).
constexpr int kTileWarps = 4;
template <int D, int KB> using AttendSmem = TileSmem<D, KB, kTileWarps, 1, 113 * 1024>;

template <typename T, int D, int KB>
__global__ void __launch_bounds__(32 * (kTileWarps + 1), 2)
    k_attend_tile(const __grid_constant__ AttendTileArgs p) {
    constexpr int W = kTileWarps;
    using S = AttendSmem<D, KB>;
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
    // the warp's Q rows; then rows r and r + 8 of its 16
    const uint32_t sq = smem + S::at_rows + warp * 16 * D * 2;
    {
        int64_t row;
        const bool live = at.row_of(p.t, len, warp * 16 + (lane & 15), row);
        fetch_rows<T, D>(sq, (const T *)a.q, live, at.offset(p.t, row, a.q_sb, a.q_st, a.q_sh));
    }
    int limit[2], qi[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        const int64_t f = at.f0 + warp * 16 + r + 8 * e;
        const int t = f < p.t.rows ? (int)(f / a.G) : at.t_first;
        qi[e] = t - at.t_first;
        limit[e] = f < p.t.rows ? blk_limit(a, len, t) : 0;
    }
    cp_wait<0>();
    __syncwarp();
    const int least_limit = __reduce_min_sync(0xffffffffu, min(limit[0], limit[1]));

    float o[D / 8][4] = {}, m[2] = {-INFINITY, -INFINITY}, l[2] = {};
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
            if (key0 + KB > len) zero_tail<D, KB>(sv, len - key0);
            float s[KB / 8][4] = {};
#pragma unroll
            for (int i = 0; i < D / 16; ++i) {
                uint32_t q[4];
                ldsm4(sq + rows_at<D>(lane & 15, 2 * i + (lane >> 4)), q);
#pragma unroll
                for (int n = 0; n < KB / 16; ++n) {
                    uint32_t x[4];
                    ldsm4(sk + panel_at<KB>(16 * n + (lane >> 4) * 8 + (lane & 7),
                                            2 * i + ((lane >> 3) & 1)), x);
                    mma16816<T>(s[2 * n], q[0], q[1], q[2], q[3], x[0], x[1]);
                    mma16816<T>(s[2 * n + 1], q[0], q[1], q[2], q[3], x[2], x[3]);
                }
            }
            // a key past some row's limit, or rows that did not choose the block
            const bool whole = key0 + KB <= least_limit;
            float corr[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float mx = -INFINITY;
#pragma unroll
                for (int n = 0; n < KB / 8; ++n)
#pragma unroll
                    for (int w = 0; w < 2; ++w) {
                        float x = s[n][2 * e + w] * scale2;
                        if (!mine[e] || (!whole && key0 + 8 * n + 2 * c + w >= limit[e]))
                            x = -INFINITY;
                        s[n][2 * e + w] = x;
                        mx = fmaxf(mx, x);
                    }
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
                mx = fmaxf(mx, m[e]);
                const float base = mx == -INFINITY ? 0.0f : mx;
                corr[e] = ex2(m[e] - base);
                m[e] = mx;
                float sum = 0.0f;
#pragma unroll
                for (int n = 0; n < KB / 8; ++n)
#pragma unroll
                    for (int w = 0; w < 2; ++w) {
                        s[n][2 * e + w] = ex2(s[n][2 * e + w] - base);
                        sum += s[n][2 * e + w];
                    }
                l[e] = fmaf(l[e], corr[e], sum);
            }
            if (__any_sync(0xffffffffu, corr[0] != 1.0f || corr[1] != 1.0f)) {
#pragma unroll
                for (int n = 0; n < D / 8; ++n) {
                    o[n][0] *= corr[0];
                    o[n][1] *= corr[0];
                    o[n][2] *= corr[1];
                    o[n][3] *= corr[1];
                }
            }
            // P is rounded to the inputs' type for the matrix instruction, as by query
            // (k_attend_rows says what that costs); l sums the unrounded weights
#pragma unroll
            for (int i = 0; i < KB / 16; ++i) {
                const uint32_t a0 = pack2<T>(s[2 * i][0], s[2 * i][1]);
                const uint32_t a1 = pack2<T>(s[2 * i][2], s[2 * i][3]);
                const uint32_t a2 = pack2<T>(s[2 * i + 1][0], s[2 * i + 1][1]);
                const uint32_t a3 = pack2<T>(s[2 * i + 1][2], s[2 * i + 1][3]);
#pragma unroll
                for (int n = 0; n < D / 16; ++n) {
                    uint32_t x[4];
                    ldsm4_t(sv + panel_at<KB>(16 * i + (lane & 15), 2 * n + (lane >> 4)), x);
                    mma16816<T>(o[2 * n], a0, a1, a2, a3, x[0], x[1]);
                    mma16816<T>(o[2 * n + 1], a0, a1, a2, a3, x[2], x[3]);
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
    unsigned redo = 0;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        l[e] += __shfl_xor_sync(0xffffffffu, l[e], 1);
        l[e] += __shfl_xor_sync(0xffffffffu, l[e], 2);
        float odd = l[e] * 0.0f;                   // NaN if anything is not finite
#pragma unroll
        for (int n = 0; n < D / 8; ++n) {
            odd = fmaf(o[n][2 * e], 0.0f, odd);
            odd = fmaf(o[n][2 * e + 1], 0.0f, odd);
        }
        const unsigned bad = __ballot_sync(0xffffffffu, odd != 0.0f && !isnan(l[e]));
        const bool live = at.f0 + warp * 16 + r + 8 * e < p.t.rows;
        redo |= __ballot_sync(0xffffffffu, c == 0 && live && (bad >> (4 * r) & 15u)) << e;
        if (!live) continue;
        const float inv = l[e] != 0.0f ? __fdiv_rn(1.0f, l[e]) : 0.0f;
        const int64_t row = at.out_row(p.t, at.f0 + warp * 16 + r + 8 * e);
        T *out = (T *)p.out + row * D + 2 * c;
#pragma unroll
        for (int n = 0; n < D / 8; ++n)
            *(uint32_t *)(out + 8 * n) = pack2<T>(o[n][2 * e] * inv, o[n][2 * e + 1] * inv);
        if (c == 0)
            p.lse[row] = l[e] != 0.0f ? ((m[e] == -INFINITY ? 0.0f : m[e]) + log2f(l[e])) * kLn2
                                      : -INFINITY;
    }
    __syncwarp();
    while (redo) {                                  // bit 4 r + e: row r + 8 e
        const int bit = __ffs(redo) - 1;
        redo &= redo - 1;
        const int64_t f = at.f0 + warp * 16 + (bit >> 2) + 8 * (bit & 1);
        const int tt = (int)(f / a.G);
        attend_row_alone<T, D>(p, at.b, at.h, tt, at.h * a.G + (int)(f - (int64_t)tt * a.G));
    }
}

// ------------------------------------------- by tile of rows, on tensor memory
// The tile's 128 rows against each block of its union: S = Q K^T and O += P V by
// tcgen05.mma, S, P and O in tensor memory, a thread per row between the two
// products. A row that did not choose a block has P = 0 there. O is rescaled only
// when a row's maximum has grown by more than 2^8 since (its P then reach 2^8 at
// most, and l and O carry the same factor). Two CTAs share an SM: one's products
// run under the other's exponentials. 291 us for 8192 queries x 32 heads of 128 over
// 4, 16 of 64-key blocks (126 GFLOP of the rows' own keys, 433 TFLOP/s; the tiles'
// unions are twice that). Bound by the chain of a step (S, the row's weights, O),
// of which two CTAs and two steps' S overlap a part: the tensor pipe computes 39%
// of the time. Q in tensor memory, which leaves room for one S only, took 421 us;
// two threads to a row, whose registers leave room for one CTA only, 531; mma.sync
// 511.
constexpr int kMmaRows = 128, kMmaKeys = 64, kMmaThreads = 192;   // 4 + producer + issuer
template <int D> using MmaSmem = TileSmem<D, kMmaKeys, 8, 1, 113 * 1024>;

template <typename T, int D>
__global__ void __launch_bounds__(kMmaThreads, 2) k_attend_mma(const __grid_constant__
                                                                  AttendTileArgs p) {
    using S = MmaSmem<D>;
    constexpr int KB = kMmaKeys, C = D / 8, panel = kMmaRows * 128;
    constexpr int kTmO = 128, columns = 256;         // S and P of two steps, then O
    extern __shared__ unsigned char smem_raw[];
    // K and V have a ring each: a step's K is read by its S alone, and the K of a
    // later step comes in its place while the step's P is still being made
    constexpr int N = S::stages;
    // (S done: ready, which is also when its K may go; P V done: done, and its V)
    __shared__ uint64_t k_full[N], v_full[N], ready[N], done[N], made[2], drained;
    __shared__ TileStage<8> info[N + 2];             // alive from a step's K to its P
    __shared__ uint32_t tmem_slot;
    const uint32_t smem = (smem_addr(smem_raw) + 1023u) & ~1023u;
    const BlkArgs &a = p.t.a;
    const TilePlace at(p.t, kMmaRows);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int len = blk_len(a, at.b);
    if (threadIdx.x == 0) {
        for (int i = 0; i < N; ++i) {
            mbar_init(&k_full[i], 1);
            mbar_init(&v_full[i], 1);
            mbar_init(&ready[i], 2);
            mbar_init(&done[i], 1);
        }
        mbar_init(&drained, 1);
        mbar_init(&made[0], kMmaRows);
        mbar_init(&made[1], kMmaRows);
        mbar_init_fence();
    }
    if (warp == 5) {
        tmem_alloc(&tmem_slot, columns);
        mma_fence_before();
    }
    const int row = threadIdx.x;                     // of warps 0 to 3
    if (warp < 4) {
        int64_t f;
        const bool live = at.row_of(p.t, len, row, f);
        const int64_t mine = live ? at.offset(p.t, f, a.q_sb, a.q_st, a.q_sh) : -1;
#pragma unroll
        for (int i = 0; i < C; ++i) {                // 32 chunks at a time
            const int r = i * (32 / C) + lane / C, ch = lane % C;
            const int64_t x = __shfl_sync(0xffffffffu, mine, r);
            cp16(smem + S::at_rows + (ch >> 3) * panel + chunk_at(warp * 32 + r, ch & 7),
                 (const T *)a.q + (x < 0 ? 0 : x + ch * 8), x >= 0);
        }
        cp_commit();
        cp_wait<0>();
        fence_proxy_async_shared();
    }
    __syncthreads();
    mma_fence_after();
    const uint32_t tmem = tmem_slot;

    const uint32_t sk = smem, sv = smem + N * S::operand;
    if (warp == 4) {
        // ------------------------------------------------ bring K, and V a step later
        TileMerge<8> merge(p.t, at, (int32_t *)(smem_raw + (smem - smem_addr(smem_raw)) +
                                                S::at_lists), S::lists);
        int j = 0, v_key0 = -1;                      // of step j - 1
        bool ok = true, last = false;
        auto bring_v = [&]() {                       // V of step j - 1
            if (v_key0 < 0) return;
            const int st = (j - 1) % N;
            ok = mbar_wait_poll(&done[st], (((j - 1) / N) & 1) ^ 1, p.t.err);
            if (ok && lane == 0) {
                mbar_arrive_expect_tx(&v_full[st], S::operand);
#pragma unroll
                for (int x = 0; x < D / 64; ++x)
                    tensor4d_g2s(sv + st * S::operand + x * KB * 128, &p.t.v_map, 64 * x, v_key0,
                                 at.h, at.b, &v_full[st]);
            }
            __syncwarp();
        };
        while (ok && !last) {
            const int least = merge.step();
            last = least == merge.kNone;
            const int parts = last ? 1 : a.block / KB;
            for (int s = 0; s < parts && ok; ++s) {
                const int key0 = last ? -1 : least * a.block + s * KB;
                if (key0 >= len) break;  // nobody sees the second half of a last, short block
                const int st = j % N;
                ok = mbar_wait_poll(&ready[st], ((j / N) & 1) ^ 1, p.t.err);
                if (!ok) break;
                if (lane == 0) {
                    TileStage<8> &x = info[j % (N + 2)];
                    x.key0 = key0;
#pragma unroll
                    for (int i = 0; i < merge.kLists; ++i) x.mask[i] = merge.mask[i];
                    if (key0 < 0) {
                        mbar_arrive(&k_full[st]);
                    } else {
                        mbar_arrive_expect_tx(&k_full[st], S::operand);
#pragma unroll
                        for (int y = 0; y < D / 64; ++y)
                            tensor4d_g2s(sk + st * S::operand + y * KB * 128, &p.t.k_map, 64 * y,
                                         key0, at.h, at.b, &k_full[st]);
                    }
                }
                __syncwarp();
                bring_v();
                v_key0 = key0;
                ++j;
            }
        }
        if (!ok) {  // somebody gave up: see the copies in flight land before the CTA ends
            for (int i = max(0, j - N); i < j; ++i) {
                mbar_wait(&k_full[i % N], (i / N) & 1, p.t.err);
                mbar_wait(&v_full[i % N], (i / N) & 1, p.t.err);
            }
        }
    } else if (warp == 5) {
        // ------------------------------------------------ issue the products
        if (lane == 0) {
            constexpr uint32_t qk = instr_f16<T>(kMmaRows, KB, false, false);
            constexpr uint32_t pv = instr_f16<T>(kMmaRows, D, false, true);
            // S of a step and O of the step before wait for different things:
            // whichever is ready goes first. S takes the columns of the P of two
            // steps before, which its product must have read: two products that
            // write different columns need not run in the order of their issue.
            bool more = true, ok = true;
            int v_key0 = -1;                         // of step j - 1
            for (int j = 0; ok && more; ++j) {
                const int st = j % N, before = (j + N - 1) % N;
                bool a_left = true, b_left = j > 0;
                int key0 = -1;
                const uint64_t t0 = global_ns();
                for (uint32_t spin = 1; a_left || b_left; ++spin) {
                    if (a_left && mbar_test(&k_full[st], (j / N) & 1) &&
                        (j < 2 || mbar_test(&done[(j - 2) % N], ((j - 2) / N) & 1))) {
                        a_left = false;
                        key0 = info[j % (N + 2)].key0;
                        more = key0 >= 0;
                        mbar_arrive(&ready[st]);  // of what the bringing warp said
                        if (more) {
                            const uint32_t k = sk + st * S::operand;
                            mma_fence_after();
#pragma unroll
                            for (int i = 0; i < D / 16; ++i)
                                mma_f16(tmem + (j & 1) * KB,
                                        desc_k(smem + S::at_rows + (i >> 2) * panel + (i & 3) * 32),
                                        desc_k(k + (i >> 2) * KB * 128 + (i & 3) * 32), qk, i > 0);
                            mma_commit(&ready[st]);
                        } else {
                            mbar_arrive(&ready[st]);
                        }
                    }
                    if (b_left && mbar_test(&made[(j - 1) & 1], ((j - 1) >> 1) & 1) &&
                        mbar_test(&v_full[before], ((j - 1) / N) & 1)) {
                        b_left = false;
                        const uint32_t v = sv + before * S::operand;
                        if (v_key0 + KB > len) {     // values past the length may be anything
                            zero_tail_one<D, KB>(v, len - v_key0);
                            fence_proxy_async_shared();
                        }
                        mma_fence_after();
#pragma unroll
                        for (int i = 0; i < KB / 16; ++i)
                            mma_f16_ta(tmem + kTmO, tmem + ((j - 1) & 1) * KB + i * 8,
                                       desc_mn(v + i * 2048, KB * 128), pv, j > 1 || i > 0);
                        mma_commit(&done[before]);
                    }
                    if (spin >= kSpinLimit || ((spin & 255) == 0 && global_ns() - t0 > kWaitLimitNs)) {
                        ok = !a_left && !b_left;
                        if (!ok) atomicOr(p.t.err + kErrTimeout, 1);
                        break;
                    }
                }
                v_key0 = key0;
            }
            if (!ok) mma_drain(&drained, p.t.err);
        }
        __syncwarp();
    } else {
        const uint32_t lanes = (uint32_t)(warp * 32) << 16;
        const int64_t f = at.f0 + row;
        const bool live = f < p.t.rows;
        const int t = live ? (int)(f / a.G) : at.t_first;
        const int limit = live ? blk_limit(a, len, t) : 0;
        const int qi = t - at.t_first;
        const float scale2 = a.scale * kLog2e;
        float m = -INFINITY, l = 0.0f;               // m: what P is relative to, in powers of 2
        int j = 0;
        bool ok = true;
        for (;; ++j) {
            ok = mbar_wait_poll(&ready[j % N], (j / N) & 1, p.t.err);
            if (!ok) break;
            mma_fence_after();
            const TileStage<8> &step = info[j % (N + 2)];
            const int key0 = step.key0;
            if (key0 < 0) break;
            const bool mine = (step.mask[qi >> 5] >> (qi & 31) & 1u) && key0 < limit;
            const uint32_t s_at = tmem + lanes + (j & 1) * KB;
            uint32_t pp[32];
            if (__any_sync(0xffffffffu, mine)) {
                uint32_t s[2][32];
                tmem_ld32(s_at, s[0]);
                tmem_ld32(s_at + 32, s[1]);
                tmem_wait_ld();
                const int seen = mine ? limit - key0 : 0;
                if (__any_sync(0xffffffffu, seen < KB)) {
#pragma unroll
                    for (int i = 0; i < KB; ++i)
                        if (i >= seen) s[i >> 5][i & 31] = 0xff800000u;   // -infinity
                }
                float mx = -INFINITY;
#pragma unroll
                for (int i = 0; i < KB; ++i) mx = fmaxf(mx, __uint_as_float(s[i >> 5][i & 31]));
                mx *= scale2;
                if (!mine) mx = -INFINITY;
                float corr = 1.0f;
                if (m == -INFINITY) {
                    m = mx;                          // nothing of this row is in O yet
                } else if (mx > m + 8.0f) {
                    corr = ex2(m - mx);
                    m = mx;
                }
                if (j > 0 && __any_sync(0xffffffffu, corr != 1.0f)) {
                    ok = mbar_wait_poll(&done[(j - 1) % N], ((j - 1) / N) & 1, p.t.err);
                    if (!ok) break;
                    mma_fence_after();
#pragma unroll
                    for (int i = 0; i < D / 32; ++i) {
                        uint32_t o[32];
                        tmem_ld32(tmem + lanes + kTmO + 32 * i, o);
                        tmem_wait_ld();
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            o[e] = __float_as_uint(__uint_as_float(o[e]) * corr);
                        tmem_st32(tmem + lanes + kTmO + 32 * i, o);
                    }
                }
                const float base = m == -INFINITY ? 0.0f : m;
                float sum = 0.0f;
#pragma unroll
                for (int i = 0; i < KB; i += 2) {
                    float x = ex2(fmaf(__uint_as_float(s[i >> 5][i & 31]), scale2, -base));
                    float y = ex2(fmaf(__uint_as_float(s[i >> 5][(i & 31) + 1]), scale2, -base));
                    if (!mine) x = y = 0.0f;
                    sum += x + y;
                    pp[i / 2] = pack2<T>(x, y);      // rounded as by query; l sums the unrounded
                }
                l = fmaf(l, corr, sum);
            } else {
#pragma unroll
                for (int i = 0; i < 32; ++i) pp[i] = 0u;
            }
            tmem_st32(s_at, pp);
            tmem_wait_st();
            mma_fence_before();
            mbar_arrive(&made[j & 1]);   // two: a warp may be a step ahead of another
        }
        if (ok && j > 0) mbar_wait_poll(&done[(j - 1) % N], ((j - 1) / N) & 1, p.t.err);
        mma_fence_after();
        float odd = l * 0.0f;                        // NaN if anything is not finite
        const float inv = l != 0.0f ? __fdiv_rn(1.0f, l) : 0.0f;
        const int64_t o_row = at.out_row(p.t, f);
#pragma unroll
        for (int i = 0; i < D / 32; ++i) {
            uint32_t o[32];
            if (j > 0) {
                tmem_ld32(tmem + lanes + kTmO + 32 * i, o);
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
                    for (int w = 0; w < 8; ++w) x[w] = __uint_as_float(o[e + w]) * inv;
                    st_pack<T, 8>((T *)p.out + o_row * D + 32 * i + e, x);
                }
            }
        }
        if (live)
            p.lse[o_row] = l != 0.0f ? ((m == -INFINITY ? 0.0f : m) + log2f(l)) * kLn2 : -INFINITY;
        unsigned redo = __ballot_sync(0xffffffffu, live && odd != 0.0f && !isnan(l));
        for (; redo; redo &= redo - 1) {
            const int64_t g = at.f0 + warp * 32 + __ffs(redo) - 1;
            const int tt = (int)(g / a.G);
            attend_row_alone<T, D>(p, at.b, at.h, tt, at.h * a.G + (int)(g - (int64_t)tt * a.G));
        }
        mma_fence_before();
    }
    __syncthreads();
    if (warp == 5) {
        mma_fence_after();
        tmem_free(tmem, columns);
    }
}

// ------------------------------------------------------------------- host
struct RowPlan {
    int nt, gt, splits;
    int64_t items;
};

// Splits of a list, a power of two up to a portable cluster's 8, while they still
// fit the SMs two at a time (a second wave costs more than longer lists do) and
// each warp keeps a slice of 16 keys.
RowPlan row_plan(const spmm_blocks_shape *s) {
    RowPlan p;
    const int64_t G = s->Hq / s->Hk;
    p.nt = G > 8 ? 2 : 1;
    p.gt = (int)((G + 8 * p.nt - 1) / (8 * p.nt));
    p.items = s->B * s->Tq * s->Hk * p.gt;
    const int64_t slices = s->n * (s->block / 16);
    p.splits = 1;
    const int64_t warps = p.nt == 1 ? kRowWarps<1> : kRowWarps<2>;
    while (p.splits < 8 && 2 * p.splits * warps <= slices && 2 * p.items * p.splits <= 152 * 2)
        p.splits *= 2;
    return p;
}

template <typename T, int D>
cudaError_t launch_rows(const RowArgs &p, const RowPlan &rp, cudaStream_t s) {
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = (unsigned)rp.splits;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)(rp.items * rp.splits));
    cfg.blockDim = dim3(32 * (rp.nt == 1 ? kRowWarps<1> : kRowWarps<2>));
    cfg.stream = s;
    cfg.attrs = &attr;
    cfg.numAttrs = rp.splits > 1 ? 1 : 0;
    count_launch();
    return rp.nt == 1 ? cudaLaunchKernelEx(&cfg, k_attend_rows<T, D, 1>, p)
                      : cudaLaunchKernelEx(&cfg, k_attend_rows<T, D, 2>, p);
}

template <typename T, int D, int KB>
cudaError_t launch_tile(AttendTileArgs &p, int64_t B, cudaStream_t s) {
    constexpr int bytes = AttendSmem<D, KB>::bytes;
    const cudaError_t e = cudaFuncSetAttribute(
        k_attend_tile<T, D, KB>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != cudaSuccess) return e;
    p.t.tiles = (int)((p.t.rows + 16 * kTileWarps - 1) / (16 * kTileWarps));
    k_attend_tile<T, D, KB><<<dim3((unsigned)p.t.tiles, (unsigned)(B * p.t.a.Hk)),
                              32 * (kTileWarps + 1), bytes, s>>>(p);
    count_launch();
    return cudaGetLastError();
}

template <typename T, int D> cudaError_t launch_mma(AttendTileArgs &p, int64_t B, cudaStream_t s) {
    constexpr int bytes = MmaSmem<D>::bytes;
    const cudaError_t e = cudaFuncSetAttribute(
        k_attend_mma<T, D>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != cudaSuccess) return e;
    p.t.tiles = (int)((p.t.rows + kMmaRows - 1) / kMmaRows);
    k_attend_mma<T, D><<<dim3((unsigned)p.t.tiles, (unsigned)(B * p.t.a.Hk)), kMmaThreads, bytes,
                         s>>>(p);
    count_launch();
    return cudaGetLastError();
}

template <typename T, int D>
cudaError_t launch_by_tile(AttendTileArgs &p, int64_t B, cudaStream_t s) {
    if (p.t.a.block == 16) return launch_tile<T, D, 16>(p, B, s);
    if (p.t.a.block == 32) return launch_tile<T, D, 32>(p, B, s);
    return launch_mma<T, D>(p, B, s);
}

// k_attend_mma takes its maxima before the scale: a scale above 0 only.
bool by_tile(const spmm_blocks_shape *s, const spmm_rows &k, const spmm_rows &v) {
    return blocks_by_tile(s, k, v) && (s->block < kMmaKeys || s->scale > 0.0f);
}

}  // namespace

cudaError_t encode_rows(const spmm_rows &r, const spmm_blocks_shape *s, int box_rows,
                        CUtensorMap *map) {
    if (!g_encode) {
        cudaDriverEntryPointQueryResult q;
        void *fn = nullptr;
        const cudaError_t e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000,
                                                               cudaEnableDefault, &q);
        if (e != cudaSuccess || q != cudaDriverEntryPointSuccess || !fn)
            return e != cudaSuccess ? e : cudaErrorNotSupported;
        g_encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
    }
    const cuuint64_t dims[4] = {(cuuint64_t)s->D, (cuuint64_t)s->Tk, (cuuint64_t)s->Hk,
                                (cuuint64_t)s->B};
    // the stride of a dimension of one means nothing, and may be any number
    const cuuint64_t strides[3] = {(cuuint64_t)(s->Tk > 1 ? r.st * 2 : 16),
                                   (cuuint64_t)(s->Hk > 1 ? r.sh * 2 : 16),
                                   (cuuint64_t)(s->B > 1 ? r.sb * 2 : 16)};
    const cuuint32_t box[4] = {64, (cuuint32_t)box_rows, 1, 1};
    const cuuint32_t estr[4] = {1, 1, 1, 1};
    const CUresult e = g_encode(
        map, s->dtype == SPMM_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
        4, const_cast<void *>(r.data), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
        CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return e == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

}  // namespace spmm

extern "C" {

spmm_status spmm_blocks_attend(const spmm_blocks_shape *s, spmm_rows q, spmm_rows k, spmm_rows v,
                               const int32_t *blocks, void *out, float *lse, void *stream) {
    using namespace spmm;
    const spmm_status st = blk_check(s, true);
    if (st != SPMM_OK) return st;
    if (s->B == 0 || s->Tq == 0) return SPMM_OK;
    if (!blocks || !lse || !out || (uintptr_t)out % 16) return SPMM_ERR_INVALID_ARG;
    if (!rows_ok(q, 2) || (s->Tk > 0 && (!rows_ok(k, 2) || !rows_ok(v, 2))))
        return SPMM_ERR_INVALID_ARG;
    cudaStream_t cs = (cudaStream_t)stream;
    RowArgs p{};
    p.a = blk_args(s, blocks);
    set_rows(p.a.q, p.a.q_sb, p.a.q_st, p.a.q_sh, q);
    set_rows(p.a.k, p.a.k_sb, p.a.k_st, p.a.k_sh, k);
    set_rows(p.a.v, p.a.v_sb, p.a.v_st, p.a.v_sh, v);
    if (by_tile(s, k, v)) {
        AttendTileArgs t{};
        t.t.a = p.a;
        t.t.rows = s->Tq * p.a.G;
        t.out = out;
        t.lse = lse;
        const int box = (int)std::min<int64_t>(s->block, 64);
        cudaError_t e = dynamic_err(cs, &t.t.err);
        if (e == cudaSuccess) e = encode_rows(k, s, box, &t.t.k_map);
        if (e == cudaSuccess) e = encode_rows(v, s, box, &t.t.v_map);
        if (e == cudaSuccess) {
            if (s->dtype == SPMM_BF16)
                e = s->D == 64 ? launch_by_tile<__nv_bfloat16, 64>(t, s->B, cs)
                               : launch_by_tile<__nv_bfloat16, 128>(t, s->B, cs);
            else
                e = s->D == 64 ? launch_by_tile<__half, 64>(t, s->B, cs)
                               : launch_by_tile<__half, 128>(t, s->B, cs);
        }
        return cuda_status(e);
    }
    const RowPlan rp = row_plan(s);
    if (rp.items * rp.splits > INT32_MAX) return SPMM_ERR_UNSUPPORTED;
    p.gt = rp.gt;
    p.splits = rp.splits;
    p.out = out;
    p.lse = lse;
    cudaError_t e;
    if (s->dtype == SPMM_BF16)
        e = s->D == 64 ? launch_rows<__nv_bfloat16, 64>(p, rp, cs)
                       : launch_rows<__nv_bfloat16, 128>(p, rp, cs);
    else
        e = s->D == 64 ? launch_rows<__half, 64>(p, rp, cs)
                       : launch_rows<__half, 128>(p, rp, cs);
    return cuda_status(e);
}

}  // extern "C"
