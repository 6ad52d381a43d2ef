// Selected-block attention, the cheap score: the mean key of each block, the
// product of every query group's summed rows with those means, and the n best
// blocks of each query.
#include "blocks.cuh"

namespace spmm {
namespace {

// ------------------------------------------------------------------ means
// A CTA per (block, sequence, kv head): D / 8 threads share a key row, the
// others take the next rows; the partial sums are added in row-group order.
// 7 us for 8192 keys x 4 heads of 128 (8 MB): a launch's latency.
constexpr int kMeanThreads = 128;

template <typename T>
__global__ void __launch_bounds__(kMeanThreads) k_block_means(BlkArgs a, int D, int new_keys,
                                                             int pair0, float *__restrict__ means) {
    __shared__ float part[kMeanThreads * 8];
    const int pair = pair0 + blockIdx.y, b = pair / a.Hk, h = pair % a.Hk;
    const int len = blk_len(a, b);
    int c = blockIdx.x;
    if (new_keys >= 0) {
        c += max(len - new_keys, 0) / a.block;
        if (c * a.block >= len) return;
    }
    if (c >= a.NB) return;
    const int units = D / 8, rows = kMeanThreads / units;
    const int u = threadIdx.x % units, g = threadIdx.x / units;
    const int k0 = c * a.block, k1 = min(k0 + a.block, len);
    float acc[8] = {};
    if (g < rows) {
        const T *k = (const T *)a.k + b * a.k_sb + h * a.k_sh + u * 8;
        for (int i = k0 + g; i < k1; i += rows) {
            float x[8];
            ld_pack<T, 8>(k + i * a.k_st, x);
#pragma unroll
            for (int e = 0; e < 8; ++e) acc[e] += x[e];
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) part[(g * units + u) * 8 + e] = acc[e];
    }
    __syncthreads();
    const float count = (float)max(k1 - k0, 1);
    for (int d = threadIdx.x; d < D; d += kMeanThreads) {
        float s = 0.0f;
        for (int i = 0; i < rows; ++i) s += part[i * D + d];
        means[(((int64_t)b * a.NB + c) * a.Hk + h) * D + d] = __fdiv_rn(s, count);
    }
}

// ----------------------------------------------------------------- scores
// score[row, c], row = (b, t - t0, h) in that order, written for the candidates only:
// causal c < position / block (the block of the position itself is always
// taken), else c < blocks that hold a key.
struct SelArgs {
    BlkArgs a;
    int D;
    int pair0;               // of the launch's (sequence, kv head) pairs, for the tiles
    int t0, nt;              // the strip's queries: t0 .. t0 + nt - 1 of each sequence
    uint32_t rows;           // B nt Hk (below 2^31)
    const float *means;
    float *score;            // [rows, NB]
    int32_t *out;
    int32_t *kept;           // [B] or NULL: a copy of lengths
};

// First block that is not a candidate; *own = the block that is always taken, or -1.
__device__ __forceinline__ int candidates(const BlkArgs &a, int b, int t, int *own) {
    const int limit = blk_limit(a, blk_len(a, b), t);
    *own = -1;
    if (limit == 0) return 0;
    if (!a.causal) return (limit + a.block - 1) / a.block;
    *own = (limit - 1) / a.block;
    return *own;
}

// Few queries: a warp per 8 blocks of one row; the lanes split D.
template <typename T>
__global__ void __launch_bounds__(128) k_score_few(SelArgs s) {
    const BlkArgs &a = s.a;
    const int lane = threadIdx.x & 31;
    const int64_t row = blockIdx.y;
    const int h = (int)(row % a.Hk);
    const int64_t bt = row / a.Hk;
    const int t = s.t0 + (int)(bt % s.nt), b = (int)(bt / s.nt);
    int own;
    const int cand = candidates(a, b, t, &own);
    const int c0 = (blockIdx.x * 4 + (threadIdx.x >> 5)) * 8;
    if (c0 >= cand) return;
    float dot[8] = {};
    for (int d = lane * 8; d < s.D; d += 256) {
        float q[8] = {};
        const T *p = (const T *)a.q + b * a.q_sb + t * a.q_st + (int64_t)h * a.G * a.q_sh + d;
        for (int g = 0; g < a.G; ++g) {
            float x[8];
            ld_pack<T, 8>(p + g * a.q_sh, x);
#pragma unroll
            for (int e = 0; e < 8; ++e) q[e] += x[e];
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if (c0 + i < cand) {
                float m[8];
                ld_pack<float, 8>(s.means + (((int64_t)b * a.NB + c0 + i) * a.Hk + h) * s.D + d, m);
#pragma unroll
                for (int e = 0; e < 8; ++e) dot[i] = fmaf(q[e], m[e], dot[i]);
            }
        }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int o = 16; o; o >>= 1) dot[i] += __shfl_xor_sync(0xffffffffu, dot[i], o);
    if (lane == 0)
        for (int i = 0; i < 8; ++i)
            if (c0 + i < cand) s.score[row * a.NB + c0 + i] = dot[i];
}

// Many queries: 64 x 128 tiles of the groups' sums times the means, fp32
// throughout (the list that a query gets must not depend on the rounding of a
// 16-bit product). The heads of a group are added as their rows are loaded, again
// for every 128 blocks: a quarter of the tile's arithmetic at 8 heads, and cheaper
// than a launch that writes the sums (20 us at 8192 x 32 heads of 128). Bound by
// the fp32 pipes and the loads of q: 47 us for 8192 queries x 4 groups x 128 blocks.
constexpr int kSt = 64, kSc = 128;      // tile of queries and of blocks
constexpr int kSk = 32;                 // depth of one step

template <typename T> __global__ void __launch_bounds__(256) k_score_tiles(SelArgs s) {
    __shared__ float qt[kSk][kSt + 4], mt[kSk][kSc + 4];
    const BlkArgs &a = s.a;
    const int pair = s.pair0 + blockIdx.z, b = pair / a.Hk, h = pair % a.Hk;
    const int t0 = s.t0 + blockIdx.y * kSt, t1 = s.t0 + s.nt, c0 = blockIdx.x * kSc;
    int own;
    if (c0 >= candidates(a, b, min(t0 + kSt, t1) - 1, &own)) return;
    const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;
    const int qr = threadIdx.x / 4, qd = threadIdx.x % 4 * 8;     // row and elements it loads
    const T *qp = (const T *)a.q + b * a.q_sb + min(t0 + qr, t1 - 1) * a.q_st +
                  (int64_t)h * a.G * a.q_sh + qd;
    float acc[4][8] = {};
    for (int d0 = 0; d0 < s.D; d0 += kSk) {
        float q[8] = {};
        if (d0 + qd < s.D) {
#pragma unroll 4
            for (int g = 0; g < a.G; ++g) {
                float x[8];
                ld_pack<T, 8>(qp + g * a.q_sh + d0, x);
#pragma unroll
                for (int e = 0; e < 8; ++e) q[e] += x[e];
            }
        }
        float4 m[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int r = (threadIdx.x + 256 * i) / 8, d = threadIdx.x % 8 * 4;
            m[i] = make_float4(0, 0, 0, 0);
            if (d0 + d < s.D && c0 + r < a.NB)
                m[i] = *(const float4 *)(s.means +
                                         (((int64_t)b * a.NB + c0 + r) * a.Hk + h) * s.D + d0 + d);
        }
        __syncthreads();
#pragma unroll
        for (int e = 0; e < 8; ++e) qt[qd + e][qr] = q[e];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int r = (threadIdx.x + 256 * i) / 8, d = threadIdx.x % 8 * 4;
            mt[d][r] = m[i].x;
            mt[d + 1][r] = m[i].y;
            mt[d + 2][r] = m[i].z;
            mt[d + 3][r] = m[i].w;
        }
        __syncthreads();
#pragma unroll
        for (int d = 0; d < kSk; ++d) {
            const float4 x = *(const float4 *)&qt[d][ty * 4];
            const float4 y = *(const float4 *)&mt[d][tx * 4], z = *(const float4 *)&mt[d][64 + tx * 4];
            const float xs[4] = {x.x, x.y, x.z, x.w};
            const float ys[8] = {y.x, y.y, y.z, y.w, z.x, z.y, z.z, z.w};
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 8; ++j) acc[i][j] = fmaf(xs[i], ys[j], acc[i][j]);
        }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int t = t0 + ty * 4 + i;
        if (t >= t1) continue;
        float *p = s.score + (((int64_t)b * s.nt + t - s.t0) * a.Hk + h) * a.NB;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int c = c0 + (j >> 2) * 64 + tx * 4 + (j & 3);
            if (c < a.NB) p[c] = acc[i][j];
        }
    }
}

// ------------------------------------------------------------------- best
// A warp per row. Scores become unsigned keys of the same order; the want-th
// largest key is found by bisection between the row's extremes, counting the
// keys at or above the middle; all keys above it and the lowest-indexed ones
// equal to it are taken, in index order. R registers a lane hold the row's keys
// when it has at most 32 R candidates; R = 0 reads them again at every step. Bound
// by the bisection's 32 dependent steps: 21 us for 32768 rows of 128 blocks.
__device__ __forceinline__ uint32_t order_key(float x) {
    if (isnan(x)) return 0u;
    x += 0.0f;                                  // -0 and +0 are equal scores
    const uint32_t u = __float_as_uint(x);
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}

template <int R> struct RowKeys {
    uint32_t key[R > 0 ? R : 1];
    const float *p;
    int cand, lane;
    __device__ __forceinline__ void load(const float *row, int cand_, int lane_) {
        p = row;
        cand = cand_;
        lane = lane_;
        if constexpr (R > 0) {
#pragma unroll
            for (int i = 0; i < R; ++i) {
                const int c = i * 32 + lane;
                key[i] = c < cand ? order_key(p[c]) : 0u;
            }
        }
    }
    __device__ __forceinline__ uint32_t at(int i) const {
        if constexpr (R > 0) return key[i];
        const int c = i * 32 + lane;
        return c < cand ? order_key(p[c]) : 0u;
    }
    // keys >= x among the candidates (x > 0)
    __device__ __forceinline__ int count(uint32_t x) const {
        int n = 0;
        if constexpr (R > 0) {
#pragma unroll
            for (int i = 0; i < R; ++i) n += key[i] >= x ? 1 : 0;
        } else {
            for (int i = 0; i * 32 < cand; ++i) n += at(i) >= x ? 1 : 0;
        }
        return __reduce_add_sync(0xffffffffu, n);
    }
    __device__ __forceinline__ void extremes(uint32_t &lo, uint32_t &hi) const {
        lo = 0xffffffffu;
        hi = 0u;
        const int steps = R > 0 ? R : (cand + 31) / 32;
#pragma unroll
        for (int i = 0; i < steps; ++i) {
            const uint32_t x = at(i);
            hi = max(hi, x);
            if (i * 32 + lane < cand) lo = min(lo, x);
        }
        lo = __reduce_min_sync(0xffffffffu, lo);
        hi = __reduce_max_sync(0xffffffffu, hi);
    }
};

// One warp writes row's list; score: the row's scores (shared or global memory).
template <int R>
__device__ __forceinline__ void best_of_row(const SelArgs &s, int64_t row, const float *score,
                                            int cand, int own) {
    const BlkArgs &a = s.a;
    const int lane = threadIdx.x & 31;
    const int want = min(cand, a.n - (own >= 0 ? 1 : 0));
    int32_t *out = s.out + row * a.n;
    int done = 0;
    if (want > 0 && want < cand) {
        RowKeys<R> keys;
        keys.load(score, cand, lane);
        // the largest x with count(keys >= x) >= want
        uint32_t lo, hi;
        keys.extremes(lo, hi);
        int n_lo = cand;                        // count(keys >= lo)
        while (lo < hi) {
            const uint32_t mid = lo + (hi - lo) / 2 + 1;
            const int n = keys.count(mid);
            if (n >= want) {
                lo = mid;
                n_lo = n;
                if (n == want) break;
            } else {
                hi = mid - 1;
            }
        }
        // exactly want keys >= lo, or lo is the want-th key and some equal ones stay out
        int spare = n_lo - want;                // of the keys equal to lo, the last ones
        int equal = 0;
        if (spare > 0) equal = n_lo - (lo == 0xffffffffu ? 0 : keys.count(lo + 1)) - spare;
        const int steps = R > 0 ? R : (cand + 31) / 32;
#pragma unroll
        for (int i = 0; i < steps; ++i) {
            const int c = i * 32 + lane;
            const uint32_t x = keys.at(i);
            bool take = c < cand && x >= lo;
            if (spare > 0) {
                const bool tie = take && x == lo;
                const unsigned ties = __ballot_sync(0xffffffffu, tie);
                if (tie && __popc(ties & ((1u << lane) - 1u)) >= equal) take = false;
                equal -= min(equal, __popc(ties));
            }
            const unsigned m = __ballot_sync(0xffffffffu, take);
            if (take) out[done + __popc(m & ((1u << lane) - 1u))] = c;
            done += __popc(m);
        }
    } else if (want > 0) {
        for (int c = lane; c < cand; c += 32) out[c] = c;
        done = cand;
    }
    if (own >= 0) {
        if (lane == 0) out[done] = own;
        ++done;
    }
    for (int j = done + lane; j < a.n; j += 32) out[j] = -1;
}

// The copy of a sequence's length, by the warp of its first list.
__device__ __forceinline__ void keep_length(const SelArgs &s, int b, int t, int h) {
    if (s.kept && (threadIdx.x & 31) == 0 && t == 0 && h == 0) s.kept[b] = s.a.lengths[b];
}

template <int R> __global__ void __launch_bounds__(128) k_best(SelArgs s) {
    const uint32_t row = blockIdx.x * 4 + (threadIdx.x >> 5);
    if (row >= s.rows) return;
    const uint32_t bt = row / (uint32_t)s.a.Hk, b = bt / (uint32_t)s.nt;
    const int t = s.t0 + (int)(bt - b * s.nt);
    int own;
    const int cand = candidates(s.a, (int)b, t, &own);
    const int h = (int)(row - bt * s.a.Hk);
    keep_length(s, (int)b, t, h);
    best_of_row<R>(s, ((int64_t)b * s.a.Tq + t) * s.a.Hk + h, s.score + (int64_t)row * s.a.NB, cand,
                   own);
}

// Few queries over at most 32 R blocks: a CTA per row, scores in shared memory,
// the list by its first warp; one launch and no scratch. Eight elements a lane:
// D / 8 lanes share a block, so a warp scores 32 / L blocks at a time, U deep.
// Bound by the latency of a few rounds of loads and then of the bisection: 16 us for
// 256 rows of up to 512 blocks of 128 (37 MB of means; at the copy rate 5.5 us).
template <typename T, int R, int L>
__global__ void __launch_bounds__(512) k_select_row(SelArgs s) {
    constexpr int kPer = 32 / L, kU = 8;
    __shared__ float score[32 * R];
    const BlkArgs &a = s.a;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
    const int64_t row = blockIdx.x;
    const int h = (int)(row % a.Hk);
    const int64_t bt = row / a.Hk;
    const int t = (int)(bt % a.Tq), b = (int)(bt / a.Tq);
    int own;
    const int cand = candidates(a, b, t, &own);
    if (cand > a.n - (own >= 0 ? 1 : 0)) {         // else every block is taken
        const int d = lane % L * 8;
        const bool live = d < s.D;
        float q[8] = {};
        const T *p = (const T *)a.q + b * a.q_sb + t * a.q_st + (int64_t)h * a.G * a.q_sh + d;
        for (int g = 0; g < a.G && live; ++g) {
            float x[8];
            ld_pack<T, 8>(p + g * a.q_sh, x);
#pragma unroll
            for (int e = 0; e < 8; ++e) q[e] += x[e];
        }
        const float *means = s.means + ((int64_t)b * a.NB * a.Hk + h) * s.D + d;
        for (int c0 = warp * kPer * kU; c0 < cand; c0 += warps * kPer * kU) {
            float dot[kU];
#pragma unroll
            for (int u = 0; u < kU; ++u) {
                const int c = c0 + u * kPer + lane / L;
                dot[u] = 0.0f;
                if (live && c < cand) {
                    float m[8];
                    ld_pack<float, 8>(means + (int64_t)c * a.Hk * s.D, m);
#pragma unroll
                    for (int e = 0; e < 8; ++e) dot[u] = fmaf(q[e], m[e], dot[u]);
                }
            }
#pragma unroll
            for (int u = 0; u < kU; ++u) {
#pragma unroll
                for (int o = L / 2; o; o >>= 1) dot[u] += __shfl_xor_sync(0xffffffffu, dot[u], o);
                const int c = c0 + u * kPer + lane / L;
                if (lane % L == 0 && c < cand) score[c] = dot[u];
            }
        }
    }
    __syncthreads();
    if (warp == 0) {
        keep_length(s, b, t, h);
        best_of_row<R>(s, row, score, cand, own);
    }
}

__global__ void k_check_lists(BlkArgs a, int64_t rows, int32_t *bad) {
    const int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
    if (i >= rows * a.n) return;
    const int j = (int)(i % a.n);
    const int c = a.blocks[i];
    bool ok = c == -1 || (unsigned)c < (unsigned)a.NB;
    if (j > 0 && c != -1) ok = ok && a.blocks[i - 1] != -1 && c > a.blocks[i - 1];
    if (!ok) *bad = 1;
}

__global__ void k_zero_word(int32_t *p) { *p = 0; }

// ------------------------------------------------------------------- host
// A CTA per row (one launch, scores in shared memory) up to 1024 rows of at most
// 1024 blocks, and for fewer than 24 queries a sequence, of which a tile of 64
// would be mostly empty; else tiles, then a warp per row. By row against by tile:
// 1024 rows (256 queries x 4 heads) of 128 blocks 17 and 26 us, 2048 rows (256 x 8)
// 20 and 18, 16384 rows (2048 x 8) 42 and 36, 32768 rows (2 x 4096 x 4) 77 and 50.
// Longer rows of few queries: a warp per 8 blocks, then a warp per row.
constexpr int64_t kTiledQueries = 24, kTiledRows = 1024, kRowBlocks = 1024;

bool tiled(const spmm_blocks_shape *s) {
    const int64_t rows = s->B * s->Tq * s->Hk;
    if (s->Tk <= kRowBlocks * s->block) return s->Tq >= kTiledQueries && rows > kTiledRows;
    return s->Tq >= kTiledQueries || rows > 65535;
}
bool by_row(const spmm_blocks_shape *s) {
    return s->Tk <= kRowBlocks * s->block && !tiled(s);
}

// Queries of each sequence whose scores are held at a time: the scores of a prompt grow
// with the square of its length, so tiles take it in strips of at most 1 GB of them (of
// kSt queries at least, and no more than a launch takes). Each strip's last CTAs leave
// SMs idle: 65536 queries x 8 kv heads of 1024 blocks (2 GB) took 4.06 ms whole, 4.27 in
// strips of 256 MB and 4.51 in strips of 64 MB.
constexpr int64_t kStripBytes = 1 << 30;
int64_t strip(const spmm_blocks_shape *s) {
    if (!tiled(s)) return s->Tq;
    const int64_t query = s->B * s->Hk * ((s->Tk + s->block - 1) / s->block) * 4;
    const int64_t tiles = std::min<int64_t>(kStripBytes / std::max<int64_t>(query, 1) / kSt, 65535);
    return std::min(s->Tq, std::max<int64_t>(tiles, 1) * kSt);
}

template <typename T>
cudaError_t launch_scores(const SelArgs &s, int64_t B, bool tiles, cudaStream_t st) {
    const BlkArgs &a = s.a;
    if (!tiles) {                // rows in grid.y
        k_score_few<T><<<dim3((unsigned)((a.NB + 31) / 32), (unsigned)s.rows), 128, 0, st>>>(s);
        count_launch();
    } else {
        SelArgs p = s;
        const int64_t pairs = B * a.Hk;
        for (int64_t i = 0; i < pairs; i += kPairs) {
            p.pair0 = (int)i;
            k_score_tiles<T><<<dim3((unsigned)((a.NB + kSc - 1) / kSc),
                                    (unsigned)((s.nt + kSt - 1) / kSt),
                                    (unsigned)std::min(kPairs, pairs - i)),
                               256, 0, st>>>(p);
            count_launch();
        }
    }
    return cudaGetLastError();
}

// A strip's scores, and the lists that they give.
template <typename T>
cudaError_t launch_lists(const SelArgs &s, int64_t B, bool tiles, cudaStream_t st) {
    const int NB = s.a.NB;
    if (NB > 0) {
        const cudaError_t e = launch_scores<T>(s, B, tiles, st);
        if (e != cudaSuccess) return e;
    }
    const unsigned grid = s.rows / 4 + (s.rows % 4 != 0);
    if (NB <= 32) k_best<1><<<grid, 128, 0, st>>>(s);
    else if (NB <= 128) k_best<4><<<grid, 128, 0, st>>>(s);
    else if (NB <= 512) k_best<16><<<grid, 128, 0, st>>>(s);
    else if (NB <= 1024) k_best<32><<<grid, 128, 0, st>>>(s);
    else k_best<0><<<grid, 128, 0, st>>>(s);
    count_launch();
    return cudaGetLastError();
}

template <typename T, int R> void launch_select_row(const SelArgs &s, int threads, cudaStream_t st) {
    if (s.D <= 64) k_select_row<T, R, 8><<<(unsigned)s.rows, threads, 0, st>>>(s);
    else if (s.D <= 128) k_select_row<T, R, 16><<<(unsigned)s.rows, threads, 0, st>>>(s);
    else k_select_row<T, R, 32><<<(unsigned)s.rows, threads, 0, st>>>(s);
    count_launch();
}

template <typename T> cudaError_t launch_select_row(const SelArgs &s, cudaStream_t st) {
    if (s.a.NB <= 128) launch_select_row<T, 4>(s, 128, st);
    else if (s.a.NB <= 512) launch_select_row<T, 16>(s, 512, st);
    else launch_select_row<T, 32>(s, 512, st);
    return cudaGetLastError();
}

}  // namespace
}  // namespace spmm

extern "C" {

spmm_status spmm_blocks_means(const spmm_blocks_shape *s, spmm_rows k, int64_t new_keys,
                              float *means, void *stream) {
    using namespace spmm;
    const spmm_status st = blk_check(s, false);
    if (st != SPMM_OK) return st;
    if (s->B == 0 || s->Tk == 0 || new_keys == 0) return SPMM_OK;
    if (!means || !rows_ok(k, dtype_bytes(s->dtype))) return SPMM_ERR_INVALID_ARG;
    BlkArgs a = blk_args(s, nullptr);
    set_rows(a.k, a.k_sb, a.k_st, a.k_sh, k);
    const int64_t most = new_keys < 0 ? a.NB : std::min<int64_t>(a.NB, new_keys / s->block + 2);
    const int nk = (int)std::min<int64_t>(new_keys, INT32_MAX);
    cudaStream_t cs = (cudaStream_t)stream;
    const int D = (int)s->D;
    const int64_t pairs = s->B * s->Hk;
    for (int64_t i = 0; i < pairs; i += kPairs) {
        const dim3 grid((unsigned)most, (unsigned)std::min(kPairs, pairs - i));
        if (s->dtype == SPMM_F32)
            k_block_means<float><<<grid, kMeanThreads, 0, cs>>>(a, D, nk, (int)i, means);
        else if (s->dtype == SPMM_BF16)
            k_block_means<__nv_bfloat16><<<grid, kMeanThreads, 0, cs>>>(a, D, nk, (int)i, means);
        else k_block_means<__half><<<grid, kMeanThreads, 0, cs>>>(a, D, nk, (int)i, means);
        count_launch();
    }
    return cuda_status(cudaGetLastError());
}

int64_t spmm_blocks_select_workspace(const spmm_blocks_shape *s) {
    using namespace spmm;
    if (blk_check(s, false) != SPMM_OK || by_row(s)) return 0;
    const int64_t NB = (s->Tk + s->block - 1) / s->block;
    return s->B * strip(s) * s->Hk * NB * 4;
}

spmm_status spmm_blocks_select(const spmm_blocks_shape *s, spmm_rows q, const float *means,
                               int32_t *blocks, void *work, int64_t work_bytes, void *stream) {
    return spmm_blocks_select_kept(s, q, means, blocks, nullptr, work, work_bytes, stream);
}

spmm_status spmm_blocks_select_kept(const spmm_blocks_shape *s, spmm_rows q, const float *means,
                                    int32_t *blocks, int32_t *kept, void *work, int64_t work_bytes,
                                    void *stream) {
    using namespace spmm;
    const spmm_status st = blk_check(s, false);
    if (st != SPMM_OK) return st;
    if (s->B == 0 || s->Tq == 0) return SPMM_OK;
    if (!blocks || !rows_ok(q, dtype_bytes(s->dtype))) return SPMM_ERR_INVALID_ARG;
    if (s->Tk > 0 && (!means || (uintptr_t)means % 16)) return SPMM_ERR_INVALID_ARG;
    const int64_t need = spmm_blocks_select_workspace(s);
    if (need && (!work || work_bytes < need)) return SPMM_ERR_INVALID_ARG;
    SelArgs g{};
    g.a = blk_args(s, nullptr);
    set_rows(g.a.q, g.a.q_sb, g.a.q_st, g.a.q_sh, q);
    g.D = (int)s->D;
    g.nt = (int)s->Tq;
    g.rows = (uint32_t)(s->B * s->Tq * s->Hk);
    g.means = means;
    g.score = (float *)work;
    g.out = blocks;
    g.kept = s->lengths ? kept : nullptr;
    cudaStream_t cs = (cudaStream_t)stream;
    cudaError_t e = cudaSuccess;
    if (by_row(s)) {
        if (s->dtype == SPMM_F32) e = launch_select_row<float>(g, cs);
        else if (s->dtype == SPMM_BF16) e = launch_select_row<__nv_bfloat16>(g, cs);
        else e = launch_select_row<__half>(g, cs);
        return cuda_status(e);
    }
    for (int64_t t0 = 0, step = strip(s); t0 < s->Tq; t0 += step) {
        g.t0 = (int)t0;
        g.nt = (int)std::min(step, s->Tq - t0);
        g.rows = (uint32_t)(s->B * g.nt * s->Hk);
        if (s->dtype == SPMM_F32) e = launch_lists<float>(g, s->B, tiled(s), cs);
        else if (s->dtype == SPMM_BF16) e = launch_lists<__nv_bfloat16>(g, s->B, tiled(s), cs);
        else e = launch_lists<__half>(g, s->B, tiled(s), cs);
        if (e != cudaSuccess) break;
    }
    return cuda_status(e);
}

spmm_status spmm_blocks_check(const spmm_blocks_shape *s, const int32_t *blocks, int32_t *bad,
                              void *stream) {
    using namespace spmm;
    const spmm_status st = blk_check(s, false);
    if (st != SPMM_OK) return st;
    const int64_t rows = s->B * s->Tq * s->Hk;
    if (!bad || (rows && !blocks)) return SPMM_ERR_INVALID_ARG;
    cudaStream_t cs = (cudaStream_t)stream;
    k_zero_word<<<1, 1, 0, cs>>>(bad);
    count_launch();
    if (rows) {
        if ((rows * s->n + 255) / 256 > INT32_MAX) return SPMM_ERR_UNSUPPORTED;
        k_check_lists<<<(unsigned)((rows * s->n + 255) / 256), 256, 0, cs>>>(
            blk_args(s, blocks), rows, bad);
        count_launch();
    }
    return cuda_status(cudaGetLastError());
}

}  // extern "C"
