// dK and dV of selected-block attention on the fifth-generation tensor cores
// (bf16, heads of 128, blocks of 64 keys and more). A CTA owns 64 keys of one
// kv head and a range of queries; the (query, head) rows that chose its block
// are gathered 128 at a time:
//   S = Q K^T, dP = dO V^T          128 rows x 64 keys, both operands K-major
//   P = exp(scale S - lse), dS = scale P (dP - delta)      a thread per row
//   dV^T += dO^T P, dK^T += Q^T dS  128 elements x 64 keys, summed over the rows
//                                   (dS as its rounded value and its rest)
// The gathered rows and P, dS serve as MN-major operands in the second pair of
// products, so nothing is transposed in memory. Eight warps gather rows by
// asynchronous copies into two stages, one thread issues the products, eight
// warps make P and dS, each half of a row's keys. 245 us for 2 x 4096 queries x 16
// heads of 128 over 2, 16 of 64-key blocks (mma.sync 852 us). Bound by the chain of
// a step (gather, first products, P and dS, second products) with room for only
// two steps' rows on chip; the tensor pipe computes 25% of the time.
#pragma once

#include "blocks_tile.cuh"
#include "umma.cuh"

namespace spmm {

// Work of k_dkdv_keys: a 64-key tile's queries in segments of at most
// kKeysSegment, an item each, so that a block which every query chose is shared
// out like the rest. tile = ((b Hk + h) NB + block) parts + part.
// (With ranges of queries instead the SMs were idle for 40% of the time.)
constexpr int kKeysSegment = 512;

struct KeyItems {
    int32_t *first;          // [tiles + 1]: a tile's first item
    int2 *item;              // (tile, segment), `first[tiles]` of them
    float *part;             // [item][dK, dV][64][D], for tiles of several items
    int64_t tiles;
};

struct BwdArgs {
    BlkArgs a;
    const void *out, *dout;
    int64_t do_sb, do_st, do_sh;
    const float *lse;
    float *delta;            // [B, Tq, Hq]
    void *dq, *dk, *dv;
    uint32_t *bits;          // [B, Hk, NB, words]
    int words;               // ceil(Tq / 32)
    int chunks;              // ranges of queries per key block
    int chunk_words;
    float *part;             // [chunks][2][B, Tk, Hk, D] when chunks > 1
    int64_t part_stride;     // B Tk Hk D
    int pair0;               // of the launch's (sequence, kv head) pairs (k_dkdv)
    int gt;
    int32_t *err;
    KeyItems keys;
};

// One key, row by row, for keys whose tile gave a result that is not finite: in
// the tile a row of q or of the gradient that is not finite, times the weight 0
// of a key that it does not see, spoils that key too. `each` calls its argument
// for every query that chose the key's block, until it returns false: when all of what
// is wanted (the gradient that is not finite; the other stands) is NaN. Lane l gets
// elements l E ..
template <typename T, int D, typename F>
__device__ __forceinline__ void dkdv_key_alone(const BwdArgs &p, int b, int h, int key, bool want_k,
                                               bool want_v, F each, float (&dk)[D / 32],
                                               float (&dv)[D / 32]) {
    const BlkArgs &a = p.a;
    constexpr int E = D / 32;
    const int lane = threadIdx.x & 31;
    const int len = blk_len(a, b);
    float k[E] = {}, v[E] = {};
    if (key < len) {
        ld_pack<T, E>((const T *)a.k + b * a.k_sb + key * a.k_st + h * a.k_sh + lane * E, k);
        ld_pack<T, E>((const T *)a.v + b * a.v_sb + key * a.v_st + h * a.v_sh + lane * E, v);
    }
#pragma unroll
    for (int e = 0; e < E; ++e) dk[e] = dv[e] = 0.0f;
    each([&](int t) {
        if (key >= blk_limit(a, len, t)) return true;
        for (int g = 0; g < a.G; ++g) {
            const int head = h * a.G + g;
            const int64_t row = ((int64_t)b * a.Tq + t) * a.Hq + head;
            float q[E], o[E], s = 0.0f, d = 0.0f;
            ld_pack<T, E>((const T *)a.q + b * a.q_sb + t * a.q_st + head * a.q_sh + lane * E, q);
            ld_pack<T, E>((const T *)p.dout + b * p.do_sb + t * p.do_st + head * p.do_sh + lane * E, o);
#pragma unroll
            for (int e = 0; e < E; ++e) {
                s = fmaf(q[e], k[e], s);
                d = fmaf(o[e], v[e], d);
            }
#pragma unroll
            for (int x = 16; x; x >>= 1) {
                s += __shfl_xor_sync(0xffffffffu, s, x);
                d += __shfl_xor_sync(0xffffffffu, d, x);
            }
            const float lse2 = p.lse[row] * kLog2e;
            if (lse2 == -INFINITY) continue;     // every score of the row is -infinity: P = 0
            const float pr = ex2(fmaf(s, a.scale * kLog2e, -lse2));
            const float ds = pr * (d - p.delta[row]) * a.scale;
#pragma unroll
            for (int e = 0; e < E; ++e) {
                dk[e] = fmaf(ds, q[e], dk[e]);
                dv[e] = fmaf(pr, o[e], dv[e]);
            }
        }
        return (want_k && !all_nan(dk)) || (want_v && !all_nan(dv));
    });
}

constexpr int kKeysD = 128;                // width of a head
constexpr int kKeysN = 64;                 // keys per CTA
constexpr int kKeysRows = 128;             // rows per step
constexpr int kKeysLoaders = 8, kKeysIssuer = 8 + kKeysLoaders;   // after 8 softmax warps
constexpr int kKeysThreads = 32 * (kKeysIssuer + 1);
constexpr int kKeysPanelK = kKeysN * 128, kKeysPanelR = kKeysRows * 128;   // bytes
constexpr int kKeysK = 0, kKeysV = 2 * kKeysPanelK, kKeysStage0 = 4 * kKeysPanelK;
constexpr int kKeysStage = 4 * kKeysPanelR;                                // Q, dO
constexpr int kKeysP = kKeysStage0 + 2 * kKeysStage, kKeysDs = kKeysP + kKeysPanelR;
constexpr int kKeysDl = kKeysDs + kKeysPanelR;                             // dS's rest
constexpr int kKeysStats = kKeysDl + kKeysPanelR;                          // [2][3][128] floats
constexpr int kKeysList = kKeysStats + 2 * 3 * kKeysRows * 4;              // the segment's queries
constexpr int kKeysSmem = kKeysList + kKeysSegment * 4 + 1024;
// tensor memory columns
constexpr int kTmS = 0, kTmDp = 64, kTmStage = 128, kTmDv = 256, kTmDk = 320, kTmColumns = 512;

template <typename T>
__global__ void __launch_bounds__(kKeysThreads, 1) k_dkdv_keys(const BwdArgs p) {
    constexpr int D = kKeysD, C = D / 8;
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    const uint32_t smem = (smem_addr(smem_raw) + 1023u) & ~1023u;
    unsigned char *sp = smem_raw + (smem - smem_addr(smem_raw));
    float *stats = (float *)(sp + kKeysStats);
    int32_t *list = (int32_t *)(sp + kKeysList);
    __shared__ uint64_t full[2], ready[2], made, done[2], drained;
    __shared__ uint32_t tmem_slot, odd[2][2];        // of dV, of dK: a bit per key
    __shared__ int n_queries;

    const BlkArgs &a = p.a;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if ((int)blockIdx.x >= p.keys.first[p.keys.tiles]) return;
    const int2 item = p.keys.item[blockIdx.x];
    const bool alone = p.keys.first[item.x + 1] - p.keys.first[item.x] == 1;
    const int parts = a.block / kKeysN;
    const int blk_id = item.x / parts, blk = blk_id % a.NB;
    const int b = blk_id / a.NB / a.Hk, h = blk_id / a.NB % a.Hk;
    const int key0 = blk * a.block + item.x % parts * kKeysN;
    if (key0 >= a.Tk) return;
    const int len = blk_len(a, b);

    if (warp == 0) {                             // the segment's queries, ascending
        const uint32_t *bits = p.bits + (int64_t)blk_id * p.words;
        const int from = item.y * kKeysSegment, to = from + kKeysSegment;
        int base = 0;
        for (int w = 0; w < p.words && base < to; w += 32) {
            const uint32_t x = w + lane < p.words ? bits[w + lane] : 0u;
            int incl = __popc(x);
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, incl, o);
                if (lane >= o) incl += y;
            }
            int at = base + incl - __popc(x);
            for (uint32_t m = x; m; m &= m - 1, ++at)
                if (at >= from && at < to) list[at - from] = (w + lane) * 32 + __ffs(m) - 1;
            base += __shfl_sync(0xffffffffu, incl, 31);
        }
        base = max(0, min(base, to) - from);
        if (lane == 0) {
            n_queries = base;
            odd[0][0] = odd[0][1] = odd[1][0] = odd[1][1] = 0;
            for (int i = 0; i < 2; ++i) {
                mbar_init(&full[i], 32 * kKeysLoaders);
                mbar_init(&ready[i], 1);
                mbar_init(&done[i], 1);
            }
            mbar_init(&made, 256);
            mbar_init(&drained, 1);
            mbar_init_fence();
        }
    } else if (warp == kKeysIssuer) {
        tmem_alloc(&tmem_slot, kTmColumns);
        mma_fence_before();
    }
    __syncthreads();
    mma_fence_after();
    const uint32_t tmem = tmem_slot;
    const int rows = n_queries * a.G;
    const int steps = (rows + kKeysRows - 1) / kKeysRows;

    if (warp >= 8 && warp < kKeysIssuer) {
        // ------------------------------------------------ gather rows
        const T *qp = (const T *)a.q + b * a.q_sb + (int64_t)h * a.G * a.q_sh;
        const T *gp = (const T *)p.dout + b * p.do_sb + (int64_t)h * a.G * p.do_sh;
        // a warp gathers kPer rows of a step; its lanes 0 .. kPer - 1 know where they are
        constexpr int kPer = kKeysRows / kKeysLoaders;
        const int i0 = threadIdx.x - 256, row0 = (warp - 8) * kPer;
        if (steps) {
            const T *kp = (const T *)a.k + b * a.k_sb + h * a.k_sh;
            const T *vp = (const T *)a.v + b * a.v_sb + h * a.v_sh;
            for (int i = i0; i < kKeysN * C; i += 32 * kKeysLoaders) {
                const int row = i / C, ch = i % C;
                const bool live = key0 + row < len;
                const int64_t key = live ? key0 + row : 0;
                const uint32_t at = (ch >> 3) * kKeysPanelK + chunk_at(row, ch & 7);
                cp16(smem + kKeysK + at, kp + key * a.k_st + ch * 8, live);
                cp16(smem + kKeysV + at, vp + key * a.v_st + ch * 8, live);
            }
        }
        for (int j = 0; j < steps; ++j) {
            const int st = j & 1;
            const int f = j * kKeysRows + row0 + lane;
            int64_t q_at = -1, g_at = 0;
            float lse2 = INFINITY, delta = 0.0f;
            int limit = 0;
            if (lane < kPer && f < rows) {
                const int q = f / a.G, g = f - q * a.G, t = list[q];
                q_at = t * a.q_st + g * a.q_sh;
                g_at = t * p.do_st + g * p.do_sh;
                const int64_t row = ((int64_t)b * a.Tq + t) * a.Hq + h * a.G + g;
                lse2 = p.lse[row] * kLog2e;
                delta = p.delta[row];
                limit = blk_limit(a, len, t);
            }
            // the stage was last read by the second products of step j - 2
            if (j >= 2 && !mbar_wait_poll(&done[st], ((j >> 1) - 1) & 1, p.err)) break;
            const uint32_t base = smem + kKeysStage0 + st * kKeysStage;
#pragma unroll
            for (int i = 0; i < kPer / 2; ++i) {
                const int row = 2 * i + (lane >> 4), ch = lane & 15;
                const int64_t x = __shfl_sync(0xffffffffu, q_at, row);
                const int64_t y = __shfl_sync(0xffffffffu, g_at, row);
                const uint32_t at = base + (ch >> 3) * kKeysPanelR + chunk_at(row0 + row, ch & 7);
                cp16(at, qp + (x < 0 ? 0 : x + ch * 8), x >= 0);
                cp16(at + 2 * kKeysPanelR, gp + (x < 0 ? 0 : y + ch * 8), x >= 0);
            }
            cp_commit();
            if (lane < kPer) {
                float *m = stats + st * 3 * kKeysRows + row0 + lane;
                m[0] = lse2 == -INFINITY ? INFINITY : lse2;  // a row without keys: P = 0
                m[kKeysRows] = delta;
                m[2 * kKeysRows] = __int_as_float(limit);
            }
            cp_wait<0>();
            fence_proxy_async_shared();
            mbar_arrive(&full[st]);
        }
    } else if (warp == kKeysIssuer) {
        // ------------------------------------------------ issue the products
        if (lane == 0) {
            constexpr uint32_t kk = instr_f16<T>(128, kKeysN, false, false);
            constexpr uint32_t mn = instr_f16<T>(128, kKeysN, true, true);
            auto second = [&](int j) {
                mma_fence_after();
                const uint32_t rows_ = smem + kKeysStage0 + (j & 1) * kKeysStage;
#pragma unroll
                for (int i = 0; i < kKeysRows / 16; ++i) {
                    mma_f16(tmem + kTmDv, desc_mn(rows_ + 2 * kKeysPanelR + i * 2048, kKeysPanelR),
                            desc_mn(smem + kKeysP + i * 2048, kKeysPanelR), mn, j > 0 || i > 0);
                    mma_f16(tmem + kTmDk, desc_mn(rows_ + i * 2048, kKeysPanelR),
                            desc_mn(smem + kKeysDs + i * 2048, kKeysPanelR), mn, j > 0 || i > 0);
                    mma_f16(tmem + kTmDk, desc_mn(rows_ + i * 2048, kKeysPanelR),
                            desc_mn(smem + kKeysDl + i * 2048, kKeysPanelR), mn, true);
                }
                mma_commit(&done[j & 1]);
            };
            auto first = [&](int j) {
                mma_fence_after();
                const uint32_t rows_ = smem + kKeysStage0 + (j & 1) * kKeysStage;
                const uint32_t tm = tmem + (j & 1) * kTmStage;
#pragma unroll
                for (int i = 0; i < D / 16; ++i) {
                    const uint32_t r = (i >> 2) * kKeysPanelR + (i & 3) * 32;
                    const uint32_t k = (i >> 2) * kKeysPanelK + (i & 3) * 32;
                    mma_f16(tm + kTmS, desc_k(rows_ + r), desc_k(smem + kKeysK + k), kk, i > 0);
                    mma_f16(tm + kTmDp, desc_k(rows_ + 2 * kKeysPanelR + r),
                            desc_k(smem + kKeysV + k), kk, i > 0);
                }
                mma_commit(&ready[j & 1]);
            };
            // A step's first products and the second ones of the step before wait for
            // different things: whichever is ready goes first (the second ones free
            // the stage that the gathering warps wait for).
            bool ok = true;
            for (int j = 0; j <= steps && ok && steps; ++j) {
                bool a_left = j < steps, b_left = j > 0;
                const uint64_t t0 = global_ns();
                for (uint32_t spin = 1; a_left || b_left; ++spin) {
                    if (a_left && mbar_test(&full[j & 1], (j >> 1) & 1)) {
                        first(j);
                        a_left = false;
                    }
                    if (b_left && mbar_test(&made, (j - 1) & 1)) {
                        second(j - 1);
                        b_left = false;
                    }
                    if (spin >= kSpinLimit || ((spin & 255) == 0 && global_ns() - t0 > kWaitLimitNs)) {
                        ok = !a_left && !b_left;
                        if (!ok) atomicOr(p.err + kErrTimeout, 1);
                        break;
                    }
                }
            }
            if (!ok) mma_drain(&drained, p.err);
        }
        __syncwarp();
    } else {
        // ------------------------------------------------ P and dS, then the result
        const int half = warp >> 2, row = (warp & 3) * 32 + lane;
        const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
        const float scale2 = a.scale * kLog2e;
        bool ok = true;
        for (int j = 0; j < steps; ++j) {
            const int st = j & 1;
            ok = mbar_wait_poll(&full[st], (j >> 1) & 1, p.err) &&
                 mbar_wait_poll(&ready[st], (j >> 1) & 1, p.err);
            if (!ok) break;
            mma_fence_after();
            uint32_t s[32], dp[32];
            tmem_ld32(tmem + lanes + st * kTmStage + kTmS + half * 32, s);
            tmem_ld32(tmem + lanes + st * kTmStage + kTmDp + half * 32, dp);
            const float *m = stats + st * 3 * kKeysRows + row;
            const float lse2 = m[0], delta = m[kKeysRows];
            const int seen = __float_as_int(m[2 * kKeysRows]) - (key0 + half * 32);
            tmem_wait_ld();
            uint32_t pp[16], dd[16], dl[16];
            const bool whole = __all_sync(0xffffffffu, seen >= 32);
            const float ds_off = -delta * a.scale;
#pragma unroll
            for (int i = 0; i < 32; i += 2) {
                float pr[2], ds[2];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    pr[e] = ex2(fmaf(__uint_as_float(s[i + e]), scale2, -lse2));
                    ds[e] = pr[e] * fmaf(__uint_as_float(dp[i + e]), a.scale, ds_off);
                    if (!whole && i + e >= seen) pr[e] = ds[e] = 0.0f;
                }
                pp[i / 2] = pack2<T>(pr[0], pr[1]);          // one part, as in k_dkdv
                split2<T>(ds[0], ds[1], dd[i / 2], dl[i / 2]);
            }
            // the products of the step before read the buffers that are written now
            if (j > 0) ok = mbar_wait_poll(&done[(j - 1) & 1], ((j - 1) >> 1) & 1, p.err);
            if (!ok) break;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint32_t at = smem + chunk_at(row, half * 4 + i);
                asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at + kKeysP),
                             "r"(pp[4 * i]), "r"(pp[4 * i + 1]), "r"(pp[4 * i + 2]),
                             "r"(pp[4 * i + 3])
                             : "memory");
                asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at + kKeysDs),
                             "r"(dd[4 * i]), "r"(dd[4 * i + 1]), "r"(dd[4 * i + 2]),
                             "r"(dd[4 * i + 3])
                             : "memory");
                asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at + kKeysDl),
                             "r"(dl[4 * i]), "r"(dl[4 * i + 1]), "r"(dl[4 * i + 2]),
                             "r"(dl[4 * i + 3])
                             : "memory");
            }
            fence_proxy_async_shared();
            mma_fence_before();
            mbar_arrive(&made);
        }
        if (ok && steps) ok = mbar_wait_poll(&done[(steps - 1) & 1], ((steps - 1) >> 1) & 1, p.err);
        mma_fence_after();
        // warps 0-3 write dV, 4-7 dK: a thread has element `row` of all 64 keys
        uint32_t x[2][32];
        uint32_t bad[2] = {0u, 0u};
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            if (steps) {
                tmem_ld32(tmem + lanes + (half ? kTmDk : kTmDv) + i * 32, x[i]);
                tmem_wait_ld();
            } else {
#pragma unroll
                for (int e = 0; e < 32; ++e) x[i][e] = 0u;
            }
#pragma unroll
            for (int e = 0; e < 32; ++e)
                if ((x[i][e] & 0x7f800000u) == 0x7f800000u) bad[i] |= 1u << e;
        }
        // to the gradients, or to the item's part of them
        const int64_t step = alone ? (int64_t)a.Hk * D : D;
        const int64_t first =
            alone ? ((int64_t)b * a.Tk + key0) * step + h * D
                  : ((int64_t)blockIdx.x * 2 + (half ? 0 : 1)) * (kKeysN * D);
        const int n = min(kKeysN, a.Tk - key0);
        T *out = (T *)(half ? p.dk : p.dv) + first + row;
        float *part = p.keys.part + first + row;
#pragma unroll
        for (int i = 0; i < kKeysN; ++i) {
            const float y = __uint_as_float(x[i >> 5][i & 31]);
            if (i >= n) break;
            if (alone) out[i * step] = from_f32<T>(y);
            else part[i * step] = y;
        }
#pragma unroll
        for (int i = 0; i < 2; ++i)
            if (bad[i]) atomicOr(&odd[half][i], bad[i]);
        asm volatile("bar.sync 1, 256;" ::: "memory");
        for (int i = warp; i < n; i += 8) {
            const bool want_v = odd[0][i >> 5] >> (i & 31) & 1u;
            const bool want_k = odd[1][i >> 5] >> (i & 31) & 1u;
            if (!want_k && !want_v) continue;
            constexpr int E = D / 32;
            float dk[E], dv[E];
            dkdv_key_alone<T, D>(
                p, b, h, key0 + i, want_k, want_v,
                [&](auto body) {
                    for (int q = 0; q < n_queries; ++q)
                        if (!body(list[q])) return;
                },
                dk, dv);
            const int64_t at = ((int64_t)b * a.Tk + key0 + i) * step + h * D + lane * E;
            float *y = p.keys.part + (int64_t)blockIdx.x * 2 * kKeysN * D + i * D + lane * E;
            if (alone) {
                if (want_k) st_pack<T, E>((T *)p.dk + at, dk);
                if (want_v) st_pack<T, E>((T *)p.dv + at, dv);
            } else {
                if (want_k) st_pack<float, E>(y, dk);
                if (want_v) st_pack<float, E>(y + kKeysN * D, dv);
            }
        }
        mma_fence_before();
    }
    __syncthreads();
    if (warp == kKeysIssuer) {
        mma_fence_after();
        tmem_free(tmem, kTmColumns);
    }
}

// Items: a warp counts a block's queries, one CTA numbers the segments.
__global__ void __launch_bounds__(256) k_key_counts(const BwdArgs p) {
    const int64_t blk = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31, parts = p.a.block / kKeysN;
    if (blk * parts >= p.keys.tiles) return;
    int n = 0;
    for (int w = lane; w < p.words; w += 32) n += __popc(p.bits[blk * p.words + w]);
    n = __reduce_add_sync(0xffffffffu, n);
    // a tile that nobody chose has an item too: it writes zeros
    if (lane < parts) p.keys.first[blk * parts + lane] = max(1, (n + kKeysSegment - 1) / kKeysSegment);
}

__global__ void __launch_bounds__(1024) k_key_items(const BwdArgs p) {
    __shared__ int warp_sum[32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    int carry = 0;
    for (int64_t i0 = 0; i0 < p.keys.tiles; i0 += 1024) {
        const int64_t i = i0 + tid;
        const int n = i < p.keys.tiles ? p.keys.first[i] : 0;
        int x = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, x, o);
            if (lane >= o) x += y;
        }
        if (lane == 31) warp_sum[warp] = x;
        __syncthreads();
        int below = 0, all = 0;
#pragma unroll
        for (int w = 0; w < 32; ++w) {
            below += w < warp ? warp_sum[w] : 0;
            all += warp_sum[w];
        }
        const int at = carry + below + x - n;
        if (i < p.keys.tiles) {
            p.keys.first[i] = at;
            for (int s = 0; s < n; ++s) p.keys.item[at + s] = make_int2((int)i, s);
        }
        carry += all;
        __syncthreads();
    }
    if (tid == 0) p.keys.first[p.keys.tiles] = carry;
}

// The parts of a tile of several items, added in the items' order.
template <typename T> __global__ void __launch_bounds__(256) k_keys_join(const BwdArgs p) {
    constexpr int D = kKeysD, U = kKeysN * D / 8;
    const BlkArgs &a = p.a;
    const int64_t tile = blockIdx.x;
    const int i0 = p.keys.first[tile], i1 = p.keys.first[tile + 1];
    if (i1 - i0 == 1) return;
    const int parts = a.block / kKeysN;
    const int64_t blk_id = tile / parts;
    const int key0 = (int)(blk_id % a.NB) * a.block + (int)(tile % parts) * kKeysN;
    const int64_t b = blk_id / a.NB / a.Hk;
    const int h = (int)(blk_id / a.NB % a.Hk);
    for (int u = blockIdx.y * 256 + threadIdx.x; u < 2 * U; u += 256 * gridDim.y) {
        const int w = u / U, key = u % U / (D / 8), d = u % (D / 8) * 8;
        if (key0 + key >= a.Tk) continue;
        float sum[8] = {};
        for (int i = i0; i < i1; ++i) {
            float x[8];
            ld_pack<float, 8>(p.keys.part + (((int64_t)i * 2 + w) * kKeysN + key) * D + d, x);
#pragma unroll
            for (int e = 0; e < 8; ++e) sum[e] += x[e];
        }
        st_pack<T, 8>((T *)(w ? p.dv : p.dk) + ((b * a.Tk + key0 + key) * a.Hk + h) * D + d, sum);
    }
}

}  // namespace spmm
