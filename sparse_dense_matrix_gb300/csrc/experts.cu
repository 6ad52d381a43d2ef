// Products grouped by expert: the slots of expert e, rows offsets[e] .. offsets[e + 1]
// of xs [P, H], times w[e] [H, F], and the gradient of w:
//   ys[s, f] = sum_h xs[s, h] w[e, h, f],   dw[e, h, f] = sum_s xs[s, h] dys[s, f].
// One kernel does both, as D[m, n] = sum_k A[m, k] B[n, k] on the tensor cores (tcgen05),
// m being the index that is adjacent in the result:
//   product    m = f, n = a slot, k = h: A = w[e]^T, B = xs. The ragged index is the
//              instruction's N, which comes in steps of 16: an expert with few slots
//              costs little, and w is read once per 256 of its slots.
//   gradient   m = f (h where h is adjacent in dw), n = h (f), k = a slot: A = dys^T,
//              B = xs^T, both MN-major. The ragged index is the summed one: rows past
//              the expert's last are the next expert's, and are set to 0 in shared
//              memory before they are used (0 times a NaN is none of this expert's). Few
//              experts with many slots are summed in parts, which a second kernel adds up.
// CTAs stay and take tiles of 128 x up to 256 in turn, or pairs of CTAs tiles of 256 x
// up to 256, of which each holds half of either operand and 128 of m of the result. A
// warp's thread copies the operands' tiles of 64 of k into a ring of stages (tensor
// copies), another (of the pair's first CTA) issues the products into one of two
// accumulators in tensor memory, and eight warps write the other one out meanwhile.
//
// Measured (bf16): 131072 slots of 128 experts that differ in popularity, 2048 x 1024, 333 us for 20
// calls in a row, 1.65 PFLOP/s, and 350 for 200 (power lowers the clock to 1.6 GHz), of the rows
// 342, of the matrices 407 (DRAM at 47%, the tensor pipe active 83% of the SMs' active cycles); one
// expert with 8192 slots, 8192 x 8192, 595, 591 and 597 us, next to 543 of the library's product of
// that size. 512 slots of 128 experts, 2048 x 768 (226 MB of matrices are reached), 41 us, 5.5
// TB/s. 8 slots of 8 experts, 2048 x 1024, 10 us (12 as a replayed graph), of which 2.4 pass before
// the first product is issued and 6 by 32 stages of one CTA after another on 64 SMs.
#include <cudaTypedefs.h>

#include "umma.cuh"

namespace spmm {
namespace {

constexpr int kSms = 152;
constexpr int kDepth = 64;           // of k in a stage: a row of 128 bytes
constexpr int kRowsM = 128;          // of m in a CTA's tile
constexpr int kResults = 8;          // warps that write results out
constexpr int kThreads = 128 + 32 * kResults;    // copies, products, tiles' list, segments' ends first
constexpr int kTilesAhead = 4;
constexpr int kSizes = 128;          // sizes that experts are sorted by (gradient)
constexpr int kSmemMax = 227 * 1024;

struct ExpertArgs {
    CUtensorMap a_map, b_map;
    const int32_t *offsets;
    void *out;
    int64_t o_se, o_ld;              // strides of e (gradient) and of n in the result
    int64_t P;
    int E, M, N, K;                  // N: gradient; K: product
    int a_step;                      // 0: one matrix for every expert
    int tiles_m, tiles_n;
    int splits;                      // gradient: parts of an expert's slots
    float *parts;                    // with more than one, [splits][E][M][N]
    int32_t *err;
};

// NT: largest n of a tile. NC: CTAs of a tile. BOX: rows of B that one copy brings.
template <int NT_, int NC_> struct ExpertShape {
    static constexpr int NT = NT_, NC = NC_, BOX = NT == 32 ? 16 : NT / NC, STEP = 16 * NC;   // of n
    static constexpr int a_bytes = kRowsM * kDepth * 2, b_bytes = NT / NC * kDepth * 2;
    static constexpr int stage = a_bytes + b_bytes;
    static constexpr int stages = 192 * 1024 / stage;
    static constexpr int columns = 2 * NT;
    // results: 32 rows of 64 bytes for each warp
    static constexpr int out_bytes = 32 * 64;
    static constexpr int at_out = stages * stage, at_offsets = at_out + kResults * out_bytes;
    static constexpr size_t bytes(int E) { return 1024 + at_offsets + sizeof(int32_t) * 2 * ((size_t)E + 1); }
};

struct ExpertTile {
    int e, n, m0, n0;                // m0, n0: first of m (of the pair's), of n (gradient)
    int r0;                          // first slot: of n (product), of k (gradient)
    int k;                           // length of k
    int part;                        // gradient: which of the expert's
};

// Shared memory's view of the experts: first slots, and the tiles of slots before each expert
// (product) or the experts in order of their slots, most first (gradient).
struct ExpertList {
    const int32_t *first, *before;
    template <bool GRAD>
    __device__ __forceinline__ int tiles(const ExpertArgs &p) const {
        return (GRAD ? p.E * p.splits * p.tiles_n : before[p.E]) * p.tiles_m;
    }
    template <typename S, bool GRAD>
    __device__ __forceinline__ ExpertTile tile(const ExpertArgs &p, int t) const {
        constexpr int NT = S::NT;
        ExpertTile x;
        x.m0 = t % p.tiles_m * (kRowsM * S::NC);
        const int u = t / p.tiles_m;
        if (GRAD) {
            const int v = u / p.tiles_n;
            x.e = before[v / p.splits];
            x.n0 = u % p.tiles_n * NT;
            x.n = min(NT, p.N - x.n0);
            x.r0 = first[x.e];
            x.k = first[x.e + 1] - first[x.e];
            x.part = v % p.splits;
            if (p.splits > 1) {                  // (whole stages, but for the last part's end)
                const int per = ((x.k + p.splits - 1) / p.splits + kDepth - 1) / kDepth * kDepth;
                const int64_t at = (int64_t)x.part * per;
                x.k = (int)max((int64_t)0, min((int64_t)per, x.k - at));
                x.r0 = (int)min(x.r0 + at, p.P);
            }
        } else {
            int lo = 0, hi = p.E - 1;            // the last expert with before[e] <= u
            while (lo < hi) {
                const int mid = (lo + hi + 1) >> 1;
                if (before[mid] <= u) lo = mid;
                else hi = mid - 1;
            }
            x.e = lo;
            x.n0 = x.part = 0;
            // an expert's slots in equal parts
            const int rows = first[lo + 1] - first[lo], parts = before[lo + 1] - before[lo];
            const int per = ((rows + parts - 1) / parts + S::STEP - 1) / S::STEP * S::STEP;
            const int at = (u - before[lo]) * per;
            x.r0 = first[lo] + at;
            x.n = min(per, rows - at);
            x.k = p.K;
        }
        return x;
    }
};

template <int NT, bool GRAD>
__device__ __forceinline__ ExpertList expert_list(const ExpertArgs &p, int32_t *smem) {
    int32_t *first = smem, *before = smem + p.E + 1;
    for (int e = threadIdx.x; e <= p.E; e += kThreads)
        first[e] = (int)min(max((int64_t)p.offsets[e], (int64_t)0), p.P);
    __syncthreads();
    if (threadIdx.x < 32) {
        // a first slot below the one before it leaves the expert without any
        int most = 0, sum = 0;
        for (int e0 = 0; e0 <= p.E; e0 += 32) {
            const int e = e0 + (int)threadIdx.x;
            int x = e <= p.E ? first[e] : 0;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, x, o);
                if ((int)threadIdx.x >= o) x = max(x, y);
            }
            x = max(x, most);
            if (e <= p.E) first[e] = x;
            most = __shfl_sync(0xffffffffu, x, 31);
        }
        __syncwarp();
        if (GRAD) {
            // A counting sort by the slots' number, to two bits behind its first: tiles of
            // like length follow one another, and CTAs that take them in turn end at about
            // the same time (65536 slots of 64 experts, the largest with 5 times the mean: 263
            // us without it, 229 with, 222 if they take them there and back).
            __shared__ int32_t keys[kSizes];
            auto key = [&](int e) {
                return kSizes - 1 - (__float_as_int((float)(first[e + 1] - first[e])) + 0x200000 -
                                    __float_as_int(1.0f)) / 0x200000;
            };
            for (int i = threadIdx.x; i < kSizes; i += 32) keys[i] = 0;
            __syncwarp();
            for (int e = threadIdx.x; e < p.E; e += 32)
                atomicAdd(&keys[min(max(key(e), 0), kSizes - 1)], 1);
            __syncwarp();
            for (int i0 = 0; i0 < kSizes; i0 += 32) {
                const int mine = keys[i0 + threadIdx.x];
                int x = mine;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const int y = __shfl_up_sync(0xffffffffu, x, o);
                    if ((int)threadIdx.x >= o) x += y;
                }
                keys[i0 + threadIdx.x] = sum + x - mine;
                sum += __shfl_sync(0xffffffffu, x, 31);
            }
            __syncwarp();
            for (int e0 = 0; e0 < p.E; e0 += 32) {
                const int e = e0 + (int)threadIdx.x;
                const int k = e < p.E ? min(max(key(e), 0), kSizes - 1) : kSizes;
                const uint32_t same = __match_any_sync(0xffffffffu, k);
                const int rank = __popc(same & ((1u << threadIdx.x) - 1));
                if (e < p.E) before[keys[k] + rank] = e;
                __syncwarp();
                if (e < p.E && rank == 0) keys[k] += __popc(same);
                __syncwarp();
            }
        } else {
            for (int e0 = 0; e0 <= p.E; e0 += 32) {
                const int e = e0 + (int)threadIdx.x;
                const int mine = e < p.E ? (first[e + 1] - first[e] + NT - 1) / NT : 0;
                int x = mine;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const int y = __shfl_up_sync(0xffffffffu, x, o);
                    if ((int)threadIdx.x >= o) x += y;
                }
                if (e <= p.E) before[e] = sum + x - mine;
                sum += __shfl_sync(0xffffffffu, x, 31);
            }
        }
    }
    __syncthreads();
    return ExpertList{first, before};
}

// Tensor copies into this CTA's shared memory; of a pair, `bar` may be the other's barrier
// (its address in the cluster's shared memory).
template <int NC>
__device__ __forceinline__ void copy3d(uint32_t dst, const CUtensorMap *map, int x, int y, int z,
                                       uint32_t bar) {
    if constexpr (NC == 1)
        asm volatile(
            "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
            " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
            "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(bar)
            : "memory");
    else
        asm volatile(
            "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.tile.mbarrier::"
            "complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
            "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(bar)
            : "memory");
}
template <int NC>
__device__ __forceinline__ void copy2d(uint32_t dst, const CUtensorMap *map, int x, int y,
                                       uint32_t bar) {
    if constexpr (NC == 1)
        asm volatile(
            "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
            " [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
            "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar)
            : "memory");
    else
        asm volatile(
            "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::"
            "complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
            "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar)
            : "memory");
}

// 16 lanes x 32 columns: with r = lane / 4 and c = lane % 4, registers 4 i and 4 i + 1
// hold row r, columns 8 i + 2 c and + 1; 4 i + 2 and 4 i + 3 those of row r + 8.
__device__ __forceinline__ void tmem_ld16x32(uint32_t addr, uint32_t (&x)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,"
        "%15}, [%16];"
        : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3]), "=r"(x[4]), "=r"(x[5]), "=r"(x[6]),
          "=r"(x[7]), "=r"(x[8]), "=r"(x[9]), "=r"(x[10]), "=r"(x[11]), "=r"(x[12]), "=r"(x[13]),
          "=r"(x[14]), "=r"(x[15])
        : "r"(addr)
        : "memory");
}

// Four 8x8 matrices, held as the matrix instruction's results are, to shared memory
// transposed: lane l gives the address of column l % 8 of matrix l / 8.
__device__ __forceinline__ void stsm4_t(uint32_t addr, uint32_t a, uint32_t b, uint32_t c,
                                        uint32_t d) {
    asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1,%2,%3,%4};" ::"r"(addr),
                 "r"(a), "r"(b), "r"(c), "r"(d)
                 : "memory");
}
__device__ __forceinline__ uint4 lds16(uint32_t addr) {
    uint4 x;
    asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w)
                 : "r"(addr));
    return x;
}

// mbar_wait by a whole warp, whose lanes then go the same way.
__device__ __forceinline__ bool warp_wait(uint64_t *bar, uint32_t parity, int32_t *err) {
    return __all_sync(0xffffffffu, mbar_wait(bar, parity, err));
}
// One thread of the warp, always the same. (Told so, the compiler keeps the thread's
// addresses and descriptors where the copies and products take them from.)
__device__ __forceinline__ bool elected() {
    uint32_t one;
    asm volatile(
        "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(one));
    return one != 0;
}

// Address of the pair's first CTA's variable.
__device__ __forceinline__ uint32_t of_first(const void *p) {
    uint32_t at;
    asm volatile("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(at) : "r"(smem_addr(p)));
    return at;
}

// The CTA's tiles in turn, worked out by a warp of their own: a search and four divisions
// take half a microsecond, in which the thread that issues the products would leave the
// tensor cores idle (they hold a product or two ahead, no more).
struct TileRing {
    ExpertTile *tile;
    uint64_t *full, *empty;
    int at;
    uint32_t parity;
    __device__ __forceinline__ void next() {
        if (++at == kTilesAhead) {
            at = 0;
            parity ^= 1;
        }
    }
    // The next tile, or false after the last; ok is false if the wait gave up.
    __device__ __forceinline__ bool take(ExpertTile &x, bool &ok, int32_t *err) {
        ok = mbar_wait(&full[at], parity, err);
        if (!ok) return false;
        x = tile[at];
        mbar_arrive(&empty[at]);
        next();
        return x.e >= 0;
    }
    __device__ __forceinline__ bool take_warp(ExpertTile &x, bool &ok, int32_t *err) {
        ok = __all_sync(0xffffffffu, mbar_wait(&full[at], parity, err));
        if (!ok) return false;
        x = tile[at];
        __syncwarp();
        if ((threadIdx.x & 31) == 0) mbar_arrive(&empty[at]);
        next();
        return x.e >= 0;
    }
};

// One arrival at the barrier of the pair's first CTA.
__device__ __forceinline__ void arrive_first(uint64_t *bar) {
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(of_first(bar))
                 : "memory");
}

__device__ __forceinline__ void arrive_first_relaxed(uint64_t *bar) {
    asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(of_first(bar))
                 : "memory");
}

// The instructions of one CTA (umma.cuh) or of a pair.
template <int NC>
__device__ __forceinline__ void product_step(uint32_t d, uint64_t a, uint64_t b, uint32_t instr,
                                             bool accumulate) {
    if constexpr (NC == 1) {
        mma_f16(d, a, b, instr, accumulate);
    } else {
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
            "l"(a), "l"(b), "r"(instr), "r"((uint32_t)accumulate)
            : "memory");
    }
}
// The barrier (of both CTAs) receives one arrival when the products issued so far are done.
template <int NC> __device__ __forceinline__ void commit_products(uint64_t *bar) {
    if constexpr (NC == 1) {
        mma_commit(bar);
    } else {
        asm volatile(
            "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster"
            ".b64 [%0], %1;" ::"r"(smem_addr(bar)),
            "h"((uint16_t)3)
            : "memory");
    }
}
template <int NC> __device__ __forceinline__ void alloc_columns(uint32_t *slot, int columns) {
    if constexpr (NC == 1) {
        tmem_alloc(slot, columns);
    } else {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                         smem_addr(slot)),
                     "r"(columns)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
}
template <int NC> __device__ __forceinline__ void free_columns(uint32_t tmem, int columns) {
    if constexpr (NC == 1)
        tmem_free(tmem, columns);
    else
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem),
                     "r"(columns)
                     : "memory");
}
// All threads of the CTA, or of the pair.
template <int NC> __device__ __forceinline__ void pair_barrier() {
    if constexpr (NC == 1)
        __syncthreads();
    else
        asm volatile("barrier.cluster.arrive.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
}

__device__ __forceinline__ void prefetch_map(const CUtensorMap *map) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(map)) : "memory");
}

// Rows [from, to) of `panels` panels of 64 rows set to 0, by one warp.
__device__ __forceinline__ void zero_rows(uint32_t operand, int panels, int from, int to) {
    const int lane = threadIdx.x & 31, n = (to - from) * 8;
    for (int q = 0; q < panels; ++q)
        for (int i = lane; i < n; i += 32)
            asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(
                             operand + q * 8192 + from * 128 + i * 16),
                         "r"(0)
                         : "memory");
}

// A_MN: A's elements adjacent in m (else in k). B is adjacent in k, in the gradient in n.
template <typename T, int NT, int NC, bool A_MN, bool GRAD>
__global__ void __launch_bounds__(kThreads, 1) k_experts(const __grid_constant__ ExpertArgs p) {
    using S = ExpertShape<NT, NC>;
    static_assert(A_MN || !GRAD, "the gradient's operands are both adjacent in m and n");
    extern __shared__ unsigned char smem_raw[];
    // last: a segment's last stage is there; mended: its rows past the end are 0, in both
    // CTAs of a pair. (These have barriers of their own, as who waits for them does not
    // follow the phases of the others.)
    __shared__ uint64_t full[S::stages], empty[S::stages], last[S::stages], mended[S::stages];
    __shared__ uint64_t ready[2], taken[2];
    __shared__ uint64_t drained, listed[kTilesAhead], read[kTilesAhead];
    __shared__ ExpertTile tile_ring[kTilesAhead];
    __shared__ uint32_t tmem_slot;
    const uint32_t smem = (smem_addr(smem_raw) + 1023u) & ~1023u;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = NC == 1 ? 0 : blockIdx.x & 1;   // in the pair
    const int first_tile = blockIdx.x / NC, step = gridDim.x / NC;
    if (threadIdx.x == 0) {
        for (int i = 0; i < S::stages; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], 1);
            mbar_init(&last[i], 1);
            mbar_init(&mended[i], NC);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&ready[i], 1);
            mbar_init(&taken[i], kResults * NC);
        }
        for (int i = 0; i < kTilesAhead; ++i) {
            mbar_init(&listed[i], 1);
            // a thread of copies, one of products, the warps of results, ends of segments
            mbar_init(&read[i], 1 + (rank == 0) + kResults + GRAD);
        }
        mbar_init(&drained, 1);
        mbar_init_fence();
    }
    if (warp == 1) {
        alloc_columns<NC>(&tmem_slot, S::columns);
        mma_fence_before();
    } else if (threadIdx.x == 64 && p.P > 0) {   // the first copies find the maps at hand
        prefetch_map(&p.a_map);
        prefetch_map(&p.b_map);
    }
    const ExpertList list = expert_list<NT, GRAD>(
        p, (int32_t *)(smem_raw + (smem - smem_addr(smem_raw)) + S::at_offsets));
    pair_barrier<NC>();
    mma_fence_after();
    const uint32_t tmem = tmem_slot;
    TileRing ring{tile_ring, listed, read, 0, 0};
    ExpertTile x;

    if (warp == 2) {
        // ------------------------------------------------------ the tiles' list
        if (lane == 0) {
            const int tiles = list.template tiles<GRAD>(p);
            ring.parity = 1;
            // there and back where lengths differ: with experts alike the tiles that share
            // operands are further apart in time then (65536 slots of 16, 4096 x 4096: 1169 us
            // for 1076)
            const bool back = GRAD && p.E > 0 &&
                              (int64_t)(list.first[list.before[0] + 1] - list.first[list.before[0]]) *
                                      p.E > 2 * (int64_t)list.first[p.E];
            for (int turn = 0;; ++turn) {
                if (!mbar_wait(&read[ring.at], ring.parity, p.err)) break;
                const int t = turn * step + (back && turn & 1 ? step - 1 - first_tile : first_tile);
                // (a turn that has none here may have been the last, or the one before it)
                const bool more = turn * (int64_t)step < tiles;
                ExpertTile &to = tile_ring[ring.at];
                if (more && t < tiles) {
                    to = list.template tile<S, GRAD>(p, t);
                } else if (more) {
                    continue;
                } else {
                    to.e = -1;
                }
                mbar_arrive(&listed[ring.at]);
                ring.next();
                if (!more) break;
            }
        }
        __syncwarp();
    } else if (warp == 0) {
        // ------------------------------------------------------ operands' tiles
        if (elected()) {
            int stage = 0;
            int64_t issued = 0;
            uint32_t parity = 1;                 // the ring starts empty
            uint32_t ends = 0;                   // a bit per stage: ends so far, mod 2
            bool ok = true;
            while (ok && ring.take(x, ok, p.err)) {
                const int m0 = x.m0 + rank * kRowsM;
                const int mine = (x.n + S::STEP - 1) / S::STEP * 16, n0 = rank * mine;   // of n
                const int boxes = GRAD ? (mine + 63) / 64 : (mine + S::BOX - 1) / S::BOX;
                const uint32_t bytes =
                    S::a_bytes + (uint32_t)boxes * (GRAD ? 8192 : S::BOX * kDepth * 2);
                for (int k0 = 0; k0 < x.k; k0 += kDepth) {
                    ok = mbar_wait(&empty[stage], parity, p.err);
                    if (!ok) break;
                    // a pair's copies are counted by its first CTA, but for a segment's end
                    const bool end = GRAD && (x.k - k0) % 16 && x.k - k0 < kDepth;
                    uint32_t bar = smem_addr(&full[stage]);
                    if (end) {
                        mbar_arrive_expect_tx(&last[stage], bytes);
                        if (rank == 0) mbar_arrive(&full[stage]);
                        bar = smem_addr(&last[stage]);
                        ends ^= 1u << stage;
                    } else if (rank == 0) {
                        mbar_arrive_expect_tx(&full[stage], NC * bytes);
                    } else {
                        bar = of_first(&full[stage]);
                    }
                    const uint32_t a = smem + stage * S::stage, b = a + S::a_bytes;
                    if (GRAD) {
                        const int r = (int)((int64_t)x.r0 + k0);
                        copy3d<NC>(a, &p.a_map, m0, r, 0, bar);
                        copy3d<NC>(a + 8192, &p.a_map, m0 + 64, r, 0, bar);
                        for (int i = 0; i < boxes; ++i)
                            copy2d<NC>(b + i * 8192, &p.b_map, x.n0 + n0 + 64 * i, r, bar);
                    } else {
                        const int z = x.e * p.a_step;
                        if (A_MN) {
                            copy3d<NC>(a, &p.a_map, m0, k0, z, bar);
                            copy3d<NC>(a + 8192, &p.a_map, m0 + 64, k0, z, bar);
                        } else {
                            copy3d<NC>(a, &p.a_map, k0, m0, z, bar);
                        }
                        for (int i = 0; i < boxes; ++i)
                            copy2d<NC>(b + i * S::BOX * 128, &p.b_map, k0,
                                       (int)((int64_t)x.r0 + n0 + i * S::BOX), bar);
                    }
                    ++issued;
                    if (++stage == S::stages) {
                        stage = 0;
                        parity ^= 1;
                    }
                }
            }
            // The last stages' products are awaited too: their arrivals at `empty` (a pair's
            // at both CTAs') are in nobody else's order, and must be there before the CTA ends.
            for (int i = 0; ok && i < S::stages; ++i) {
                ok = mbar_wait(&empty[stage], parity, p.err);
                if (++stage == S::stages) {
                    stage = 0;
                    parity ^= 1;
                }
            }
            // another thread gave up: see the copies in flight land before the CTA ends
            // (those of a pair's second CTA are counted by the first: it waits for a while)
            if (!ok && rank == 1) mbar_wait(&drained, 0, p.err);
            for (int64_t i = 0; !ok && i < S::stages; ++i) {
                const int64_t at = issued - 1 - i;
                if (rank == 0 && at >= 0)
                    mbar_wait(&full[at % S::stages], (uint32_t)(at / S::stages) & 1, p.err);
                if (GRAD) mbar_wait(&last[i], (ends >> i & 1) ^ 1, p.err);
            }
        }
        __syncwarp();
    } else if (warp == 1) {
        // ------------------------------------------------------ products
        if (rank == 0 && elected()) {
            int stage = 0, acc = 0;
            uint32_t parity = 0, free_parity = 1;    // both accumulators start free
            uint32_t ends = 0;                       // a bit per stage: ends so far, mod 2
            bool ok = true, more = ring.take(x, ok, p.err);
            while (more) {
                ExpertTile y;                    // the next tile, taken while this one's products run
                if (x.k == 0) {
                    more = ring.take(x, ok, p.err);
                    continue;
                }
                ok = mbar_wait(&taken[acc], free_parity, p.err);
                if (!ok) break;
                const int mine = (x.n + S::STEP - 1) / S::STEP * 16;
                const uint32_t d = tmem + acc * NT;
                const uint32_t instr = instr_f16<T>(kRowsM * NC, mine * NC, A_MN, GRAD);
                const int whole = x.k / kDepth, rest = x.k % kDepth;
                for (int i = 0; i < whole; ++i) {
                    ok = mbar_wait(&full[stage], parity, p.err);
                    if (!ok) break;
                    mma_fence_after();
                    const uint32_t a = smem + stage * S::stage, b = a + S::a_bytes;
                    uint64_t da = A_MN ? desc_mn(a, 8192) : desc_k(a);
                    uint64_t db = GRAD ? desc_mn(b, 8192) : desc_k(b);
#pragma unroll
                    for (int j = 0; j < kDepth / 16; ++j) {
                        product_step<NC>(d, da, db, instr, i > 0 || j > 0);
                        da += (A_MN ? 2048 : 32) >> 4;
                        db += (GRAD ? 2048 : 32) >> 4;
                    }
                    commit_products<NC>(&empty[stage]);
                    if (++stage == S::stages) {
                        stage = 0;
                        parity ^= 1;
                    }
                    if (i == 0) more = ring.take(y, ok, p.err);
                    if (!ok) break;
                }
                if (!ok) break;
                if (rest) {
                    const int steps = (rest + 15) / 16;
                    const uint32_t a = smem + stage * S::stage, b = a + S::a_bytes;
                    ok = mbar_wait(&full[stage], parity, p.err);
                    if (ok && GRAD && rest % 16) {
                        ok = mbar_wait(&mended[stage], ends >> stage & 1, p.err);
                        if (NC == 2) asm volatile("fence.acq_rel.cluster;" ::: "memory");
                        ends ^= 1u << stage;
                    }
                    if (!ok) break;
                    mma_fence_after();
                    for (int i = 0; i < steps; ++i)
                        product_step<NC>(d, A_MN ? desc_mn(a + i * 2048, 8192) : desc_k(a + i * 32),
                                         GRAD ? desc_mn(b + i * 2048, 8192) : desc_k(b + i * 32),
                                         instr, whole > 0 || i > 0);
                    commit_products<NC>(&empty[stage]);
                    if (++stage == S::stages) {
                        stage = 0;
                        parity ^= 1;
                    }
                }
                commit_products<NC>(&ready[acc]);
                acc ^= 1;
                free_parity ^= acc == 0;
                if (whole == 0) more = ring.take(y, ok, p.err);
                x = y;
            }
            if (!ok) {
                commit_products<NC>(&drained);
                mbar_wait_poll(&drained, 0, p.err);
            }
        }
        __syncwarp();
    } else if (warp == 3) {
        // ------------------------------------------------------ ends of segments
        // rows of k past the expert's last, up to a step of products, are set to 0
        uint32_t count = 0, ends = 0;            // stages so far
        bool ok = true;
        while (GRAD && ok && ring.take_warp(x, ok, p.err)) {
            count += x.k / kDepth;
            const int rest = x.k % kDepth, stage = count % S::stages;
            if (rest % 16) {
                ok = warp_wait(&last[stage], ends >> stage & 1, p.err);
                if (!ok) break;
                ends ^= 1u << stage;
                const int to = (rest + 15) & ~15, mine = (x.n + S::STEP - 1) / S::STEP * 16;
                const uint32_t a = smem + stage * S::stage;
                zero_rows(a, 2, rest, to);
                zero_rows(a + S::a_bytes, (mine + 63) / 64, rest, to);
                fence_proxy_async_shared();
                __syncwarp();
                if (lane == 0) {
                    if (rank == 0) mbar_arrive(&mended[stage]);
                    else arrive_first(&mended[stage]);
                }
            }
            count += rest > 0;
        }
        __syncwarp();
    } else {
        // ------------------------------------------------------ results
        // two warps to a quarter of tensor memory's lanes (a warp reads those of its number mod
        // 4), each every other 32 columns
        const int quarter = warp & 3, c0 = (warp - 4) / 4 * 32;
        // A row's four 16-byte chunks are permuted by half its number, so that eight rows' fall in
        // different banks, and two whole rows'.
        const uint32_t out_smem = smem + S::at_out + (warp - 4) * S::out_bytes;
        auto chunk = [&](int row, int c) {
            return out_smem + row * 64 + (((c ^ (row >> 1)) & 3) << 4);
        };
        const int put_row = (lane >> 4) * 8 + (lane & 7), put_c = (lane >> 3) & 1;
        int acc = 0;
        uint32_t parity = 0;
        bool ok = true;
        while (ring.take_warp(x, ok, p.err)) {
            const int m = x.m0 + rank * kRowsM + quarter * 32 + (lane & 3) * 8;
            T *out = (T *)p.out + (GRAD ? x.e * p.o_se + x.n0 * p.o_ld : (int64_t)x.r0 * p.o_ld) + m;
            if (GRAD && p.splits > 1) {
                // fp32, as the registers hold them: two adjacent n of a row of m
                float *part = p.parts + ((int64_t)x.part * p.E + x.e) * p.M * p.N + x.n0;
                const int row = x.m0 + rank * kRowsM + quarter * 32 + (lane >> 2);
                if (x.k > 0) {
                    if (!warp_wait(&ready[acc], parity, p.err)) break;
                    mma_fence_after();
                }
                const uint32_t d = tmem + acc * NT + ((uint32_t)quarter << 21);
                for (int c = c0; c < x.n; c += 64) {
                    uint32_t v[2][16] = {};
                    if (x.k > 0) {
                        tmem_ld16x32(d + c, v[0]);
                        tmem_ld16x32(d + (16u << 16) + c, v[1]);
                        tmem_wait_ld();
                    }
#pragma unroll
                    for (int h = 0; h < 2; ++h)
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            const int m = row + 16 * h + 8 * (i & 1);
                            const int n = c + 8 * (i >> 1) + 2 * (lane & 3);
                            if (m < p.M && n < x.n)
                                *(float2 *)(part + (int64_t)m * p.N + n) =
                                    make_float2(__uint_as_float(v[h][2 * i]),
                                                __uint_as_float(v[h][2 * i + 1]));
                        }
                }
                if (x.k > 0) {
                    mma_fence_before();
                    __syncwarp();
                    if (lane == 0) {
                        if (rank == 0) mbar_arrive(&taken[acc]);
                        else arrive_first_relaxed(&taken[acc]);
                    }
                    acc ^= 1;
                    parity ^= acc == 0;
                }
                continue;
            }
            if (x.k == 0) {
                for (int n = c0 / 4 + (lane >> 2); m < p.M && n < x.n; n += 16)
                    *(uint4 *)(out + n * p.o_ld) = make_uint4(0, 0, 0, 0);
                continue;
            }
            if (!warp_wait(&ready[acc], parity, p.err)) break;
            mma_fence_after();
            const uint32_t d = tmem + acc * NT + ((uint32_t)quarter << 21);
            uint32_t v[2][16];
            if (c0 < x.n) {
                tmem_ld16x32(d + c0, v[0]);
                tmem_ld16x32(d + (16u << 16) + c0, v[1]);
            }
            // handed back as soon as the last columns are in registers; no memory is (a release
            // would wait for the stores)
            auto hand_back = [&] {
                mma_fence_before();
                __syncwarp();
                if (lane == 0) {
                    if (rank == 0) mbar_arrive(&taken[acc]);
                    else arrive_first_relaxed(&taken[acc]);
                }
            };
            if (c0 >= x.n) hand_back();
            for (int c = c0; c < x.n; c += 64) {
                tmem_wait_ld();
                uint32_t y[2][8];
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        y[h][i] = pack2<T>(__uint_as_float(v[h][2 * i]),
                                           __uint_as_float(v[h][2 * i + 1]));
                if (c + 64 < x.n) {              // on their way while these are written
                    tmem_ld16x32(d + c + 64, v[0]);
                    tmem_ld16x32(d + (16u << 16) + c + 64, v[1]);
                } else {
                    hand_back();
                }
                __syncwarp();                    // the rows before are read
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int i = 0; i < 4; i += 2)
                        stsm4_t(chunk(put_row + i * 8, put_c + 2 * h), y[h][2 * i], y[h][2 * i + 1],
                                y[h][2 * i + 2], y[h][2 * i + 3]);
                __syncwarp();
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int n = c + i * 8 + (lane >> 2);
                    const uint4 z = lds16(chunk(i * 8 + (lane >> 2), lane & 3));
                    if (m < p.M && n < x.n) *(uint4 *)(out + n * p.o_ld) = z;
                }
            }
            acc ^= 1;
            parity ^= acc == 0;
        }
        if (!GRAD) {                             // the rows of no pair
            const int64_t kept = list.first[p.E];
            uint4 *out = (uint4 *)((T *)p.out + kept * p.o_ld);
            const int64_t n = (p.P - kept) * p.o_ld / 8;
            constexpr int threads = 32 * kResults;
            for (int64_t i = (int64_t)blockIdx.x * threads + threadIdx.x - 128; i < n;
                 i += (int64_t)gridDim.x * threads)
                out[i] = make_uint4(0, 0, 0, 0);
        }
        __syncwarp();
    }
    // (of a pair: neither leaves, or gives its tensor memory back, before both are done)
    pair_barrier<NC>();
    if (warp == 1) free_columns<NC>(tmem, S::columns);
}

// dw[e, n, m] (m adjacent, strides o_se and o_ld) = the sum of the parts [splits][E][M][N], in
// their order: 32 x 32 elements a CTA, turned over in shared memory.
template <typename T>
__global__ void __launch_bounds__(256) k_experts_sum(const float *parts, int splits, int E, int M,
                                                     int N, T *out, int64_t o_se, int64_t o_ld) {
    __shared__ float tile[32][33];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int tiles_n = (N + 31) / 32, m0 = blockIdx.x / tiles_n * 32, n0 = blockIdx.x % tiles_n * 32;
    const int64_t e = blockIdx.y, one = (int64_t)M * N;
    for (int i = warp; i < 32; i += 8) {
        const int m = m0 + i, n = n0 + lane;
        float x = 0.0f;
        if (m < M && n < N) {
            const float *p = parts + e * one + (int64_t)m * N + n;
#pragma unroll 4
            for (int j = 0; j < splits; ++j) x += p[j * E * one];
        }
        tile[i][lane] = x;
    }
    __syncthreads();
    for (int i = warp; i < 32; i += 8) {
        const int n = n0 + i, m = m0 + lane;
        if (m < M && n < N) out[e * o_se + n * o_ld + m] = from_f32<T>(tile[lane][i]);
    }
}

// ------------------------------------------------------------------- host
bool aligned(const void *p) { return p && (uintptr_t)p % 16 == 0; }

spmm_status check_sizes(int dtype, const int32_t *offsets, int64_t P, int64_t E, int64_t H,
                        int64_t F) {
    if (!dtype_ok(dtype) || !offsets || P < 0 || E < 0 || H < 0 || F < 0)
        return SPMM_ERR_INVALID_ARG;
    if (dtype == SPMM_F32 || H % 8 || F % 8 || H > (1 << 20) || F > (1 << 20) ||
        E > SPMM_ROUTES_MAX_EXPERTS || P > INT32_MAX - 65536)   // (slots and a tile: 32 bits)
        return SPMM_ERR_UNSUPPORTED;
    return SPMM_OK;
}

// Strides of [E, H, F] matrices, one of the last two adjacent.
bool strides_ok(int64_t se, int64_t sh, int64_t sf) {
    if (se < 0 || se % 8) return false;
    return (sf == 1 && sh > 0 && sh % 8 == 0) || (sh == 1 && sf > 0 && sf % 8 == 0);
}
bool strides_far(int64_t se, int64_t sh, int64_t sf) {
    return std::max(se, std::max(sh, sf)) >= (int64_t)1 << 38;   // a tensor map's are below 2^40 bytes
}

PFN_cuTensorMapEncodeTiled_v12000 encoder() {
    static const PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
        cudaDriverEntryPointQueryResult q;
        void *f = nullptr;
        const cudaError_t e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000,
                                                               cudaEnableDefault, &q);
        return e == cudaSuccess && q == cudaDriverEntryPointSuccess
                   ? reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f)
                   : nullptr;
    }();
    return fn;
}

// [n2, n1, n0] elements with adjacent n0; copies of box1 rows of 64.
cudaError_t encode(CUtensorMap *map, int dtype, int rank, const void *p, int64_t n0, int64_t n1,
                   int64_t n2, int64_t s1, int64_t s2, int box1) {
    if (!encoder()) return cudaErrorNotSupported;
    const cuuint64_t dims[3] = {(cuuint64_t)n0, (cuuint64_t)n1, (cuuint64_t)n2};
    const cuuint64_t strides[2] = {(cuuint64_t)s1 * 2, (cuuint64_t)s2 * 2};
    const cuuint32_t box[3] = {kDepth, (cuuint32_t)box1, 1}, step[3] = {1, 1, 1};
    const CUresult e = encoder()(
        map, dtype == SPMM_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
        (cuuint32_t)rank, const_cast<void *>(p), dims, strides, box, step,
        CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return e == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

template <typename T, int NT, int NC, bool A_MN, bool GRAD>
cudaError_t launch(const ExpertArgs &p, int64_t most, cudaStream_t s) {
    using S = ExpertShape<NT, NC>;
    // the kernel's limit is the process's: always the largest, as another thread may set it
    // (besides: barriers, the tiles' ring, the tensor memory's address, the sort's sizes)
    constexpr size_t fixed = sizeof(uint64_t) * (4 * S::stages + 2 * 2 + 1 + 2 * kTilesAhead) +
                             sizeof(ExpertTile) * kTilesAhead + 16 + GRAD * sizeof(int32_t) * kSizes;
    static_assert(S::bytes(SPMM_ROUTES_MAX_EXPERTS) + fixed <= kSmemMax, "fits");
    // (and once for each device)
    static std::atomic<uint64_t> done{0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    const uint64_t bit = 1ull << (dev & 63);
    if (e == cudaSuccess && (dev > 63 || !(done.load(std::memory_order_relaxed) & bit))) {
        e = cudaFuncSetAttribute(k_experts<T, NT, NC, A_MN, GRAD>,
                                 cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 (int)S::bytes(SPMM_ROUTES_MAX_EXPERTS));
        if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_relaxed);
    }
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t c{};
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = NC;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    c.gridDim = dim3((unsigned)std::max<int64_t>(1, std::min<int64_t>(most, kSms / NC)) * NC);
    c.blockDim = dim3(kThreads);
    c.dynamicSmemBytes = S::bytes(p.E);
    c.stream = s;
    c.attrs = &attr;
    c.numAttrs = NC > 1;
    e = cudaLaunchKernelEx(&c, k_experts<T, NT, NC, A_MN, GRAD>, p);
    count_launch();
    return e;
}

template <int NT, int NC, bool A_MN, bool GRAD>
cudaError_t launch(int dtype, const ExpertArgs &p, int64_t most, cudaStream_t s) {
    return dtype == SPMM_BF16 ? launch<__nv_bfloat16, NT, NC, A_MN, GRAD>(p, most, s)
                              : launch<__half, NT, NC, A_MN, GRAD>(p, most, s);
}

// Tiles of up to 32 slots while the experts have no more than 8 on average. A product is then
// bound by the matrices' bytes and by the latency of its copies: tiles of one CTA give twice
// as many of them. Measured, in microseconds, against the pairs' tiles of 256 (2048 x 1024): 8
// slots of 64 experts 10.0 and 12.0, 512 of 64 32.4 and 35.6; 16 on average, 2048 slots of 128
// (2048 x 768), 53.1 and 50.9; 64 on average, 512 of 8 (2048 x 2048), 16.1 and 11.5.
bool few_slots(int64_t P, int64_t E) { return P <= 8 * E; }

template <int NT, int NC>
cudaError_t product(int dtype, ExpertArgs &p, const void *xs, const void *w, int64_t se,
                    int64_t sh, int64_t sf, cudaStream_t s) {
    using S = ExpertShape<NT, NC>;
    const int64_t n2 = p.a_step ? p.E : 1, s2 = p.a_step ? se : 8;
    const bool mn = sf == 1;
    cudaError_t e = mn ? encode(&p.a_map, dtype, 3, w, p.M, p.K, n2, sh, s2, 64)
                       : encode(&p.a_map, dtype, 3, w, p.K, p.M, n2, sf, s2, kRowsM);
    if (e == cudaSuccess) e = encode(&p.b_map, dtype, 2, xs, p.K, p.P, 1, p.K, 8, S::BOX);
    if (e != cudaSuccess) return e;
    p.tiles_m = (p.M + kRowsM * NC - 1) / (kRowsM * NC);
    const int64_t most = (p.P / NT + std::min<int64_t>(p.E, p.P)) * p.tiles_m;
    return mn ? launch<NT, NC, true, false>(dtype, p, most, s)
              : launch<NT, NC, false, false>(dtype, p, most, s);
}

template <int NC>
cudaError_t weights(int dtype, ExpertArgs &p, cudaStream_t s) {
    constexpr int NT = 256;
    p.tiles_m = (p.M + kRowsM * NC - 1) / (kRowsM * NC);
    p.tiles_n = (p.N + NT - 1) / NT;
    cudaError_t e = launch<NT, NC, true, true>(
        dtype, p, (int64_t)p.E * p.splits * p.tiles_m * p.tiles_n, s);
    if (e != cudaSuccess || p.splits == 1) return e;
    const dim3 grid((unsigned)(((p.M + 31) / 32) * ((p.N + 31) / 32)), (unsigned)p.E);
    if (dtype == SPMM_BF16)
        k_experts_sum<<<grid, 256, 0, s>>>(p.parts, p.splits, p.E, p.M, p.N, (__nv_bfloat16 *)p.out,
                                           p.o_se, p.o_ld);
    else
        k_experts_sum<<<grid, 256, 0, s>>>(p.parts, p.splits, p.E, p.M, p.N, (__half *)p.out, p.o_se,
                                           p.o_ld);
    count_launch();
    return cudaGetLastError();
}

// Parts of an expert's slots in the gradient: the number that is done soonest by an estimate,
// in microseconds, for experts alike: a pair's 64 slots of a tile take 0.31, a tile's beginning
// and end 1; parts take a launch more (4) and are written and read once at 5 TB/s.
// Measured with one part and with this many: 65536 slots of one expert, 256 x 256, 276 us and 36
// (54 parts), 2048 x 1024, 277 and 168 (7); 16384 of four experts, 512 x 512, 24 and 19 (4); 4096
// of one, 256 x 256, 24 and 16 (13), 1024 x 1024, 24 and 20 (4).
// However the slots are spread, no part has more than kPartSlots: one expert may hold all of them,
// and who waits for a tile's sum waits for all of its stages, 0.08 s of a limit of 0.5.
constexpr int64_t kPartSlots = (int64_t)1 << 24;
int64_t weight_splits(int64_t P, int64_t E, int64_t H, int64_t F) {
    if (E == 0 || H == 0 || F == 0) return 1;
    constexpr int64_t pairs = kSms / 2;
    const int64_t fewest = std::max<int64_t>(1, (P + kPartSlots - 1) / kPartSlots);
    const int64_t tiles = E * ((H + 255) / 256) * ((F + 255) / 256), slots = P / E;
    if (tiles >= 2 * pairs) return fewest;
    int64_t best = fewest;
    double least = 0.0;
    for (int64_t n = fewest; n == fewest || (n <= pairs && n * 128 <= slots); ++n) {
        const double us = (double)((tiles * n + pairs - 1) / pairs) *
                              ((double)((slots / n + 63) / 64) * 0.31 + 1.0) +
                          (n > 1 ? 4.0 + (double)(n * E * H * F) * 1.6e-6 : 0.0);
        if (n == fewest || us < least) {
            best = n;
            least = us;
        }
    }
    return best;
}

}  // namespace
}  // namespace spmm

extern "C" {

spmm_status spmm_routes_product(int dtype, const void *xs, const void *w, int64_t w_se,
                                int64_t w_sh, int64_t w_sf, const int32_t *offsets, int64_t P,
                                int64_t E, int64_t H, int64_t F, void *ys, void *stream) {
    using namespace spmm;
    const spmm_status st = check_sizes(dtype, offsets, P, E, H, F);
    if (st != SPMM_OK) return st;
    if (P == 0 || F == 0) return SPMM_OK;
    if (!aligned(ys)) return SPMM_ERR_INVALID_ARG;
    cudaStream_t s = (cudaStream_t)stream;
    if (E == 0 || H == 0)                        // nothing to add up
        return cuda_status(cudaMemsetAsync(ys, 0, (size_t)P * F * 2, s));
    if (!aligned(xs) || !aligned(w) || !strides_ok(w_se, w_sh, w_sf)) return SPMM_ERR_INVALID_ARG;
    ExpertArgs p{};
    if (strides_far(w_se, w_sh, w_sf) || (P / 32 + E) * ((F + kRowsM - 1) / kRowsM) > (1 << 30))
        return SPMM_ERR_UNSUPPORTED;
    p.offsets = offsets;
    p.out = ys;
    p.o_ld = F;
    p.P = P;
    p.E = (int)E;
    p.M = (int)F;
    p.K = (int)H;
    p.a_step = E > 1 && w_se > 0;
    cudaError_t e = dynamic_err(s, &p.err);
    if (e == cudaSuccess)
        e = few_slots(P, E) ? product<32, 1>(dtype, p, xs, w, w_se, w_sh, w_sf, s)
            : F > kRowsM    ? product<256, 2>(dtype, p, xs, w, w_se, w_sh, w_sf, s)
                            : product<256, 1>(dtype, p, xs, w, w_se, w_sh, w_sf, s);
    return cuda_status(e);
}

int64_t spmm_routes_product_weights_workspace(int64_t P, int64_t E, int64_t H, int64_t F) {
    using namespace spmm;
    if (P < 0 || E < 0 || H < 0 || F < 0 || E > SPMM_ROUTES_MAX_EXPERTS || H > (1 << 20) ||
        F > (1 << 20) || P > INT32_MAX)
        return 0;
    const int64_t splits = weight_splits(P, E, H, F);
    return splits > 1 ? splits * E * H * F * (int64_t)sizeof(float) : 0;
}

spmm_status spmm_routes_product_weights(int dtype, const void *xs, const void *dys,
                                        const int32_t *offsets, int64_t P, int64_t E, int64_t H,
                                        int64_t F, void *dw, int64_t dw_se, int64_t dw_sh,
                                        int64_t dw_sf, void *work, int64_t work_bytes,
                                        void *stream) {
    using namespace spmm;
    const spmm_status st = check_sizes(dtype, offsets, P, E, H, F);
    if (st != SPMM_OK) return st;
    if (E == 0 || H == 0 || F == 0) return SPMM_OK;
    if (!aligned(dw) || !strides_ok(dw_se, dw_sh, dw_sf) || (E > 1 && dw_se == 0) ||
        (dw_sf == 1 ? dw_sh < F : dw_sf < H))    // rows on top of one another
        return SPMM_ERR_INVALID_ARG;
    if (P && (!aligned(xs) || !aligned(dys))) return SPMM_ERR_INVALID_ARG;
    const int64_t need = spmm_routes_product_weights_workspace(P, E, H, F);
    if (need && (!aligned(work) || work_bytes < need)) return SPMM_ERR_INVALID_ARG;
    const bool by_f = dw_sf == 1;                // m = f, else m = h
    ExpertArgs p{};
    p.splits = (int)weight_splits(P, E, H, F);
    p.parts = (float *)work;
    p.M = (int)(by_f ? F : H);
    p.N = (int)(by_f ? H : F);
    if (E * p.splits * ((p.M + kRowsM - 1) / kRowsM) * ((p.N + 255) / 256) > (1 << 30))
        return SPMM_ERR_UNSUPPORTED;
    p.offsets = offsets;
    p.out = dw;
    p.o_se = dw_se;
    p.o_ld = by_f ? dw_sh : dw_sf;
    p.P = P;
    p.E = (int)E;
    cudaStream_t s = (cudaStream_t)stream;
    cudaError_t e = dynamic_err(s, &p.err);
    const void *a = by_f ? dys : xs, *b = by_f ? xs : dys;
    if (e == cudaSuccess && P) {
        e = encode(&p.a_map, dtype, 3, a, p.M, P, 1, p.M, 8, kDepth);
        if (e == cudaSuccess) e = encode(&p.b_map, dtype, 2, b, p.N, P, 1, p.N, 8, kDepth);
    }
    if (e == cudaSuccess)
        e = p.M > kRowsM ? weights<2>(dtype, p, s) : weights<1>(dtype, p, s);
    return cuda_status(e);
}

}  // extern "C"
