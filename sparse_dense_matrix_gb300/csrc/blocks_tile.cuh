// Selected-block attention by tile of rows: R = 16 W adjacent (query, head) rows
// of one kv head per CTA, a consumer warp per 16 rows. A producer warp merges
// the lists of the tile's queries (all ascending, so the next block is the
// smallest of the lists' heads) and has the tensor-copy engine bring each block
// of the union once into a ring of shared-memory stages, with the bits of the
// queries that chose it; a consumer warp skips a block that none of its rows
// chose. Neighbouring queries choose alike, so a block's keys and values are
// read once for many rows, and nothing is written but the result.
#pragma once

#include "blocks.cuh"

namespace spmm {

constexpr int kTileWarps = 8;                      // consumer warps
constexpr int kTileRows = 16 * kTileWarps;
constexpr int kTileThreads = 32 * (kTileWarps + 1);
constexpr int kTileLists = kTileRows / 32;         // lists per producer lane, words of bits

struct TileStage {
    int key0;                                      // first key, or -1: no more blocks
    uint32_t mask[kTileLists];                     // bit of each query of the tile
};

// Shared memory: `stages` of K then V, KB keys each, as D / 64 panels of KB rows
// of 128 bytes, the 16-byte chunks of a row permuted by the copy's 128-byte
// swizzle; then the barriers and what the producer says of each stage.
template <int D, int KB> struct TileSmem {
    static constexpr int operand = KB * D * 2;
    static constexpr int stage = 2 * operand;
    static constexpr int stages = (D == 128 ? 6 : 8) * 64 / KB > 16 ? 16 : (D == 128 ? 6 : 8) * 64 / KB;
    static constexpr int bytes = stages * stage + 1024 /* alignment */;
};

template <int KB> __device__ __forceinline__ uint32_t panel_at(int row, int chunk) {
    return (uint32_t)((chunk >> 3) * KB * 128 + row * 128 + (((chunk ^ row) & 7) << 4));
}

// A K or V tile whose first coordinate is a 64-element panel.
__device__ __forceinline__ void tensor4d_g2s(uint32_t dst, const CUtensorMap *map, int x, int y,
                                             int z, int w, uint64_t *bar) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4, %5}], [%6];"
        ::"r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(w),
          "r"(smem_addr(bar))
        : "memory");
}

struct TileArgs {
    BlkArgs a;
    CUtensorMap k_map, v_map;
    int64_t rows;            // Tq G rows of one kv head
    int tiles;               // ceil(rows / kTileRows)
    int32_t *err;
};

// Which rows a CTA owns. Later tiles see more keys: they are started first.
struct TilePlace {
    int b, h;
    int64_t f0;              // first row, f = t G + g
    int t_first, nq;         // the tile's queries
    __device__ __forceinline__ TilePlace(const TileArgs &p) {
        const int hb = blockIdx.y;
        h = hb % p.a.Hk;
        b = hb / p.a.Hk;
        f0 = (int64_t)(p.tiles - 1 - (int)blockIdx.x) * kTileRows;
        const int64_t f1 = min(p.rows, f0 + kTileRows) - 1;
        t_first = (int)(f0 / p.a.G);
        nq = (int)(f1 / p.a.G) - t_first + 1;
    }
};

template <int D, int KB>
__device__ __forceinline__ void tile_produce(const TileArgs &p, const TilePlace &at,
                                             uint32_t smem, uint64_t *full, uint64_t *empty,
                                             TileStage *info) {
    using S = TileSmem<D, KB>;
    const BlkArgs &a = p.a;
    const int lane = threadIdx.x & 31;
    const int len = blk_len(a, at.b);
    constexpr int kNone = INT_MAX;
    const int32_t *list[kTileLists];
    int j[kTileLists], head[kTileLists], end[kTileLists];     // end: first block out of sight
    auto next = [&](int i) {
        // entries below the one before them or out of range are skipped
        head[i] = kNone;
        while (j[i] < a.n) {
            const int at_ = j[i]++;
            if (blk_entry_ok(list[i], at_, a.NB)) {
                const int c = list[i][at_];
                if (c < end[i]) head[i] = c;
                break;
            }
        }
    };
#pragma unroll
    for (int i = 0; i < kTileLists; ++i) {
        const int q = i * 32 + lane;
        j[i] = a.n;
        end[i] = 0;
        list[i] = a.blocks;
        if (q < at.nq) {
            const int t = at.t_first + q;
            list[i] = a.blocks + (((int64_t)at.b * a.Tq + t) * a.Hk + at.h) * a.n;
            j[i] = 0;
            end[i] = (blk_limit(a, len, t) + a.block - 1) / a.block;
        }
        next(i);
    }
    int stage = 0, issued = 0;
    uint32_t parity = 1;                           // the ring starts empty
    bool ok = true;
    while (ok) {
        int least = head[0];
#pragma unroll
        for (int i = 1; i < kTileLists; ++i) least = min(least, head[i]);
        least = __reduce_min_sync(0xffffffffu, least);
        uint32_t mask[kTileLists];
#pragma unroll
        for (int i = 0; i < kTileLists; ++i) {
            const bool mine = least != kNone && head[i] == least;
            mask[i] = __ballot_sync(0xffffffffu, mine);
            if (mine) next(i);
        }
        const int parts = least == kNone ? 1 : a.block / KB;
        for (int s = 0; s < parts; ++s) {
            const int key0 = least == kNone ? -1 : least * a.block + s * KB;
            if (key0 >= a.Tk) break;               // the second half of a last, short block
            ok = mbar_wait(&empty[stage], parity, p.err);
            if (!ok) break;
            if (lane == 0) {
                info[stage].key0 = key0;
#pragma unroll
                for (int i = 0; i < kTileLists; ++i) info[stage].mask[i] = mask[i];
                if (key0 < 0) {
                    mbar_arrive(&full[stage]);
                } else {
                    mbar_arrive_expect_tx(&full[stage], S::stage);
                    const uint32_t dst = smem + stage * S::stage;
#pragma unroll
                    for (int x = 0; x < D / 64; ++x) {
                        tensor4d_g2s(dst + x * KB * 128, &p.k_map, 64 * x, key0, at.h, at.b,
                                     &full[stage]);
                        tensor4d_g2s(dst + S::operand + x * KB * 128, &p.v_map, 64 * x, key0, at.h,
                                     at.b, &full[stage]);
                    }
                }
            }
            __syncwarp();
            ++issued;
            if (++stage == S::stages) {
                stage = 0;
                parity ^= 1;
            }
        }
        if (least == kNone) break;
    }
    if (!ok) {      // a consumer gave up: see the copies in flight land before the CTA ends
        for (int i = 0; i < S::stages && i < issued; ++i) {
            const int last = issued - 1 - i;
            mbar_wait(&full[last % S::stages], (last / S::stages) & 1, p.err);
        }
    }
}

// Keys of a stage at or past the sequence's length may hold anything: zero their
// values (0 times what lies there might be NaN). Every consumer warp that uses
// the stage writes the same zeros before it reads.
template <int D, int KB>
__device__ __forceinline__ void zero_tail(uint32_t operand, int from) {
    const int lane = threadIdx.x & 31;
    for (int i = from * (D / 8) + lane; i < KB * (D / 8); i += 32)
        asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(
                         operand + panel_at<KB>(i / (D / 8), i % (D / 8))),
                     "r"(0)
                     : "memory");
    __syncwarp();
}

// A fragments (16 rows x D) of two strided rows per lane, straight from memory.
template <typename T, int D>
__device__ __forceinline__ void load_row_frags(uint32_t (&x)[D / 16][4], const T *r0, const T *r1,
                                               int c) {
#pragma unroll
    for (int i = 0; i < D / 16; ++i) {
        x[i][0] = r0 ? __ldg((const uint32_t *)(r0 + 16 * i + 2 * c)) : 0u;
        x[i][1] = r1 ? __ldg((const uint32_t *)(r1 + 16 * i + 2 * c)) : 0u;
        x[i][2] = r0 ? __ldg((const uint32_t *)(r0 + 16 * i + 8 + 2 * c)) : 0u;
        x[i][3] = r1 ? __ldg((const uint32_t *)(r1 + 16 * i + 8 + 2 * c)) : 0u;
    }
}

// ------------------------------------------------------------------- host
cudaError_t encode_rows(const spmm_rows &r, const spmm_blocks_shape *s, int box_rows,
                        CUtensorMap *map);

// Device word that a bounded wait which gave up sets (spmm_dynamic_sync reads it).
cudaError_t dynamic_err(int32_t **err);

}  // namespace spmm
