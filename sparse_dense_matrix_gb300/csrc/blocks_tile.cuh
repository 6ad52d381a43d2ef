// Selected-block attention by tile of rows: 16 W adjacent (query, head) rows
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

template <int W> struct TileStage {
    int key0;                                      // first key, or -1: no more blocks
    uint32_t mask[(W + 1) / 2];                    // bit of each query of the tile
};

// Shared memory: `stages` of K then V, KB keys each, as D / 64 panels of KB rows
// of 128 bytes, the 16-byte chunks of a row permuted by the copy's 128-byte
// swizzle; then `tiles` operands of 16 W rows. `budget` bytes in all.
template <int D, int KB, int W, int tiles, int budget> struct TileSmem {
    static constexpr int operand = KB * D * 2;
    static constexpr int stage = 2 * operand;
    static constexpr int rows = 16 * W * D * 2;    // one operand of the tile's own rows
    // the lists of the tile's queries, when they fit: 16 entries for each of 16 W
    static constexpr int lists = 16 * W * 16 * 4;
    static constexpr int fit = (budget - 1024 /* alignment */ - lists - tiles * rows) / stage;
    static constexpr int stages = fit > 16 ? 16 : fit;
    static constexpr int at_rows = stages * stage, at_lists = at_rows + tiles * rows;
    static constexpr int bytes = at_lists + lists + 1024;
    static_assert(stages >= 2, "the ring needs two stages");
};

// 16-byte chunk `chunk` of row `row` of a [rows][D] operand that threads fill:
// eight consecutive rows' chunks fall in different banks.
template <int D> __device__ __forceinline__ uint32_t rows_at(int row, int chunk) {
    return (uint32_t)(row * D * 2 + ((chunk ^ (row & 7)) << 4));
}

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
    int tiles;               // of rows per kv head
    int32_t *err;
};

// Which rows a CTA owns. Later tiles see more keys: they are started first.
struct TilePlace {
    int b, h;
    int64_t f0;              // first row, f = t G + g
    int t_first, nq;         // the tile's queries
    __device__ __forceinline__ TilePlace(const TileArgs &p, int tile_rows) {
        const int hb = blockIdx.y;
        h = hb % p.a.Hk;
        b = hb / p.a.Hk;
        f0 = (int64_t)(p.tiles - 1 - (int)blockIdx.x) * tile_rows;
        const int64_t f1 = min(p.rows, f0 + tile_rows) - 1;
        t_first = (int)(f0 / p.a.G);
        nq = (int)(f1 / p.a.G) - t_first + 1;
    }
    // Row `i` of the tile as a row of [B, Tq, Hq]; whether it sees any key.
    __device__ __forceinline__ int64_t out_row(const TileArgs &p, int64_t f) const {
        return (int64_t)b * p.a.Tq * p.a.Hq + f / p.a.G * p.a.Hq + h * p.a.G + f % p.a.G;
    }
    __device__ __forceinline__ bool row_of(const TileArgs &p, int len, int i, int64_t &f) const {
        f = f0 + i;
        return f < p.rows && blk_limit(p.a, len, (int)(f / p.a.G)) > 0;
    }
    // Element offset of that row in a strided [B, Tq, Hq, D] tensor.
    __device__ __forceinline__ int64_t offset(const TileArgs &p, int64_t f, int64_t sb, int64_t st,
                                              int64_t sh) const {
        return b * sb + f / p.a.G * st + (h * p.a.G + f % p.a.G) * sh;
    }
};

// The merge of a tile's lists, by one warp: step() gives the next block of the
// union (kNone after the last) and the bits of the queries that chose it. All
// lists are ascending, so that is the smallest of their heads. The lists go to
// shared memory first where they fit: a step then waits for no load from global
// memory (about 700 cycles, more than a step's arithmetic).
template <int W> struct TileMerge {
    static constexpr int kLists = (W + 1) / 2;     // lists per lane, words of bits
    static constexpr int kNone = INT_MAX;
    const int32_t *list[kLists];                   // the next entry
    int left[kLists], head[kLists], prev[kLists];
    int end[kLists];                               // first block out of sight
    int nq, NB;
    uint32_t mask[kLists];

    __device__ __forceinline__ void advance(int i) {
        // entries below the one before them or out of range are skipped
        int c = kNone;
        while (left[i] > 0) {
            --left[i];
            const int x = *list[i]++;
            const bool ok = (unsigned)x < (unsigned)NB && x > prev[i];
            prev[i] = x;
            if (ok) {
                c = x < end[i] ? x : kNone;
                break;
            }
        }
        head[i] = c;
    }

    __device__ __forceinline__ TileMerge(const TileArgs &p, const TilePlace &at, int32_t *lists,
                                         int lists_bytes) {
        const BlkArgs &a = p.a;
        const int lane = threadIdx.x & 31, len = blk_len(a, at.b);
        nq = at.nq;
        NB = a.NB;
        const int32_t *base =
            a.blocks + (((int64_t)at.b * a.Tq + at.t_first) * a.Hk + at.h) * a.n;
        const int64_t pitch = (int64_t)a.Hk * a.n;
        const bool staged = (int64_t)nq * a.n * 4 <= lists_bytes;
        if (staged) {
            for (int q = lane; q < nq; q += 32) {
#pragma unroll 8
                for (int j = 0; j < a.n; ++j) lists[q * a.n + j] = base[q * pitch + j];
            }
            __syncwarp();
        }
#pragma unroll
        for (int i = 0; i < kLists; ++i) {
            const int q = i * 32 + lane;
            left[i] = end[i] = 0;
            head[i] = kNone;
            prev[i] = -1;
            list[i] = lists;
            if (q < nq) {
                list[i] = staged ? lists + q * a.n : base + q * pitch;
                left[i] = a.n;
                end[i] = (blk_limit(a, len, at.t_first + q) + a.block - 1) / a.block;
                advance(i);
            }
        }
    }

    __device__ __forceinline__ int step() {
        int least = head[0];
#pragma unroll
        for (int i = 1; i < kLists; ++i)
            if (32 * i < nq) least = min(least, head[i]);
        least = __reduce_min_sync(0xffffffffu, least);
#pragma unroll
        for (int i = 0; i < kLists; ++i) {
            mask[i] = 0;
            if (32 * i >= nq) continue;            // usually all but the first 32 queries
            const bool mine = least != kNone && head[i] == least;
            mask[i] = __ballot_sync(0xffffffffu, mine);
            if (mine) advance(i);
        }
        return least;
    }
};

template <typename S, int D, int KB, int W>
__device__ __forceinline__ void tile_produce(const TileArgs &p, const TilePlace &at,
                                             uint32_t smem, uint64_t *full, uint64_t *empty,
                                             TileStage<W> *info, int32_t *lists) {
    const BlkArgs &a = p.a;
    const int lane = threadIdx.x & 31, len = blk_len(a, at.b);
    TileMerge<W> merge(p, at, lists, S::lists);
    int stage = 0, issued = 0;
    uint32_t parity = 1;                           // the ring starts empty
    bool ok = true;
    while (ok) {
        const int least = merge.step();
        const bool last = least == merge.kNone;
        const int parts = last ? 1 : a.block / KB;
        for (int s = 0; s < parts; ++s) {
            const int key0 = last ? -1 : least * a.block + s * KB;
            if (key0 >= len) break;    // nobody sees the second half of a last, short block
            ok = mbar_wait(&empty[stage], parity, p.err);
            if (!ok) break;
            if (lane == 0) {
                info[stage].key0 = key0;
#pragma unroll
                for (int i = 0; i < merge.kLists; ++i) info[stage].mask[i] = merge.mask[i];
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
        if (last) break;
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

// The same by one thread, for the threads that issue the products.
template <int D, int KB> __device__ __forceinline__ void zero_tail_one(uint32_t operand, int from) {
    for (int i = max(from, 0) * (D / 8); i < KB * (D / 8); ++i)
        asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(
                         operand + panel_at<KB>(i / (D / 8), i % (D / 8))),
                     "r"(0)
                     : "memory");
}

// One warp's 16 rows of a strided tensor into its part of shared memory: lanes
// 0 to 15 say of rows 0 to 15 where they start; a row that is not live is 0.
template <typename T, int D>
__device__ __forceinline__ void fetch_rows(uint32_t dst, const T *p, bool live, int64_t offset) {
    const int lane = threadIdx.x & 31;
    const int64_t mine = live ? offset : -1;
#pragma unroll
    for (int i = 0; i < D / 16; ++i) {             // 32 chunks at a time
        const int row = i * 32 / (D / 8) + lane / (D / 8), chunk = lane % (D / 8);
        const int64_t at = __shfl_sync(0xffffffffu, mine, row);
        cp16(dst + rows_at<D>(row, chunk), p + (at < 0 ? 0 : at + chunk * 8), at >= 0);
    }
    cp_commit();
}

// ------------------------------------------------------------------- host
cudaError_t encode_rows(const spmm_rows &r, const spmm_blocks_shape *s, int box_rows,
                        CUtensorMap *map);

// By query or by tile: the smaller of two estimates, in microseconds.
// By query, a list costs 12 ns and 0.31 ns per 1000 elements of its keys (on all
// SMs together). By tile, a CTA walks the union of its queries' lists, of which
// neighbours share what they share, at worst all blocks, at 1 us a step, two CTAs
// to an SM. Either takes some 8 us around that. Measured with lists that share
// nothing, by query against by tile: 16 queries x 8 heads x 4 over a cache of
// 8192 keys (16 of 64-key blocks, heads of 128) 17 and 112 us, 256 of them 93 and
// 116; 4 x 777 queries, one head each, 7 of 32-key blocks 190 and 27; 3 x 333
// queries x 3 heads 71 and 41; 2048 queries x 4 heads x 8, 16 of 32-key blocks
// 622 and 133.
constexpr int kTileRows = 128;       // of the tensor-memory kernels; the others' are 64

inline bool blocks_by_tile(const spmm_blocks_shape *s, const spmm_rows &k, const spmm_rows &v) {
    if (s->Tk == 0 || s->B * s->Hk > 65535) return false;
    // a tensor map steps forward, by less than 2^40 bytes: a row shared by several
    // keys, heads or sequences (stride 0) goes by query
    auto mapped = [&](int64_t n, int64_t stride) {
        return n <= 1 || (stride > 0 && stride < ((int64_t)1 << 39));
    };
    for (const spmm_rows &r : {k, v})
        if (!mapped(s->Tk, r.st) || !mapped(s->Hk, r.sh) || !mapped(s->B, r.sb)) return false;
    const int64_t G = s->Hq / s->Hk, parts = s->block > 64 ? s->block / 64 : 1;
    const int64_t NB = (s->Tk + s->block - 1) / s->block;
    const int64_t tiles = s->B * s->Hk * ((s->Tq * G + kTileRows - 1) / kTileRows);
    const int64_t queries = std::min<int64_t>(s->Tq, (kTileRows + G - 1) / G + 1);
    const int64_t steps = parts * std::min<int64_t>(NB, queries * std::min<int64_t>(s->n, NB));
    const double tile_us = (double)steps * (double)((tiles + 303) / 304);
    const double lists = (double)s->B * s->Tq * s->Hk * ((G + 15) / 16);
    const double keys = (double)std::min<int64_t>(s->n * s->block, s->Tk);
    return tile_us < lists * (0.012 + keys * s->D * 0.31e-6);
}

}  // namespace spmm
