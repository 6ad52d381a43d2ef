// Shared by the selected-block attention kernels: the problem as they see it,
// fragments of the 16x8x16 matrix instruction, and the host's checks.
#pragma once

#include "dyn.cuh"
#include "tma.cuh"

namespace spmm {

// What a kernel needs of spmm_blocks_shape; strides in elements.
struct BlkArgs {
    int Tq, Tk, Hq, Hk, G, n, block, NB;
    int causal;
    float scale;
    const int32_t *lengths, *blocks;
    const void *q, *k, *v;
    int64_t q_sb, q_st, q_sh, k_sb, k_st, k_sh, v_sb, v_st, v_sh;
};

__device__ __forceinline__ int blk_len(const BlkArgs &a, int b) {
    return a.lengths ? min(max(a.lengths[b], 0), a.Tk) : a.Tk;
}

// Keys that query t of a sequence of `len` keys sees: [0, blk_limit).
__device__ __forceinline__ int blk_limit(const BlkArgs &a, int len, int t) {
    return a.causal ? max(len - a.Tq + t + 1, 0) : len;
}

// An entry of a list counts if it is in range and above the entry before it.
__device__ __forceinline__ bool blk_entry_ok(const int32_t *list, int j, int NB) {
    const int c = list[j];
    return (unsigned)c < (unsigned)NB && (j == 0 || c > list[j - 1]);
}

// D += A B on one warp: A 16x16 (row), B 16x8 (col), fp32 accumulators. With
// r = lane / 4 and c = lane % 4 a lane holds of A rows r, r + 8 and columns
// 2c, 2c+1, 2c+8, 2c+9; of B rows 2c, 2c+1 | 2c+8, 2c+9 of column r; of D
// columns 2c, 2c+1 of rows r and r + 8.
template <typename T>
__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
    if constexpr (std::is_same<T, __half>::value) {
        asm(
            "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
            "{%8,%9}, {%0,%1,%2,%3};\n"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    } else {
        asm(
            "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
            "{%8,%9}, {%0,%1,%2,%3};\n"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    }
}

template <typename T> __device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    if constexpr (std::is_same<T, __half>::value) {
        const __half2 h = __floats2half2_rn(lo, hi);
        return *reinterpret_cast<const uint32_t *>(&h);
    } else {
        const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
        return *reinterpret_cast<const uint32_t *>(&h);
    }
}

// Two values as the pair of their rounded parts and the pair of what that left out
// (itself rounded): together 16 bits and more of each.
template <typename T>
__device__ __forceinline__ void split2(float x, float y, uint32_t &hi, uint32_t &lo) {
    hi = pack2<T>(x, y);
    if constexpr (std::is_same<T, __half>::value) {
        const float2 r = __half22float2(*reinterpret_cast<const __half2 *>(&hi));
        lo = pack2<T>(x - r.x, y - r.y);
    } else {
        lo = pack2<T>(x - __uint_as_float(hi << 16), y - __uint_as_float(hi & 0xffff0000u));
    }
}

// Transpose of an 8x8 matrix of 16-bit elements held two adjacent ones per lane.
__device__ __forceinline__ uint32_t movmatrix(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;\n" : "=r"(y) : "r"(x));
    return y;
}

// Four 8x8 matrices from shared memory, lane l giving the address of row l % 8
// of matrix l / 8; `trans` hands each lane the transposed matrices' elements.
__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&x)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];\n"
                 : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3])
                 : "r"(addr));
}
__device__ __forceinline__ void ldsm4_t(uint32_t addr, uint32_t (&x)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];\n"
                 : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3])
                 : "r"(addr));
}

// 16 bytes global -> shared, asynchronously; zeros when !live (src is not read).
__device__ __forceinline__ void cp16(uint32_t dst, const void *src, bool live) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;\n" ::"r"(dst), "l"(src),
                 "r"(live ? 16 : 0));
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;\n"); }
template <int N> __device__ __forceinline__ void cp_wait() {
    asm volatile("cp.async.wait_group %0;\n" ::"n"(N));
}

// 2^x to about 2^-22 of itself, results below 2^-126 as 0: nothing next to the rounding
// that the weights get as operands (2^-8 of itself in bf16, 2^-11 in fp16).
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm volatile("ex2.approx.ftz.f32 %0, %1;\n" : "=f"(y) : "f"(x));
    return y;
}

// Whether the warp's elements are all NaN: no further term of a sum changes them.
template <int E> __device__ __forceinline__ bool all_nan(const float (&x)[E]) {
    bool y = true;
#pragma unroll
    for (int e = 0; e < E; ++e) y = y && isnan(x[e]);
    return __all_sync(0xffffffffu, y);
}

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// ------------------------------------------------------------------- host
inline bool rows_ok(const spmm_rows &r, int64_t e) {
    return r.data && (uintptr_t)r.data % 16 == 0 && r.sb * e % 16 == 0 && r.st * e % 16 == 0 &&
           r.sh * e % 16 == 0 && r.sb >= 0 && r.st >= 0 && r.sh >= 0;
}

// Everything but the tensors. `attend`: the limits of the matrix kernels too.
inline spmm_status blk_check(const spmm_blocks_shape *s, bool attend) {
    if (!s || s->B < 0 || s->Tq < 0 || s->Tk < 0 || s->Hq < 1 || s->Hk < 1 || s->D < 1 || s->n < 1)
        return SPMM_ERR_INVALID_ARG;
    if (!dtype_ok(s->dtype) || s->Hq % s->Hk) return SPMM_ERR_INVALID_ARG;
    if (s->block != 16 && s->block != 32 && s->block != 64 && s->block != 128)
        return SPMM_ERR_UNSUPPORTED;
    if (s->D % 8 || s->D > 256) return SPMM_ERR_UNSUPPORTED;
    if (attend && ((s->D != 64 && s->D != 128) || s->dtype == SPMM_F32)) return SPMM_ERR_UNSUPPORTED;
    // positions, lists and rows are indexed with 32 bits; offsets of elements with 64
    if (s->Tq > (1 << 26) || s->Tk > (1 << 26) || s->Hq > 65535 || s->n > (1 << 20) ||
        s->B > INT32_MAX)
        return SPMM_ERR_UNSUPPORTED;
    // (and sizes that are multiples of all keys' bytes stay far below 2^63)
    if (s->B * s->Hk > ((int64_t)1 << 40) / std::max<int64_t>(s->Tk, 1)) return SPMM_ERR_UNSUPPORTED;
    if (s->B && s->Hq * std::max<int64_t>(s->Tq, 1) > (int64_t)INT32_MAX / s->B)
        return SPMM_ERR_UNSUPPORTED;
    return SPMM_OK;
}

inline BlkArgs blk_args(const spmm_blocks_shape *s, const int32_t *blocks) {
    BlkArgs a{};
    a.Tq = (int)s->Tq;
    a.Tk = (int)s->Tk;
    a.Hq = (int)s->Hq;
    a.Hk = (int)s->Hk;
    a.G = (int)(s->Hq / s->Hk);
    a.n = (int)s->n;
    a.block = (int)s->block;
    a.NB = (int)((s->Tk + s->block - 1) / s->block);
    a.causal = s->causal ? 1 : 0;
    a.scale = s->scale;
    a.lengths = s->lengths;
    a.blocks = blocks;
    return a;
}

inline void set_rows(const void *&p, int64_t &sb, int64_t &st, int64_t &sh, const spmm_rows &r) {
    p = r.data;
    sb = r.sb;
    st = r.st;
    sh = r.sh;
}

// (Sequence, kv head) pairs that one launch takes in its y or z dimension; for more of
// them there are several launches.
constexpr int64_t kPairs = 65535;

inline int64_t round_up(int64_t x, int64_t m) { return (x + m - 1) / m * m; }

}  // namespace spmm
