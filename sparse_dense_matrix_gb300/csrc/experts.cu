// Products grouped by expert: the slots of expert e, rows offsets[e] .. offsets[e + 1]
// of xs [P, H], times w[e] [H, F], and the gradient of w:
//   ys[s, f] = sum_h xs[s, h] w[e, h, f],   dw[e, h, f] = sum_s xs[s, h] dys[s, f].
// The simplest form: 64 x 64 outputs a CTA, 4 x 4 a thread, operands in shared memory
// as fp32.
#include "blocks.cuh"

namespace spmm {
namespace {

constexpr int kTile = 64, kDepth = 16, kThreads = 256;

struct ExpertArgs {
    const void *a, *b;               // xs and w, or xs and dys
    void *out;
    const int32_t *offsets;
    int64_t se, sh, sf;              // strides of w or dw
    int64_t P;
    int E, H, F;
};

struct Segment {
    int64_t begin, end;
};
__device__ __forceinline__ Segment segment(const ExpertArgs &p, int e) {
    Segment s;
    s.begin = min(max((int64_t)p.offsets[e], (int64_t)0), p.P);
    s.end = min(max((int64_t)p.offsets[e + 1], s.begin), p.P);
    return s;
}

// c[4][4] += the tile's product over `n` of the summed index; at(i, j) and bt(i, j) give
// the elements (summed index, row) and (summed index, column).
template <typename FA, typename FB>
__device__ __forceinline__ void tile_product(float (&c)[4][4], int64_t n, FA at, FB bt) {
    __shared__ float sa[kDepth][kTile + 4], sb[kDepth][kTile + 4];
    const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;
    for (int64_t k0 = 0; k0 < n; k0 += kDepth) {
        for (int i = threadIdx.x; i < kDepth * kTile; i += kThreads) {
            const int64_t k = k0 + i / kTile;
            sa[i / kTile][i % kTile] = k < n ? at(k, i % kTile) : 0.0f;
            sb[i / kTile][i % kTile] = k < n ? bt(k, i % kTile) : 0.0f;
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < kDepth; ++k)
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    c[i][j] = fmaf(sa[k][ty * 4 + i], sb[k][tx * 4 + j], c[i][j]);
        __syncthreads();
    }
}

// CTA y takes the y-th tile of 64 slots of the experts in turn, then of the rows behind.
template <typename T> __global__ void __launch_bounds__(kThreads) k_product(const ExpertArgs p) {
    __shared__ int which;
    __shared__ int64_t first;
    if (threadIdx.x == 0) {
        int64_t left = blockIdx.y;
        int e = 0;
        for (; e < p.E; ++e) {
            const Segment s = segment(p, e);
            const int64_t tiles = (s.end - s.begin + kTile - 1) / kTile;
            if (left < tiles) break;
            left -= tiles;
        }
        which = e;
        first = (e < p.E ? segment(p, e).begin : min(max((int64_t)p.offsets[p.E], (int64_t)0), p.P)) +
                left * kTile;
    }
    __syncthreads();
    const int e = which;
    const int64_t r0 = first, r1 = min(e < p.E ? segment(p, e).end : p.P, r0 + kTile);
    const int f0 = blockIdx.x * kTile;
    if (r0 >= r1) return;
    const T *xs = (const T *)p.a, *w = (const T *)p.b + e * p.se;
    float c[4][4] = {};
    if (e < p.E)
        tile_product(
            c, p.H,
            [&](int64_t k, int i) { return r0 + i < r1 ? to_f32(xs[(r0 + i) * p.H + k]) : 0.0f; },
            [&](int64_t k, int j) {
                return f0 + j < p.F ? to_f32(w[k * p.sh + (f0 + j) * p.sf]) : 0.0f;
            });
    const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;
    for (int i = 0; i < 4; ++i)
        for (int j = 0; j < 4; ++j) {
            const int64_t r = r0 + ty * 4 + i;
            const int f = f0 + tx * 4 + j;
            if (r < r1 && f < p.F) ((T *)p.out)[r * p.F + f] = from_f32<T>(c[i][j]);
        }
}

template <typename T> __global__ void __launch_bounds__(kThreads) k_weights(const ExpertArgs p) {
    const int e = blockIdx.z;
    const Segment s = segment(p, e);
    const int h0 = blockIdx.y * kTile, f0 = blockIdx.x * kTile;
    const T *xs = (const T *)p.a + s.begin * p.H, *dys = (const T *)p.b + s.begin * p.F;
    float c[4][4] = {};
    tile_product(
        c, s.end - s.begin,
        [&](int64_t k, int i) { return h0 + i < p.H ? to_f32(xs[k * p.H + h0 + i]) : 0.0f; },
        [&](int64_t k, int j) { return f0 + j < p.F ? to_f32(dys[k * p.F + f0 + j]) : 0.0f; });
    const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;
    for (int i = 0; i < 4; ++i)
        for (int j = 0; j < 4; ++j) {
            const int h = h0 + ty * 4 + i, f = f0 + tx * 4 + j;
            if (h < p.H && f < p.F)
                ((T *)p.out)[e * p.se + h * p.sh + f * p.sf] = from_f32<T>(c[i][j]);
        }
}

// ------------------------------------------------------------------- host
bool aligned(const void *p) { return p && (uintptr_t)p % 16 == 0; }

spmm_status check_sizes(int dtype, const int32_t *offsets, int64_t P, int64_t E, int64_t H,
                        int64_t F) {
    if (!dtype_ok(dtype) || !offsets || P < 0 || E < 0 || H < 0 || F < 0)
        return SPMM_ERR_INVALID_ARG;
    if (dtype == SPMM_F32 || H % 8 || F % 8 || H > (1 << 20) || F > (1 << 20) ||
        E > SPMM_ROUTES_MAX_EXPERTS || P > INT32_MAX)
        return SPMM_ERR_UNSUPPORTED;
    return SPMM_OK;
}

// Strides of [E, H, F] matrices, one of the last two adjacent.
bool strides_ok(int64_t se, int64_t sh, int64_t sf) {
    if (se < 0 || se % 8) return false;
    return (sf == 1 && sh > 0 && sh % 8 == 0) || (sh == 1 && sf > 0 && sf % 8 == 0);
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
    if (!aligned(ys) || (H && (!aligned(xs) || (E && (!aligned(w) || !strides_ok(w_se, w_sh, w_sf))))))
        return SPMM_ERR_INVALID_ARG;
    const ExpertArgs p{xs, w, ys, offsets, w_se, w_sh, w_sf, P, (int)E, (int)H, (int)F};
    const dim3 grid((unsigned)((F + kTile - 1) / kTile), (unsigned)(P / kTile + E + 1));
    if (dtype == SPMM_BF16)
        k_product<__nv_bfloat16><<<grid, kThreads, 0, (cudaStream_t)stream>>>(p);
    else
        k_product<__half><<<grid, kThreads, 0, (cudaStream_t)stream>>>(p);
    count_launch();
    return cuda_status(cudaGetLastError());
}

spmm_status spmm_routes_product_weights(int dtype, const void *xs, const void *dys,
                                        const int32_t *offsets, int64_t P, int64_t E, int64_t H,
                                        int64_t F, void *dw, int64_t dw_se, int64_t dw_sh,
                                        int64_t dw_sf, void *stream) {
    using namespace spmm;
    const spmm_status st = check_sizes(dtype, offsets, P, E, H, F);
    if (st != SPMM_OK) return st;
    if (E == 0 || H == 0 || F == 0) return SPMM_OK;
    if (!aligned(dw) || !strides_ok(dw_se, dw_sh, dw_sf) || (E > 1 && dw_se == 0))
        return SPMM_ERR_INVALID_ARG;
    if (P && (!aligned(xs) || !aligned(dys))) return SPMM_ERR_INVALID_ARG;
    const ExpertArgs p{xs, dys, dw, offsets, dw_se, dw_sh, dw_sf, P, (int)E, (int)H, (int)F};
    const dim3 grid((unsigned)((F + kTile - 1) / kTile), (unsigned)((H + kTile - 1) / kTile),
                    (unsigned)E);
    if (dtype == SPMM_BF16)
        k_weights<__nv_bfloat16><<<grid, kThreads, 0, (cudaStream_t)stream>>>(p);
    else
        k_weights<__half><<<grid, kThreads, 0, (cudaStream_t)stream>>>(p);
    count_launch();
    return cuda_status(cudaGetLastError());
}

}  // extern "C"
