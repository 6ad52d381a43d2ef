// Expert routes: the tokens x slots matrix that a router picks anew in every
// call. ids[t, j] names the expert of token t's j-th choice; the kept pairs
// (t, j), in order of (expert, t, j), get the slots 0, 1, 2, ... With s the
// slot of (t, j), w its weight and R the matrix with R[t, s] = w:
//   dispatch            xs[s] = x[t]                 (pattern of R^T times x)
//   combine             out[t] = sum_j w y[s]        (R y)
//   combine_backward    dy[s] = w dout[t], dw[t, j] = <dout[t], y[s]>
//   dispatch_backward   dx[t] = sum_j dxs[s]         (pattern of R times dxs)
// Each product is walked by token: a token's row of R is its k slots, so every
// row of x, dout and out moves once, every slot's row once, and nothing is
// accumulated across threads that own different tokens (no atomics).
#include "dyn.cuh"

namespace spmm {
namespace {

// ------------------------------------------------------------------ sort
// A stable counting sort of the P = T k pairs by expert. The pairs are cut into
// tiles, a tile into one contiguous run per warp, so a pair's slot is
//   offsets[e] + pairs of e in earlier tiles + in earlier warps' runs
//              + among the earlier pairs of the warp's own run,
// all exact integers: the last by __match_any_sync 32 pairs at a time, the
// third from a [warp][expert] table in shared memory, the first two from the
// tiles' histograms. With one tile they are in the same table and a single
// launch does it all (P <= 8192, the range where a second launch costs more
// than the idle SMs do). Bound by latency: 4 us for 32 pairs, 15 us in two launches
// for 131072 pairs of 128 experts, next to the products' 370 us.
constexpr int kSortThreads = 512;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int64_t kSortOneTile = 8192;
constexpr int64_t kSortTile = 2048;
constexpr int kSortMaxTiles = 512;

__device__ __forceinline__ bool kept(int id, int E) { return (unsigned)id < (unsigned)E; }

__global__ void __launch_bounds__(kSortThreads) k_route_hist(const int32_t *__restrict__ ids,
                                                            int64_t P, int E, int64_t tile,
                                                            int32_t *__restrict__ hist) {
    extern __shared__ int32_t count[];
    for (int e = threadIdx.x; e < E; e += kSortThreads) count[e] = 0;
    __syncthreads();
    const int64_t p0 = blockIdx.x * tile, p1 = min(P, p0 + tile);
    for (int64_t p = p0 + threadIdx.x; p < p1; p += kSortThreads) {
        const int id = ids[p];
        if (kept(id, E)) atomicAdd(&count[id], 1);   // integer count: order-independent
    }
    __syncthreads();
    for (int e = threadIdx.x; e < E; e += kSortThreads) hist[(int64_t)blockIdx.x * E + e] = count[e];
}

__global__ void __launch_bounds__(kSortThreads) k_route_sort(
    const int32_t *__restrict__ ids, int64_t P, int E, int64_t tile, int tiles,
    const int32_t *__restrict__ hist, int32_t *__restrict__ slots, int32_t *__restrict__ offsets) {
    extern __shared__ int32_t sh[];
    int32_t *run = sh;                       // [kSortWarps][E]: next slot of (warp, expert)
    int32_t *total = sh + kSortWarps * E;    // [E + 1]: pairs per expert, then its first slot
    __shared__ int32_t scan_warp[kSortWarps];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int64_t p0 = blockIdx.x * tile, p1 = min(P, p0 + tile);
    const int64_t per = ((tile + kSortWarps - 1) / kSortWarps + 31) / 32 * 32;
    const int64_t q0 = min(p1, p0 + warp * per), q1 = min(p1, q0 + per);
    int32_t *mine = run + warp * E;

    for (int e = tid; e < kSortWarps * E; e += kSortThreads) run[e] = 0;
    __syncthreads();
    for (int64_t p = q0 + lane; p < q1; p += 32) {
        const int id = ids[p];
        if (kept(id, E)) atomicAdd(&mine[id], 1);
    }
    __syncthreads();
    // per expert: pairs before this tile, and in all tiles
    for (int e = tid; e < E; e += kSortThreads) {
        int before = 0, all = 0;
        if (tiles > 1) {
            for (int b = 0; b < tiles; ++b) {
                const int c = hist[(int64_t)b * E + e];
                if (b < (int)blockIdx.x) before += c;
                all += c;
            }
        }
        for (int w = 0; w < kSortWarps; ++w) {
            const int c = run[w * E + e];
            run[w * E + e] = before;
            before += c;
        }
        total[e] = tiles > 1 ? all : before;
    }
    __syncthreads();
    // exclusive scan of total over the experts, kSortThreads at a time
    int carry = 0;
    for (int e0 = 0; e0 < E; e0 += kSortThreads) {
        const int e = e0 + tid;
        const int v = e < E ? total[e] : 0;
        int x = v;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, x, o);
            if (lane >= o) x += y;
        }
        if (lane == 31) scan_warp[warp] = x;
        __syncthreads();
        int below = 0, sum = 0;
        for (int w = 0; w < kSortWarps; ++w) {
            const int c = scan_warp[w];
            if (w < warp) below += c;
            sum += c;
        }
        if (e < E) total[e] = carry + below + x - v;
        carry += sum;
        __syncthreads();
    }
    if (blockIdx.x == 0) {
        for (int e = tid; e < E; e += kSortThreads) offsets[e] = total[e];
        if (tid == 0) offsets[E] = carry;
    }
    for (int64_t base = q0; base < q1; base += 32) {
        const int64_t p = base + lane;
        const int id = p < q1 ? ids[p] : -1;
        const bool k = kept(id, E);
        const unsigned same = __match_any_sync(0xffffffffu, k ? id : -1);
        const int before = __popc(same & ((1u << lane) - 1u));
        int slot = -1;
        if (k) slot = total[id] + mine[id] + before;
        __syncwarp();
        if (k && before == 0) mine[id] += __popc(same);
        __syncwarp();
        if (p < q1) slots[p] = slot;
    }
}

// ------------------------------------------------------------ row products
// blockDim.x threads share a token's row, V elements per access; blockDim.y
// tokens per CTA. Rows of slots past the last kept pair hold nothing and are
// set to 0: row r by the CTA of token r / k, so no further launch is needed.
// All of them are bound by memory; bytes over time in bf16: dispatch 16384 tokens x
// 8 x 4096 178 us, 6.8 TB/s (all that a copy reaches); combine the same 193 us, 6.3
// TB/s; combine's gradient 8192 x 8 x 2048 100 us, 5.7 TB/s.
struct RouteArgs {
    const int32_t *slots;    // [T, k]
    const int32_t *n_kept;   // offsets + E
    const float *w;          // [T, k] or NULL (all 1)
    int64_t T, H;
    int64_t ldx;             // elements between rows of the per-token input
    int k;
};

template <typename U>
__global__ void __launch_bounds__(256) k_dispatch(RouteArgs a, const U *__restrict__ x,
                                                 U *__restrict__ xs) {
    const int64_t t = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
    if (t >= a.T) return;
    const int32_t *slots = a.slots + t * a.k;
    const int64_t n_kept = *a.n_kept;
    for (int64_t c = threadIdx.x; c < a.H; c += blockDim.x) {
        const U v = x[t * a.ldx + c];
        for (int j = 0; j < a.k; ++j) {
            const int s = slots[j];
            if (s >= 0) xs[(int64_t)s * a.H + c] = v;
        }
        for (int64_t r = max(n_kept, t * a.k); r < (t + 1) * a.k; ++r) xs[r * a.H + c] = U{};
    }
}

template <typename T, int V>
__global__ void __launch_bounds__(256) k_combine(RouteArgs a, const T *__restrict__ y,
                                                T *__restrict__ out) {
    const int64_t t = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
    if (t >= a.T) return;
    const int32_t *slots = a.slots + t * a.k;
    const float *w = a.w ? a.w + t * a.k : nullptr;
    for (int64_t c = (int64_t)threadIdx.x * V; c < a.H; c += (int64_t)blockDim.x * V) {
        float acc[V];
#pragma unroll
        for (int i = 0; i < V; ++i) acc[i] = 0.0f;
        for (int j = 0; j < a.k; ++j) {
            const int s = slots[j];
            if (s < 0) continue;      // a dropped pair is skipped, not multiplied by 0
            float v[V];
            ld_pack<T, V>(y + (int64_t)s * a.H + c, v);
            const float wj = w ? w[j] : 1.0f;
#pragma unroll
            for (int i = 0; i < V; ++i) acc[i] = fmaf(wj, v[i], acc[i]);
        }
        st_pack<T, V>(out + t * a.H + c, acc);
    }
}

// The dot products of a token's choices meet in shared memory once per kGroup of
// them: one pair of barriers each, not one per choice (122 us at 8192 tokens x 8
// x 2048 in bf16; holding eight rows of y in registers at once instead costs the
// occupancy that hides the loads, 171 us).
constexpr int kGroup = 64;

template <typename T, int V>
__global__ void __launch_bounds__(256) k_combine_bwd(RouteArgs a, const T *__restrict__ dout,
                                                    const T *__restrict__ y, T *__restrict__ dy,
                                                    float *__restrict__ dw) {
    __shared__ float part[kGroup][8];            // [choice][warp]
    const int64_t t = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
    const int lanes = blockDim.x, warp = (threadIdx.y * lanes + threadIdx.x) >> 5;
    const bool live = t < a.T;
    const int32_t *slots = a.slots + t * a.k;
    for (int j0 = 0; j0 < a.k; j0 += kGroup) {
        const int j1 = min(a.k, j0 + kGroup);
        for (int j = j0; j < j1 && live; ++j) {
            const int s = slots[j];
            float dot = 0.0f;
            if (s >= 0) {
                const float wj = a.w ? a.w[t * a.k + j] : 1.0f;
                for (int64_t c = (int64_t)threadIdx.x * V; c < a.H; c += (int64_t)lanes * V) {
                    float d[V], v[V];
                    ld_pack<T, V>(dout + t * a.ldx + c, d);
                    ld_pack<T, V>(y + (int64_t)s * a.H + c, v);
#pragma unroll
                    for (int i = 0; i < V; ++i) {
                        dot = fmaf(d[i], v[i], dot);
                        d[i] *= wj;
                    }
                    st_pack<T, V>(dy + (int64_t)s * a.H + c, d);
                }
            }
            if (dw) {
#pragma unroll
                for (int o = 16; o; o >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, o);
                if ((threadIdx.x & 31) == 0) part[j - j0][warp] = dot;
            }
        }
        if (dw) {
            __syncthreads();
            const int per = lanes / 32, first = threadIdx.y * per;
            for (int j = j0 + threadIdx.x; j < j1 && live; j += lanes) {
                float sum = 0.0f;
                for (int i = 0; i < per; ++i) sum += part[j - j0][first + i];
                dw[t * a.k + j] = sum;
            }
            __syncthreads();
        }
    }
    if (!live) return;
    const int64_t n_kept = *a.n_kept;
    const float zero[V] = {};
    for (int64_t r = max(n_kept, t * a.k); r < (t + 1) * a.k; ++r)
        for (int64_t c = (int64_t)threadIdx.x * V; c < a.H; c += (int64_t)lanes * V)
            st_pack<T, V>(dy + r * a.H + c, zero);
}

// ------------------------------------------------------------------- host
// threads per token: enough for one access each, 32 to 256
dim3 row_block(int64_t accesses) {
    int x = 32;
    while (x < 256 && x < accesses) x <<= 1;
    return dim3((unsigned)x, (unsigned)(256 / x));
}

unsigned row_grid(int64_t T, const dim3 &b) { return (unsigned)((T + b.y - 1) / b.y); }

bool wide_ok(int dtype, int64_t H, int64_t ldx, std::initializer_list<const void *> ptrs) {
    const int e = dtype_bytes(dtype);
    if (H * e % 16 || ldx * e % 16) return false;
    for (const void *p : ptrs)
        if ((uintptr_t)p % 16) return false;
    return true;
}

spmm_status check_rows(int dtype, const int32_t *slots, const int32_t *offsets, int64_t T,
                       int64_t k, int64_t E, int64_t H, int64_t ldx) {
    if (!dtype_ok(dtype) || T < 0 || k < 0 || E < 0 || H < 0) return SPMM_ERR_INVALID_ARG;
    if (T == 0 || k == 0) return SPMM_OK;
    if (!slots || !offsets) return SPMM_ERR_INVALID_ARG;
    if (ldx < 0) return SPMM_ERR_INVALID_ARG;
    if (T > INT32_MAX / k || H >= INT32_MAX / 4 || E > SPMM_ROUTES_MAX_EXPERTS)
        return SPMM_ERR_UNSUPPORTED;
    return SPMM_OK;
}

template <typename F> void by_type(int dtype, F f) {
    if (dtype == SPMM_F32) f(float{}, std::integral_constant<int, 4>{});
    else if (dtype == SPMM_BF16) f(__nv_bfloat16{}, std::integral_constant<int, 8>{});
    else f(__half{}, std::integral_constant<int, 8>{});
}

cudaError_t launch_combine(int dtype, const RouteArgs &a, const void *y, void *out,
                           cudaStream_t s) {
    const bool wide = wide_ok(dtype, a.H, 0, {y, out});
    by_type(dtype, [&](auto t, auto v) {
        using T = decltype(t);
        constexpr int V = decltype(v)::value;
        const dim3 b = row_block(wide ? a.H / V : a.H);
        if (wide) k_combine<T, V><<<row_grid(a.T, b), b, 0, s>>>(a, (const T *)y, (T *)out);
        else k_combine<T, 1><<<row_grid(a.T, b), b, 0, s>>>(a, (const T *)y, (T *)out);
    });
    count_launch();
    return cudaGetLastError();
}

int64_t sort_tiles(int64_t P) {
    if (P <= kSortOneTile) return 1;
    return std::min<int64_t>(kSortMaxTiles, (P + kSortTile - 1) / kSortTile);
}

// the warps' counters and the experts' first slots
size_t sort_smem(int64_t E) { return sizeof(int32_t) * (size_t)(kSortWarps * E + E + 1); }

}  // namespace
}  // namespace spmm

extern "C" {

int64_t spmm_routes_workspace(int64_t T, int64_t k, int64_t E) {
    using namespace spmm;
    if (T <= 0 || k <= 0 || E <= 0 || T > INT32_MAX / k || E > SPMM_ROUTES_MAX_EXPERTS) return 0;
    const int64_t tiles = sort_tiles(T * k);
    return tiles > 1 ? tiles * E * (int64_t)sizeof(int32_t) : 0;
}

spmm_status spmm_routes_sort(const int32_t *ids, int64_t T, int64_t k, int64_t E, int32_t *slots,
                             int32_t *offsets, void *work, int64_t work_bytes, void *stream) {
    using namespace spmm;
    if (T < 0 || k < 0 || E < 0 || !offsets) return SPMM_ERR_INVALID_ARG;
    if (E > SPMM_ROUTES_MAX_EXPERTS) return SPMM_ERR_UNSUPPORTED;
    const int64_t P = k && T > INT32_MAX / k ? -1 : T * k;
    if (P < 0) return SPMM_ERR_UNSUPPORTED;
    if (P > 0 && (!ids || !slots)) return SPMM_ERR_INVALID_ARG;
    const int64_t need = spmm_routes_workspace(T, k, E);
    if (need && (!work || work_bytes < need)) return SPMM_ERR_INVALID_ARG;
    cudaStream_t s = (cudaStream_t)stream;
    const int64_t tiles = sort_tiles(P);
    const int64_t tile = (P + tiles - 1) / tiles;
    cudaError_t e = cudaSuccess;
    if (tiles > 1) {
        k_route_hist<<<(unsigned)tiles, kSortThreads, sizeof(int32_t) * (size_t)E, s>>>(
            ids, P, (int)E, tile, (int32_t *)work);
        count_launch();
        e = cudaGetLastError();
        if (e != cudaSuccess) return cuda_status(e);
    }
    const size_t smem = sort_smem(E);
    if (smem > 48 * 1024) {
        // the kernel's limit is the process's: always the largest, so that another
        // thread's call cannot lower it between here and the launch
        e = cudaFuncSetAttribute(k_route_sort, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 (int)sort_smem(SPMM_ROUTES_MAX_EXPERTS));
        if (e != cudaSuccess) return cuda_status(e);
    }
    k_route_sort<<<(unsigned)tiles, kSortThreads, smem, s>>>(ids, P, (int)E, tile, (int)tiles,
                                                            (const int32_t *)work, slots, offsets);
    count_launch();
    return cuda_status(cudaGetLastError());
}

spmm_status spmm_routes_dispatch(int dtype, const void *x, int64_t ldx, const int32_t *slots,
                                 const int32_t *offsets, int64_t T, int64_t k, int64_t E,
                                 int64_t H, void *xs, void *stream) {
    using namespace spmm;
    const spmm_status st = check_rows(dtype, slots, offsets, T, k, E, H, ldx);
    if (st != SPMM_OK) return st;
    if (T == 0 || k == 0 || H == 0) return SPMM_OK;
    if (!x || !xs) return SPMM_ERR_INVALID_ARG;
    cudaStream_t s = (cudaStream_t)stream;
    RouteArgs a{slots, offsets + E, nullptr, T, H, ldx, (int)k};
    const int e = dtype_bytes(dtype);
    if (wide_ok(dtype, H, ldx, {x, xs})) {     // a copy: the type does not matter
        a.H = H * e / 16;
        a.ldx = ldx * e / 16;
        const dim3 b = row_block(a.H);
        k_dispatch<uint4><<<row_grid(T, b), b, 0, s>>>(a, (const uint4 *)x, (uint4 *)xs);
    } else if (e == 4) {
        const dim3 b = row_block(H);
        k_dispatch<uint32_t><<<row_grid(T, b), b, 0, s>>>(a, (const uint32_t *)x, (uint32_t *)xs);
    } else {
        const dim3 b = row_block(H);
        k_dispatch<uint16_t><<<row_grid(T, b), b, 0, s>>>(a, (const uint16_t *)x, (uint16_t *)xs);
    }
    count_launch();
    return cuda_status(cudaGetLastError());
}

spmm_status spmm_routes_combine(int dtype, const void *y, const float *w, const int32_t *slots,
                                const int32_t *offsets, int64_t T, int64_t k, int64_t E,
                                int64_t H, void *out, void *stream) {
    using namespace spmm;
    const spmm_status st = check_rows(dtype, slots, offsets, T, k, E, H, H);
    if (st != SPMM_OK) return st;
    if (T == 0 || H == 0) return SPMM_OK;
    if (!out || (k > 0 && !y)) return SPMM_ERR_INVALID_ARG;
    const RouteArgs a{slots, k ? offsets + E : nullptr, w, T, H, H, (int)k};
    return cuda_status(launch_combine(dtype, a, y, out, (cudaStream_t)stream));
}

spmm_status spmm_routes_combine_backward(int dtype, const void *dout, int64_t lddout,
                                         const void *y, const float *w, const int32_t *slots,
                                         const int32_t *offsets, int64_t T, int64_t k, int64_t E,
                                         int64_t H, void *dy, float *dw, void *stream) {
    using namespace spmm;
    const spmm_status st = check_rows(dtype, slots, offsets, T, k, E, H, lddout);
    if (st != SPMM_OK) return st;
    if (T == 0 || k == 0) return SPMM_OK;
    if (H > 0 && (!dout || !y || !dy)) return SPMM_ERR_INVALID_ARG;
    if (H == 0 && !dw) return SPMM_OK;
    cudaStream_t s = (cudaStream_t)stream;
    const RouteArgs a{slots, offsets + E, w, T, H, lddout, (int)k};
    const bool wide = wide_ok(dtype, H, lddout, {dout, y, dy});
    by_type(dtype, [&](auto t, auto v) {
        using T_ = decltype(t);
        constexpr int V = decltype(v)::value;
        const dim3 b = row_block(wide ? H / V : H);
        if (wide)
            k_combine_bwd<T_, V><<<row_grid(T, b), b, 0, s>>>(a, (const T_ *)dout, (const T_ *)y,
                                                              (T_ *)dy, dw);
        else
            k_combine_bwd<T_, 1><<<row_grid(T, b), b, 0, s>>>(a, (const T_ *)dout, (const T_ *)y,
                                                              (T_ *)dy, dw);
    });
    count_launch();
    return cuda_status(cudaGetLastError());
}

}  // extern "C"
