// Shared by the operators whose pattern is chosen at run time (expert routes,
// selected key blocks): element types and their packed loads and stores. Sums
// are always formed in fp32; a value is rounded to its 16-bit type once, where
// it is stored.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "common.cuh"
#include "spmm_dynamic.h"

namespace spmm {

__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_f32(__half x) { return __half2float(x); }

template <typename T> __device__ __forceinline__ T from_f32(float x);
template <> __device__ __forceinline__ float from_f32<float>(float x) { return x; }
template <> __device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float x) {
    return __float2bfloat16_rn(x);
}
template <> __device__ __forceinline__ __half from_f32<__half>(float x) {
    return __float2half_rn(x);
}

// V elements of type T moved by one access: 16 bytes, or a single element when
// a row's start or length rules the wide access out.
template <typename T, int V>
struct alignas(sizeof(T) * V < 16 ? sizeof(T) * V : 16) Pack {
    T e[V];
};

template <typename T, int V>
__device__ __forceinline__ void ld_pack(const T *p, float (&x)[V]) {
    const Pack<T, V> v = *reinterpret_cast<const Pack<T, V> *>(p);
#pragma unroll
    for (int i = 0; i < V; ++i) x[i] = to_f32(v.e[i]);
}

template <typename T, int V>
__device__ __forceinline__ void st_pack(T *p, const float (&x)[V]) {
    Pack<T, V> v;
#pragma unroll
    for (int i = 0; i < V; ++i) v.e[i] = from_f32<T>(x[i]);
    *reinterpret_cast<Pack<T, V> *>(p) = v;
}

inline int dtype_bytes(int dtype) { return dtype == SPMM_F32 ? 4 : 2; }
inline bool dtype_ok(int dtype) {
    return dtype == SPMM_F32 || dtype == SPMM_BF16 || dtype == SPMM_F16;
}

inline spmm_status cuda_status(cudaError_t e) {
    if (e == cudaSuccess) return SPMM_OK;
    return e == cudaErrorMemoryAllocation ? SPMM_ERR_OOM : SPMM_ERR_CUDA;
}

// The current device's word that a bounded wait which gave up sets, for a launch on
// `s` (spmm_dynamic_sync reads it).
cudaError_t dynamic_err(cudaStream_t s, int32_t **err);

}  // namespace spmm
