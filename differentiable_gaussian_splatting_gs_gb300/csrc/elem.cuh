// Element types of the decoder operators (layer norm, cross attention): float, __half and
// __nv_bfloat16 values in memory, float32 in registers.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace gs {

__device__ __forceinline__ float to_float(float v) { return v; }
__device__ __forceinline__ float to_float(__half v) { return __half2float(v); }
__device__ __forceinline__ float to_float(__nv_bfloat16 v) { return __bfloat162float(v); }

template <class T>
__device__ __forceinline__ T from_float(float v);
template <>
__device__ __forceinline__ float from_float<float>(float v) { return v; }
template <>
__device__ __forceinline__ __half from_float<__half>(float v) { return __float2half_rn(v); }
template <>
__device__ __forceinline__ __nv_bfloat16 from_float<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

// VEC consecutive elements moved with one access (VEC * sizeof(T) is 2, 4 or 16 bytes, aligned to it).
template <class T, int VEC>
struct alignas(sizeof(T) * VEC) Pack {
    T v[VEC];
};

// x[i] of an array whose element type is known at run time (dtype: GS_DTYPE_*).
__device__ __forceinline__ float load_elem(const void* x, long long i, int dtype) {
    if (dtype == 0) return static_cast<const float*>(x)[i];
    if (dtype == 1) return __half2float(static_cast<const __half*>(x)[i]);
    return __bfloat162float(static_cast<const __nv_bfloat16*>(x)[i]);
}

__device__ __forceinline__ void store_elem(void* x, long long i, int dtype, float v) {
    if (dtype == 0) static_cast<float*>(x)[i] = v;
    else if (dtype == 1) static_cast<__half*>(x)[i] = __float2half_rn(v);
    else static_cast<__nv_bfloat16*>(x)[i] = __float2bfloat16_rn(v);
}

}  // namespace gs
