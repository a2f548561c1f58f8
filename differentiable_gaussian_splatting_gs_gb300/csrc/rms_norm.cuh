// What the forward and the backward root-mean-square norm kernels share beside the layer norm's (layer_norm.cuh).
#pragma once

#include "fp8.cuh"
#include "layer_norm.cuh"

namespace gs {

// The vector of the row that thread l holds as its i-th. Rows read an element at a time keep 128 consecutive elements,
// which share a scale in 8 bits, in one warp: 4 in turn of each thread.
template <int VEC, int NV, int LPR>
__device__ __forceinline__ int vec_at(int l, int i) {
    if (VEC == 1 && NV % 4 == 0 && LPR > 32) return (i / 4) * 4 * LPR + (l / 32) * 128 + (i % 4) * 32 + (l & 31);
    return l + i * LPR;
}

template <class T, int VEC, int NV, int LPR, int FULL>
__device__ __forceinline__ void load_vecs(Pack<T, VEC> (&raw)[NV], const T* row, int l, int nvec, bool live) {
    static_assert(VEC > 1 || NV % 4 != 0 || LPR <= 32 || FULL % 4 == 0, "a row's first FULL vectors are whole turns of four");
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int v = vec_at<VEC, NV, LPR>(l, i);
        if (live && (i < FULL || v < nvec)) raw[i] = *reinterpret_cast<const Pack<T, VEC>*>(row + (size_t)v * VEC);
    }
}

// Rows of more than kNormMaxCols elements belong to a block, which takes kLongTurn columns of VEC x 4 to a thread at a time and
// has the four loads under way together. Where the j-th of them lies, from the turn's first column on: 128 consecutive elements
// to neighbouring lanes of one warp, either way.
constexpr int kLongLoads = 4;
template <int VEC>
constexpr int kLongTurn = kNormBlock * kLongLoads * VEC;
template <int VEC>
__device__ __forceinline__ int long_at(int c0, int j) {
    const int t = threadIdx.x;
    return VEC == 1 ? c0 + (t / 32) * kQBlock + j * 32 + t % 32 : c0 + (j * kNormBlock + t) * VEC;
}
template <class T, int VEC>
__device__ __forceinline__ void load_long(Pack<T, VEC> (&p)[kLongLoads], const T* row, int c0, int cols) {
#pragma unroll
    for (int j = 0; j < kLongLoads; ++j)
        if (long_at<VEC>(c0, j) < cols) p[j] = *reinterpret_cast<const Pack<T, VEC>*>(row + long_at<VEC>(c0, j));
}
// VEC weights from column c on (VEC > 1: they lie on 16 bytes), 1 without.
template <int VEC>
__device__ __forceinline__ void load_weights(float (&w)[VEC], const void* weight, int dtype, int c) {
    if (!weight) {
#pragma unroll
        for (int k = 0; k < VEC; ++k) w[k] = 1.f;
    } else if constexpr (VEC == 1) {
        w[0] = load_elem(weight, c, dtype);
    } else if (dtype == GS_DTYPE_F32) {
#pragma unroll
        for (int k = 0; k < VEC; k += 4) {
            const float4 v = *reinterpret_cast<const float4*>(static_cast<const float*>(weight) + c + k);
            w[k] = v.x, w[k + 1] = v.y, w[k + 2] = v.z, w[k + 3] = v.w;
        }
    } else if constexpr (VEC == 8) {
        if (dtype == GS_DTYPE_F16) unpack<__half, 8>(*reinterpret_cast<const Pack<__half, 8>*>(static_cast<const __half*>(weight) + c), w);
        else unpack<__nv_bfloat16, 8>(*reinterpret_cast<const Pack<__nv_bfloat16, 8>*>(static_cast<const __nv_bfloat16*>(weight) + c), w);
    }
}

}  // namespace gs
