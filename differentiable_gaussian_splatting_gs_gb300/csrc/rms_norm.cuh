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
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int v = vec_at<VEC, NV, LPR>(l, i);
        if (live && (i < FULL || v < nvec)) raw[i] = *reinterpret_cast<const Pack<T, VEC>*>(row + (size_t)v * VEC);
    }
}

}  // namespace gs
