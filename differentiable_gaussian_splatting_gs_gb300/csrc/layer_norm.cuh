// What the forward and the backward layer-norm kernels share: how a row is laid over threads, and
// sums over a row.
#pragma once

#include "elem.cuh"
#include "gs_common.cuh"
#include "gs_internal.h"

namespace gs {

// A row belongs to LPR threads: a part of a warp (8 or 16 lanes), a warp, or a block of kNormBlock
// threads. Thread l holds the vectors l, l + LPR, ..., l + (NV - 1) LPR of the row, VEC elements each,
// in registers, so that every pass over the row after the first reads no memory.
constexpr int kNormBlock = 256;   // threads per block of the row kernels
constexpr int kNormMaxElems = 32; // elements of a row per thread
constexpr int kNormMaxCols = kNormBlock * kNormMaxElems;  // longer rows are read again in each pass

// Sum of N values over the LPR threads of a row, the same in all of them. For LPR > 32, `buf` is
// shared memory of 2 * N * 8 floats used alternately (flip by `phase`), so one barrier per sum is enough.
template <int LPR, int N>
__device__ __forceinline__ void row_sum(float (&s)[N], float* buf, int& phase) {
    constexpr int kLanes = LPR < 32 ? LPR : 32;
#pragma unroll
    for (int o = kLanes / 2; o > 0; o >>= 1)
#pragma unroll
        for (int i = 0; i < N; ++i) s[i] += __shfl_xor_sync(0xffffffffu, s[i], o);
    if (LPR > 32) {
        constexpr int kWarps = LPR / 32;
        float* b = buf + phase * (N * kWarps);
        phase ^= 1;
        if ((threadIdx.x & 31) == 0)
#pragma unroll
            for (int i = 0; i < N; ++i) b[i * kWarps + (threadIdx.x >> 5)] = s[i];
        __syncthreads();
#pragma unroll
        for (int i = 0; i < N; ++i) {
            float t = 0.f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) t += b[i * kWarps + w];
            s[i] = t;
        }
    }
}

template <class T, int VEC, int NV, int LPR>
__device__ __forceinline__ void load_row(Pack<T, VEC> (&raw)[NV], const T* row, int l, int nvec, bool live) {
#pragma unroll
    for (int i = 0; i < NV; ++i)
        if (live && l + i * LPR < nvec) raw[i] = *reinterpret_cast<const Pack<T, VEC>*>(row + (size_t)(l + i * LPR) * VEC);
}

// Calls f with the layout's constants for rows of `nvec` vectors of VEC elements of type T, at most
// kNormMaxElems elements per thread. Parts of a warp for rows of up to 8 or 16 vectors, a warp as long
// as its 32 elements per lane reach (a shuffle reduction needs no barrier), then a block.
template <int NV_, int LPR_>
struct NormShape {
    static constexpr int NV = NV_, LPR = LPR_;
};

template <int VEC, class F>
cudaError_t norm_dispatch(int nvec, F&& f) {
    if constexpr (VEC > 1) {
        if (nvec <= 8) return f(NormShape<1, 8>());
        if (nvec <= 16) return f(NormShape<1, 16>());
        if (nvec <= 32) return f(NormShape<1, 32>());
        if (nvec <= 64) return f(NormShape<2, 32>());
        if (nvec <= 96) return f(NormShape<3, 32>());
        if (nvec <= 128) return f(NormShape<4, 32>());
        if constexpr (VEC == 4) {
            if (nvec <= 192) return f(NormShape<6, 32>());
            if (nvec <= 256) return f(NormShape<8, 32>());
        }
        if (nvec <= 256) return f(NormShape<1, 256>());
        if (nvec <= 512) return f(NormShape<2, 256>());
        if constexpr (VEC == 8) return f(NormShape<4, 256>());
        if (nvec <= 1024) return f(NormShape<4, 256>());
        return f(NormShape<8, 256>());
    } else {
        if (nvec <= 32) return f(NormShape<1, 32>());
        if (nvec <= 64) return f(NormShape<2, 32>());
        if (nvec <= 128) return f(NormShape<4, 32>());
        if (nvec <= 256) return f(NormShape<8, 32>());
        if (nvec <= 384) return f(NormShape<12, 32>());
        if (nvec <= 512) return f(NormShape<16, 32>());
        if (nvec <= 768) return f(NormShape<24, 32>());
        if (nvec <= 1024) return f(NormShape<32, 32>());
        if (nvec <= 2048) return f(NormShape<8, 256>());
        if (nvec <= 4096) return f(NormShape<16, 256>());
        return f(NormShape<32, 256>());
    }
}

}  // namespace gs
