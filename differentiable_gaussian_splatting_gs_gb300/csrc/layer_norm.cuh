// What the forward and the backward layer-norm kernels share: how a row is laid over threads, and
// sums over a row.
#pragma once

#include "elem.cuh"
#include "gs_common.cuh"
#include "gs_internal.h"
#include "norm_ring.cuh"

namespace gs {

// A row belongs to LPR threads: a part of a warp (4, 8 or 16 lanes), or 1, 2, 4 or 8 warps of a block of kNormBlock
// threads. Thread l holds the vectors l, l + LPR, ..., l + (NV - 1) LPR of the row, VEC elements each,
// in registers, so that every pass over the row after the first reads no memory.
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
        const int group = threadIdx.x / LPR;
        float* b = buf + (group * 2 + phase) * (N * kWarps);
        phase ^= 1;
        if ((threadIdx.x & 31) == 0)
#pragma unroll
            for (int i = 0; i < N; ++i) b[i * kWarps + (threadIdx.x % LPR >> 5)] = s[i];
        asm volatile("bar.sync %0, %1;" ::"r"(1 + group), "n"(LPR) : "memory");
#pragma unroll
        for (int i = 0; i < N; ++i) {
            float t = 0.f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) t += b[i * kWarps + w];
            s[i] = t;
        }
    }
}

template <class T, int VEC, int NV, int LPR, int FULL>
__device__ __forceinline__ void load_row(Pack<T, VEC> (&raw)[NV], const T* row, int l, int nvec, bool live) {
#pragma unroll
    for (int i = 0; i < NV; ++i)
        if (live && (i < FULL || l + i * LPR < nvec)) raw[i] = *reinterpret_cast<const Pack<T, VEC>*>(row + (size_t)(l + i * LPR) * VEC);
}

// The weights as floats in shared memory, `missing` where there are none. (In registers they would take as many
// as the row itself does in the forward, and keep the warps from being many enough to cover the memory's latency.)
// Element j of vector v lies where consecutive threads, which hold consecutive vectors, meet no bank twice: fours of
// a vector's elements as planes.
template <int VEC>
__device__ __forceinline__ int plane_at(int c, int nvec) {
    constexpr int P = VEC % 4 == 0 ? 4 : 1;
    return ((c % VEC) / P * nvec + c / VEC) * P + c % P;
}

template <int VEC>
__device__ __forceinline__ void stage_weights(float* dst, const void* w, int dtype, int cols, float missing) {
    for (int c = threadIdx.x; c < cols; c += blockDim.x) dst[plane_at<VEC>(c, cols / VEC)] = w ? load_elem(w, c, dtype) : missing;
}

template <class T, int VEC>
__device__ __forceinline__ void unpack(const Pack<T, VEC>& p, float (&f)[VEC]) {
#pragma unroll
    for (int k = 0; k < VEC; ++k) f[k] = to_float(p.v[k]);
}
template <class T, int VEC>
__device__ __forceinline__ Pack<T, VEC> repack(const float (&f)[VEC]) {
    Pack<T, VEC> p;
#pragma unroll
    for (int k = 0; k < VEC; ++k) p.v[k] = from_float<T>(f[k]);
    return p;
}

// Vector v of an array of floats in shared memory.
template <int VEC>
__device__ __forceinline__ void load_floats(float (&f)[VEC], const float* p, int v, int nvec) {
    if constexpr (VEC == 1) {
        f[0] = p[v];
    } else {
#pragma unroll
        for (int j = 0; j < VEC; j += 4) {
            const float4 q = reinterpret_cast<const float4*>(p)[j / 4 * nvec + v];
            f[j] = q.x, f[j + 1] = q.y, f[j + 2] = q.z, f[j + 3] = q.w;
        }
    }
}
template <int VEC>
__device__ __forceinline__ void store_floats(const float (&f)[VEC], float* p, int v, int nvec) {
    if constexpr (VEC == 1) {
        p[v] = f[0];
    } else {
#pragma unroll
        for (int j = 0; j < VEC; j += 4) reinterpret_cast<float4*>(p)[j / 4 * nvec + v] = make_float4(f[j], f[j + 1], f[j + 2], f[j + 3]);
    }
}

constexpr unsigned kNormSpin = 1u << 18;  // polls before a wait gives up
// Rows that come through the ring: 16-byte vectors, several per thread of a warp, or a block's. (Rows read an element at a
// time took longer through it, copied with the 16-byte pieces they begin and end in: 100,000 x 127 bfloat16,
// backward, 38 us against 23.)
template <int VEC, int NV, int LPR>
constexpr bool norm_ring = VEC > 1 && (LPR > 32 || (LPR == 32 && NV > 1));

template <int BARS>
__device__ __forceinline__ void init_ring_bars(uint64_t* bars) {
    if (threadIdx.x == 0) {
        for (int i = 0; i < BARS; ++i) mbar_init(bars + i, 1);
        fence_mbar_init();
    }
    __syncthreads();
}

// Calls f with the layout's constants for rows of `nvec` vectors of VEC elements of type T: as few threads as hold
// the row with MOST vectors each (a sum over a warp needs no barrier), or up to kNormMaxElems elements in the
// longest rows.
template <int NV_, int LPR_, int FULL_>
struct NormShape {
    static constexpr int NV = NV_, LPR = LPR_;
    static constexpr int FULL = FULL_;  // the thread's first vectors, which every row of this shape has
};

template <int VEC, int MOST, class F>
cudaError_t norm_dispatch(int nvec, F&& f) {
    if constexpr (VEC > 1) {
        if (nvec <= 4) return f(NormShape<1, 4, 0>());
        if (nvec <= 8) return f(NormShape<1, 8, 0>());
        if (nvec <= 16) return f(NormShape<1, 16, 0>());
        if (nvec <= 32) return f(NormShape<1, 32, 0>());
        if (nvec <= 64) return f(NormShape<2, 32, 1>());
        if constexpr (MOST >= 4) {
            if (nvec <= 96) return f(NormShape<3, 32, 2>());
            if (nvec <= 128) return f(NormShape<4, 32, 3>());
        }
        if constexpr (MOST >= 8) {
            if (nvec <= 192) return f(NormShape<6, 32, 4>());
            if (nvec <= 256) return f(NormShape<8, 32, 6>());
        }
        if (nvec <= 64 * MOST) return f(NormShape<MOST, 64, MOST / 2>());
        if (nvec <= 128 * MOST) return f(NormShape<MOST, 128, MOST / 2>());
        if (nvec <= 256 * MOST) return f(NormShape<MOST, 256, MOST / 2>());
        return f(NormShape<kNormMaxElems / VEC, 256, MOST>());
    } else {
        if (nvec <= 32) return f(NormShape<1, 32, 0>());
        if (nvec <= 64) return f(NormShape<2, 32, 1>());
        if (nvec <= 128) return f(NormShape<4, 32, 2>());
        if (nvec <= 256) return f(NormShape<8, 32, 4>());
        if (nvec <= 384) return f(NormShape<12, 32, 8>());
        if (nvec <= 512) return f(NormShape<16, 32, 12>());
        if (nvec <= 1024) return f(NormShape<16, 64, 8>());
        if (nvec <= 2048) return f(NormShape<16, 128, 8>());
        if (nvec <= 4096) return f(NormShape<16, 256, 8>());
        return f(NormShape<32, 256, 16>());
    }
}

}  // namespace gs
