// 8-bit values with a scale for each block of 128: q = e4m3(x / scale), scale = max |x| of the block / 448, which the
// block's largest element meets exactly. A block without elements above 448 2^-126 has scale 1 (its elements become 0), so
// that no scale is 0 or subnormal. Magnitudes are compared as integers, where NaN is the largest: a block with one has a NaN
// scale and NaN elements, one with an infinity an infinite scale, which nothing finite can stand beside.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "gs_common.cuh"

namespace gs {

constexpr int kQBlock = 128;  // columns (or rows and columns) that share a scale

__device__ __forceinline__ unsigned magnitude(float v) { return __float_as_uint(v) & 0x7fffffffu; }

// The largest of LANES neighbouring lanes' magnitudes.
template <int LANES>
__device__ __forceinline__ unsigned lanes_top(unsigned m) {
    if constexpr (LANES == 32) {
        return __reduce_max_sync(0xffffffffu, m);
    } else {
#pragma unroll
        for (int o = LANES / 2; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
        return m;
    }
}

// A product with 1/448, within an ulp of the quotient: a division for each 128 elements in every lane took a third of the
// quantizing kernels' instructions.
__device__ __forceinline__ float block_scale(unsigned top) {
    const float s = __uint_as_float(top) * (1.f / 448.f);
    return s < 1.17549435e-38f ? 1.f : s;
}
// The scale's reciprocal to an ulp: a quotient moves by 1.5 ulps of float32. That changes one value in a million of float32 inputs.
// Quotients of 16-bit ones often lie halfway between two 8-bit values exactly (one in 2,000 of a norm's), where either is as near:
// there the last bits decide, in one of 10,000 otherwise than a division's. (Quotients corrected by their remainder, which round as a
// division does: 17,384 x 4096 bfloat16 37 us instead of 33, by 128 x 128 51 instead of 40, the norm to 8 bits 3 to 7% more.)
__device__ __forceinline__ float scale_back(float scale) { return rcp_approx(scale); }

// Four values times the scale's reciprocal, the first in the lowest byte.
__device__ __forceinline__ uint32_t quantize4(float a, float b, float c, float d, float inv) {
    uint16_t lo, hi;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b * inv), "f"(a * inv));
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d * inv), "f"(c * inv));
    return (uint32_t)lo | (uint32_t)hi << 16;
}
__device__ __forceinline__ uint8_t quantize1(float a, float inv) {
    uint16_t lo;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(0.f), "f"(a * inv));
    return (uint8_t)lo;
}

// Where a scale is: scale[row * row_stride + block * block_stride].
struct ScaleAt {
    float* p;
    long long row, block;
    __device__ __forceinline__ float& at(long long r, long long b) const { return p[r * row + b * block]; }
};

}  // namespace gs
