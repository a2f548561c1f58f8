// Values of x in 8 bits with a scale for each 1 x 128 or 128 x 128 block (fp8.cuh).
//
// Bound by memory: x is read once and a byte written for each element. Two forms, by the direction in which x is contiguous:
// along its rows, as activations and weights are, or down its columns (the transpose of such a tensor, whose scales then
// run along what were its rows: the operands of a weight's gradient). Both hold a block's elements in registers between the
// maximum and the rounding.
#include "elem.cuh"
#include "fp8.cuh"
#include "gs_common.cuh"
#include "gs_internal.h"

namespace gs {

struct QuantArgs {
    const void* x;
    uint8_t* q;
    ScaleAt scale;
    long long rows, x_stride, q_stride;  // x_stride: of rows, or of columns where these are contiguous
    int cols;
};

constexpr int kQuantBlock = 256;
constexpr int kQuantRows = 8;  // rows of a warp

// Rows of 128 columns, 4 to a lane: 8 rows of a warp, whose loads are all under way together. BLOCK: the 128 rows of a
// block of 16 warps share a scale.
template <class T, bool VEC, bool BLOCK>
__global__ void __launch_bounds__(BLOCK ? 512 : kQuantBlock) k_quantize_rows(const QuantArgs a) {
    pdl_entry();
    __shared__ unsigned tops[16];
    const int lane = threadIdx.x & 31, warp = threadIdx.x / 32, blocks = (a.cols + kQBlock - 1) / kQBlock;
    // neighbouring warps take neighbouring columns of the same rows, or the rows of one block
    const long long turn = BLOCK ? blockIdx.x : (long long)blockIdx.x * (kQuantBlock / 32) + warp;
    const long long row0 = turn / blocks * (BLOCK ? kQBlock : kQuantRows) + (BLOCK ? warp * kQuantRows : 0);
    const int block = (int)(turn % blocks), c = block * kQBlock + (VEC ? 4 * lane : lane);
    const T* x = static_cast<const T*>(a.x) + row0 * a.x_stride + c;
    float v[kQuantRows][4];
#pragma unroll
    for (int r = 0; r < kQuantRows; ++r) {
        if (VEC) {
            Pack<T, 4> p = {};
            if (row0 + r < a.rows && c < a.cols) p = *reinterpret_cast<const Pack<T, 4>*>(x + r * a.x_stride);
#pragma unroll
            for (int j = 0; j < 4; ++j) v[r][j] = to_float(p.v[j]);
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) v[r][j] = row0 + r < a.rows && c + 32 * j < a.cols ? to_float(x[r * a.x_stride + 32 * j]) : 0.f;
        }
    }
    float scale[kQuantRows];
    unsigned all = 0;
#pragma unroll
    for (int r = 0; r < kQuantRows; ++r) {
        unsigned top = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) top = max(top, magnitude(v[r][j]));
        if (BLOCK) all = max(all, top);
        else scale[r] = block_scale(__reduce_max_sync(0xffffffffu, top));
    }
    if (BLOCK) {
        all = __reduce_max_sync(0xffffffffu, all);
        if (lane == 0) tops[warp] = all;
        __syncthreads();
        all = __reduce_max_sync(0xffffffffu, tops[lane & 15]);
#pragma unroll
        for (int r = 0; r < kQuantRows; ++r) scale[r] = block_scale(all);
    }
    uint8_t* q = a.q + row0 * a.q_stride + c;
#pragma unroll
    for (int r = 0; r < kQuantRows; ++r) {
        if (row0 + r >= a.rows) break;
        const float back = 1.f / scale[r];
        if (VEC) {
            if (c < a.cols) *reinterpret_cast<uint32_t*>(q + r * a.q_stride) = quantize4(v[r][0], v[r][1], v[r][2], v[r][3], back);
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (c + 32 * j < a.cols) q[r * a.q_stride + 32 * j] = quantize1(v[r][j], back);
        }
        if (lane == r && !BLOCK) a.scale.at(row0 + r, block) = scale[r];
    }
    if (BLOCK && threadIdx.x == 0) a.scale.at(row0 / kQBlock, block) = scale[0];
}

// Columns are contiguous: a thread takes PER neighbouring rows and all 128 columns of their block, so that a row's maximum
// needs no other thread and its 128 bytes go out 16 at a time. A block of threads has 128 rows. PER is 2 where two rows'
// 16-bit elements are one word, so that the block's 128 columns take 128 registers whatever the element's size.
template <class T, int PER, bool BLOCK>
__global__ void __launch_bounds__(kQBlock / PER) k_quantize_cols(const QuantArgs a) {
    pdl_entry();
    __shared__ unsigned tops[4];
    const int blocks = (a.cols + kQBlock - 1) / kQBlock;
    // neighbouring blocks of threads take neighbouring rows of the same columns
    const long long tiles = (a.rows + kQBlock - 1) / kQBlock, row0 = blockIdx.x % tiles * kQBlock + threadIdx.x * PER;
    const int block = (int)(blockIdx.x / tiles), c0 = block * kQBlock, n = min(kQBlock, a.cols - c0);
    const T* x = static_cast<const T*>(a.x) + (long long)c0 * a.x_stride + row0;
    Pack<T, PER> v[kQBlock];
    const bool live = row0 < a.rows;  // with PER = 2 the rows are even
#pragma unroll
    for (int c = 0; c < kQBlock; ++c) {
        v[c] = Pack<T, PER>{};
        if (live && c < n) v[c] = *reinterpret_cast<const Pack<T, PER>*>(x + c * a.x_stride);
    }
    unsigned top[PER];
#pragma unroll
    for (int r = 0; r < PER; ++r) {
        top[r] = 0;
#pragma unroll
        for (int c = 0; c < kQBlock; ++c) top[r] = max(top[r], magnitude(to_float(v[c].v[r])));
    }
    if (BLOCK) {
        unsigned all = top[0];
        if (PER == 2) all = max(all, top[PER - 1]);
        all = __reduce_max_sync(0xffffffffu, all);
        if ((threadIdx.x & 31) == 0) tops[threadIdx.x / 32] = all;
        __syncthreads();
        all = tops[0];
#pragma unroll
        for (int w = 1; w < kQBlock / PER / 32; ++w) all = max(all, tops[w]);
#pragma unroll
        for (int r = 0; r < PER; ++r) top[r] = all;
    }
    if (!live) return;
#pragma unroll
    for (int r = 0; r < PER; ++r) {
        const float scale = block_scale(top[r]), back = 1.f / scale;
        uint8_t* q = a.q + (row0 + r) * a.q_stride + c0;
#pragma unroll
        for (int c = 0; c < kQBlock; c += 16) {  // rows of q start on 16 bytes; what lies behind the columns is left as it was
            uint4 w;
            uint32_t* p = &w.x;
#pragma unroll
            for (int j = 0; j < 4; ++j)
                p[j] = quantize4(to_float(v[c + 4 * j].v[r]), to_float(v[c + 4 * j + 1].v[r]), to_float(v[c + 4 * j + 2].v[r]),
                                 to_float(v[c + 4 * j + 3].v[r]), back);
            if (c + 16 <= n) {
                *reinterpret_cast<uint4*>(q + c) = w;
            } else {
#pragma unroll
                for (int j = 0; j < 16; ++j)
                    if (c + j < n) q[c + j] = (uint8_t)(p[j / 4] >> (8 * (j % 4)));
            }
        }
        if (!BLOCK) a.scale.at(row0 + r, block) = scale;
        else if (threadIdx.x == 0 && r == 0) a.scale.at(row0 / kQBlock, block) = scale;
    }
}

namespace {

cudaError_t go(void (*kernel)(const QuantArgs), long long blocks, int threads, const QuantArgs& a, cudaStream_t st) {
    if (blocks > 0x7fffffffll) return cudaErrorInvalidConfiguration;
    count_launches(1);
    return launch_pdl(kernel, dim3((unsigned)blocks), dim3(threads), 0, st, a);
}

template <class T>
cudaError_t run(const QuantArgs& a, bool by_cols, bool block, cudaStream_t st) {
    const long long blocks = (a.cols + kQBlock - 1) / kQBlock;
    const uintptr_t x = reinterpret_cast<uintptr_t>(a.x);
    if (by_cols) {
        const long long tiles = (a.rows + kQBlock - 1) / kQBlock * blocks;
        if constexpr (sizeof(T) == 2)
            if (a.rows % 2 == 0 && a.x_stride % 2 == 0 && x % 4 == 0)
                return go(block ? k_quantize_cols<T, 2, true> : k_quantize_cols<T, 2, false>, tiles, kQBlock / 2, a, st);
        return go(block ? k_quantize_cols<T, 1, true> : k_quantize_cols<T, 1, false>, tiles, kQBlock, a, st);
    }
    const bool vec = a.cols % 4 == 0 && a.x_stride % 4 == 0 && x % (4 * sizeof(T)) == 0;
    if (block) return go(vec ? k_quantize_rows<T, true, true> : k_quantize_rows<T, false, true>, (a.rows + kQBlock - 1) / kQBlock * blocks, 512, a, st);
    const long long warps = (a.rows + kQuantRows - 1) / kQuantRows * blocks;
    return go(vec ? k_quantize_rows<T, true, false> : k_quantize_rows<T, false, false>, (warps + kQuantBlock / 32 - 1) / (kQuantBlock / 32),
              kQuantBlock, a, st);
}

}  // namespace

cudaError_t launch_quantize(int dtype, const void* x, long long x_stride, bool by_cols, long long rows, int cols, bool block, void* q,
                            long long q_stride, float* scale, long long scale_row, long long scale_block, cudaStream_t st) {
    if (rows == 0 || cols == 0) return cudaSuccess;
    const QuantArgs a{x, static_cast<uint8_t*>(q), {scale, scale_row, scale_block}, rows, x_stride, q_stride, cols};
    if (dtype == GS_DTYPE_F32) return run<float>(a, by_cols, block, st);
    if (dtype == GS_DTYPE_F16) return run<__half>(a, by_cols, block, st);
    return run<__nv_bfloat16>(a, by_cols, block, st);
}

}  // namespace gs
