// Values of x in 8 bits with a scale for each 1 x 128 or 128 x 128 block (fp8.cuh).
//
// Bound by memory: x is read once and a byte written for each element. Two forms, by the direction in which x is contiguous:
// along its rows, as activations and weights are, or down its columns (the transpose of such a tensor, whose scales then
// run along what were its rows: the operands of a weight's gradient). Both hold a block's elements in registers between the
// maximum and the rounding. Times in a graph: 17,384 x 4096 bfloat16 33 us (6.4 TB/s, 94% of the measured copy rate), 4096 x 17,384 transposed
// 42 us (5.1 TB/s), 4096 x 1024 float32 by 128 x 128 3.5 us; rows that do not lie on 16 bytes 47 us (4,097 x 17,383 bfloat16,
// transposed 61).
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
    int beside;  // log2 of the warps of a block of threads that lie along the columns, where each has rows of its own
};

constexpr int kQuantBlock = 256;  // threads

template <class T>
struct QuantBits {
    typedef uint16_t type;
};
template <>
struct QuantBits<float> {
    typedef uint32_t type;
};

// Both halves of a word at once, as integers, in the order of their magnitudes.
template <int N>
__device__ __forceinline__ unsigned halves_top(const uint32_t (&w)[N]) {
    unsigned t = 0;
#pragma unroll
    for (int i = 0; i < N; ++i) t = __vmaxu2(t, w[i] & 0x7fff7fffu);
    return max(t & 0xffffu, t >> 16);
}

// Rows, each block of 128 columns by neighbouring lanes with VEC elements in 16 bytes: a half warp (16-bit types) or a warp. A warp
// has kRows rows, whose kLoads loads are all under way together. BLOCK: 128 rows, a block of threads', share a scale. (17,384 x 4096
// bfloat16: elements unpacked before the comparison, 8 bytes to a lane, a division for each row 75 us; 8 loads in 99 registers 45; 4
// loads and 6 blocks of threads on an SM 33. With scales for 128 x 128 those registers are needed: 40, float32 58 with 8 loads and 72
// with 4.)
template <class T, bool BLOCK>
struct QuantRows {
    static constexpr int kVec = 16 / (int)sizeof(T), kLanes = kQBlock / kVec, kLoads = BLOCK && sizeof(T) == 4 ? 8 : 4, kBeside = 32 / kLanes, kRows = kLoads * kBeside;
};
template <class T, bool BLOCK>
__global__ void __launch_bounds__(BLOCK ? kQBlock / QuantRows<T, BLOCK>::kRows * 32 : kQuantBlock, !BLOCK && sizeof(T) == 2 ? 6 : 0) k_quantize_rows(const QuantArgs a) {
    using R = QuantRows<T, BLOCK>;
    constexpr int kWarps = BLOCK ? kQBlock / R::kRows : kQuantBlock / 32;
    pdl_entry();
    __shared__ unsigned tops[kWarps];
    const int lane = threadIdx.x & 31, warp = threadIdx.x / 32, l = lane % R::kLanes, beside = lane / R::kLanes;
    const int blocks = (a.cols + kQBlock - 1) / kQBlock;
    // a block's warps take neighbouring columns of the same rows (few columns: the next rows'), or the rows of one block
    const int across = BLOCK ? 1 : 1 << a.beside, up = BLOCK ? warp : warp >> a.beside;
    const long long row0 = (BLOCK ? (long long)blockIdx.x * kQBlock : (long long)blockIdx.x * (kWarps >> a.beside) * R::kRows) + up * R::kRows + beside;
    for (int block = blockIdx.y * across + (BLOCK ? 0 : warp & (across - 1)); block < blocks; block += gridDim.y * across) {
        const int c = block * kQBlock + l * R::kVec;
        const bool in = c < a.cols;
        const T* x = static_cast<const T*>(a.x) + row0 * a.x_stride + c;
        Pack<uint32_t, 4> v[R::kLoads];
#pragma unroll
        for (int i = 0; i < R::kLoads; ++i) {
            v[i] = Pack<uint32_t, 4>{};
            if (in && row0 + i * R::kBeside < a.rows) v[i] = *reinterpret_cast<const Pack<uint32_t, 4>*>(x + i * R::kBeside * a.x_stride);
        }
        auto top_of = [](const Pack<uint32_t, 4>& p) {
            if (sizeof(T) == 2) return magnitude(to_float(__builtin_bit_cast(T, (typename QuantBits<T>::type)halves_top(p.v))));
            return max(max(p.v[0] & 0x7fffffffu, p.v[1] & 0x7fffffffu), max(p.v[2] & 0x7fffffffu, p.v[3] & 0x7fffffffu));
        };
        unsigned all = 0;
        if (BLOCK) {
#pragma unroll
            for (int i = 0; i < R::kLoads; ++i) all = max(all, top_of(v[i]));
            all = __reduce_max_sync(0xffffffffu, all);
            __syncthreads();  // the turn before has read them
            if (lane == 0) tops[warp] = all;
            __syncthreads();
            all = __reduce_max_sync(0xffffffffu, tops[lane % kWarps]);
        }
        uint8_t* q = a.q + row0 * a.q_stride + c;
        float kept = 0.f;
#pragma unroll
        for (int i = 0; i < R::kLoads; ++i) {
            const float scale = block_scale(BLOCK ? all : lanes_top<R::kLanes>(top_of(v[i]))), back = scale_back(scale);
            if (l == i) kept = scale;
            if (!in || row0 + i * R::kBeside >= a.rows) continue;
            const Pack<T, R::kVec> e = __builtin_bit_cast(Pack<T, R::kVec>, v[i]);
            Pack<uint32_t, R::kVec / 4> out;
#pragma unroll
            for (int k = 0; k < R::kVec; k += 4) out.v[k / 4] = quantize4(to_float(e.v[k]), to_float(e.v[k + 1]), to_float(e.v[k + 2]), to_float(e.v[k + 3]), back);
            *reinterpret_cast<Pack<uint32_t, R::kVec / 4>*>(q + i * R::kBeside * a.q_stride) = out;
        }
        // lane i of a row's has the scale of its i-th row
        if (!BLOCK && l < R::kLoads && row0 + l * R::kBeside < a.rows) a.scale.at(row0 + l * R::kBeside, block) = kept;
        if (BLOCK && threadIdx.x == 0) a.scale.at(blockIdx.x, block) = block_scale(all);
    }
}

// Rows that do not lie on 16 bytes, or do not end there: an element at a time, 8 rows of a warp.
constexpr int kQuantRows = 8;
template <class T, bool BLOCK>
__global__ void __launch_bounds__(BLOCK ? 512 : kQuantBlock) k_quantize_rows_odd(const QuantArgs a) {
    pdl_entry();
    __shared__ unsigned tops[16];
    const int lane = threadIdx.x & 31, warp = threadIdx.x / 32, blocks = (a.cols + kQBlock - 1) / kQBlock;
    constexpr int kWarps = kQuantBlock / 32;
    const int across = BLOCK ? 1 : 1 << a.beside, up = BLOCK ? warp : warp >> a.beside;
    const long long row0 = (BLOCK ? (long long)blockIdx.x * kQBlock : (long long)blockIdx.x * (kWarps >> a.beside) * kQuantRows) + up * kQuantRows;
    for (int block = blockIdx.y * across + (BLOCK ? 0 : warp & (across - 1)); block < blocks; block += gridDim.y * across) {
        const int c = block * kQBlock + lane;
        const T* x = static_cast<const T*>(a.x) + row0 * a.x_stride + c;
        T v[kQuantRows][4];
        const int rows = (int)min((long long)kQuantRows, a.rows - row0);
        unsigned all = 0, top[kQuantRows];
#pragma unroll
        for (int r = 0; r < kQuantRows; ++r)
#pragma unroll
            for (int j = 0; j < 4; ++j) v[r][j] = r < rows && c + 32 * j < a.cols ? x[r * a.x_stride + 32 * j] : from_float<T>(0.f);
#pragma unroll
        for (int r = 0; r < kQuantRows; ++r) {
            top[r] = 0;
#pragma unroll
            for (int j = 0; j < 4; ++j) top[r] = max(top[r], magnitude(to_float(v[r][j])));
            all = max(all, top[r]);
        }
        if (BLOCK) {
            all = __reduce_max_sync(0xffffffffu, all);
            __syncthreads();
            if (lane == 0) tops[warp] = all;
            __syncthreads();
            all = __reduce_max_sync(0xffffffffu, tops[lane & 15]);
        }
        uint8_t* q = a.q + row0 * a.q_stride + c;
        float kept = 0.f;
#pragma unroll
        for (int r = 0; r < kQuantRows; ++r) {
            const float scale = block_scale(BLOCK ? all : __reduce_max_sync(0xffffffffu, top[r])), back = scale_back(scale);
            if (lane == r) kept = scale;
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (r < rows && c + 32 * j < a.cols) q[r * a.q_stride + 32 * j] = quantize1(to_float(v[r][j]), back);
        }
        if (!BLOCK && lane < rows) a.scale.at(row0 + lane, block) = kept;
        if (BLOCK && threadIdx.x == 0) a.scale.at(blockIdx.x, block) = block_scale(all);
    }
}

// What a thread holds of a column in the form below: one row, or the two neighbouring rows of a 16-bit word, kept as bits so
// that 128 of them take 128 registers.
template <class T, int PER>
struct QuantWord;
template <>
struct QuantWord<float, 1> {
    typedef uint32_t Bits;
    static __device__ __forceinline__ float value(uint32_t w, int) { return __uint_as_float(w); }
    static __device__ __forceinline__ uint32_t larger(uint32_t top, uint32_t w) { return max(top, w & 0x7fffffffu); }
    static __device__ __forceinline__ unsigned top(uint32_t t, int) { return t; }
};
template <class T>
struct QuantWord<T, 1> {
    typedef uint16_t Bits;
    static __device__ __forceinline__ float value(uint32_t w, int) { return to_float(__builtin_bit_cast(T, (uint16_t)w)); }
    static __device__ __forceinline__ uint32_t larger(uint32_t top, uint32_t w) { return max(top, w & 0x7fffu); }
    static __device__ __forceinline__ unsigned top(uint32_t t, int r) { return magnitude(value(t, r)); }
};
template <class T>
struct QuantWord<T, 2> {
    typedef uint32_t Bits;
    static __device__ __forceinline__ float value(uint32_t w, int r) { return to_float(__builtin_bit_cast(T, (uint16_t)(r ? w >> 16 : w & 0xffffu))); }
    static __device__ __forceinline__ uint32_t larger(uint32_t top, uint32_t w) { return __vmaxu2(top, w & 0x7fff7fffu); }  // both rows' magnitudes
    static __device__ __forceinline__ unsigned top(uint32_t t, int r) { return magnitude(value(t, r)); }
};

// Columns are contiguous: four threads share PER neighbouring rows, 32 columns of their block each, and their maxima through
// shared memory. A block of threads has 128 rows; their bytes go through shared memory too, so that a row's 128 are written at
// once. (Written by each thread as it has them, 16 at a time: 4096 x 17,384 bfloat16 88 us; with one thread for all 128
// columns, 168 registers, 60 us.)
constexpr int kQuantPart = 32;
template <class T, int PER, bool BLOCK>
__global__ void __launch_bounds__(4 * kQBlock / PER) k_quantize_cols(const QuantArgs a) {
    using W = QuantWord<T, PER>;
    constexpr int kThreads = kQBlock / PER;  // along the rows
    pdl_entry();
    __shared__ uint32_t tops[4][kThreads];
    __shared__ uint4 tile[kQBlock][8];  // 16 bytes of row r at [r][c ^ r / PER % 8]: no bank twice, written or read
    const int t = threadIdx.x % kThreads, part = threadIdx.x / kThreads, blocks = (a.cols + kQBlock - 1) / kQBlock;
    const long long row0 = (long long)blockIdx.x * kQBlock + t * PER;
    const bool live = row0 < a.rows;  // with PER = 2 the rows are even
    for (int block = blockIdx.y; block < blocks; block += gridDim.y) {
        const int c0 = block * kQBlock + part * kQuantPart, n = min(kQuantPart, a.cols - c0);
        const T* x = static_cast<const T*>(a.x) + (long long)c0 * a.x_stride + row0;
        uint32_t v[kQuantPart], all = 0;
#pragma unroll
        for (int c = 0; c < kQuantPart; ++c) v[c] = live && c < n ? *reinterpret_cast<const typename W::Bits*>(x + c * a.x_stride) : 0u;
#pragma unroll
        for (int c = 0; c < kQuantPart; ++c) all = W::larger(all, v[c]);
        __syncthreads();  // the turn before has read them
        tops[part][t] = all;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 4; ++i) all = W::larger(all, tops[i][t]);
        unsigned top[PER];
#pragma unroll
        for (int r = 0; r < PER; ++r) top[r] = W::top(all, r);
        if (BLOCK) {
            unsigned m = __reduce_max_sync(0xffffffffu, max(top[0], top[PER - 1]));
            __syncthreads();
            if ((threadIdx.x & 31) == 0) tops[0][threadIdx.x / 32] = m;
            __syncthreads();
#pragma unroll
            for (int w = 0; w < kThreads / 32; ++w) m = max(m, tops[0][w]);  // the first part's warps have every row
            top[0] = top[PER - 1] = m;
        }
#pragma unroll
        for (int r = 0; r < PER; ++r) {
            const float scale = block_scale(top[r]), back = scale_back(scale);
            if (part == 0 && (BLOCK ? threadIdx.x == 0 && r == 0 : live)) a.scale.at(BLOCK ? blockIdx.x : row0 + r, block) = scale;
#pragma unroll
            for (int c = 0; c < kQuantPart; c += 16) {
                uint32_t p[4];
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    p[j] = quantize4(W::value(v[c + 4 * j], r), W::value(v[c + 4 * j + 1], r), W::value(v[c + 4 * j + 2], r), W::value(v[c + 4 * j + 3], r), back);
                tile[t * PER + r][(part * 2 + c / 16) ^ (t & 7)] = make_uint4(p[0], p[1], p[2], p[3]);
            }
        }
        __syncthreads();
        // rows of q start on 16 bytes; what lies behind the columns is left as it was
        const int left = a.cols - block * kQBlock - threadIdx.x % 8 * 16;
        for (int r = threadIdx.x / 8; r < kQBlock; r += 4 * kThreads / 8) {
            const long long row = (long long)blockIdx.x * kQBlock + r;
            if (row >= a.rows || left <= 0) break;
            const uint4 w = tile[r][threadIdx.x % 8 ^ (r / PER & 7)];
            uint8_t* q = a.q + row * a.q_stride + block * kQBlock + threadIdx.x % 8 * 16;
            if (left >= 16) {
                *reinterpret_cast<uint4*>(q) = w;
            } else {
                const uint32_t p[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                for (int j = 0; j < 16; ++j)
                    if (j < left) q[j] = (uint8_t)(p[j / 4] >> (8 * (j % 4)));
            }
        }
    }
}

namespace {

// `up` blocks of rows by `across` of columns (a block of threads takes several of these where the grid ends).
cudaError_t go(void (*kernel)(const QuantArgs), long long up, long long across, int threads, const QuantArgs& a, cudaStream_t st) {
    if (up > 0x7fffffffll) return cudaErrorInvalidConfiguration;
    count_launches(1);
    return launch_pdl(kernel, dim3((unsigned)up, (unsigned)(across < 65535 ? across : 65535)), dim3(threads), 0, st, a);
}

template <class T>
cudaError_t run(QuantArgs a, bool by_cols, bool block, cudaStream_t st) {
    auto over = [](long long n, long long m) { return (n + m - 1) / m; };
    const long long across = over(a.cols, kQBlock), tiles = over(a.rows, kQBlock);
    const uintptr_t x = reinterpret_cast<uintptr_t>(a.x);
    if (by_cols) {
        if constexpr (sizeof(T) == 2)
            if (a.rows % 2 == 0 && a.x_stride % 2 == 0 && x % 4 == 0)
                return go(block ? k_quantize_cols<T, 2, true> : k_quantize_cols<T, 2, false>, tiles, across, 2 * kQBlock, a, st);
        return go(block ? k_quantize_cols<T, 1, true> : k_quantize_cols<T, 1, false>, tiles, across, 4 * kQBlock, a, st);
    }
    using R = QuantRows<T, false>;
    constexpr int kWarps = kQuantBlock / 32;
    while (1 << a.beside < across && 1 << a.beside < kWarps) ++a.beside;
    const long long up = kWarps >> a.beside;  // (139,072 x 100 bfloat16: 19 us with all warps along the columns)
    const bool vec = a.cols % R::kVec == 0 && a.x_stride % R::kVec == 0 && x % 16 == 0;
    if (vec) return block ? go(k_quantize_rows<T, true>, tiles, across, kQBlock / QuantRows<T, true>::kRows * 32, a, st)
                          : go(k_quantize_rows<T, false>, over(a.rows, up * R::kRows), over(across, 1 << a.beside), kQuantBlock, a, st);
    return block ? go(k_quantize_rows_odd<T, true>, tiles, across, 512, a, st)
                 : go(k_quantize_rows_odd<T, false>, over(a.rows, up * kQuantRows), over(across, 1 << a.beside), kQuantBlock, a, st);
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
