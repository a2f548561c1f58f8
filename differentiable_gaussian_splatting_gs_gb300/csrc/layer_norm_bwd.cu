// Layer norm, backward. With xhat = (x - mean) rstd and g = w dy, per row
//   dx = rstd (g - mean(g) - xhat mean(g xhat)),
// and over the rows dw = sum dy xhat, db = sum dy.
//
// Bound by memory: x and dy are read once, dx is written once. A row's elements stay in registers, and
// so do the thread's columns of dw and db: the grid is persistent, each thread adds up the rows it
// meets, the block adds its threads' sums in shared memory and leaves them in the workspace, and a
// second kernel adds the blocks'. All in a fixed order, so the same call gives the same bits.
#include "layer_norm.cuh"

namespace gs {

struct NormBwdArgs {
    const void *dy, *x, *weight;
    const float *mean, *rstd;
    void* dx;
    float* part;  // [blocks][2][cols]: each block's share of dw and db
    long long rows, dy_stride, x_stride, dx_stride;
    int cols, wdtype;
};

template <class T, int VEC, int NV, int LPR>
__global__ void __launch_bounds__(kNormBlock) k_norm_bwd(const NormBwdArgs a) {
    pdl_entry();
    extern __shared__ float share[];  // rows per block x 2 x cols: the block's sums (LPR < 256)
    __shared__ float buf[2 * 2 * kNormBlock / 32];
    int phase = 0;
    constexpr int kRows = kNormBlock / LPR, E = NV * VEC;
    const int l = threadIdx.x % LPR, nvec = a.cols / VEC;
    const float inv = 1.f / (float)a.cols;
    float w[E], dw[E], db[E];
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
            const int c = (l + i * LPR) * VEC + j;
            w[i * VEC + j] = a.weight && c < a.cols ? load_elem(a.weight, c, a.wdtype) : 1.f;
            dw[i * VEC + j] = db[i * VEC + j] = 0.f;
        }
    const T *x = static_cast<const T*>(a.x), *dy = static_cast<const T*>(a.dy);
    T* dx = static_cast<T*>(a.dx);
    const long long step = (long long)gridDim.x * kRows;
    for (long long base = (long long)blockIdx.x * kRows; base < a.rows; base += step) {
        const long long row = base + threadIdx.x / LPR;
        const bool live = row < a.rows;
        Pack<T, VEC> rx[NV], rd[NV];
        load_row<T, VEC, NV, LPR>(rx, x + row * a.x_stride, l, nvec, live);
        load_row<T, VEC, NV, LPR>(rd, dy + row * a.dy_stride, l, nvec, live);
        const float mean = live ? a.mean[row] : 0.f, rstd = live ? a.rstd[row] : 0.f;
        float s[2] = {0.f, 0.f};
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (live && l + i * LPR < nvec)
#pragma unroll
                for (int j = 0; j < VEC; ++j) {
                    const int e = i * VEC + j;
                    const float d = to_float(rd[i].v[j]), h = (to_float(rx[i].v[j]) - mean) * rstd, g = d * w[e];
                    dw[e] = fmaf(d, h, dw[e]);
                    db[e] += d;
                    s[0] += g;
                    s[1] = fmaf(g, h, s[1]);
                }
        row_sum<LPR>(s, buf, phase);
        if (!live) continue;
        const float m0 = s[0] * inv, m1 = s[1] * inv;
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (l + i * LPR < nvec) {
                Pack<T, VEC> o;
#pragma unroll
                for (int j = 0; j < VEC; ++j) {
                    const float h = (to_float(rx[i].v[j]) - mean) * rstd, g = to_float(rd[i].v[j]) * w[i * VEC + j];
                    o.v[j] = from_float<T>(rstd * (g - m0 - h * m1));
                }
                *reinterpret_cast<Pack<T, VEC>*>(dx + row * a.dx_stride + (size_t)(l + i * LPR) * VEC) = o;
            }
    }
    if (!a.part) return;
    float* part = a.part + (size_t)blockIdx.x * 2 * a.cols;
    if (LPR == kNormBlock) {
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int j = 0; j < VEC; ++j) {
                const int c = (l + i * LPR) * VEC + j;
                if (c < a.cols) {
                    part[c] = dw[i * VEC + j];
                    part[a.cols + c] = db[i * VEC + j];
                }
            }
        return;
    }
    float* mine = share + (size_t)(threadIdx.x / LPR) * 2 * a.cols;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
            const int c = (l + i * LPR) * VEC + j;
            if (c < a.cols) {
                mine[c] = dw[i * VEC + j];
                mine[a.cols + c] = db[i * VEC + j];
            }
        }
    __syncthreads();
    for (int c = threadIdx.x; c < 2 * a.cols; c += kNormBlock) {
        float t = 0.f;
        for (int r = 0; r < kRows; ++r) t += share[(size_t)r * 2 * a.cols + c];
        part[c] = t;
    }
}

// Rows of more than kNormMaxCols elements: a block per row for dx, which reads the row twice.
template <class T>
__global__ void __launch_bounds__(kNormBlock) k_norm_bwd_long(const NormBwdArgs a) {
    pdl_entry();
    __shared__ float buf[2 * 2 * kNormBlock / 32];
    int phase = 0;
    for (long long row = blockIdx.x; row < a.rows; row += gridDim.x) {
        const T* x = static_cast<const T*>(a.x) + row * a.x_stride;
        const T* dy = static_cast<const T*>(a.dy) + row * a.dy_stride;
        T* dx = static_cast<T*>(a.dx) + row * a.dx_stride;
        const float mean = a.mean[row], rstd = a.rstd[row];
        float s[2] = {0.f, 0.f};
        for (int c = threadIdx.x; c < a.cols; c += kNormBlock) {
            const float g = to_float(dy[c]) * (a.weight ? load_elem(a.weight, c, a.wdtype) : 1.f);
            s[0] += g;
            s[1] = fmaf(g, (to_float(x[c]) - mean) * rstd, s[1]);
        }
        row_sum<kNormBlock>(s, buf, phase);
        const float m0 = s[0] / (float)a.cols, m1 = s[1] / (float)a.cols;
        for (int c = threadIdx.x; c < a.cols; c += kNormBlock) {
            const float g = to_float(dy[c]) * (a.weight ? load_elem(a.weight, c, a.wdtype) : 1.f);
            dx[c] = from_float<T>(rstd * (g - m0 - (to_float(x[c]) - mean) * rstd * m1));
        }
    }
}

// ... and dw, db of such rows: a thread per column over the block's share of the rows.
template <class T>
__global__ void __launch_bounds__(kNormBlock) k_norm_bwd_long_cols(const NormBwdArgs a) {
    pdl_entry();
    const int c = blockIdx.x * kNormBlock + threadIdx.x;
    if (c >= a.cols) return;
    const long long per = (a.rows + gridDim.y - 1) / gridDim.y, r0 = blockIdx.y * per;
    const long long r1 = r0 + per < a.rows ? r0 + per : a.rows;
    const T *x = static_cast<const T*>(a.x) + c, *dy = static_cast<const T*>(a.dy) + c;
    float dw = 0.f, db = 0.f;
    for (long long r = r0; r < r1; ++r) {
        const float d = to_float(dy[r * a.dy_stride]);
        dw = fmaf(d, (to_float(x[r * a.x_stride]) - a.mean[r]) * a.rstd[r], dw);
        db += d;
    }
    float* part = a.part + (size_t)blockIdx.y * 2 * a.cols;
    part[c] = dw;
    part[a.cols + c] = db;
}

// dw, db = the sums of the blocks' shares: a warp per 32 columns and slice of the shares, eight slices
// to a block, in order.
__global__ void __launch_bounds__(256) k_norm_bwd_sum(const float* part, int blocks, int cols, void* dweight, void* dbias,
                                                      int wdtype) {
    pdl_entry();
    __shared__ float share[8][33];
    const int c = blockIdx.x * 32 + (threadIdx.x & 31), s = threadIdx.x >> 5;  // c counts dw's columns, then db's
    float t = 0.f;
    if (c < 2 * cols) {
#pragma unroll 8
        for (int b = s; b < blocks; b += 8) t += part[(size_t)b * 2 * cols + c];
    }
    share[s][threadIdx.x & 31] = t;
    __syncthreads();
    if (s != 0 || c >= 2 * cols) return;
#pragma unroll
    for (int i = 1; i < 8; ++i) t += share[i][threadIdx.x & 31];
    if (c < cols) {
        if (dweight) store_elem(dweight, c, wdtype, t);
    } else if (dbias) {
        store_elem(dbias, c - cols, wdtype, t);
    }
}

namespace {

constexpr int kMaxShares = 1024;  // blocks that leave a share of dw and db in the workspace

long long shares(long long rows) { return rows < kMaxShares ? rows : kMaxShares; }

template <class T, int VEC>
cudaError_t run(const NormBwdArgs& a, int* blocks, cudaStream_t st) {
    return norm_dispatch<VEC>(a.cols / VEC, [&](auto shape) {
        using S = decltype(shape);
        constexpr int kRows = kNormBlock / S::LPR;
        static std::atomic<int> cache[256] = {};
        auto* kernel = k_norm_bwd<T, VEC, S::NV, S::LPR>;
        // at most 2 x 8 x 1024 floats (a warp's row) or 2 x 32 x 8 VEC (8 lanes' row)
        const size_t smem = kRows > 1 ? (size_t)kRows * 2 * a.cols * sizeof(float) : 0;
        constexpr int kMost = kRows > 1 ? kRows * 2 * S::NV * S::LPR * VEC * (int)sizeof(float) : 0;
        if (kMost > 48 * 1024) {
            cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMost);
            if (e) return e;
        }
        int most = resident_blocks(kernel, kNormBlock, kMost, cache);
        if (most > kMaxShares) most = kMaxShares;
        const long long want = (a.rows + kRows - 1) / kRows;
        *blocks = (int)(want < most ? want : most);
        count_launches(1);
        return launch_pdl(kernel, dim3((unsigned)*blocks), dim3(kNormBlock), smem, st, a);
    });
}

template <class T>
cudaError_t run_typed(const NormBwdArgs& a, int* blocks, cudaStream_t st) {
    constexpr int V = 16 / (int)sizeof(T);
    if (a.cols > kNormMaxCols) {
        static std::atomic<int> cache[256] = {};
        const int most = resident_blocks(k_norm_bwd_long<T>, kNormBlock, 0, cache);
        count_launches(1);
        cudaError_t e = launch_pdl(k_norm_bwd_long<T>, dim3((unsigned)(a.rows < most ? a.rows : most)), dim3(kNormBlock), 0, st, a);
        if (e || !a.part) return e;
        *blocks = (int)(shares(a.rows) < 64 ? shares(a.rows) : 64);
        count_launches(1);
        return launch_pdl(k_norm_bwd_long_cols<T>, dim3((a.cols + kNormBlock - 1) / kNormBlock, *blocks), dim3(kNormBlock), 0, st, a);
    }
    const bool vec = a.cols % V == 0 && a.x_stride % V == 0 && a.dy_stride % V == 0 && a.dx_stride % V == 0 &&
                     (reinterpret_cast<uintptr_t>(a.x) | reinterpret_cast<uintptr_t>(a.dy) |
                      reinterpret_cast<uintptr_t>(a.dx)) % 16 == 0;
    return vec ? run<T, V>(a, blocks, st) : run<T, 1>(a, blocks, st);
}

}  // namespace

size_t norm_bwd_workspace_bytes(long long rows, int cols) { return (size_t)shares(rows) * 2 * cols * sizeof(float); }

cudaError_t launch_norm_bwd(int dtype, const void* dy, long long dy_stride, const void* x, long long x_stride,
                            long long rows, int cols, const float* mean, const float* rstd, const void* weight,
                            int wdtype, void* dx, long long dx_stride, void* dweight, void* dbias, float* workspace,
                            cudaStream_t st) {
    const bool sums = dweight || dbias;
    const NormBwdArgs a{dy, x, weight, mean, rstd, dx, sums ? workspace : nullptr, rows, dy_stride, x_stride, dx_stride, cols, wdtype};
    int blocks = 0;
    cudaError_t e = cudaSuccess;
    if (rows > 0) {
        if (dtype == GS_DTYPE_F32) e = run_typed<float>(a, &blocks, st);
        else if (dtype == GS_DTYPE_F16) e = run_typed<__half>(a, &blocks, st);
        else e = run_typed<__nv_bfloat16>(a, &blocks, st);
    }
    if (e || !sums) return e;
    count_launches(1);
    return launch_pdl(k_norm_bwd_sum, dim3((unsigned)((2ll * cols + 31) / 32)), dim3(256), 0, st, (const float*)workspace, blocks,
                      cols, dweight, dbias, wdtype);
}

}  // namespace gs
