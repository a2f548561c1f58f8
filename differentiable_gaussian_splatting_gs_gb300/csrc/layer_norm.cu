// Layer norm, forward: y = (x - mean) rstd w + b over each row, with rstd = 1 / sqrt(var + eps).
//
// The work is bound by memory: x is read once and y written once. A row stays in the registers of
// the threads it is laid over (layer_norm.cuh), where the mean is formed first and the variance then
// from the centred values: sum(x^2) - sum(x)^2 / C in one pass would lose the variance of channels
// whose mean is large. The grid is persistent, so the weights are read into registers once, and each
// thread loads its next row before it reduces the present one.
#include "layer_norm.cuh"

namespace gs {

struct NormFwdArgs {
    const void *x, *weight, *bias;
    void* y;
    float *mean, *rstd;
    long long rows, x_stride, y_stride;
    int cols, wdtype;
    float eps;
};

template <class T, int VEC, int NV, int LPR>
__global__ void __launch_bounds__(kNormBlock) k_norm_fwd(const NormFwdArgs a) {
    pdl_entry();
    __shared__ float buf[2 * kNormBlock / 32];
    int phase = 0;
    constexpr int kRows = kNormBlock / LPR;  // rows of a block at a time
    const int l = threadIdx.x % LPR, nvec = a.cols / VEC;
    const float inv = 1.f / (float)a.cols;
    float w[NV * VEC], b[NV * VEC];
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
            const int c = (l + i * LPR) * VEC + j;
            w[i * VEC + j] = a.weight && c < a.cols ? load_elem(a.weight, c, a.wdtype) : 1.f;
            b[i * VEC + j] = a.bias && c < a.cols ? load_elem(a.bias, c, a.wdtype) : 0.f;
        }
    const T* x = static_cast<const T*>(a.x);
    T* y = static_cast<T*>(a.y);
    const long long step = (long long)gridDim.x * kRows;
    long long base = (long long)blockIdx.x * kRows;  // uniform over the block: all lanes take part in the sums
    Pack<T, VEC> raw[NV];
    load_row<T, VEC, NV, LPR>(raw, x + (base + threadIdx.x / LPR) * a.x_stride, l, nvec, base + threadIdx.x / LPR < a.rows);
    for (; base < a.rows; base += step) {
        const long long row = base + threadIdx.x / LPR;
        const bool live = row < a.rows;
        float v[NV * VEC];
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int j = 0; j < VEC; ++j)
                v[i * VEC + j] = live && l + i * LPR < nvec ? to_float(raw[i].v[j]) : 0.f;
        load_row<T, VEC, NV, LPR>(raw, x + (row + step) * a.x_stride, l, nvec, row + step < a.rows);
        float s[1] = {0.f};
#pragma unroll
        for (int i = 0; i < NV * VEC; ++i) s[0] += v[i];
        row_sum<LPR>(s, buf, phase);
        const float mean = s[0] * inv;
        s[0] = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (l + i * LPR < nvec)
#pragma unroll
                for (int j = 0; j < VEC; ++j) {
                    v[i * VEC + j] -= mean;
                    s[0] = fmaf(v[i * VEC + j], v[i * VEC + j], s[0]);
                }
        row_sum<LPR>(s, buf, phase);
        const float rstd = 1.f / sqrtf(s[0] * inv + a.eps);
        if (!live) continue;
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (l + i * LPR < nvec) {
                Pack<T, VEC> o;
#pragma unroll
                for (int j = 0; j < VEC; ++j)
                    o.v[j] = from_float<T>(fmaf(v[i * VEC + j] * rstd, w[i * VEC + j], b[i * VEC + j]));
                *reinterpret_cast<Pack<T, VEC>*>(y + row * a.y_stride + (size_t)(l + i * LPR) * VEC) = o;
            }
        if (l == 0) {
            a.mean[row] = mean;
            a.rstd[row] = rstd;
        }
    }
}

// Rows of more than kNormMaxCols elements: a block per row, which reads it again for each pass (the
// second and third from the L2 or the L1).
template <class T>
__global__ void __launch_bounds__(kNormBlock) k_norm_fwd_long(const NormFwdArgs a) {
    pdl_entry();
    __shared__ float buf[2 * kNormBlock / 32];
    int phase = 0;
    for (long long row = blockIdx.x; row < a.rows; row += gridDim.x) {
        const T* x = static_cast<const T*>(a.x) + row * a.x_stride;
        T* y = static_cast<T*>(a.y) + row * a.y_stride;
        float s[1] = {0.f};
        for (int c = threadIdx.x; c < a.cols; c += kNormBlock) s[0] += to_float(x[c]);
        row_sum<kNormBlock>(s, buf, phase);
        const float mean = s[0] / (float)a.cols;
        s[0] = 0.f;
        for (int c = threadIdx.x; c < a.cols; c += kNormBlock) {
            const float d = to_float(x[c]) - mean;
            s[0] = fmaf(d, d, s[0]);
        }
        row_sum<kNormBlock>(s, buf, phase);
        const float rstd = 1.f / sqrtf(s[0] / (float)a.cols + a.eps);
        for (int c = threadIdx.x; c < a.cols; c += kNormBlock) {
            const float w = a.weight ? load_elem(a.weight, c, a.wdtype) : 1.f;
            const float b = a.bias ? load_elem(a.bias, c, a.wdtype) : 0.f;
            y[c] = from_float<T>(fmaf((to_float(x[c]) - mean) * rstd, w, b));
        }
        if (threadIdx.x == 0) {
            a.mean[row] = mean;
            a.rstd[row] = rstd;
        }
    }
}

namespace {

template <class T, int VEC>
cudaError_t run(const NormFwdArgs& a, cudaStream_t st) {
    return norm_dispatch<VEC>(a.cols / VEC, [&](auto shape) {
        using S = decltype(shape);
        static std::atomic<int> cache[256] = {};
        auto* kernel = k_norm_fwd<T, VEC, S::NV, S::LPR>;
        const int most = resident_blocks(kernel, kNormBlock, 0, cache);
        const long long want = (a.rows + kNormBlock / S::LPR - 1) / (kNormBlock / S::LPR);
        count_launches(1);
        return launch_pdl(kernel, dim3((unsigned)(want < most ? want : most)), dim3(kNormBlock), 0, st, a);
    });
}

template <class T>
cudaError_t run_typed(const NormFwdArgs& a, cudaStream_t st) {
    constexpr int V = 16 / (int)sizeof(T);
    if (a.cols > kNormMaxCols) {
        static std::atomic<int> cache[256] = {};
        const int most = resident_blocks(k_norm_fwd_long<T>, kNormBlock, 0, cache);
        count_launches(1);
        return launch_pdl(k_norm_fwd_long<T>, dim3((unsigned)(a.rows < most ? a.rows : most)), dim3(kNormBlock), 0, st, a);
    }
    // 16-byte accesses when every row starts on a 16-byte boundary and ends with a whole vector
    const bool vec = a.cols % V == 0 && a.x_stride % V == 0 && a.y_stride % V == 0 &&
                     (reinterpret_cast<uintptr_t>(a.x) | reinterpret_cast<uintptr_t>(a.y)) % 16 == 0;
    return vec ? run<T, V>(a, st) : run<T, 1>(a, st);
}

}  // namespace

cudaError_t launch_norm_fwd(int dtype, const void* x, long long x_stride, long long rows, int cols, const void* weight,
                            const void* bias, int wdtype, float eps, void* y, long long y_stride, float* mean,
                            float* rstd, cudaStream_t st) {
    if (rows == 0) return cudaSuccess;
    const NormFwdArgs a{x, weight, bias, y, mean, rstd, rows, x_stride, y_stride, cols, wdtype, eps};
    if (dtype == GS_DTYPE_F32) return run_typed<float>(a, st);
    if (dtype == GS_DTYPE_F16) return run_typed<__half>(a, st);
    return run_typed<__nv_bfloat16>(a, st);
}

}  // namespace gs
