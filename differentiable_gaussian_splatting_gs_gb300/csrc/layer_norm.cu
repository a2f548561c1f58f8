// Layer norm, forward: y = (x - mean) rstd w + b over each row, with rstd = 1 / sqrt(var + eps).
//
// The work is bound by memory: x is read once and y written once. A row stays in the registers of
// the threads it is laid over (layer_norm.cuh), in its own type, where the mean is formed first and the variance
// then from the centred values: sum(x^2) - sum(x)^2 / C in one pass would lose the variance of channels
// whose mean is large. The grid is persistent, with the weights in shared memory, and each thread loads its next
// row before it reduces the present one; rows of more than a vector per thread come through shared memory (NormRing).
#include "layer_norm.cuh"

namespace gs {

struct NormFwdArgs {
    const void *x, *weight, *bias;
    void* y;
    float *mean, *rstd;
    long long rows, x_stride, y_stride;
    int cols, wdtype;
    float eps;
    unsigned* err;
};

template <class T, int VEC, int NV, int LPR, int FULL>
__global__ void __launch_bounds__(kNormBlock) k_norm_fwd(const NormFwdArgs a) {
    pdl_entry();
    extern __shared__ __align__(16) float weights[];  // w, then b
    __shared__ float buf[2 * kNormBlock / 32];
    int phase = 0;
    constexpr int kRows = kNormBlock / LPR;  // rows of a block at a time
    const int l = threadIdx.x % LPR, nvec = a.cols / VEC;
    const float inv = 1.f / (float)a.cols;
    auto in = [&](int i) { return i < FULL || l + i * LPR < nvec; };
    const T* x = static_cast<const T*>(a.x);
    T* y = static_cast<T*>(a.y);
    const long long step = (long long)gridDim.x * kRows;
    long long base = (long long)blockIdx.x * kRows;  // uniform over the block: all lanes take part in the sums
    constexpr bool kRing = norm_ring<VEC, NV, LPR>;
    Pack<T, VEC> raw[NV], next[NV];
    constexpr int kStages = norm_stages<NV, LPR>;
    __shared__ uint64_t bars[kRing ? kRows * kStages : 1];
    NormRing<1, kRing ? LPR : 32, kStages> ring;
    if constexpr (kRing) {
        init_ring_bars<kRows * kStages>(bars);
        ring.src[0] = reinterpret_cast<const char*>(x);
        ring.stride[0] = a.x_stride * (long long)sizeof(T);
        ring.start(reinterpret_cast<unsigned char*>(weights + 2 * a.cols), bars, a.cols, sizeof(T),
                   base + threadIdx.x / LPR, a.rows, step, kNormSpin, a.err);
    } else {
        load_row<T, VEC, NV, LPR, FULL>(next, x + (base + threadIdx.x / LPR) * a.x_stride, l, nvec, base + threadIdx.x / LPR < a.rows);
    }
    stage_weights<VEC>(weights, a.weight, a.wdtype, a.cols, 1.f);
    stage_weights<VEC>(weights + a.cols, a.bias, a.wdtype, a.cols, 0.f);
    __syncthreads();
    for (; base < a.rows; base += step) {
        const long long row = base + threadIdx.x / LPR;
        const bool live = row < a.rows;
        if (VEC == 1 && !live) break;  // the same in all threads of the row
        if constexpr (kRing) {
            if (live) {
                ring.wait();
                load_row<T, VEC, NV, LPR, FULL>(raw, reinterpret_cast<const T*>(ring.at(0)), l, nvec, true);
            }
        } else {
#pragma unroll
            for (int i = 0; i < NV; ++i) raw[i] = next[i];
            load_row<T, VEC, NV, LPR, FULL>(next, x + (row + step) * a.x_stride, l, nvec, row + step < a.rows);
        }
        // A row read an element at a time takes a register for each whatever its type: converted once.
        float f[VEC], t[2] = {0.f, 0.f}, one[VEC == 1 ? NV : 1];
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (live && in(i)) {
                unpack<T, VEC>(raw[i], f);
                if (VEC == 1) one[i] = f[0];
#pragma unroll
                for (int k = 0; k < VEC; ++k) t[(VEC == 1 ? i : k) & 1] += f[k];
            }
        float s[1] = {t[0] + t[1]};
        row_sum<LPR>(s, buf, phase);
        if (kRing && live) {
            __syncwarp();
            ring.next();
        }
        const float mean = s[0] * inv;
        t[0] = t[1] = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (live && in(i)) {
                if (VEC == 1) f[0] = one[i];
                else unpack<T, VEC>(raw[i], f);
#pragma unroll
                for (int k = 0; k < VEC; ++k) {
                    const float d = f[k] - mean;
                    if (VEC == 1) one[i] = d;
                    t[(VEC == 1 ? i : k) & 1] = fmaf(d, d, t[(VEC == 1 ? i : k) & 1]);
                }
            }
        s[0] = t[0] + t[1];
        row_sum<LPR>(s, buf, phase);
        const float rstd = 1.f / sqrtf(s[0] * inv + a.eps);
        if (!live) continue;
        T* to = y + row * a.y_stride + l * VEC;
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (in(i)) {
                float w[VEC], b[VEC];
                load_floats<VEC>(w, weights, l + i * LPR, nvec);
                load_floats<VEC>(b, weights + a.cols, l + i * LPR, nvec);
                if (VEC > 1) unpack<T, VEC>(raw[i], f);
#pragma unroll
                for (int k = 0; k < VEC; ++k) f[k] = fmaf((VEC == 1 ? one[i] : f[k] - mean) * rstd, w[k], b[k]);
                *reinterpret_cast<Pack<T, VEC>*>(to + i * LPR * VEC) = repack<T, VEC>(f);
            }
        if (l == 0) {
            a.mean[row] = mean;
            a.rstd[row] = rstd;
        }
    }
    if constexpr (kRing) ring.finish();
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
    // 32 elements a thread: each sum is a shuffle reduction and, over several warps, a barrier
    return norm_dispatch<VEC, VEC == 8 ? 4 : 8>(a.cols / VEC, [&](auto shape) {
        using S = decltype(shape);
        static std::atomic<int> cache[256] = {};
        // vectors tested against the row's end although it has them: 139,072 x 1024 bfloat16 93.8 us, 100.4 without the test
        // (the loads are then issued in another order); 20,000 x 4096, whose rows take the block, 69.1 and 65.1 us
        auto* kernel = k_norm_fwd<T, VEC, S::NV, S::LPR, VEC == 1 || S::LPR == 256 ? S::FULL : 0>;
        constexpr bool kRing = norm_ring<VEC, S::NV, S::LPR>;
        constexpr int kCols = S::NV * S::LPR * VEC;
        auto smem_of = [&](int cols) {
            return 2 * cols * sizeof(float) + (kRing ? NormRing<1, kRing ? S::LPR : 32, norm_stages<S::NV, S::LPR>>::smem(cols, sizeof(T)) : 0);
        };
        const int kMost = (int)smem_of(kCols);
        if (kMost > 48 * 1024) {
            cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMost);
            if (e) return e;
        }
        const int most = resident_blocks(kernel, kNormBlock, kMost, cache);
        const size_t smem = smem_of(a.cols);
        const long long want = (a.rows + kNormBlock / S::LPR - 1) / (kNormBlock / S::LPR);
        count_launches(1);
        return launch_pdl(kernel, dim3((unsigned)(want < most ? want : most)), dim3(kNormBlock), smem, st, a);
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
                            float* rstd, unsigned* err, cudaStream_t st) {
    if (rows == 0) return cudaSuccess;
    const NormFwdArgs a{x, weight, bias, y, mean, rstd, rows, x_stride, y_stride, cols, wdtype, eps, err};
    if (dtype == GS_DTYPE_F32) return run_typed<float>(a, st);
    if (dtype == GS_DTYPE_F16) return run_typed<__half>(a, st);
    return run_typed<__nv_bfloat16>(a, st);
}

}  // namespace gs
