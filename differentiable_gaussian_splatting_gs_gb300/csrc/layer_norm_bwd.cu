// Layer norm, backward. With xhat = (x - mean) rstd and g = w dy, per row
//   dx = rstd (g - mean(g) - xhat mean(g xhat)),
// and over the rows dw = sum dy xhat, db = sum dy.
//
// Bound by memory: x and dy are read once, dx is written once. A row's elements stay in registers, and
// so do the thread's columns of dw and db: the grid is persistent, each thread adds up the rows it
// meets, the block adds its threads' sums in shared memory and leaves them in the workspace, and a
// second kernel adds the blocks'. All in a fixed order, so the same call gives the same bits. The sums leave
// no registers for loads ahead: rows of more than a vector per thread come through shared memory (NormRing).
#include "layer_norm.cuh"

namespace gs {

struct NormBwdArgs {
    const void *dy, *x, *weight;
    const float *mean, *rstd;
    void* dx;
    float* part;  // [blocks][2][cols]: each block's share of dw and db
    long long rows, dy_stride, x_stride, dx_stride;
    int cols, wdtype;
    unsigned* err;
};

template <class T, int VEC, int NV, int LPR, int FULL>
__global__ void __launch_bounds__(kNormBlock, NV * VEC >= 12 && NV * VEC <= 16 ? 2 : 1) k_norm_bwd(const NormBwdArgs a) {
    pdl_entry();
    extern __shared__ __align__(16) float share[];  // w; at the end the block's sums, 2 x cols
    __shared__ float buf[2 * 2 * kNormBlock / 32];
    int phase = 0;
    constexpr int kRows = kNormBlock / LPR;
    const int l = threadIdx.x % LPR, nvec = a.cols / VEC;
    const float inv = 1.f / (float)a.cols;
    float dw[NV][VEC], db[NV][VEC];
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int k = 0; k < VEC; ++k) dw[i][k] = db[i][k] = 0.f;
    auto in = [&](int i) { return i < FULL || l + i * LPR < nvec; };
    stage_weights<VEC>(share, a.weight, a.wdtype, a.cols, 1.f);
    __syncthreads();
    const T *x = static_cast<const T*>(a.x), *dy = static_cast<const T*>(a.dy);
    T* dx = static_cast<T*>(a.dx);
    const long long step = (long long)gridDim.x * kRows;
    constexpr bool kRing = norm_ring<VEC, NV, LPR>;
    constexpr int kStages = norm_stages<NV, LPR>;
    __shared__ uint64_t bars[kRing ? kRows * kStages : 1];
    NormRing<2, kRing ? LPR : 32, kStages> ring;
    if constexpr (kRing) {
        init_ring_bars<kRows * kStages>(bars);
        ring.src[0] = reinterpret_cast<const char*>(x);
        ring.src[1] = reinterpret_cast<const char*>(dy);
        ring.stride[0] = a.x_stride * (long long)sizeof(T);
        ring.stride[1] = a.dy_stride * (long long)sizeof(T);
        ring.start(reinterpret_cast<unsigned char*>(share + 2 * a.cols), bars, a.cols, sizeof(T),
                   (long long)blockIdx.x * kRows + threadIdx.x / LPR, a.rows, step, kNormSpin, a.err);
    }
    const long long first = (long long)blockIdx.x * kRows + threadIdx.x / LPR;
    float next_m = first < a.rows ? a.mean[first] : 0.f, next_r = first < a.rows ? a.rstd[first] : 0.f;
    for (long long base = (long long)blockIdx.x * kRows; base < a.rows; base += step) {
        const long long row = base + threadIdx.x / LPR;
        const bool live = row < a.rows;
        if (LPR >= 32 && !live) break;  // the same in all threads of the row
        const float m = next_m, r = next_r;
        if (row + step < a.rows) {
            next_m = a.mean[row + step];
            next_r = a.rstd[row + step];
        }
        Pack<T, VEC> rx[NV], rd[NV];
        if constexpr (kRing) {
            if (live) {
                ring.wait();
                load_row<T, VEC, NV, LPR, FULL>(rx, reinterpret_cast<const T*>(ring.at(0)), l, nvec, true);
                load_row<T, VEC, NV, LPR, FULL>(rd, reinterpret_cast<const T*>(ring.at(1)), l, nvec, true);
            }
        } else {
            load_row<T, VEC, NV, LPR, FULL>(rx, x + row * a.x_stride, l, nvec, live);
            load_row<T, VEC, NV, LPR, FULL>(rd, dy + row * a.dy_stride, l, nvec, live);
        }
        // xhat and w dy of a 16-bit row, or of one read an element at a time, stay as floats: 139,072 x 1024 bfloat16
        // takes 170 us when both are formed again for dx, 137 us so. Float32 vectors would take more registers than x and dy.
        constexpr bool kKeep = VEC == 1 || sizeof(T) == 2;
        float h[kKeep ? NV : 1][VEC], g[kKeep ? NV : 1][VEC], s[2] = {0.f, 0.f};
        auto form = [&](int i, float (&hi)[VEC], float (&gi)[VEC], float (&d)[VEC]) {
            load_floats<VEC>(gi, share, l + i * LPR, nvec);
            unpack<T, VEC>(rx[i], hi);
            unpack<T, VEC>(rd[i], d);
#pragma unroll
            for (int k = 0; k < VEC; ++k) {
                hi[k] = (hi[k] - m) * r;
                gi[k] *= d[k];
            }
        };
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (live && in(i)) {
                float d[VEC];
                auto &hi = h[kKeep ? i : 0], &gi = g[kKeep ? i : 0];
                form(i, hi, gi, d);
#pragma unroll
                for (int k = 0; k < VEC; ++k) {
                    dw[i][k] = fmaf(d[k], hi[k], dw[i][k]);
                    db[i][k] += d[k];
                    s[0] += gi[k];
                    s[1] = fmaf(gi[k], hi[k], s[1]);
                }
            }
        row_sum<LPR>(s, buf, phase);
        if (!live) continue;
        if constexpr (kRing) {
            __syncwarp();
            ring.next();
        }
        // rstd (g - mean(g) - xhat mean(g xhat))
        const float c0 = -s[0] * inv * r, c1 = -s[1] * inv * r;
        T* to = dx + row * a.dx_stride + l * VEC;
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (in(i)) {
                float o[VEC];
                auto &hi = h[kKeep ? i : 0], &gi = g[kKeep ? i : 0];
                if (!kKeep) form(i, hi, gi, o);
#pragma unroll
                for (int k = 0; k < VEC; ++k) o[k] = fmaf(gi[k], r, fmaf(hi[k], c1, c0));
                *reinterpret_cast<Pack<T, VEC>*>(to + i * LPR * VEC) = repack<T, VEC>(o);
            }
    }
    if constexpr (kRing) ring.finish();
    if (!a.part) return;
    float* part = a.part + (size_t)blockIdx.x * 2 * a.cols;
    // the rows' threads one after the other
#pragma unroll 1
    for (int r = 0; r < kRows; ++r) {
        __syncthreads();
        if ((int)threadIdx.x / LPR != r) continue;
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (in(i)) {
                if (r > 0) {
                    float u[VEC], v[VEC];
                    load_floats<VEC>(u, share, l + i * LPR, nvec);
                    load_floats<VEC>(v, share + a.cols, l + i * LPR, nvec);
#pragma unroll
                    for (int k = 0; k < VEC; ++k) {
                        dw[i][k] = u[k] + dw[i][k];
                        db[i][k] = v[k] + db[i][k];
                    }
                }
                store_floats<VEC>(dw[i], share, l + i * LPR, nvec);
                store_floats<VEC>(db[i], share + a.cols, l + i * LPR, nvec);
            }
    }
    __syncthreads();
    for (int c = threadIdx.x; c < a.cols; c += kNormBlock) {
        part[c] = share[plane_at<VEC>(c, nvec)];
        part[a.cols + c] = share[a.cols + plane_at<VEC>(c, nvec)];
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

// ... and, before it, dw and db of such rows: a thread per column over the block's share of the rows.
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

// dw, db = the sums of the blocks' shares: 32 columns to a block, whose 32 warps take the shares in turn, in order.
__global__ void __launch_bounds__(1024) k_norm_bwd_sum(const float* part, int blocks, int cols, void* dweight, void* dbias,
                                                       int wdtype) {
    pdl_entry();
    __shared__ float share[32][33];
    const int c = blockIdx.x * 32 + (threadIdx.x & 31), s = threadIdx.x >> 5;  // c counts dw's columns, then db's
    float t = 0.f;
    if (c < 2 * cols) {
#pragma unroll 8
        for (int b = s; b < blocks; b += 32) t += part[(size_t)b * 2 * cols + c];
    }
    share[s][threadIdx.x & 31] = t;
    __syncthreads();
    t = share[threadIdx.x & 31][s];  // a warp per column
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
    const int col = blockIdx.x * 32 + s;
    if ((threadIdx.x & 31) != 0 || col >= 2 * cols) return;
    if (col < cols) {
        if (dweight) store_elem(dweight, col, wdtype, t);
    } else if (dbias) {
        store_elem(dbias, col - cols, wdtype, t);
    }
}

namespace {

constexpr int kMaxShares = 1024;  // blocks that leave a share of dw and db in the workspace

long long shares(long long rows) { return rows < kMaxShares ? rows : kMaxShares; }

template <class T, int VEC>
cudaError_t run(const NormBwdArgs& a, int* blocks, cudaStream_t st) {
    // 16 elements a thread. 139,072 x 1024 bfloat16: 137 us; with 32 (two sums each leave registers for 8 warps an
    // SM) and with 8 (a barrier of four warps for each row) 1.4 and 1.5 times as long
    return norm_dispatch<VEC, VEC == 8 ? 2 : 4>(a.cols / VEC, [&](auto shape) {
        using S = decltype(shape);
        constexpr int kRows = kNormBlock / S::LPR;
        static std::atomic<int> cache[256] = {};
        auto* kernel = k_norm_bwd<T, VEC, S::NV, S::LPR, S::FULL>;
        constexpr bool kRing = norm_ring<VEC, S::NV, S::LPR>;
        auto smem_of = [&](int cols) {
            return 2 * cols * sizeof(float) + (kRing ? NormRing<2, kRing ? S::LPR : 32, norm_stages<S::NV, S::LPR>>::smem(cols, sizeof(T)) : 0);
        };
        const int kMost = (int)smem_of(S::NV * S::LPR * VEC);
        const size_t smem = smem_of(a.cols);
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
        if (a.part) {  // first: dx may overwrite dy or x
            *blocks = (int)(shares(a.rows) < 64 ? shares(a.rows) : 64);
            count_launches(1);
            const cudaError_t e = launch_pdl(k_norm_bwd_long_cols<T>, dim3((a.cols + kNormBlock - 1) / kNormBlock, *blocks), dim3(kNormBlock), 0, st, a);
            if (e) return e;
        }
        static std::atomic<int> cache[256] = {};
        const int most = resident_blocks(k_norm_bwd_long<T>, kNormBlock, 0, cache);
        count_launches(1);
        return launch_pdl(k_norm_bwd_long<T>, dim3((unsigned)(a.rows < most ? a.rows : most)), dim3(kNormBlock), 0, st, a);
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
                            unsigned* err, cudaStream_t st) {
    const bool sums = dweight || dbias;
    const NormBwdArgs a{dy, x, weight, mean, rstd, dx, sums ? workspace : nullptr, rows, dy_stride, x_stride, dx_stride, cols, wdtype, err};
    int blocks = 0;
    cudaError_t e = cudaSuccess;
    if (rows > 0) {
        if (dtype == GS_DTYPE_F32) e = run_typed<float>(a, &blocks, st);
        else if (dtype == GS_DTYPE_F16) e = run_typed<__half>(a, &blocks, st);
        else e = run_typed<__nv_bfloat16>(a, &blocks, st);
    }
    if (e || !sums) return e;
    count_launches(1);
    return launch_pdl(k_norm_bwd_sum, dim3((unsigned)((2ll * cols + 31) / 32)), dim3(1024), 0, st, (const float*)workspace, blocks,
                      cols, dweight, dbias, wdtype);
}

}  // namespace gs
