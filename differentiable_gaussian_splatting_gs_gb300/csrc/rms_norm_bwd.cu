// Root-mean-square norm, backward. With hhat = h rstd and g = w dy, per row
//   dx = rstd (g - hhat mean(g hhat)) + dh,
// the gradient of x and of the residual alike (dh: h's own gradient, from what reads the sum besides the norm), and over
// the rows dw = sum dy hhat.
//
// Bound by memory: h, dy and dh are read once, dx is written once. As the layer norm's backward: a row's elements and the
// thread's columns of dw stay in registers, the grid is persistent, a block leaves its sums in the workspace and a
// second kernel adds the blocks', all in a fixed order; rows of more than a vector per thread come through the ring. Times in a graph:
// 139,072 x 1024 bfloat16 with dh 164 us (7.0 TB/s: the L2 keeps the end of what is written), 20,001 x 333 float16 12.7 us.
#include <algorithm>

#include "rms_norm.cuh"

namespace gs {

struct RmsBwdArgs {
    const void *dy, *h, *dh, *weight;
    const float* rstd;
    void* dx;
    float* part;  // [blocks][cols]: each block's share of dw
    long long rows, dy_stride, h_stride, dh_stride, dx_stride;
    int cols, wdtype;
    unsigned* err;
};

// Blocks of an SM at least (0: as the registers come out; 1 leaves the compiler more of them than that), where that was faster: rows of one
// vector to a thread (200,000 x 128 float16 41 us, so 35; with dh 46, 42), and few single elements without dh (200,000 x 135 bfloat16
// 57 us, so 50; with dh 60, and 65 so). Rows of a whole warp with dh would
// spill, and of 8 lanes and fewer there was nothing to gain (200,000 x 64 bfloat16 15 us, and 17 so).
template <int VEC, int NV, int LPR, bool DH>
constexpr int kRmsBwdBlocks = NV * VEC >= 12 && NV * VEC <= 16 ? 2 : VEC > 1 && NV == 1 && (LPR == 16 || (LPR == 32 && !DH)) ? 3 : VEC == 1 && NV <= 8 && !DH ? 0 : 1;

template <class T, int VEC, int NV, int LPR, int FULL, bool DH>
__global__ void __launch_bounds__(kNormBlock, kRmsBwdBlocks<VEC, NV, LPR, DH>) k_rms_bwd(const RmsBwdArgs a) {
    pdl_entry();
    extern __shared__ __align__(16) float share[];  // w; at the end the block's sums
    __shared__ float buf[2 * kNormBlock / 32];
    int phase = 0;
    constexpr int kRows = kNormBlock / LPR;
    const int l = threadIdx.x % LPR, nvec = a.cols / VEC;
    const float inv = 1.f / (float)a.cols;
    float dw[NV][VEC];
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int k = 0; k < VEC; ++k) dw[i][k] = 0.f;
    auto in = [&](int i) { return i < FULL || l + i * LPR < nvec; };
    stage_weights<VEC>(share, a.weight, a.wdtype, a.cols, 1.f);
    __syncthreads();
    const T *h = static_cast<const T*>(a.h), *dy = static_cast<const T*>(a.dy), *dh = static_cast<const T*>(a.dh);
    T* dx = static_cast<T*>(a.dx);
    const long long step = (long long)gridDim.x * kRows;
    constexpr bool kRing = norm_ring<VEC, NV, LPR>;
    constexpr int kArrays = DH ? 3 : 2, kStages = norm_stages<NV, LPR>;
    __shared__ uint64_t bars[kRing ? kRows * kStages : 1];
    NormRing<kArrays, kRing ? LPR : 32, kStages> ring;
    const long long first = (long long)blockIdx.x * kRows + threadIdx.x / LPR;
    if constexpr (kRing) {
        init_ring_bars<kRows * kStages>(bars);
        ring.src[0] = reinterpret_cast<const char*>(h);
        ring.src[1] = reinterpret_cast<const char*>(dy);
        ring.stride[0] = a.h_stride * (long long)sizeof(T);
        ring.stride[1] = a.dy_stride * (long long)sizeof(T);
        if constexpr (DH) {
            ring.src[2] = reinterpret_cast<const char*>(dh);
            ring.stride[2] = a.dh_stride * (long long)sizeof(T);
        }
        ring.start(reinterpret_cast<unsigned char*>(share + (a.cols + 3) / 4 * 4), bars, a.cols, sizeof(T), first, a.rows, step,
                   kNormSpin, a.err);
    }
    float next_r = first < a.rows ? a.rstd[first] : 0.f;
    // Of the other rows those of one vector to a thread are loaded a turn ahead (200,000 x 64 bfloat16 with dh: 28.9 us without, 22.6
    // so); rows read an element at a time have no registers for it (60,000 x 1001 float32 with dh: 146 us without, 214 so).
    constexpr bool kAhead = !kRing && (VEC > 1 || NV <= 4);
    Pack<T, VEC> nh[kAhead ? NV : 1], nd[kAhead ? NV : 1], ne[kAhead && DH ? NV : 1];
    auto ask = [&](long long row) {
        if constexpr (kAhead) {
            load_row<T, VEC, NV, LPR, FULL>(nh, h + row * a.h_stride, l, nvec, row < a.rows);
            load_row<T, VEC, NV, LPR, FULL>(nd, dy + row * a.dy_stride, l, nvec, row < a.rows);
            if constexpr (DH) load_row<T, VEC, NV, LPR, FULL>(ne, dh + row * a.dh_stride, l, nvec, row < a.rows);
        }
    };
    ask(first);
    for (long long base = (long long)blockIdx.x * kRows; base < a.rows; base += step) {
        const long long row = base + threadIdx.x / LPR;
        const bool live = row < a.rows;
        if (LPR >= 32 && !live) break;  // the same in all threads of the row
        const float r = next_r;
        if (row + step < a.rows) next_r = a.rstd[row + step];
        Pack<T, VEC> rh[NV], rd[NV], re[DH ? NV : 1];
        if constexpr (kRing) {
            if (live) {
                ring.wait();
                load_row<T, VEC, NV, LPR, FULL>(rh, reinterpret_cast<const T*>(ring.at(0)), l, nvec, true);
                load_row<T, VEC, NV, LPR, FULL>(rd, reinterpret_cast<const T*>(ring.at(1)), l, nvec, true);
                if constexpr (DH) load_row<T, VEC, NV, LPR, FULL>(re, reinterpret_cast<const T*>(ring.at(kArrays - 1)), l, nvec, true);
            }
        } else if constexpr (kAhead) {
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                rh[i] = nh[i];
                rd[i] = nd[i];
                if constexpr (DH) re[i] = ne[i];
            }
            ask(row + step);
        } else {
            load_row<T, VEC, NV, LPR, FULL>(rh, h + row * a.h_stride, l, nvec, live);
            load_row<T, VEC, NV, LPR, FULL>(rd, dy + row * a.dy_stride, l, nvec, live);
            if constexpr (DH) load_row<T, VEC, NV, LPR, FULL>(re, dh + row * a.dh_stride, l, nvec, live);
        }
        // hhat and w dy of a 16-bit row, or of one read an element at a time, stay as floats (as in the layer norm's backward)
        constexpr bool kKeep = VEC == 1 || sizeof(T) == 2;
        float hh[kKeep ? NV : 1][VEC], g[kKeep ? NV : 1][VEC], s[1] = {0.f};
        auto form = [&](int i, float (&hi)[VEC], float (&gi)[VEC], float (&d)[VEC]) {
            load_floats<VEC>(gi, share, l + i * LPR, nvec);
            unpack<T, VEC>(rh[i], hi);
            unpack<T, VEC>(rd[i], d);
#pragma unroll
            for (int k = 0; k < VEC; ++k) {
                hi[k] *= r;
                gi[k] *= d[k];
            }
        };
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (live && in(i)) {
                float d[VEC];
                auto &hi = hh[kKeep ? i : 0], &gi = g[kKeep ? i : 0];
                form(i, hi, gi, d);
#pragma unroll
                for (int k = 0; k < VEC; ++k) {
                    dw[i][k] = fmaf(d[k], hi[k], dw[i][k]);
                    s[0] = fmaf(gi[k], hi[k], s[0]);
                }
            }
        row_sum<LPR>(s, buf, phase);
        if (!live) continue;
        if constexpr (kRing) {
            __syncwarp();
            ring.next();
        }
        const float c = -s[0] * inv * r;
        T* to = dx + row * a.dx_stride + l * VEC;
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (in(i)) {
                float o[VEC], e[VEC];
                auto &hi = hh[kKeep ? i : 0], &gi = g[kKeep ? i : 0];
                if (!kKeep) form(i, hi, gi, o);
                if constexpr (DH) unpack<T, VEC>(re[i], e);
#pragma unroll
                for (int k = 0; k < VEC; ++k) o[k] = fmaf(gi[k], r, DH ? fmaf(hi[k], c, e[k]) : hi[k] * c);
                *reinterpret_cast<Pack<T, VEC>*>(to + i * LPR * VEC) = repack<T, VEC>(o);
            }
    }
    if constexpr (kRing) ring.finish();
    if (!a.part) return;
    // the rows' threads one after the other
#pragma unroll 1
    for (int r = 0; r < kRows; ++r) {
        __syncthreads();
        if ((int)threadIdx.x / LPR != r) continue;
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (in(i)) {
                if (r > 0) {
                    float u[VEC];
                    load_floats<VEC>(u, share, l + i * LPR, nvec);
#pragma unroll
                    for (int k = 0; k < VEC; ++k) dw[i][k] = u[k] + dw[i][k];
                }
                store_floats<VEC>(dw[i], share, l + i * LPR, nvec);
            }
    }
    __syncthreads();
    float* part = a.part + (size_t)blockIdx.x * a.cols;
    for (int c = threadIdx.x; c < a.cols; c += kNormBlock) part[c] = share[plane_at<VEC>(c, nvec)];
}

// Rows of more than kNormMaxCols elements: a block per row for dx, which reads the row twice. (2000 x 20,000 with dh: bfloat16 155 us,
// float32 190; an element at a time 360 and 337.)
template <class T, int VEC, bool DH>
__global__ void __launch_bounds__(kNormBlock) k_rms_bwd_long(const RmsBwdArgs a) {
    pdl_entry();
    __shared__ float buf[2 * kNormBlock / 32];
    int phase = 0;
    for (long long row = blockIdx.x; row < a.rows; row += gridDim.x) {
        const T *h = static_cast<const T*>(a.h) + row * a.h_stride, *dy = static_cast<const T*>(a.dy) + row * a.dy_stride;
        const T* dh = static_cast<const T*>(a.dh) + (DH ? row * a.dh_stride : 0);
        T* dx = static_cast<T*>(a.dx) + row * a.dx_stride;
        const float rstd = a.rstd[row];
        Pack<T, VEC> ph[kLongLoads], pd[kLongLoads], pe[DH ? kLongLoads : 1];
        float s[1] = {0.f}, u[VEC], v[VEC], w[VEC];
        for (int c0 = 0; c0 < a.cols; c0 += kLongTurn<VEC>) {
            load_long<T, VEC>(ph, h, c0, a.cols);
            load_long<T, VEC>(pd, dy, c0, a.cols);
#pragma unroll
            for (int j = 0; j < kLongLoads; ++j) {
                if (long_at<VEC>(c0, j) >= a.cols) continue;
                load_weights<VEC>(w, a.weight, a.wdtype, long_at<VEC>(c0, j));
                unpack<T, VEC>(ph[j], u);
                unpack<T, VEC>(pd[j], v);
#pragma unroll
                for (int k = 0; k < VEC; ++k) s[0] = fmaf(v[k] * w[k], u[k] * rstd, s[0]);
            }
        }
        row_sum<kNormBlock>(s, buf, phase);
        const float m = s[0] / (float)a.cols;
        for (int c0 = 0; c0 < a.cols; c0 += kLongTurn<VEC>) {
            load_long<T, VEC>(ph, h, c0, a.cols);
            load_long<T, VEC>(pd, dy, c0, a.cols);
            if constexpr (DH) load_long<T, VEC>(pe, dh, c0, a.cols);
#pragma unroll
            for (int j = 0; j < kLongLoads; ++j) {
                const int c = long_at<VEC>(c0, j);
                if (c >= a.cols) continue;
                float e[VEC];
                load_weights<VEC>(w, a.weight, a.wdtype, c);
                unpack<T, VEC>(ph[j], u);
                unpack<T, VEC>(pd[j], v);
                if constexpr (DH) unpack<T, VEC>(pe[j], e);
#pragma unroll
                for (int k = 0; k < VEC; ++k) v[k] = fmaf(rstd, v[k] * w[k] - u[k] * rstd * m, DH ? e[k] : 0.f);
                *reinterpret_cast<Pack<T, VEC>*>(dx + c) = repack<T, VEC>(v);
            }
        }
    }
}

// ... and, before it, dw of such rows: VEC columns to a thread over the block's share of the rows.
template <class T, int VEC>
__global__ void __launch_bounds__(kNormBlock) k_rms_bwd_long_cols(const RmsBwdArgs a) {
    pdl_entry();
    const int c = (blockIdx.x * kNormBlock + threadIdx.x) * VEC;
    if (c >= a.cols) return;
    const long long per = (a.rows + gridDim.y - 1) / gridDim.y, r0 = blockIdx.y * per;
    const long long r1 = r0 + per < a.rows ? r0 + per : a.rows;
    const T *h = static_cast<const T*>(a.h) + c, *dy = static_cast<const T*>(a.dy) + c;
    float dw[VEC];
#pragma unroll
    for (int k = 0; k < VEC; ++k) dw[k] = 0.f;
#pragma unroll 4
    for (long long r = r0; r < r1; ++r) {
        const float rstd = a.rstd[r];
        float u[VEC], v[VEC];
        unpack<T, VEC>(*reinterpret_cast<const Pack<T, VEC>*>(h + r * a.h_stride), u);
        unpack<T, VEC>(*reinterpret_cast<const Pack<T, VEC>*>(dy + r * a.dy_stride), v);
#pragma unroll
        for (int k = 0; k < VEC; ++k) dw[k] = fmaf(v[k], u[k] * rstd, dw[k]);
    }
    float* part = a.part + (size_t)blockIdx.y * a.cols + c;
#pragma unroll
    for (int k = 0; k < VEC; ++k) part[k] = dw[k];
}

// dw = the sum of the blocks' shares: 32 columns to a block, whose 32 warps take the shares in turn, in order.
__global__ void __launch_bounds__(1024) k_rms_bwd_sum(const float* part, int blocks, int cols, void* dweight, int wdtype) {
    pdl_entry();
    __shared__ float share[32][33];
    const int lane = threadIdx.x & 31, c = blockIdx.x * 32 + lane, s = threadIdx.x >> 5;
    float t = 0.f;
    if (c < cols) {
#pragma unroll 8
        for (int b = s; b < blocks; b += 32) t += part[(size_t)b * cols + c];
    }
    share[s][lane] = t;
    __syncthreads();
    t = share[lane][s];  // a warp per column
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
    const int col = blockIdx.x * 32 + s;
    if (lane == 0 && col < cols) store_elem(dweight, col, wdtype, t);
}

namespace {

constexpr int kMaxShares = 1024;  // blocks that leave a share of dw in the workspace

long long shares(long long rows) { return rows < kMaxShares ? rows : kMaxShares; }

template <class T, int VEC, bool DH>
cudaError_t run(const RmsBwdArgs& a, int* blocks, cudaStream_t st) {
    return norm_dispatch<VEC, VEC == 8 ? 2 : 4>(a.cols / VEC, [&](auto shape) {
        using S = decltype(shape);
        constexpr int kRows = kNormBlock / S::LPR;
        static std::atomic<int> cache[256] = {};
        auto* kernel = k_rms_bwd<T, VEC, S::NV, S::LPR, S::FULL, DH>;
        constexpr bool kRing = norm_ring<VEC, S::NV, S::LPR>;
        auto smem_of = [&](int cols) {
            return (cols + 3) / 4 * 4 * sizeof(float) +
                   (kRing ? NormRing<DH ? 3 : 2, kRing ? S::LPR : 32, norm_stages<S::NV, S::LPR>>::smem(cols, sizeof(T)) : 0);
        };
        const int kMost = (int)smem_of(S::NV * S::LPR * VEC);
        if (kMost > 48 * 1024) {
            cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMost);
            if (e) return e;
        }
        int most = resident_blocks(kernel, kNormBlock, kMost, cache);
        if (most > kMaxShares) most = kMaxShares;
        const long long want = (a.rows + kRows - 1) / kRows;
        *blocks = (int)(want < most ? want : most);
        count_launches(1);
        return launch_pdl(kernel, dim3((unsigned)*blocks), dim3(kNormBlock), smem_of(a.cols), st, a);
    });
}

template <class T, int VEC, bool DH>
cudaError_t run_long(const RmsBwdArgs& a, int* blocks, cudaStream_t st) {
    if (a.part) {  // first: dx may overwrite dy or h
        const int across = (int)((a.cols + (long long)kNormBlock * VEC - 1) / (kNormBlock * VEC));
        const long long up = 8 * device_sm_count() / across;  // two thousand threads to an SM
        *blocks = (int)std::min(shares(a.rows), up > 64 ? up : 64);
        count_launches(1);
        const cudaError_t e = launch_pdl(k_rms_bwd_long_cols<T, VEC>, dim3(across, *blocks), dim3(kNormBlock), 0, st, a);
        if (e) return e;
    }
    static std::atomic<int> cache[256] = {};
    auto* kernel = k_rms_bwd_long<T, VEC, DH>;
    const int most = resident_blocks(kernel, kNormBlock, 0, cache);
    count_launches(1);
    return launch_pdl(kernel, dim3((unsigned)(a.rows < most ? a.rows : most)), dim3(kNormBlock), 0, st, a);
}

template <class T, int VEC>
cudaError_t run_vec(const RmsBwdArgs& a, int* blocks, cudaStream_t st) {
    if (a.cols > kNormMaxCols) return a.dh ? run_long<T, VEC, true>(a, blocks, st) : run_long<T, VEC, false>(a, blocks, st);
    return a.dh ? run<T, VEC, true>(a, blocks, st) : run<T, VEC, false>(a, blocks, st);
}

template <class T>
cudaError_t run_typed(const RmsBwdArgs& a, int* blocks, cudaStream_t st) {
    constexpr int V = 16 / (int)sizeof(T);
    auto fine = [](const void* p, long long stride) { return !p || (stride % V == 0 && reinterpret_cast<uintptr_t>(p) % 16 == 0); };
    const bool vec = a.cols % V == 0 && fine(a.h, a.h_stride) && fine(a.dy, a.dy_stride) && fine(a.dx, a.dx_stride) && fine(a.dh, a.dh_stride) &&
                     (a.cols <= kNormMaxCols || fine(a.weight, 0));
    return vec ? run_vec<T, V>(a, blocks, st) : run_vec<T, 1>(a, blocks, st);
}

}  // namespace

size_t rms_bwd_workspace_bytes(long long rows, int cols) { return (size_t)shares(rows) * cols * sizeof(float); }

cudaError_t launch_rms_bwd(int dtype, const RmsTensors& t, const void* dy, long long dy_stride, const void* dh, long long dh_stride,
                           long long rows, int cols, int wdtype, void* dx, long long dx_stride, void* dweight, float* workspace,
                           unsigned* err, cudaStream_t st) {
    const RmsBwdArgs a{dy, t.h, dh, t.weight, t.rstd, dx, dweight ? workspace : nullptr, rows, dy_stride, t.h_stride, dh_stride, dx_stride,
                       cols, wdtype, err};
    int blocks = 0;
    cudaError_t e = cudaSuccess;
    if (rows > 0) {
        if (dtype == GS_DTYPE_F32) e = run_typed<float>(a, &blocks, st);
        else if (dtype == GS_DTYPE_F16) e = run_typed<__half>(a, &blocks, st);
        else e = run_typed<__nv_bfloat16>(a, &blocks, st);
    }
    if (e || !dweight) return e;
    count_launches(1);
    return launch_pdl(k_rms_bwd_sum, dim3((unsigned)((cols + 31) / 32)), dim3(1024), 0, st, (const float*)workspace, blocks, cols, dweight, wdtype);
}

}  // namespace gs
