// Root-mean-square norm with the residual's addition, forward: h = x + r (rounded to the tensors' type), y = h rstd w
// with rstd = 1 / sqrt(mean of h^2 + eps); y in the tensors' type, or in 8 bits with a scale for each 128 columns (fp8.cuh).
//
// Bound by memory: x and r are read once, h and y written once. The layout is the layer norm's (layer_norm.cuh): a row
// stays in the registers of the threads it is laid over, the grid is persistent, weights lie in shared memory, rows of
// more than a vector per thread come through the ring of bulk copies. A block's 128 columns belong to neighbouring lanes of
// one warp, so that its maximum is a few shuffles. Times in a graph: 139,072 x 1024 bfloat16 with a residual 165 us to 8 bits
// (6.1 TB/s, 89% of the measured copy rate), 185 us to bfloat16; 1 x 1024 2.9 us (a call of its own 7 to 8, the host's); rows that do
// not lie on 16 bytes 4.3 to 5.3 TB/s in 16 bits, 6.1 to 6.6 in float32.
#include "rms_norm.cuh"

namespace gs {

struct RmsFwdArgs {
    const void *x, *r, *weight;
    void *h, *y;
    uint8_t* q;
    ScaleAt scale;
    float* rstd;
    long long rows, x_stride, r_stride, h_stride, y_stride;  // y_stride: of y or q
    int cols, wdtype;
    float eps;
    unsigned* err;
};

// Blocks of an SM at least (0: as the registers come out), where that was faster: of rows read an element at a time the longest (8000 x
// 8191 float16 with a residual 153 us, so 134; to 8 bits 202, 155), but for bfloat16 with a residual, which would spill (157 us, and 174
// so); and, without a residual, those of 12 and 16 to a thread (200,000 x 333 float16 57 us, so 53; with one 107, and 127 with a fourth
// block).
template <class T, int VEC, int NV, bool RES>
constexpr int kRmsFwdBlocks = VEC > 1 ? 0 : NV > 16 ? RES && std::is_same_v<T, __nv_bfloat16> ? 0 : 2 : NV >= 12 && !RES ? 3 : 0;

template <class T, int VEC, int NV, int LPR, int FULL, bool RES>
__global__ void __launch_bounds__(kNormBlock, kRmsFwdBlocks<T, VEC, NV, RES>) k_rms_fwd(const RmsFwdArgs a) {
    pdl_entry();
    extern __shared__ __align__(16) float weights[];
    __shared__ float buf[2 * kNormBlock / 32];
    int phase = 0;
    constexpr int kRows = kNormBlock / LPR;  // rows of a block at a time
    const int l = threadIdx.x % LPR, nvec = a.cols / VEC;
    const float inv = 1.f / (float)a.cols;
    auto at = [&](int i) { return vec_at<VEC, NV, LPR>(l, i); };
    auto in = [&](int i) { return i < FULL || at(i) < nvec; };
    const T *x = static_cast<const T*>(a.x), *r = static_cast<const T*>(a.r);
    const long long step = (long long)gridDim.x * kRows;
    long long base = (long long)blockIdx.x * kRows;  // uniform over the block: all lanes take part in the sums
    constexpr bool kRing = norm_ring<VEC, NV, LPR>;
    constexpr int kArrays = RES ? 2 : 1, kStages = norm_stages<NV, LPR>;
    Pack<T, VEC> raw[NV], add[RES ? NV : 1], next[NV], next_r[RES ? NV : 1];
    __shared__ uint64_t bars[kRing ? kRows * kStages : 1];
    NormRing<kArrays, kRing ? LPR : 32, kStages> ring;
    const long long first = base + threadIdx.x / LPR;
    if constexpr (kRing) {
        init_ring_bars<kRows * kStages>(bars);
        ring.src[0] = reinterpret_cast<const char*>(x);
        ring.stride[0] = a.x_stride * (long long)sizeof(T);
        if constexpr (RES) {
            ring.src[1] = reinterpret_cast<const char*>(r);
            ring.stride[1] = a.r_stride * (long long)sizeof(T);
        }
        ring.start(reinterpret_cast<unsigned char*>(weights + (a.cols + 3) / 4 * 4), bars, a.cols, sizeof(T), first, a.rows, step,
                   kNormSpin, a.err);
    } else {
        load_vecs<T, VEC, NV, LPR, FULL>(next, x + first * a.x_stride, l, nvec, first < a.rows);
        if constexpr (RES) load_vecs<T, VEC, NV, LPR, FULL>(next_r, r + first * a.r_stride, l, nvec, first < a.rows);
    }
    stage_weights<VEC>(weights, a.weight, a.wdtype, a.cols, 1.f);
    __syncthreads();
    for (; base < a.rows; base += step) {
        const long long row = base + threadIdx.x / LPR;
        const bool live = row < a.rows;
        if constexpr (kRing) {
            if (live) {
                ring.wait();
                load_vecs<T, VEC, NV, LPR, FULL>(raw, reinterpret_cast<const T*>(ring.at(0)), l, nvec, true);
                if constexpr (RES) load_vecs<T, VEC, NV, LPR, FULL>(add, reinterpret_cast<const T*>(ring.at(kArrays - 1)), l, nvec, true);
            }
        } else {
            const bool more = row + step < a.rows;
#pragma unroll
            for (int i = 0; i < NV; ++i) raw[i] = next[i];
            load_vecs<T, VEC, NV, LPR, FULL>(next, x + (row + step) * a.x_stride, l, nvec, more);
            if constexpr (RES) {
#pragma unroll
                for (int i = 0; i < NV; ++i) add[i] = next_r[i];
                load_vecs<T, VEC, NV, LPR, FULL>(next_r, r + (row + step) * a.r_stride, l, nvec, more);
            }
        }
        float f[VEC], t[2] = {0.f, 0.f};
        T* h = static_cast<T*>(a.h) + row * a.h_stride;
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (live && in(i)) {
                unpack<T, VEC>(raw[i], f);
                if constexpr (RES) {  // the norm is of h as it is stored, which the backward reads
                    float g[VEC];
                    unpack<T, VEC>(add[i], g);
#pragma unroll
                    for (int k = 0; k < VEC; ++k) f[k] += g[k];
                    raw[i] = repack<T, VEC>(f);
                    unpack<T, VEC>(raw[i], f);
                }
#pragma unroll
                for (int k = 0; k < VEC; ++k) t[(VEC == 1 ? i : k) & 1] = fmaf(f[k], f[k], t[(VEC == 1 ? i : k) & 1]);
            }
        float s[1] = {t[0] + t[1]};
        row_sum<LPR>(s, buf, phase);
        if (kRing && live) {
            __syncwarp();
            ring.next();
        }
        const float rstd = 1.f / sqrtf(s[0] * inv + a.eps);
        if constexpr (RES) {
#pragma unroll
            for (int i = 0; i < NV; ++i)
                if (live && in(i)) *reinterpret_cast<Pack<T, VEC>*>(h + at(i) * VEC) = raw[i];
        }
        if (live && l == 0) a.rstd[row] = rstd;
        auto norm = [&](int i) {
            float w[VEC];
            load_floats<VEC>(w, weights, at(i), nvec);
            unpack<T, VEC>(raw[i], f);
#pragma unroll
            for (int k = 0; k < VEC; ++k) f[k] *= rstd * w[k];
        };
        if (!a.q) {
            T* y = static_cast<T*>(a.y) + row * a.y_stride;
#pragma unroll
            for (int i = 0; i < NV; ++i)
                if (live && in(i)) {
                    norm(i);
                    *reinterpret_cast<Pack<T, VEC>*>(y + at(i) * VEC) = repack<T, VEC>(f);
                }
            continue;
        }
        uint8_t* q = a.q + row * a.y_stride;
        if constexpr (VEC > 1) {
            constexpr int kLanes = kQBlock / VEC < LPR ? kQBlock / VEC : LPR;
#pragma unroll
            for (int i = 0; i < NV; ++i) {  // all lanes take part in the shuffles
                const bool mine = live && in(i);
                unsigned top = 0;
                if (mine) {
                    norm(i);
#pragma unroll
                    for (int k = 0; k < VEC; ++k) top = max(top, magnitude(f[k]));
                }
                const float scale = block_scale(lanes_top<kLanes>(top));
                if (mine) {
                    const float back = scale_back(scale);
                    Pack<uint32_t, VEC / 4> out;
#pragma unroll
                    for (int k = 0; k < VEC; k += 4) out.v[k / 4] = quantize4(f[k], f[k + 1], f[k + 2], f[k + 3], back);
                    *reinterpret_cast<Pack<uint32_t, VEC / 4>*>(q + at(i) * VEC) = out;
                    if (l % kLanes == 0) a.scale.at(row, at(i) * VEC / kQBlock) = scale;
                }
            }
        } else {
            constexpr int kTurn = NV < 4 ? NV : 4;
#pragma unroll
            for (int i0 = 0; i0 < NV; i0 += kTurn) {
                float y[kTurn];
                unsigned top = 0;
#pragma unroll
                for (int j = 0; j < kTurn; ++j) {
                    y[j] = 0.f;
                    if (live && in(i0 + j)) {
                        norm(i0 + j);
                        y[j] = f[0];
                        top = max(top, magnitude(f[0]));
                    }
                }
                const float scale = block_scale(lanes_top<32>(top)), back = scale_back(scale);
#pragma unroll
                for (int j = 0; j < kTurn; ++j)
                    if (live && in(i0 + j)) q[at(i0 + j)] = quantize1(y[j], back);
                if (live && (l & 31) == 0 && at(i0) < nvec) a.scale.at(row, at(i0) / kQBlock) = scale;
            }
        }
    }
    if constexpr (kRing) ring.finish();
}

// Rows of more than kNormMaxCols elements: a block per row, which reads it again for y (from the L2 or the L1), or h, which
// each thread reads as it wrote it. (2000 x 20,000 with a residual: bfloat16 72 us, float32 113; an element at a time, one after the
// other, 190 and 285.)
template <class T, int VEC, bool RES>
__global__ void __launch_bounds__(kNormBlock) k_rms_fwd_long(const RmsFwdArgs a) {
    pdl_entry();
    __shared__ float buf[2 * kNormBlock / 32];
    int phase = 0;
    constexpr int kLanes = kQBlock / VEC < 32 ? kQBlock / VEC : 32;  // that share a scale
    for (long long row = blockIdx.x; row < a.rows; row += gridDim.x) {
        const T *x = static_cast<const T*>(a.x) + row * a.x_stride, *r = static_cast<const T*>(a.r) + (RES ? row * a.r_stride : 0);
        T* h = static_cast<T*>(a.h) + (RES ? row * a.h_stride : 0);
        Pack<T, VEC> p[kLongLoads], add[RES ? kLongLoads : 1];
        float s[1] = {0.f}, f[VEC];
        for (int c0 = 0; c0 < a.cols; c0 += kLongTurn<VEC>) {
            load_long<T, VEC>(p, x, c0, a.cols);
            if constexpr (RES) load_long<T, VEC>(add, r, c0, a.cols);
#pragma unroll
            for (int j = 0; j < kLongLoads; ++j) {
                const int c = long_at<VEC>(c0, j);
                if (c >= a.cols) continue;
                unpack<T, VEC>(p[j], f);
                if constexpr (RES) {
                    float g[VEC];
                    unpack<T, VEC>(add[j], g);
#pragma unroll
                    for (int k = 0; k < VEC; ++k) f[k] += g[k];
                    p[j] = repack<T, VEC>(f);
                    *reinterpret_cast<Pack<T, VEC>*>(h + c) = p[j];
                    unpack<T, VEC>(p[j], f);
                }
#pragma unroll
                for (int k = 0; k < VEC; ++k) s[0] = fmaf(f[k], f[k], s[0]);
            }
        }
        row_sum<kNormBlock>(s, buf, phase);
        const float rstd = 1.f / sqrtf(s[0] / (float)a.cols + a.eps);
        if (threadIdx.x == 0) a.rstd[row] = rstd;
        for (int c0 = 0; c0 < a.cols; c0 += kLongTurn<VEC>) {
            load_long<T, VEC>(p, RES ? h : x, c0, a.cols);
            // the j-th y, and the largest of its magnitudes
            auto norm = [&](int j, float (&y)[VEC]) {
                const int c = long_at<VEC>(c0, j);
                unsigned top = 0;
                if (c < a.cols) {
                    float w[VEC];
                    load_weights<VEC>(w, a.weight, a.wdtype, c);
                    unpack<T, VEC>(p[j], y);
#pragma unroll
                    for (int k = 0; k < VEC; ++k) {
                        y[k] *= rstd * w[k];
                        top = max(top, magnitude(y[k]));
                    }
                }
                return top;
            };
            if (!a.q) {
#pragma unroll
                for (int j = 0; j < kLongLoads; ++j) {
                    norm(j, f);
                    if (long_at<VEC>(c0, j) < a.cols)
                        *reinterpret_cast<Pack<T, VEC>*>(static_cast<T*>(a.y) + row * a.y_stride + long_at<VEC>(c0, j)) = repack<T, VEC>(f);
                }
                continue;
            }
            uint8_t* q = a.q + row * a.y_stride;
            if constexpr (VEC == 1) {  // the four share a scale
                float y[kLongLoads][1];
                unsigned top = 0;
#pragma unroll
                for (int j = 0; j < kLongLoads; ++j) top = max(top, norm(j, y[j]));
                const float scale = block_scale(lanes_top<32>(top)), back = scale_back(scale);
                const int c = long_at<1>(c0, 0);
                if (threadIdx.x % 32 == 0 && c < a.cols) a.scale.at(row, c / kQBlock) = scale;
#pragma unroll
                for (int j = 0; j < kLongLoads; ++j)
                    if (c + 32 * j < a.cols) q[c + 32 * j] = quantize1(y[j][0], back);
            } else {
#pragma unroll
                for (int j = 0; j < kLongLoads; ++j) {  // all lanes take part in the shuffles
                    const int c = long_at<VEC>(c0, j);
                    const float scale = block_scale(lanes_top<kLanes>(norm(j, f))), back = scale_back(scale);
                    if (c >= a.cols) continue;
                    if (threadIdx.x % kLanes == 0) a.scale.at(row, c / kQBlock) = scale;
                    Pack<uint32_t, VEC / 4> out;
#pragma unroll
                    for (int k = 0; k < VEC; k += 4) out.v[k / 4] = quantize4(f[k], f[k + 1], f[k + 2], f[k + 3], back);
                    *reinterpret_cast<Pack<uint32_t, VEC / 4>*>(q + c) = out;
                }
            }
        }
    }
}

namespace {

template <class T, int VEC, bool RES>
cudaError_t run(const RmsFwdArgs& a, cudaStream_t st) {
    return norm_dispatch<VEC, VEC == 8 ? 4 : 8>(a.cols / VEC, [&](auto shape) {
        using S = decltype(shape);
        static std::atomic<int> cache[256] = {};
        auto* kernel = k_rms_fwd<T, VEC, S::NV, S::LPR, VEC == 1 || S::LPR == 256 ? S::FULL : 0, RES>;
        constexpr bool kRing = norm_ring<VEC, S::NV, S::LPR>;
        constexpr int kCols = S::NV * S::LPR * VEC;
        auto smem_of = [&](int cols) {
            return (cols + 3) / 4 * 4 * sizeof(float) +
                   (kRing ? NormRing<RES ? 2 : 1, kRing ? S::LPR : 32, norm_stages<S::NV, S::LPR>>::smem(cols, sizeof(T)) : 0);
        };
        const int kMost = (int)smem_of(kCols);
        if (kMost > 48 * 1024) {
            cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMost);
            if (e) return e;
        }
        const int most = resident_blocks(kernel, kNormBlock, kMost, cache);
        const long long want = (a.rows + kNormBlock / S::LPR - 1) / (kNormBlock / S::LPR);
        count_launches(1);
        return launch_pdl(kernel, dim3((unsigned)(want < most ? want : most)), dim3(kNormBlock), smem_of(a.cols), st, a);
    });
}

template <class T, int VEC, bool RES>
cudaError_t run_long(const RmsFwdArgs& a, cudaStream_t st) {
    static std::atomic<int> cache[256] = {};
    auto* kernel = k_rms_fwd_long<T, VEC, RES>;
    const int most = resident_blocks(kernel, kNormBlock, 0, cache);
    count_launches(1);
    return launch_pdl(kernel, dim3((unsigned)(a.rows < most ? a.rows : most)), dim3(kNormBlock), 0, st, a);
}

template <class T, int VEC>
cudaError_t run_vec(const RmsFwdArgs& a, cudaStream_t st) {
    if (a.cols > kNormMaxCols) return a.r ? run_long<T, VEC, true>(a, st) : run_long<T, VEC, false>(a, st);
    return a.r ? run<T, VEC, true>(a, st) : run<T, VEC, false>(a, st);
}

template <class T>
cudaError_t run_typed(const RmsFwdArgs& a, cudaStream_t st) {
    constexpr int V = 16 / (int)sizeof(T);
    // 16-byte accesses (8-bit results: as many elements at a time) when every row starts and ends on a whole one
    auto fine = [](const void* p, long long stride, int elems, int bytes) {
        return !p || (stride % elems == 0 && reinterpret_cast<uintptr_t>(p) % bytes == 0);
    };
    const bool vec = a.cols % V == 0 && fine(a.x, a.x_stride, V, 16) && fine(a.r, a.r_stride, V, 16) &&
                     (!a.r || fine(a.h, a.h_stride, V, 16)) && fine(a.y, a.y_stride, V, 16) && fine(a.q, a.y_stride, V, V) &&
                     (a.cols <= kNormMaxCols || fine(a.weight, 0, 1, 16));
    return vec ? run_vec<T, V>(a, st) : run_vec<T, 1>(a, st);
}

}  // namespace

cudaError_t launch_rms_fwd(int dtype, const RmsTensors& t, long long rows, int cols, int wdtype, float eps, unsigned* err, cudaStream_t st) {
    if (rows == 0) return cudaSuccess;
    const RmsFwdArgs a{t.x, t.r, t.weight, t.h, t.y, static_cast<uint8_t*>(t.q), {t.scale, t.scale_row, t.scale_block}, t.rstd,
                       rows, t.x_stride, t.r_stride, t.h_stride, t.q ? t.q_stride : t.y_stride, cols, wdtype, eps, err};
    if (dtype == GS_DTYPE_F32) return run_typed<float>(a, st);
    if (dtype == GS_DTYPE_F16) return run_typed<__half>(a, st);
    return run_typed<__nv_bfloat16>(a, st);
}

}  // namespace gs
