// Cross attention on the float32 pipes, for what the tensor-core kernels do not take: float32 heads above 128 (backward:
// above 64) and the backward of 16-bit heads above 128. Every stride, mask and length; products and sums in float32.
// Calls without a query or without a key, of any type, have only zeros (and an lse of -inf) to write.
//
// Forward: a block of 256 threads per 64 queries of a head. It walks the keys in tiles of 64 with the
// running maximum and sum of the softmax, so scores stay on chip. Backward: a block per 64 (heads above 128: 32) keys
// (dk, dv; walks the queries of all heads that share the key head) and one per as many queries (dq; walks
// the keys). Each output is summed by one block in a fixed order: no atomics, the same bits every time,
// at the price of forming S and dP twice. Bound by the reads of shared memory (69% of their rate) beside the multiply-adds
// (54%), with eight warps an SM: 2 x 8 heads of 128, 2000 x 2500 float32, backward 4.1 ms (4.7 in two
// launches; 5.7 with single multiply-adds and tiles staged an element at a time too).
#include "attention.cuh"

namespace gs {

namespace {

constexpr int kFM = 64, kFN = 64;  // tile of the forward kernel
// side of the backward kernels' tile: four operands' rows and two tiles of gradients share shared memory
template <int DP>
constexpr int kSide = DP <= 128 ? 64 : 32;
constexpr int kThreads = 256;

// rows x DP floats of shared memory (row stride DP + 4) from rows first .. of a head's tensor; rows that
// do not take part and columns from d on become 0.
template <class T, int DP, int ROWS, bool KEYS>
__device__ __forceinline__ void stage(float* dst, const AttnTensor& t, const AttnArgs& a, int b, int h, int first, int len) {
    const T* src = head_base<T>(t, b, h);
    constexpr int V = 16 / (int)sizeof(T), kVectors = ROWS * DP / V / kThreads;
    if (kVectors > 0 && a.d % V == 0 && t.len_stride % V == 0 && reinterpret_cast<uintptr_t>(src) % 16 == 0) {
        constexpr int kTurn = kVectors > 8 ? 8 : kVectors > 0 ? kVectors : 1;  // loads under way together
        static_assert(kVectors % kTurn == 0);
#pragma unroll 1
        for (int v0 = 0; v0 < kVectors; v0 += kTurn) {
            Pack<T, V> w[kTurn];
#pragma unroll
            for (int u = 0; u < kTurn; ++u) {
                const int e = (threadIdx.x + (v0 + u) * kThreads) * V, c = e % DP, row = first + e / DP;
                const bool in = c < a.d && (KEYS ? key_valid(a, b, row, len) : row < len);
#pragma unroll
                for (int k = 0; k < V; ++k) w[u].v[k] = from_float<T>(0.f);
                if (in) w[u] = *reinterpret_cast<const Pack<T, V>*>(src + row * t.len_stride + c);
            }
#pragma unroll
            for (int u = 0; u < kTurn; ++u) {
                const int e = (threadIdx.x + (v0 + u) * kThreads) * V;
#pragma unroll
                for (int k = 0; k < V; k += 4)
                    *reinterpret_cast<float4*>(dst + e / DP * (DP + 4) + e % DP + k) =
                        make_float4(to_float(w[u].v[k]), to_float(w[u].v[k + 1]), to_float(w[u].v[k + 2]), to_float(w[u].v[k + 3]));
            }
        }
        return;
    }
    constexpr int kBatch = 16;  // loads under way together
    static_assert(ROWS * DP % (kBatch * kThreads) == 0);
#pragma unroll 1
    for (int e0 = threadIdx.x; e0 < ROWS * DP; e0 += kBatch * kThreads) {
        float v[kBatch];
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            const int e = e0 + u * kThreads, c = e % DP, row = first + e / DP;
            const bool in = c < a.d && (KEYS ? key_valid(a, b, row, len) : row < len);
            v[u] = 0.f;
            if (in) v[u] = to_float(src[row * t.len_stride + c]);
        }
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            const int e = e0 + u * kThreads;
            dst[e / DP * (DP + 4) + e % DP] = v[u];
        }
    }
}

// acc[i][j] = row (ty * R + i) of x . row (tx + 16 j) of y; multiply-adds in pairs, of even and of odd elements.
template <int DP, int R, int C>
__device__ __forceinline__ void dots(const float* x, const float* y, int ty, int tx, float (&acc)[R][C]) {
    f32x2 sum[R][C];
#pragma unroll
    for (int i = 0; i < R; ++i)
#pragma unroll
        for (int j = 0; j < C; ++j) sum[i][j] = f2_pack(0.f, 0.f);
#pragma unroll 4
    for (int d = 0; d < DP; d += 4) {
        ulonglong2 u[R], v[C];
#pragma unroll
        for (int i = 0; i < R; ++i) u[i] = *reinterpret_cast<const ulonglong2*>(x + (ty * R + i) * (DP + 4) + d);
#pragma unroll
        for (int j = 0; j < C; ++j) v[j] = *reinterpret_cast<const ulonglong2*>(y + (tx + 16 * j) * (DP + 4) + d);
#pragma unroll
        for (int i = 0; i < R; ++i)
#pragma unroll
            for (int j = 0; j < C; ++j) sum[i][j] = f2_fma(u[i].x, v[j].x, f2_fma(u[i].y, v[j].y, sum[i][j]));
    }
#pragma unroll
    for (int i = 0; i < R; ++i)
#pragma unroll
        for (int j = 0; j < C; ++j) {
            const float2 t = f2_unpack(sum[i][j]);
            acc[i][j] = t.x + t.y;
        }
}

// A tile of probabilities or of dS: rows of N elements, each TWICE (a pair for f2_fma) where shared memory has the room.
template <int N, bool TWICE>
constexpr int kTileRow = (N + 4) * (TWICE ? 2 : 1);
template <int N, bool TWICE>
__device__ __forceinline__ void put(float* p, int row, int n, float v) {
    if (TWICE) *reinterpret_cast<float2*>(p + row * kTileRow<N, TWICE> + 2 * n) = make_float2(v, v);
    else p[row * kTileRow<N, TWICE> + n] = v;
}

// acc[i][m] += sum over n of p[ty * R + i][n] times elements 2 (tx + 16 m) and the next of y's row n (y: row stride DP + 4)
template <int DP, int N, bool TWICE, int R>
__device__ __forceinline__ void accumulate(const float* p, const float* y, int ty, int tx, f32x2 (&acc)[R][DP / 32]) {
#pragma unroll 1
    for (int n0 = 0; n0 < N; n0 += 4) {
        f32x2 u[R][4];
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const float* from = p + (ty * R + i) * kTileRow<N, TWICE> + n0 * (TWICE ? 2 : 1);
            if (TWICE) {
                const ulonglong2 w0 = *reinterpret_cast<const ulonglong2*>(from), w1 = *reinterpret_cast<const ulonglong2*>(from + 4);
                u[i][0] = w0.x, u[i][1] = w0.y, u[i][2] = w1.x, u[i][3] = w1.y;
            } else {
                const float4 w = *reinterpret_cast<const float4*>(from);
                u[i][0] = f2_pack(w.x, w.x), u[i][1] = f2_pack(w.y, w.y), u[i][2] = f2_pack(w.z, w.z), u[i][3] = f2_pack(w.w, w.w);
            }
        }
#pragma unroll
        for (int k = 0; k < 4; ++k)
#pragma unroll
            for (int m = 0; m < DP / 32; ++m) {
                const f32x2 v = *reinterpret_cast<const f32x2*>(y + (n0 + k) * (DP + 4) + 2 * (tx + 16 * m));
#pragma unroll
                for (int i = 0; i < R; ++i) acc[i][m] = f2_fma(u[i][k], v, acc[i][m]);
            }
    }
}

template <int DP, int R>
__device__ __forceinline__ void clear(f32x2 (&acc)[R][DP / 32]) {
#pragma unroll
    for (int i = 0; i < R; ++i)
#pragma unroll
        for (int m = 0; m < DP / 32; ++m) acc[i][m] = f2_pack(0.f, 0.f);
}

template <class T, int DP, int R>
__device__ __forceinline__ void store_rows(const AttnTensor& t, int d, int b, int h, int first, int len, int ty, int tx,
                                           const f32x2 (&acc)[R][DP / 32], const float (&f)[R]) {
    T* dst = static_cast<T*>(t.data) + b * t.batch_stride + h * t.head_stride;
#pragma unroll
    for (int i = 0; i < R; ++i) {
        const int row = first + ty * R + i;
        if (row >= len) continue;
#pragma unroll
        for (int m = 0; m < DP / 32; ++m) {
            const float2 v = f2_unpack(acc[i][m]);
            const int c = 2 * (tx + 16 * m);
            if (c < d) dst[row * t.len_stride + c] = from_float<T>(v.x * f[i]);
            if (c + 1 < d) dst[row * t.len_stride + c + 1] = from_float<T>(v.y * f[i]);
        }
    }
}

struct Where {
    int b, h, tile;
};
__device__ __forceinline__ Where where(int block, int tiles, int heads) {
    const int bh = block / tiles;
    return {bh / heads, bh % heads, block % tiles};
}

}  // namespace

template <class T, int DP>
__global__ void __launch_bounds__(kThreads) k_attn_fwd_simt(const AttnArgs a, int tiles) {
    pdl_entry();
    extern __shared__ float sm[];
    constexpr bool kTwice = false;  // heads of 256 leave no room for pairs
    float *sq = sm, *sk = sq + kFM * (DP + 4), *sv = sk + kFN * (DP + 4), *sp = sv + kFN * (DP + 4);
    const Where w = where(blockIdx.x, tiles, a.heads);
    const int hk = w.h / (a.heads / a.kv_heads), ty = threadIdx.x / 16, tx = threadIdx.x % 16;
    const int len = key_count(a, w.b);
    stage<T, DP, kFM, false>(sq, a.q, a, w.b, w.h, w.tile * kFM, a.len_q);
    f32x2 o[4][DP / 32];
    float top[4], sum[4];
    clear<DP>(o);
#pragma unroll
    for (int i = 0; i < 4; ++i) top[i] = -INFINITY, sum[i] = 0.f;
    for (int n0 = 0; n0 < len; n0 += kFN) {
        __syncthreads();
        stage<T, DP, kFN, true>(sk, a.k, a, w.b, hk, n0, len);
        stage<T, DP, kFN, true>(sv, a.v, a, w.b, hk, n0, len);
        __syncthreads();
        float s[4][4];
        dots<DP>(sq, sk, ty, tx, s);
        bool in[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) in[j] = key_valid(a, w.b, n0 + tx + 16 * j, len);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float m = top[i];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                s[i][j] = in[j] ? s[i][j] * a.scale : -INFINITY;
                m = fmaxf(m, s[i][j]);
            }
#pragma unroll
            for (int k = 8; k > 0; k >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, k));
            const float base = m == -INFINITY ? 0.f : m;  // no key so far: every term is exp(-inf) = 0
            const float keep = expf(top[i] - base);
            float t = 0.f;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float p = expf(s[i][j] - base);
                t += p;
                put<kFN, kTwice>(sp, ty * 4 + i, tx + 16 * j, p);
            }
#pragma unroll
            for (int k = 8; k > 0; k >>= 1) t += __shfl_xor_sync(0xffffffffu, t, k);
            sum[i] = sum[i] * keep + t;
            top[i] = m;
#pragma unroll
            for (int c = 0; c < DP / 32; ++c) o[i][c] = f2_mul(o[i][c], f2_pack(keep, keep));
        }
        __syncwarp();  // a row's probabilities are written and read by the same half warp
        accumulate<DP, kFN, kTwice>(sp, sv, ty, tx, o);
    }
    float f[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[i] = sum[i] == 0.f ? 0.f : 1.f / sum[i];
        const int row = w.tile * kFM + ty * 4 + i;
        if (tx == 0 && row < a.len_q)
            a.lse[((long long)w.b * a.heads + w.h) * a.len_q + row] = sum[i] == 0.f ? -INFINITY : top[i] + logf(sum[i]);
    }
    store_rows<T, DP>(a.out, a.d, w.b, w.h, w.tile * kFM, a.len_q, ty, tx, o, f);
}

// P and dS of a square tile (queries x keys, or transposed for the dk/dv kernel) into shared memory.
template <int DP, bool T_>
__device__ __forceinline__ void tile_gradient(const AttnArgs& a, const float* sq, const float* sdo, const float* sk, const float* sv,
                                              float* sp, float* sds, const float* lse, const float* delta, int b, int q0,
                                              int n0, int len, int ty, int tx) {
    constexpr int M = kSide<DP>, R = M / 16;
    float s[R][R], dp[R][R];
    dots<DP>(T_ ? sk : sq, T_ ? sq : sk, ty, tx, s);
    dots<DP>(T_ ? sv : sdo, T_ ? sdo : sv, ty, tx, dp);
#pragma unroll
    for (int i = 0; i < R; ++i)
#pragma unroll
        for (int j = 0; j < R; ++j) {
            const int r = ty * R + i, c = tx + 16 * j, qi = q0 + (T_ ? c : r), n = n0 + (T_ ? r : c);
            const bool in = qi < a.len_q && key_valid(a, b, n, len);
            const float p = in ? expf(s[i][j] * a.scale - lse[qi]) : 0.f;
            if (T_) put<M, true>(sp, r, c, p);
            put<M, true>(sds, r, c, in ? p * (dp[i][j] - delta[qi]) * a.scale : 0.f);
        }
}

template <class T, int DP>
__device__ __forceinline__ void dkv_block(const AttnArgs& a, int block, int tiles, float* sm) {
    constexpr int M = kSide<DP>, R = M / 16, kRow = M * (DP + 4);
    float *sk = sm, *sv = sk + kRow, *sq = sv + kRow, *sdo = sq + kRow, *sp = sdo + kRow, *sds = sp + M * kTileRow<M, true>;
    const Where w = where(block, tiles, a.kv_heads);
    const int share = a.heads / a.kv_heads, ty = threadIdx.x / 16, tx = threadIdx.x % 16, n0 = w.tile * M;
    const int len = key_count(a, w.b);
    f32x2 dk[R][DP / 32], dv[R][DP / 32];
    clear<DP>(dk);
    clear<DP>(dv);
    if (n0 < len) {
        stage<T, DP, M, true>(sk, a.k, a, w.b, w.h, n0, len);
        stage<T, DP, M, true>(sv, a.v, a, w.b, w.h, n0, len);
        for (int h = w.h * share; h < (w.h + 1) * share; ++h) {
            const long long row = ((long long)w.b * a.heads + h) * a.len_q;
            for (int q0 = 0; q0 < a.len_q; q0 += M) {
                __syncthreads();
                stage<T, DP, M, false>(sq, a.q, a, w.b, h, q0, a.len_q);
                stage<T, DP, M, false>(sdo, a.dout, a, w.b, h, q0, a.len_q);
                __syncthreads();
                tile_gradient<DP, true>(a, sq, sdo, sk, sv, sp, sds, a.lse + row, a.delta + row, w.b, q0, n0, len, ty, tx);
                __syncwarp();
                accumulate<DP, M, true>(sp, sdo, ty, tx, dv);
                accumulate<DP, M, true>(sds, sq, ty, tx, dk);
            }
        }
    }
    float one[R];
#pragma unroll
    for (int i = 0; i < R; ++i) one[i] = 1.f;
    store_rows<T, DP>(a.dk, a.d, w.b, w.h, n0, a.len_k, ty, tx, dk, one);
    store_rows<T, DP>(a.dv, a.d, w.b, w.h, n0, a.len_k, ty, tx, dv, one);
}

template <class T, int DP>
__device__ __forceinline__ void dq_block(const AttnArgs& a, int block, int tiles, float* sm) {
    constexpr int M = kSide<DP>, R = M / 16, kRow = M * (DP + 4);
    float *sk = sm, *sv = sk + kRow, *sq = sv + kRow, *sdo = sq + kRow, *sds = sdo + kRow;
    const Where w = where(block, tiles, a.heads);
    const int hk = w.h / (a.heads / a.kv_heads), ty = threadIdx.x / 16, tx = threadIdx.x % 16, q0 = w.tile * M;
    const int len = key_count(a, w.b);
    const long long row = ((long long)w.b * a.heads + w.h) * a.len_q;
    stage<T, DP, M, false>(sq, a.q, a, w.b, w.h, q0, a.len_q);
    stage<T, DP, M, false>(sdo, a.dout, a, w.b, w.h, q0, a.len_q);
    f32x2 dq[R][DP / 32];
    clear<DP>(dq);
    for (int n0 = 0; n0 < len; n0 += M) {
        __syncthreads();
        stage<T, DP, M, true>(sk, a.k, a, w.b, hk, n0, len);
        stage<T, DP, M, true>(sv, a.v, a, w.b, hk, n0, len);
        __syncthreads();
        tile_gradient<DP, false>(a, sq, sdo, sk, sv, nullptr, sds, a.lse + row, a.delta + row, w.b, q0, n0, len, ty, tx);
        __syncwarp();
        accumulate<DP, M, true>(sds, sk, ty, tx, dq);
    }
    float one[R];
#pragma unroll
    for (int i = 0; i < R; ++i) one[i] = 1.f;
    store_rows<T, DP>(a.dq, a.d, w.b, w.h, q0, a.len_q, ty, tx, dq, one);
}

// The dk, dv blocks, then the dq blocks, which fill the SMs that the others' last round leaves.
template <class T, int DP>
__global__ void __launch_bounds__(kThreads) k_attn_bwd_simt(const AttnArgs a, int tiles_k, int tiles_q) {
    pdl_entry();
    extern __shared__ float sm[];
    const int block = blockIdx.x, keys = tiles_k * a.kv_heads * a.batch;
    if (block < keys) dkv_block<T, DP>(a, block, tiles_k, sm);
    else dq_block<T, DP>(a, block - keys, tiles_q, sm);
}

// delta = sum over the head's elements of dout out, a warp per query and head.
template <class T>
__global__ void __launch_bounds__(kThreads) k_attn_delta(const AttnArgs a) {
    pdl_entry();
    const long long rows = (long long)a.batch * a.heads * a.len_q;
    const long long warp = ((long long)blockIdx.x * kThreads + threadIdx.x) / 32;
    if (warp >= rows) return;
    const int lane = threadIdx.x & 31, i = (int)(warp % a.len_q);
    const long long bh = warp / a.len_q;
    const int b = (int)(bh / a.heads), h = (int)(bh % a.heads);
    const T* o = head_base<T>(a.out, b, h) + i * a.out.len_stride;
    const T* d = head_base<T>(a.dout, b, h) + i * a.dout.len_stride;
    float s = 0.f;
    for (int c = lane; c < a.d; c += 32) s = fmaf(to_float(o[c]), to_float(d[c]), s);
#pragma unroll
    for (int k = 16; k > 0; k >>= 1) s += __shfl_xor_sync(0xffffffffu, s, k);
    if (lane == 0) a.delta[warp] = s;
}

// Zeros, and an lse of -inf where there is one: a warp per row of a head.
template <class T>
__global__ void __launch_bounds__(kThreads) k_attn_zero(const AttnTensor t, int heads, int len, int d, long long rows, float* lse) {
    pdl_entry();
    const int lane = threadIdx.x & 31;
    for (long long row = ((long long)blockIdx.x * kThreads + threadIdx.x) / 32; row < rows; row += (long long)gridDim.x * (kThreads / 32)) {
        const long long bh = row / len;
        T* to = static_cast<T*>(t.data) + bh / heads * t.batch_stride + bh % heads * t.head_stride + row % len * t.len_stride;
        for (int c = lane; c < d; c += 32) to[c] = T(0);
        if (lse && lane == 0) lse[row] = -INFINITY;
    }
}

namespace {

template <class K, class... A>
cudaError_t launch_blocks(K kernel, long long blocks, size_t smem, cudaStream_t st, const A&... args) {
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e) return e;
    if (blocks == 0) return cudaSuccess;
    if (blocks > 0x7fffffffll) return cudaErrorInvalidConfiguration;
    count_launches(1);
    return launch_pdl(kernel, dim3((unsigned)blocks), dim3(kThreads), smem, st, args...);
}

template <class T, int DP>
cudaError_t fwd(const AttnArgs& a, cudaStream_t st) {
    const size_t smem = sizeof(float) * ((kFM + 2 * kFN) * (DP + 4) + kFM * kTileRow<kFN, DP <= 128>);
    const int tiles = (a.len_q + kFM - 1) / kFM;
    return launch_blocks(k_attn_fwd_simt<T, DP>, (long long)tiles * a.heads * a.batch, smem, st, a, tiles);
}

template <class T, int DP>
cudaError_t bwd(const AttnArgs& a, cudaStream_t st) {
    constexpr int M = kSide<DP>;
    const size_t smem = sizeof(float) * (4 * M * (DP + 4) + 2 * M * kTileRow<M, true>);
    const int tiles_k = (a.len_k + M - 1) / M, tiles_q = (a.len_q + M - 1) / M;
    const long long blocks = (long long)tiles_k * a.kv_heads * a.batch + (long long)tiles_q * a.heads * a.batch;
    return launch_blocks(k_attn_bwd_simt<T, DP>, blocks, smem, st, a, tiles_k, tiles_q);
}

}  // namespace

cudaError_t launch_attn_delta(const AttnArgs& a, cudaStream_t st) {
    const long long rows = (long long)a.batch * a.heads * a.len_q;
    if (rows == 0) return cudaSuccess;
    const long long blocks = (rows + kThreads / 32 - 1) / (kThreads / 32);
    if (blocks > 0x7fffffffll) return cudaErrorInvalidConfiguration;
    count_launches(1);
    auto* kernel = a.dtype == GS_DTYPE_F32 ? k_attn_delta<float> : a.dtype == GS_DTYPE_F16 ? k_attn_delta<__half> : k_attn_delta<__nv_bfloat16>;
    return launch_pdl(kernel, dim3((unsigned)blocks), dim3(kThreads), 0, st, a);
}

cudaError_t launch_attn_fwd_simt(const AttnArgs& a, cudaStream_t st) { return fwd<float, 256>(a, st); }

cudaError_t launch_attn_bwd_simt(const AttnArgs& a, cudaStream_t st) {
    if (a.dtype == GS_DTYPE_F32) return a.d <= 128 ? bwd<float, 128>(a, st) : bwd<float, 256>(a, st);
    return a.dtype == GS_DTYPE_F16 ? bwd<__half, 256>(a, st) : bwd<__nv_bfloat16, 256>(a, st);
}

cudaError_t launch_attn_zero(const AttnArgs& a, const AttnTensor& t, int heads, int len, float* lse, cudaStream_t st) {
    const long long rows = (long long)a.batch * heads * len;
    if (rows == 0) return cudaSuccess;
    const long long blocks = (rows + kThreads / 32 - 1) / (kThreads / 32);
    count_launches(1);
    auto* kernel = a.dtype == GS_DTYPE_F32 ? k_attn_zero<float> : k_attn_zero<unsigned short>;  // zero is all bits zero
    return launch_pdl(kernel, dim3((unsigned)(blocks < 65536 ? blocks : 65536)), dim3(kThreads), 0, st, t, heads, len, a.d, rows, lse);
}

}  // namespace gs
