// The global 2-norm of many gradients, and their clipping: norm = sqrt(sum of g^2 over all tensors),
// g' = g min(1, max_norm / (norm + eps)).
//
// Bound by memory: the norm reads every gradient once, the clipping reads and writes them. Two launches: the first leaves a
// sum for each of its blocks, the second's blocks add all of these in one order (the same bits every time, no atomics) and
// multiply. The second starts at the end of what the first read, which the L2 still holds. A tensor is cut into chunks, and a
// block finds its chunk's tensor by bisection in a table that is part of the launch's arguments, so that no copy precedes it.
//
// Squares are added in float32 over one chunk and thread (64 elements), in float64 from there on. A chunk whose float32 sum
// leaves 1e-25 .. 1e37, where squares overflow or are lost below the subnormals, is added again in float64.
#include <cmath>

#include "elem.cuh"
#include "gs_common.cuh"
#include "gs_internal.h"

namespace gs {

constexpr int kClipBlock = 256;
constexpr int kClipChunk = 16384;  // elements

struct ClipTensor {
    const void* g;
    void* out;
    long long n;
    unsigned first;  // its first chunk
    int dtype;
};
template <int MOST>
struct ClipTable {
    ClipTensor t[MOST];
    int tensors;
    unsigned chunks;
};

// The tensor that has chunk c: the last whose first chunk is not behind it. (Empty tensors have none.)
template <int MOST>
__device__ __forceinline__ const ClipTensor& tensor_of(const ClipTable<MOST>& a, unsigned c) {
    int lo = 0, hi = a.tensors - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) / 2;
        if (a.t[mid].first <= c) lo = mid;
        else hi = mid - 1;
    }
    return a.t[lo];
}

// f(i, v) for the chunk's elements v at i, 16 bytes at a time where the tensor allows, else one.
template <class T, class F>
__device__ __forceinline__ void each(const ClipTensor& t, long long at, int n, F&& f) {
    constexpr int V = 16 / (int)sizeof(T);
    const T* g = static_cast<const T*>(t.g) + at;
    int done = 0;
    if (reinterpret_cast<uintptr_t>(t.g) % 16 == 0 && reinterpret_cast<uintptr_t>(t.out) % 16 == 0) {
        done = n / V * V;
        int i = threadIdx.x * V;
        for (; i + 3 * kClipBlock * V < done; i += 4 * kClipBlock * V) {  // (loads would not move over f's stores by themselves)
            Pack<T, V> p[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) p[j] = *reinterpret_cast<const Pack<T, V>*>(g + i + j * kClipBlock * V);
#pragma unroll
            for (int j = 0; j < 4; ++j) f(i + j * kClipBlock * V, p[j]);
        }
        for (; i < done; i += kClipBlock * V) f(i, *reinterpret_cast<const Pack<T, V>*>(g + i));
    }
    for (int i = done + threadIdx.x; i < n; i += kClipBlock) f(i, *reinterpret_cast<const Pack<T, 1>*>(g + i));
}

template <class F>
__device__ __forceinline__ void each_of(const ClipTensor& t, long long at, int n, F&& f) {
    if (t.dtype == GS_DTYPE_F32) each<float>(t, at, n, f);
    else if (t.dtype == GS_DTYPE_F16) each<__half>(t, at, n, f);
    else each<__nv_bfloat16>(t, at, n, f);
}

// Sum over the block, the same in all threads.
template <class S>
__device__ __forceinline__ S block_sum(S s, S* buf) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) buf[threadIdx.x / 32] = s;
    __syncthreads();
    s = S(0);
#pragma unroll
    for (int w = 0; w < kClipBlock / 32; ++w) s += buf[w];
    return s;
}

template <int MOST>
__global__ void __launch_bounds__(kClipBlock) k_grad_squares(const __grid_constant__ ClipTable<MOST> a, double* part) {
    pdl_entry();
    __shared__ double buf[kClipBlock / 32];
    double sum = 0.0;
    for (unsigned c = blockIdx.x; c < a.chunks; c += gridDim.x) {
        const ClipTensor& t = tensor_of(a, c);
        const long long at = (long long)(c - t.first) * kClipChunk;
        const int n = (int)min((long long)kClipChunk, t.n - at);
        float s[4] = {0.f, 0.f, 0.f, 0.f};
        each_of(t, at, n, [&](int, const auto& p) {
#pragma unroll
            for (int k = 0; k < (int)(sizeof(p.v) / sizeof(p.v[0])); ++k) {
                const float v = to_float(p.v[k]);
                s[k & 3] = fmaf(v, v, s[k & 3]);
            }
        });
        const float mine = (s[0] + s[1]) + (s[2] + s[3]);
        const double chunk = block_sum((double)mine, buf);
        if (chunk > 1e-25 && chunk < 1e37) {
            sum += chunk;
            continue;
        }
        double d = 0.0;
        each_of(t, at, n, [&](int, const auto& p) {
#pragma unroll
            for (int k = 0; k < (int)(sizeof(p.v) / sizeof(p.v[0])); ++k) {
                const double v = to_float(p.v[k]);
                d = fma(v, v, d);
            }
        });
        sum += block_sum(d, buf);
    }
    if (threadIdx.x == 0) part[blockIdx.x] = sum;
}

// The norm from the first launches' sums, the same in all threads and blocks.
__device__ __forceinline__ double norm_of(const double* part, int parts, double* buf) {
    double s = 0.0;
    for (int i = threadIdx.x; i < parts; i += kClipBlock) s += part[i];
    return sqrt(block_sum(s, buf));
}

__global__ void __launch_bounds__(kClipBlock) k_grad_norm(const double* part, int parts, float* norm) {
    pdl_entry();
    __shared__ double buf[kClipBlock / 32];
    const double n = norm_of(part, parts, buf);
    if (threadIdx.x == 0) *norm = (float)n;
}

template <int MOST>
__global__ void __launch_bounds__(kClipBlock) k_grad_scale(const __grid_constant__ ClipTable<MOST> a, const double* part, int parts,
                                                           double max_norm, double eps, float* norm) {
    pdl_entry();
    __shared__ double buf[kClipBlock / 32];
    const double n = norm_of(part, parts, buf), f = n + eps == 0.0 ? 1.0 : max_norm / (n + eps);
    const float factor = f > 1.0 ? 1.f : (float)f;  // NaN stays
    if (norm && blockIdx.x == 0 && threadIdx.x == 0) *norm = (float)n;
    for (unsigned k = blockIdx.x; k < a.chunks; k += gridDim.x) {
        const unsigned c = a.chunks - 1 - k;
        const ClipTensor& t = tensor_of(a, c);
        if (factor == 1.f && t.g == t.out) continue;
        const long long at = (long long)(c - t.first) * kClipChunk;
        const int count = (int)min((long long)kClipChunk, t.n - at);
        each_of(t, at, count, [&](int i, const auto& p) {
            using P = std::remove_const_t<std::remove_reference_t<decltype(p)>>;
            using T = std::remove_const_t<std::remove_reference_t<decltype(p.v[0])>>;
            P q;
#pragma unroll
            for (int j = 0; j < (int)(sizeof(p.v) / sizeof(p.v[0])); ++j) q.v[j] = from_float<T>(to_float(p.v[j]) * factor);
            *reinterpret_cast<P*>(static_cast<T*>(t.out) + at + i) = q;
        });
    }
}

namespace {

constexpr int kClipMost = 512;  // tensors of a launch (its arguments end at 32,764 bytes)

long long chunks_of(long long n) { return (n + kClipChunk - 1) / kClipChunk; }

// A launch's tensors from `from` on; where the next launch's begin.
template <int MOST>
int fill(ClipTable<MOST>& a, const gs_gradient* g, int n, int from) {
    a.tensors = 0;
    a.chunks = 0;
    int i = from;
    for (; i < n && a.tensors < MOST; ++i) {
        const long long c = chunks_of(g[i].n);
        if (c == 0) continue;
        if (a.chunks + c > 0x7fffffffll) break;
        a.t[a.tensors++] = ClipTensor{g[i].grad, g[i].out ? g[i].out : g[i].grad, g[i].n, a.chunks, g[i].dtype};
        a.chunks += (unsigned)c;
    }
    return i;
}

int blocks_of(unsigned chunks) {
    const unsigned most = (unsigned)(device_sm_count() * 8);  // of 256 threads
    return (int)(chunks < most ? chunks : most);
}

template <int MOST>
cudaError_t run(const gs_gradient* g, int n, bool clip, double max_norm, double eps, double* part, float* norm, cudaStream_t st) {
    ClipTable<MOST> a;
    int parts = 0;
    cudaError_t e;
    for (int i = 0; i < n;) {
        i = fill(a, g, n, i);
        if (a.chunks == 0) continue;
        const int blocks = blocks_of(a.chunks);
        count_launches(1);
        if ((e = launch_pdl(k_grad_squares<MOST>, dim3(blocks), dim3(kClipBlock), 0, st, a, part + parts))) return e;
        parts += blocks;
    }
    if (!clip || parts == 0) {
        count_launches(1);
        return launch_pdl(k_grad_norm, dim3(1), dim3(kClipBlock), 0, st, (const double*)part, parts, norm);
    }
    for (int i = 0; i < n;) {
        const int next = fill(a, g, n, i);
        if (a.chunks > 0) {
            count_launches(1);
            if ((e = launch_pdl(k_grad_scale<MOST>, dim3(blocks_of(a.chunks)), dim3(kClipBlock), 0, st, a, (const double*)part, parts,
                                max_norm, eps, norm)))
                return e;
            norm = nullptr;
        }
        i = next;
    }
    return cudaSuccess;
}

}  // namespace

size_t clip_workspace_bytes(const gs_gradient* g, int n) {
    size_t parts = 0;
    ClipTable<1> one;
    for (int i = 0; i < n; ++i) {  // a launch's blocks are at most the tensors' alone
        fill(one, g, i + 1, i);
        parts += (size_t)blocks_of(one.chunks);
    }
    const size_t most = (size_t)device_sm_count() * 8 * ((size_t)n / 32 + 1);
    return (parts < most ? parts : most) * sizeof(double);
}

cudaError_t launch_clip(const gs_gradient* g, int n, bool clip, double max_norm, double eps, void* workspace, float* norm, cudaStream_t st) {
    double* part = static_cast<double*>(workspace);
    return n <= 32 ? run<32>(g, n, clip, max_norm, eps, part, norm, st) : run<kClipMost>(g, n, clip, max_norm, eps, part, norm, st);
}

}  // namespace gs
