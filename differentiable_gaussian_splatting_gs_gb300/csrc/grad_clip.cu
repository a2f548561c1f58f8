// The global 2-norm of many gradients, and their clipping: norm = sqrt(sum of g^2 over all tensors),
// g' = g min(1, max_norm / (norm + eps)).
//
// Bound by memory: the norm reads every gradient once, the clipping reads and writes them. Two launches: the first leaves a
// sum for each of its blocks, the second's blocks add all of these in one order (the same bits every time, no atomics) and
// multiply. The second starts at the end of what the first read, which the L2 still holds. A tensor is cut into chunks, and a
// block finds its chunk's tensor by bisection in a table that is part of the launch's arguments, so that no copy precedes it.
// Times in a graph: 94.4 million float32 in 5 tensors 187 us (three passes at the measured copy rate: 167), the norm alone 64 (5.9
// TB/s); 14 tensors of 1.1 million elements 9.0 us, two launches' latency and the joining of the sums (called 12 to 14, the host's).
//
// Squares are added in float32 over one chunk and thread (up to 64 elements), from there on as pairs of float32 whose sum has
// twice the bits. (Double precision, of which an SM does two operations a cycle, took 10 of 28 us for 14 tensors of 1.1 million
// elements.) A thread whose sum leaves 1e-25 .. 1e25, where squares are lost below the subnormals, or overflow in the sum of
// all threads' (3e13 of them would), adds its elements again in double precision, unless all are zeros (as those of hidden
// Gaussians are); such sums are kept apart, and all others join them in the end.
#include <cmath>

#include "elem.cuh"
#include "gs_common.cuh"
#include "gs_internal.h"

namespace gs {

constexpr int kClipBlock = 256;
constexpr int kClipMostChunk = 16384, kClipLeastChunk = 2048;  // elements

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
    int tensors, chunk;  // chunk: elements of one
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

// f(i, v) for the chunk's elements v at i: 16 bytes at a time between the first and the last whole ones, else one. WRITES: f writes
// the same place of `out`, which may lie on 16 bytes elsewhere; then one at a time.
template <class T, bool WRITES, class F>
__device__ __forceinline__ void each(const ClipTensor& t, long long at, int n, F&& f) {
    constexpr int V = 16 / (int)sizeof(T);
    const T* g = static_cast<const T*>(t.g) + at;
    int done = 0;
    if (!WRITES || (reinterpret_cast<uintptr_t>(t.g) - reinterpret_cast<uintptr_t>(t.out)) % 16 == 0) {
        const int head = min(n, (int)(-reinterpret_cast<uintptr_t>(g) % 16 / sizeof(T)));
        if (threadIdx.x < head) f((int)threadIdx.x, *reinterpret_cast<const Pack<T, 1>*>(g + threadIdx.x));
        done = head + (n - head) / V * V;
        int i = head + threadIdx.x * V;
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

template <bool WRITES, class F>
__device__ __forceinline__ void each_of(const ClipTensor& t, long long at, int n, F&& f) {
    if (t.dtype == GS_DTYPE_F32) each<float, WRITES>(t, at, n, f);
    else if (t.dtype == GS_DTYPE_F16) each<__half, WRITES>(t, at, n, f);
    else each<__nv_bfloat16, WRITES>(t, at, n, f);
}

// A sum as two floats, and what did not fit them.
struct SquareSum {
    float hi, lo;
    double wide;
};

// (hi, lo) + v, exact up to the bits below lo (Knuth's sum of two numbers and its error).
__device__ __forceinline__ void add_to(float& hi, float& lo, float v, float v_lo = 0.f) {
    const float s = hi + v, b = s - hi;
    lo += ((hi - (s - b)) + (v - b)) + v_lo;
    hi = s;
}

// The block's sum, in thread 0 (wide: where any thread has some).
__device__ __forceinline__ SquareSum block_sum(SquareSum s, SquareSum* buf) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) add_to(s.hi, s.lo, __shfl_xor_sync(0xffffffffu, s.hi, o), __shfl_xor_sync(0xffffffffu, s.lo, o));
    const bool wide = __any_sync(0xffffffffu, __double_as_longlong(s.wide) != 0);
    if (wide)
        for (int o = 16; o > 0; o >>= 1) s.wide += __shfl_xor_sync(0xffffffffu, s.wide, o);
    if ((threadIdx.x & 31) == 0) buf[threadIdx.x / 32] = s;
    __syncthreads();
    if (threadIdx.x == 0)
        for (int w = 1; w < kClipBlock / 32; ++w) {
            add_to(s.hi, s.lo, buf[w].hi, buf[w].lo);
            if (__double_as_longlong(buf[w].wide) != 0) s.wide += buf[w].wide;
        }
    return s;
}

template <int MOST>
__global__ void __launch_bounds__(kClipBlock) k_grad_squares(const __grid_constant__ ClipTable<MOST> a, SquareSum* part) {
    pdl_entry();
    __shared__ SquareSum buf[kClipBlock / 32];
    SquareSum sum{0.f, 0.f, 0.0};
    for (unsigned c = blockIdx.x; c < a.chunks; c += gridDim.x) {
        const ClipTensor& t = tensor_of(a, c);
        const long long at = (long long)(c - t.first) * a.chunk;
        const int n = (int)min((long long)a.chunk, t.n - at);
        float s[4] = {0.f, 0.f, 0.f, 0.f};
        unsigned any = 0;
        each_of<false>(t, at, n, [&](int, const auto& p) {
#pragma unroll
            for (int k = 0; k < (int)(sizeof(p.v) / sizeof(p.v[0])); ++k) {
                const float v = to_float(p.v[k]);
                s[k & 3] = fmaf(v, v, s[k & 3]);
                any |= __float_as_uint(v);
            }
        });
        const float mine = (s[0] + s[1]) + (s[2] + s[3]);
        if (mine > 1e-25f && mine < 1e25f) {
            add_to(sum.hi, sum.lo, mine);
        } else if (any << 1) {
            each_of<false>(t, at, n, [&](int, const auto& p) {
#pragma unroll
                for (int k = 0; k < (int)(sizeof(p.v) / sizeof(p.v[0])); ++k) {
                    const double v = to_float(p.v[k]);
                    sum.wide = fma(v, v, sum.wide);
                }
            });
        }
    }
    sum = block_sum(sum, buf);
    if (threadIdx.x == 0) part[blockIdx.x] = sum;
}

// The norm from the first launches' sums, and the factor of the gradients, in thread 0.
__device__ __forceinline__ void norm_of(const SquareSum* part, int parts, double max_norm, double eps, SquareSum* buf, float& norm, float& factor) {
    SquareSum s{0.f, 0.f, 0.0};
    for (int i = threadIdx.x; i < parts; i += kClipBlock) {
        const SquareSum p = part[i];
        add_to(s.hi, s.lo, p.hi, p.lo);
        if (__double_as_longlong(p.wide) != 0) s.wide += p.wide;
    }
    s = block_sum(s, buf);
    if (threadIdx.x != 0) return;
    if (__double_as_longlong(s.wide) == 0 && s.hi < 1e37f) {
        // sqrt(hi + lo) from sqrt(hi): one step of Newton's, whose error is of the order of the root's own rounding squared
        const float r = sqrtf(s.hi);
        norm = r > 0.f ? r + (fmaf(-r, r, s.hi) + s.lo) / (2.f * r) : 0.f;
        const float e = norm + (float)eps;
        factor = e == 0.f ? 1.f : (float)max_norm / e;
    } else {
        const double n = sqrt((double)s.hi + (double)s.lo + s.wide), e = n + eps;
        norm = (float)n;
        factor = e == 0.0 ? 1.f : (float)(max_norm / e);
    }
    if (factor > 1.f) factor = 1.f;  // NaN stays
}

__global__ void __launch_bounds__(kClipBlock) k_grad_norm(const SquareSum* part, int parts, float* norm) {
    pdl_entry();
    __shared__ SquareSum buf[kClipBlock / 32];
    float n, factor;
    norm_of(part, parts, 0.0, 0.0, buf, n, factor);
    if (threadIdx.x == 0) *norm = n;
}

template <int MOST>
__global__ void __launch_bounds__(kClipBlock) k_grad_scale(const __grid_constant__ ClipTable<MOST> a, const SquareSum* part, int parts,
                                                           double max_norm, double eps, float* norm) {
    pdl_entry();
    __shared__ SquareSum buf[kClipBlock / 32];
    __shared__ float shared_factor;
    float n, mine;
    norm_of(part, parts, max_norm, eps, buf, n, mine);
    if (threadIdx.x == 0) {
        shared_factor = mine;
        if (norm && blockIdx.x == 0) *norm = n;
    }
    __syncthreads();
    const float factor = shared_factor;
    for (unsigned k = blockIdx.x; k < a.chunks; k += gridDim.x) {
        const unsigned c = a.chunks - 1 - k;
        const ClipTensor& t = tensor_of(a, c);
        if (factor == 1.f && t.g == t.out) continue;
        const long long at = (long long)(c - t.first) * a.chunk;
        const int count = (int)min((long long)a.chunk, t.n - at);
        each_of<true>(t, at, count, [&](int i, const auto& p) {
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

int resident() { return device_sm_count() * 8; }  // blocks of 256 threads

// Elements of a chunk: few where all gradients are few, so that every SM has some (14 tensors of 1.1 million: 16,384
// elements 10.0 us).
int chunk_of(const gs_gradient* g, int n) {
    double total = 0.0;
    for (int i = 0; i < n; ++i) total += (double)g[i].n;
    int c = kClipLeastChunk;
    while (c < kClipMostChunk && total > (double)c * resident()) c *= 2;
    return c;
}

// A launch's tensors from `from` on; where the next launch's begin.
template <int MOST>
int fill(ClipTable<MOST>& a, const gs_gradient* g, int n, int from) {
    a.tensors = 0;
    a.chunks = 0;
    int i = from;
    for (; i < n && a.tensors < MOST; ++i) {
        const long long c = (g[i].n + a.chunk - 1) / a.chunk;
        if (c == 0) continue;
        if (a.chunks + c > 0x7fffffffll) break;
        a.t[a.tensors++] = ClipTensor{g[i].grad, g[i].out ? g[i].out : g[i].grad, g[i].n, a.chunks, g[i].dtype};
        a.chunks += (unsigned)c;
    }
    return i;
}

int blocks_of(unsigned chunks) {
    const unsigned most = (unsigned)resident();
    return (int)(chunks < most ? chunks : most);
}

template <int MOST>
cudaError_t run(const gs_gradient* g, int n, bool clip, double max_norm, double eps, SquareSum* part, float* norm, cudaStream_t st) {
    ClipTable<MOST> a;
    a.chunk = chunk_of(g, n);
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
        return launch_pdl(k_grad_norm, dim3(1), dim3(kClipBlock), 0, st, (const SquareSum*)part, parts, norm);
    }
    for (int i = 0; i < n;) {
        const int next = fill(a, g, n, i);
        if (a.chunks > 0) {
            count_launches(1);
            if ((e = launch_pdl(k_grad_scale<MOST>, dim3(blocks_of(a.chunks)), dim3(kClipBlock), 0, st, a, (const SquareSum*)part, parts,
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
    one.chunk = chunk_of(g, n);
    for (int i = 0; i < n; ++i) {  // a launch's blocks are at most the tensors' alone
        fill(one, g, i + 1, i);
        parts += (size_t)blocks_of(one.chunks);
    }
    const size_t most = (size_t)resident() * ((size_t)n / 32 + 1);
    return (parts < most ? parts : most) * sizeof(SquareSum);
}

cudaError_t launch_clip(const gs_gradient* g, int n, bool clip, double max_norm, double eps, void* workspace, float* norm, cudaStream_t st) {
    SquareSum* part = static_cast<SquareSum*>(workspace);
    return n <= 32 ? run<32>(g, n, clip, max_norm, eps, part, norm, st) : run<kClipMost>(g, n, clip, max_norm, eps, part, norm, st);
}

}  // namespace gs
