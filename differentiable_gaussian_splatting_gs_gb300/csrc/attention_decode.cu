// Cross attention, forward, for one query whose heads share no keys (the single-token form). Every key and value is
// read once, so the memory bounds it, and the tensor cores' tiles of 128 queries would be empty. The keys are split over
// blocks until every SM has some, and the shares joined by k_attn_combine. With more rows to a key head (queries x
// sharing heads) the dot products take longer than the memory, and tiles are faster: bfloat16, 4346 keys, heads of 64,
// one row: 16 heads 7.9 us here and 12.1 on the tensor cores, 16 x 16 heads 45 (6.3 TB/s) and 61; two rows 19 and 11.
//
// A group of LPK lanes takes a key: eight elements of it to a lane, the dot products summed by shuffles, and each
// group has the running maximum, sum and output of its own keys, in registers, which meet at the end: over the warp by
// shuffles, over the block in shared memory. A masked key is read too, so that all loads of a turn are under way together
// (with a branch around each they followed one another: 90 us for 8 x 16 heads of 4346 keys, now 28), and replaced by 0
// only in turns that may have one: a select for every element, and single multiply-adds instead of pairs, took 41 us.
#include "attention_tc.cuh"

namespace gs {

namespace {

constexpr int kWarps = 8, kAhead = 8;  // warps of a block; keys that a group has in flight

// Eight elements as they lie in memory, the first `left` of them where not VEC.
template <class T, bool VEC>
struct Eight {
    static constexpr int V = VEC ? 16 / (int)sizeof(T) : 1;
    Pack<T, V> w[8 / V];
    __device__ __forceinline__ void load(const T* p, int left) {
#pragma unroll
        for (int e = 0; e < 8; e += V)
            if (VEC || e < left) w[e / V] = *reinterpret_cast<const Pack<T, V>*>(p + e);
    }
    __device__ __forceinline__ f32x2 two(int e, int left) const {
        return f2_pack(VEC || e < left ? to_float(w[e / V].v[e % V]) : 0.f, VEC || e + 1 < left ? to_float(w[(e + 1) / V].v[(e + 1) % V]) : 0.f);
    }
    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int e = 0; e < 8; ++e) w[e / V].v[e % V] = from_float<T>(0.f);
    }
};

}  // namespace

template <class T, int LPK, bool VEC>
__global__ void __launch_bounds__(kWarps * 32, VEC ? 2 : 1) k_attn_decode(const AttnArgs a, int splits, int dp, float* part, float* part_lse) {
    pdl_entry();
    constexpr int kGroups = 32 / LPK;
    __shared__ float meet[kWarps][LPK * 8 + 2];
    int at = blockIdx.x;
    const int split = at % splits;
    at /= splits;
    const int h = at % a.heads, b = at / a.heads;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, group = lane / LPK, c0 = lane % LPK * 8, left = a.d - c0;
    const int len = key_count(a, b);
    const int per = (a.len_k + splits - 1) / splits, k0 = split * per, k1 = min(k0 + per, len);
    const float c = a.scale * 1.4426950408889634f;  // scores in units of log2
    // lanes beyond the head's elements load its first ones, against a q of 0 and into no output
    const int cl = left > 0 ? c0 : 0;
    const T *qb = head_base<T>(a.q, b, h) + c0, *kb = head_base<T>(a.k, b, h) + cl, *vb = head_base<T>(a.v, b, h) + cl;
    f32x2 q2[4], o2[4];
    float top = -INFINITY, sum = 0.f;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        q2[e] = f2_pack(2 * e < left ? to_float(qb[2 * e]) * c : 0.f, 2 * e + 1 < left ? to_float(qb[2 * e + 1]) * c : 0.f);
        o2[e] = f2_pack(0.f, 0.f);
    }
    for (int base = k0 + warp * kGroups * kAhead; base < k1; base += kWarps * kGroups * kAhead) {
        Eight<T, VEC> k[kAhead], v[kAhead];
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            const int key = min(base + u * kGroups + group, a.len_k - 1);
            k[u].load(kb + key * a.k.len_stride, left);
            v[u].load(vb + key * a.v.len_stride, left);
        }
        float s[kAhead], m = top;
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            f32x2 x = f2_mul(q2[0], k[u].two(0, left));
#pragma unroll
            for (int e = 1; e < 4; ++e) x = f2_fma(q2[e], k[u].two(2 * e, left), x);
            const float2 y = f2_unpack(x);
            s[u] = left > 0 ? y.x + y.y : 0.f;
        }
#pragma unroll
        for (int x = LPK / 2; x > 0; x >>= 1)
#pragma unroll
            for (int u = 0; u < kAhead; ++u) s[u] += __shfl_xor_sync(0xffffffffu, s[u], x);
        if (a.key_mask || base + kGroups * kAhead > k1) {
#pragma unroll
            for (int u = 0; u < kAhead; ++u) {
                const int key = base + u * kGroups + group;
                if (key < k1 && key_valid(a, b, key, len)) continue;
                s[u] = -INFINITY;
                v[u].clear();  // it may hold NaN
            }
        }
#pragma unroll
        for (int u = 0; u < kAhead; ++u) m = fmaxf(m, s[u]);
        const float zero = m == -INFINITY ? 0.f : m;  // no key so far: exp(-inf) = 0
        const float keep = ex2_approx(top - zero);
        top = m;
        sum *= keep;
        const f32x2 keep2 = f2_pack(keep, keep);
#pragma unroll
        for (int e = 0; e < 4; ++e) o2[e] = f2_mul(o2[e], keep2);
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            const float p = ex2_approx(s[u] - zero);
            sum += p;
            const f32x2 p2 = f2_pack(p, p);
#pragma unroll
            for (int e = 0; e < 4; ++e) o2[e] = f2_fma(p2, v[u].two(2 * e, left), o2[e]);
        }
    }
    float o[8];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const float2 y = f2_unpack(o2[e]);
        o[2 * e] = y.x, o[2 * e + 1] = y.y;
    }
    // the warp's groups
#pragma unroll
    for (int x = LPK; x < 32; x <<= 1) {
        const float m = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x)), keep = ex2_approx(top - (m == -INFINITY ? 0.f : m));
        top = m;
        sum *= keep;
        sum += __shfl_xor_sync(0xffffffffu, sum, x);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            o[e] *= keep;
            o[e] += __shfl_xor_sync(0xffffffffu, o[e], x);
        }
    }
    if (group == 0) {
#pragma unroll
        for (int e = 0; e < 8; ++e) meet[warp][c0 + e] = o[e];
        if (lane == 0) meet[warp][LPK * 8] = top, meet[warp][LPK * 8 + 1] = sum;
    }
    __syncthreads();
    // the block's warps
    float m = -INFINITY, total = 0.f, keep[kWarps];
#pragma unroll
    for (int w = 0; w < kWarps; ++w) m = fmaxf(m, meet[w][LPK * 8]);
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        keep[w] = ex2_approx(meet[w][LPK * 8] - (m == -INFINITY ? 0.f : m));
        total = fmaf(keep[w], meet[w][LPK * 8 + 1], total);
    }
    const long long qrow = (long long)b * a.heads + h, prow = (long long)split * a.batch * a.heads + qrow;
    const float f = total == 0.f ? 0.f : 1.f / total;
    T* dst = static_cast<T*>(a.out.data) + b * a.out.batch_stride + h * a.out.head_stride;
    for (int col = threadIdx.x; col < a.d; col += kWarps * 32) {
        float x = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) x = fmaf(keep[w], meet[w][col], x);
        if (part) part[prow * dp + col] = x * f;
        else dst[col] = from_float<T>(x * f);
    }
    if (threadIdx.x == 0) (part ? part_lse[prow] : a.lse[qrow]) = total == 0.f ? -INFINITY : (m + log2f(total)) * 0.6931471805599453f;
}

namespace {

template <class T, int LPK>
cudaError_t run(const AttnArgs& a, int splits, int dp, float* part, float* part_lse, cudaStream_t st) {
    const unsigned blocks = (unsigned)(splits * a.heads * a.batch);
    constexpr int V = 16 / (int)sizeof(T);
    auto aligned = [&](const AttnTensor& t) {
        return reinterpret_cast<uintptr_t>(t.data) % 16 == 0 && t.batch_stride % V == 0 && t.len_stride % V == 0 && t.head_stride % V == 0;
    };
    const bool vec = a.d % 8 == 0 && aligned(a.k) && aligned(a.v);
    count_launches(1);
    return launch_pdl(vec ? k_attn_decode<T, LPK, true> : k_attn_decode<T, LPK, false>, dim3(blocks), dim3(kWarps * 32), 0, st, a, splits,
                      dp, part, part_lse);
}

template <class T>
cudaError_t typed(const AttnArgs& a, int splits, int dp, float* part, float* part_lse, cudaStream_t st) {
    if (a.d <= 32) return run<T, 4>(a, splits, dp, part, part_lse, st);
    if (a.d <= 64) return run<T, 8>(a, splits, dp, part, part_lse, st);
    if (a.d <= 128) return run<T, 16>(a, splits, dp, part, part_lse, st);
    return run<T, 32>(a, splits, dp, part, part_lse, st);
}

}  // namespace

cudaError_t launch_attn_decode(const AttnArgs& a, int splits, int dp, float* part, float* part_lse, cudaStream_t st) {
    if (a.dtype == GS_DTYPE_F32) return typed<float>(a, splits, dp, part, part_lse, st);
    if (a.dtype == GS_DTYPE_F16) return typed<__half>(a, splits, dp, part, part_lse, st);
    return typed<__nv_bfloat16>(a, splits, dp, part, part_lse, st);
}

}  // namespace gs
