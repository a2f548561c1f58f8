// Cross attention: laying tensors out in the workspace for the tensor-core kernels, and joining the shares of
// a walk that was split. All of it moves memory once with 16-byte accesses where the rows allow them.
#include "attention_tc.cuh"

namespace gs {

// A block per batch entry, a thread per key of each chunk: ballots within a warp, the warps' counts summed.
__global__ void __launch_bounds__(1024) k_attn_index(const AttnArgs a, int* count, int* index) {
    pdl_entry();
    __shared__ int warps[2][32];
    const int b = blockIdx.x, len = key_count(a, b), warp = threadIdx.x >> 5;
    int* out = index + (long long)b * a.len_k;
    int done = 0, phase = 0;
    for (int n0 = 0; n0 < len; n0 += 1024, phase ^= 1) {
        const int key = n0 + threadIdx.x;
        const bool in = key < len && a.key_mask[b * a.mask_stride + key] != 0;
        const unsigned votes = __ballot_sync(0xffffffffu, in);
        if ((threadIdx.x & 31) == 0) warps[phase][warp] = __popc(votes);
        __syncthreads();
        int before = 0, total = 0;
#pragma unroll
        for (int w = 0; w < 32; ++w) {
            const int c = warps[phase][w];
            before += w < warp ? c : 0;
            total += c;
        }
        if (in) out[done + before + __popc(votes & lanemask_lt())] = key;
        done += total;
    }
    if (threadIdx.x == 0) count[b] = done;
}

// A thread per eight elements of a packed row, all tensors of a call in one launch (blockIdx.z).
struct PackJobs {
    PackJob job[4];
};
template <class T, int PL>
__global__ void __launch_bounds__(256) k_attn_pack(const AttnArgs a, const PackJobs jobs, const int* count, const int* index, int dp) {
    pdl_entry();
    const PackJob& j = jobs.job[blockIdx.z];
    const AttnTensor& t = j.t;
    const int heads = j.heads, keys = j.keys, per = dp / 8;
    const long long rows = j.rows;
    __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(j.dst);
    for (long long bh = blockIdx.y; bh < (long long)a.batch * heads; bh += gridDim.y) {
        const int b = (int)(bh / heads), h = (int)(bh % heads);
        const int live = !keys ? j.len : count ? count[b] : key_count(a, b);
        const int last = keys ? (live + kTileRows - 1) / kTileRows * kTileRows : live;  // rows that are read
        for (long long i = (long long)blockIdx.x * 256 + threadIdx.x; i < (long long)last * per; i += (long long)gridDim.x * 256) {
            const int row = (int)(i / per), c = (int)(i % per) * 8;
            float x[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] = 0.f;
            if (row < live) {
                const int src = index && keys ? index[(long long)b * a.len_k + row] : row;
                const T* p = head_base<T>(t, b, h) + src * t.len_stride + c;
                if (c + 8 <= a.d && reinterpret_cast<uintptr_t>(p) % 16 == 0) {
                    constexpr int V = 16 / (int)sizeof(T);
#pragma unroll
                    for (int e = 0; e < 8; e += V) {
                        const Pack<T, V> w = *reinterpret_cast<const Pack<T, V>*>(p + e);
#pragma unroll
                        for (int k = 0; k < V; ++k) x[e + k] = to_float(w.v[k]);
                    }
                } else {
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        if (c + e < a.d) x[e] = to_float(p[e]);
                }
            }
#pragma unroll
            for (int q = 0; q < PL; ++q) {
                uint32_t w[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    if (PL == 1) {
                        w[e] = pack2<typename std::conditional<sizeof(T) == 4, __nv_bfloat16, T>::type>(x[2 * e], x[2 * e + 1]);
                    } else {
                        w[e] = pack2<__nv_bfloat16>(x[2 * e], x[2 * e + 1]);
                        x[2 * e] -= __uint_as_float(w[e] << 16);
                        x[2 * e + 1] -= __uint_as_float(w[e] & 0xffff0000u);
                    }
                }
                *reinterpret_cast<uint4*>(dst + ((bh * PL + q) * rows + row) * dp + c) = make_uint4(w[0], w[1], w[2], w[3]);
            }
        }
    }
}

// The shares weighted by exp(lse - max lse), WARPS warps to a query and head, each with its part of the shares; they are
// joined in order.
template <class T, int WARPS>
__global__ void __launch_bounds__(256) k_attn_combine(const AttnArgs a, const float* part, const float* part_lse, int splits,
                                                      int dp) {
    pdl_entry();
    __shared__ float meet[WARPS > 1 ? WARPS : 1][256 + 2];
    const long long rows = (long long)a.batch * a.heads * a.len_q;
    const long long row = ((long long)blockIdx.x * 256 + threadIdx.x) / (32 * WARPS);
    if (row >= rows) return;
    const int lane = threadIdx.x & 31, warp = WARPS > 1 ? threadIdx.x >> 5 : 0, i = (int)(row % a.len_q);
    const long long bh = row / a.len_q;
    const int b = (int)(bh / a.heads), h = (int)(bh % a.heads);
    constexpr int kMost = 8, kAhead = 4;  // columns of a lane (heads of up to 256), shares under way
    float o[kMost] = {}, total = 0.f, top = -INFINITY;
    for (int s0 = warp; s0 < splits; s0 += WARPS * kAhead) {
        float l[kAhead], x[kAhead][kMost], m = top;
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            const int s = s0 + u * WARPS;
            l[u] = s < splits ? part_lse[s * rows + row] : -INFINITY;
#pragma unroll
            for (int k = 0; k < kMost; ++k)
                if (s < splits && lane + 32 * k < a.d) x[u][k] = part[(s * rows + row) * dp + lane + 32 * k];
        }
#pragma unroll
        for (int u = 0; u < kAhead; ++u) m = fmaxf(m, l[u]);
        const float zero = m == -INFINITY ? 0.f : m, keep = expf(top - zero);
        top = m;
        total *= keep;
#pragma unroll
        for (int k = 0; k < kMost; ++k) o[k] *= keep;
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            const float w = expf(l[u] - zero);
            total += w;
#pragma unroll
            for (int k = 0; k < kMost; ++k)
                if (lane + 32 * k < a.d) o[k] += l[u] == -INFINITY ? 0.f : w * x[u][k];  // a share without keys was not written
        }
    }
    if (WARPS > 1) {
#pragma unroll
        for (int k = 0; k < kMost; ++k) meet[warp][lane + 32 * k] = o[k];
        if (lane == 0) meet[warp][256] = top, meet[warp][257] = total;
        __syncthreads();
        if (warp != 0) return;
        float m = -INFINITY;
#pragma unroll
        for (int w = 0; w < WARPS; ++w) m = fmaxf(m, meet[w][256]);
        total = 0.f;
        top = m;
#pragma unroll
        for (int k = 0; k < kMost; ++k) o[k] = 0.f;
#pragma unroll
        for (int w = 0; w < WARPS; ++w) {
            const float keep = expf(meet[w][256] - (m == -INFINITY ? 0.f : m));
            total = fmaf(keep, meet[w][257], total);
#pragma unroll
            for (int k = 0; k < kMost; ++k) o[k] = fmaf(keep, meet[w][lane + 32 * k], o[k]);
        }
    }
    T* dst = static_cast<T*>(a.out.data) + b * a.out.batch_stride + h * a.out.head_stride + i * a.out.len_stride;
#pragma unroll
    for (int k = 0; k < kMost; ++k)
        if (lane + 32 * k < a.d) dst[lane + 32 * k] = from_float<T>(total == 0.f ? 0.f : o[k] / total);
    if (lane == 0) a.lse[row] = total == 0.f ? -INFINITY : top + logf(total);
}

cudaError_t launch_attn_index(const AttnArgs& a, int* count, int* index, cudaStream_t st) {
    count_launches(1);
    return launch_pdl(k_attn_index, dim3(a.batch), dim3(1024), 0, st, a, count, index);
}

cudaError_t launch_attn_pack(const AttnArgs& a, const PackJob* jobs, int n, const int* count, const int* index, int planes, int dp,
                             cudaStream_t st) {
    if (n == 0) return cudaSuccess;
    PackJobs all{};
    long long x = 1, y = 1;
    for (int i = 0; i < n; ++i) {
        all.job[i] = jobs[i];
        const long long blocks = (jobs[i].rows * (dp / 8) + 255) / 256, bh = (long long)a.batch * jobs[i].heads;
        x = blocks > x ? blocks : x;
        y = bh > y ? bh : y;
    }
    const dim3 grid((unsigned)(x < 4096 ? x : 4096), (unsigned)(y < 32768 ? y : 32768), (unsigned)n);
    auto* kernel = planes == 3 ? k_attn_pack<float, 3> : a.dtype == GS_DTYPE_F16 ? k_attn_pack<__half, 1> : k_attn_pack<__nv_bfloat16, 1>;
    count_launches(1);
    return launch_pdl(kernel, grid, dim3(256), 0, st, a, all, count, index, dp);
}

cudaError_t launch_attn_combine(const AttnArgs& a, const float* part, const float* part_lse, int splits, int dp, cudaStream_t st) {
    const bool many = splits > 4;  // a block per row: eight times four shares under way together
    const long long rows = (long long)a.batch * a.heads * a.len_q, blocks = many ? rows : (rows + 7) / 8;
    auto* kernel = a.dtype == GS_DTYPE_F32   ? (many ? k_attn_combine<float, 8> : k_attn_combine<float, 1>)
                   : a.dtype == GS_DTYPE_F16 ? (many ? k_attn_combine<__half, 8> : k_attn_combine<__half, 1>)
                                             : (many ? k_attn_combine<__nv_bfloat16, 8> : k_attn_combine<__nv_bfloat16, 1>);
    count_launches(1);
    return launch_pdl(kernel, dim3((unsigned)blocks), dim3(256), 0, st, a, part, part_lse, splits, dp);
}

}  // namespace gs
