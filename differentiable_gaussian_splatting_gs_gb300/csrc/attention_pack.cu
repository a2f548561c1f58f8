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

// The shares weighted by exp(lse - max lse): 2^log_lanes threads to a query and head, four columns each, GROUPS times,
// each group with every GROUPS-th share; the groups are joined in order. Eight shares are under way together: the loads'
// latency bounds it (18,432 rows of two shares, or 4,096 of nine, of 64 columns: 5 us).
template <class T, int GROUPS>
__global__ void __launch_bounds__(256) k_attn_combine(const TcArgs t, int per, int dp, int log_lanes) {
    pdl_entry();
    constexpr int kAhead = 8;
    __shared__ float meet[GROUPS > 1 ? 6 : 1][256];
    const AttnArgs& a = t.a;
    const long long rows = (long long)t.tail * per;
    const unsigned unit = blockIdx.x * (256u >> log_lanes) + (threadIdx.x >> log_lanes), row = unit / GROUPS;
    const int group = unit % GROUPS, col = (threadIdx.x & ((1 << log_lanes) - 1)) * 4;
    const int block = t.whole + (int)(row / per), x = (int)(row % per), r = x % kTileRows, groups = a.heads / t.fold;
    const int b = block / t.tiles / groups, h0 = block / t.tiles % groups * t.fold, h = h0 + r / t.fold_rows;
    const int i = (block % t.tiles * (per / kTileRows) + x / kTileRows) * t.fold_rows + r % t.fold_rows;
    const bool in = row < rows && i < a.len_q && h < h0 + t.fold && col < a.d;
    float o[4] = {}, total = 0.f, top = -INFINITY;
    for (int s0 = group; s0 < t.splits && in; s0 += GROUPS * kAhead) {
        float l[kAhead], m = top;
        float4 x[kAhead];
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            const int s = min(s0 + u * GROUPS, t.splits - 1);
            l[u] = t.part_lse[s * rows + row];
            x[u] = *reinterpret_cast<const float4*>(t.part + (s * rows + row) * dp + col);
        }
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            if (s0 + u * GROUPS >= t.splits) l[u] = -INFINITY;
            m = fmaxf(m, l[u]);
        }
        const float zero = m == -INFINITY ? 0.f : m, keep = expf(top - zero);
        top = m;
        total *= keep;
#pragma unroll
        for (int k = 0; k < 4; ++k) o[k] *= keep;
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            if (l[u] == -INFINITY) continue;  // a share without keys was not written
            const float w = expf(l[u] - zero);
            total += w;
            o[0] += w * x[u].x, o[1] += w * x[u].y, o[2] += w * x[u].z, o[3] += w * x[u].w;
        }
    }
    if (GROUPS > 1) {
#pragma unroll
        for (int k = 0; k < 4; ++k) meet[k][threadIdx.x] = o[k];
        meet[4][threadIdx.x] = top;
        meet[5][threadIdx.x] = total;
        __syncthreads();
        if (group != 0) return;
#pragma unroll
        for (int g = 1; g < GROUPS; ++g) top = fmaxf(top, meet[4][threadIdx.x + (g << log_lanes)]);
        total = o[0] = o[1] = o[2] = o[3] = 0.f;
#pragma unroll
        for (int g = 0; g < GROUPS; ++g) {
            const int at = threadIdx.x + (g << log_lanes);
            const float keep = expf(meet[4][at] - (top == -INFINITY ? 0.f : top));
            total = fmaf(keep, meet[5][at], total);
#pragma unroll
            for (int k = 0; k < 4; ++k) o[k] = fmaf(keep, meet[k][at], o[k]);
        }
    }
    if (!in) return;
    T* dst = static_cast<T*>(a.out.data) + b * a.out.batch_stride + h * a.out.head_stride + i * a.out.len_stride;
#pragma unroll
    for (int k = 0; k < 4; ++k)
        if (col + k < a.d) dst[col + k] = from_float<T>(total == 0.f ? 0.f : o[k] / total);
    if (col == 0) a.lse[((long long)b * a.heads + h) * a.len_q + i] = total == 0.f ? -INFINITY : top + logf(total);
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

cudaError_t launch_attn_combine(const TcArgs& t, int rows, int dp, cudaStream_t st) {
    const bool many = t.splits > 8;  // more than are under way together
    int log_lanes = 0;
    while (4 << log_lanes < dp) ++log_lanes;
    const long long threads = ((long long)t.tail * rows * (many ? 4 : 1)) << log_lanes;
    const int type = t.a.dtype;
    auto* kernel = type == GS_DTYPE_F32   ? (many ? k_attn_combine<float, 4> : k_attn_combine<float, 1>)
                   : type == GS_DTYPE_F16 ? (many ? k_attn_combine<__half, 4> : k_attn_combine<__half, 1>)
                                          : (many ? k_attn_combine<__nv_bfloat16, 4> : k_attn_combine<__nv_bfloat16, 1>);
    count_launches(1);
    return launch_pdl(kernel, dim3((unsigned)((threads + 255) / 256)), dim3(256), 0, st, t, rows, dp, log_lanes);
}

}  // namespace gs
