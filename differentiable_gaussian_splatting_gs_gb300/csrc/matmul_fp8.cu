// Matrix product of 8-bit values with a scale for each block of 128:
//   out[m, n] = sum over blocks of sa[m, block] sb[n, block] sum over the block of a[m, k] b[n, k].
//
// The tensor cores multiply a block of 128 of the inner dimension at a time (four products of 32, float32 in tensor memory
// from zero), and the elementwise warps add it, times its scales, to float32 sums in registers: a block's scales are the
// same for all its products, which therefore need no scaling of their own.
//
// One operand's rows lie along the 128 lanes of tensor memory (P), the other's along its columns (Q, TN of them). Where a
// has many rows it is P; with up to 64 rows b is, so that no lane is empty, and a's rows are the few columns. A lane's thread
// multiplies all its columns by the lane's scale; scales that differ by column (COLS) take one more multiplication, read
// from shared memory, where columns of the same block of 128 share one (b's 128 x 128 blocks).
//
// A warp copies tiles (128 bytes of inner dimension, 128-byte swizzle), one issues the products, the others multiply and
// add; accumulators alternate between two places, so that a block's products run beside the additions of the one before.
// Blocks of threads take tiles in turn, and go on copying and multiplying while the result of the last one is stored.
// Where tiles are few, a cluster of up to 8 blocks shares the inner dimension of one, joined through their shared
// memory in a fixed order.
#include <cudaTypedefs.h>

#include <algorithm>

#include "elem.cuh"
#include "fp8.cuh"
#include "gs_internal.h"
#include "tcgen05.cuh"

namespace gs {

constexpr int kMmRows = 128;   // lanes: rows of P in a tile
constexpr int kMmBlock = 128;  // inner dimension of a block, bytes

struct MmArgs {
    CUtensorMap p, q;
    const float *p_scale, *q_scale;
    long long p_row, p_block, q_row, q_block;  // strides of the scales
    int p_shift, q_shift;                      // 2^shift rows share a scale
    void* out;
    long long out_p, out_q;  // strides of the result, one of them 1
    int dtype, wide, np, nq, blocks, tiles_p, tiles, splits;  // wide: rows of the result lie in whole 32 bytes
    unsigned limit, *err;
};

__device__ __forceinline__ void mma8_ss(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, bool add) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 da, db;\n\tsetp.ne.b32 p, %4, 0;\n\tmov.b64 da, {%1, %5};\n\tmov.b64 db, {%2, %5};\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], da, db, %3, p;\n\t}" ::"r"(d),
        "r"(a), "r"(b), "r"(idesc), "r"((uint32_t)add), "r"(kTileDescHi)
        : "memory");
}

__device__ __forceinline__ void tile_load2(uint32_t dst, const CUtensorMap* map, int c0, int c1, uint64_t* bar) {
    asm volatile("cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4}], [%2];" ::"r"(dst),
                 "l"(map), "r"(smem_u32(bar)), "r"(c0), "r"(c1)
                 : "memory");
}

__device__ __forceinline__ void tmem_ld16(uint32_t addr, uint32_t (&v)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]),
          "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
        : "r"(addr));
}
__device__ __forceinline__ void tmem_wait_ld16(uint32_t (&v)[16]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(v[0]), "+r"(v[1]), "+r"(v[2]), "+r"(v[3]), "+r"(v[4]), "+r"(v[5]), "+r"(v[6]), "+r"(v[7]), "+r"(v[8]),
                   "+r"(v[9]), "+r"(v[10]), "+r"(v[11]), "+r"(v[12]), "+r"(v[13]), "+r"(v[14]), "+r"(v[15])::"memory");
}

// All threads of the cluster's blocks: what they wrote before to shared memory is seen by the others after.
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ unsigned cluster_rank() {
    unsigned r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
// A float of block `rank`'s shared memory at this block's address p.
__device__ __forceinline__ float peer_float(const float* p, unsigned rank) {
    float v;
    asm volatile("{\n\t.reg .b32 a;\n\tmapa.shared::cluster.u32 a, %1, %2;\n\tld.shared::cluster.f32 %0, [a];\n\t}"
                 : "=f"(v)
                 : "r"(smem_u32(p)), "r"(rank)
                 : "memory");
    return v;
}

// What the sizes of a tile decide.
template <int TN>
struct MmShape {
    static constexpr int kCols = TN == 256 ? 128 : TN < 64 ? TN : 64;  // columns of an elementwise warp
    static constexpr int kWarps = 4 * (TN / kCols);             // elementwise
    static constexpr int kThreads = 32 * (kWarps + 4);          // and a warpgroup for the copies and the products
    // Registers, where a warp's sums are 128 columns: of what the launch gives each thread (168), the third warpgroup
    // leaves all but 24, and the elementwise two take 240: 128 x 24 + 256 x 240 = 384 x 168.
    static constexpr bool kShift = kCols == 128;
    static constexpr int kLaunch = 168, kFew = 24, kMany = 240;
    static_assert(!kShift || 128 * kFew + (kThreads - 128) * kMany <= kThreads * kLaunch);
    static constexpr int kBytes = (kMmRows + TN) * kMmBlock;    // a stage: both operands' tiles
    static constexpr int kResident = TN >= 128 ? 1 : 2;         // blocks of threads on an SM
    static constexpr int kStages = TN == 256 ? 4 : TN == 128 ? 6 : TN == 64 ? 4 : 5;
    static constexpr int kBufs = TN == 128 ? 4 : 2;             // accumulators
    static constexpr int kTmem = kBufs * TN;
    static constexpr int kSmem = 1024 + kStages * kBytes;
    static_assert(kTmem >= 32 && kResident * kTmem <= 512 && (kTmem & (kTmem - 1)) == 0);
    static_assert(kStages * kBytes >= kMmRows * TN * 4, "a cluster's sums take the tiles' place");
};

// 32 bytes of a row of the result at once: whole sectors of the L2, which 16 bytes of a thread's own row each are not.
__device__ __forceinline__ void store32(void* to, const uint32_t (&v)[8]) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(to), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]),
                 "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                 : "memory");
}

// The thread's row of a tile, COLS columns that end at `left`: 32 bytes at a time where the result allows (`wide`).
template <int COLS>
__device__ __forceinline__ void store_row(const MmArgs& a, const f32x2 (&acc)[COLS / 2], long long at, int left) {
    const int size = a.dtype == GS_DTYPE_F32 ? 4 : 2;
    if (a.wide && left >= COLS) {
        char* to = static_cast<char*>(a.out) + at * size;
        if (a.dtype == GS_DTYPE_F32) {
#pragma unroll
            for (int c = 0; c < COLS; c += 8) {
                uint32_t v[8];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float2 f = f2_unpack(acc[c / 2 + i]);
                    v[2 * i] = __float_as_uint(f.x);
                    v[2 * i + 1] = __float_as_uint(f.y);
                }
                store32(to + c * 4, v);
            }
        } else {
#pragma unroll
            for (int c = 0; c < COLS; c += 16) {
                uint32_t v[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float2 f = f2_unpack(acc[c / 2 + i]);
                    v[i] = a.dtype == GS_DTYPE_F16 ? pack2<__half>(f.x, f.y) : pack2<__nv_bfloat16>(f.x, f.y);
                }
                store32(to + c * 2, v);
            }
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < COLS / 2; ++i) {
        const float2 v = f2_unpack(acc[i]);
        if (2 * i < left) store_elem(a.out, at + 2 * i * a.out_q, a.dtype, v.x);
        if (2 * i + 1 < left) store_elem(a.out, at + (2 * i + 1) * a.out_q, a.dtype, v.y);
    }
}

template <int TN, bool COLS>
__global__ void __launch_bounds__(MmShape<TN>::kThreads, MmShape<TN>::kResident) k_matmul_fp8(const __grid_constant__ MmArgs a) {
    using S = MmShape<TN>;
    constexpr int kStages = S::kStages, kBufs = S::kBufs, kCols = S::kCols, kPart = kCols < 32 || kCols == 128 ? 16 : 32;
    extern __shared__ unsigned char dynamic[];
    __shared__ uint64_t full[kStages], empty[kStages], done[kBufs], drained[kBufs], last;
    __shared__ uint32_t tmem_at;
    __shared__ __align__(16) float col_scales[COLS ? S::kWarps : 1][2][COLS ? kCols : 4];
    const uint32_t tiles = (smem_u32(dynamic) + 1023) & ~1023u;
    const int warp = threadIdx.x / 32, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int i = 0; i < kStages; ++i) {
            mbar_init(full + i, 1);
            mbar_init(empty + i, 1);
        }
        for (int i = 0; i < kBufs; ++i) {
            mbar_init(done + i, 1);
            mbar_init(drained + i, S::kWarps);
        }
        mbar_init(&last, 1);
        fence_mbar_init();
    }
    // Tensor memory is taken once the kernel before has given up its own, and before the next one's blocks may come, which
    // would otherwise hold what a block of this or of that one waits for.
    pdl_wait();
    if (warp == S::kWarps + 1) tmem_alloc<S::kTmem>(&tmem_at);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    pdl_launch_dependents();
    const uint32_t tmem = tmem_at;
    // this block's tiles and its share of their inner dimension
    const int rank = blockIdx.x % a.splits, step = gridDim.x / a.splits;
    const int k0 = (int)((long long)a.blocks * rank / a.splits), k1 = (int)((long long)a.blocks * (rank + 1) / a.splits);
    if (warp >= S::kWarps) {
        if constexpr (S::kShift) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(S::kFew));
        if (warp == S::kWarps) {
            // ---- copies ----
            int turn = 0;
            if (elect_one()) {
                bool ok = true;
                for (int t = blockIdx.x / a.splits; t < a.tiles && ok; t += step) {
                    const int p0 = t % a.tiles_p * kMmRows, q0 = t / a.tiles_p * TN;
                    for (int k = k0; k < k1 && ok; ++k, ++turn) {
                        const int s = turn % kStages;
                        if (turn >= kStages && !mbar_wait_bounded(empty + s, (turn / kStages - 1) & 1, a.limit, a.err)) {
                            ok = false;
                            break;
                        }
                        const uint32_t at = tiles + s * S::kBytes;
                        mbar_arrive_expect_tx(full + s, S::kBytes);
                        tile_load2(at, &a.p, k * kMmBlock, p0, full + s);
                        tile_load2(at + kMmRows * kMmBlock, &a.q, k * kMmBlock, q0, full + s);
                    }
                }
                // every copy has landed before the block ends
                for (int i = turn > kStages ? turn - kStages : 0; i < turn; ++i) mbar_drain(full + i % kStages, (i / kStages) & 1, a.err);
            }
            __syncwarp();
        } else if (warp == S::kWarps + 1) {
            // ---- products ----
            constexpr uint32_t idesc = (1u << 4) | ((uint32_t)(TN >> 3) << 17) | ((128u >> 4) << 24);  // e4m3 x e4m3, float32
            int turn = 0;
            bool ok = true;
            for (int t = blockIdx.x / a.splits; t < a.tiles && ok; t += step)
                for (int k = k0; k < k1 && ok; ++k, ++turn) {
                    const int s = turn % kStages, b = turn % kBufs;
                    if (turn >= kBufs) ok = warp_wait(drained + b, (turn / kBufs - 1) & 1, a.limit, a.err);
                    ok = ok && warp_wait(full + s, (turn / kStages) & 1, a.limit, a.err);
                    if (!ok) break;
                    tc_fence_after();
                    if (elect_one()) {
                        const uint32_t at = tiles + s * S::kBytes, p = tile_desc(at), q = tile_desc(at + kMmRows * kMmBlock);
#pragma unroll
                        for (int j = 0; j < 4; ++j) mma8_ss(tmem + b * TN, p + 2 * j, q + 2 * j, idesc, j > 0);
                        mma_commit(empty + s);
                        mma_commit(done + b);
                    }
                    __syncwarp();
                }
            // every product is complete before the tensor memory is freed
            if (elect_one()) {
                mma_commit(&last);
                mbar_drain(&last, 0, a.err);
            }
            __syncwarp();
        }
    } else {
        if constexpr (S::kShift) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(S::kMany));
        // ---- scales and sums ----
        const int row = warp % 4 * 32 + lane, c0 = warp / 4 * kCols;
        const uint32_t from = tmem + ((uint32_t)(warp % 4 * 32) << 16) + c0;
        int turn = 0;
        bool ok = true;
        for (int t = blockIdx.x / a.splits; t < a.tiles; t += step) {
            const int p0 = t % a.tiles_p * kMmRows, q0 = t / a.tiles_p * TN + c0;
            const float* ps = a.p_scale + (long long)(min(p0 + row, a.np - 1) >> a.p_shift) * a.p_row;
            // columns that share a scale: one for all of the warp's; else the lane's of them
            constexpr int kMine = COLS ? (kCols + 31) / 32 : 1;
            const float* qs[kMine];
#pragma unroll
            for (int j = 0; j < kMine; ++j)
                qs[j] = a.q_scale + (long long)(min(q0 + (COLS ? 32 * j + lane : 0), a.nq - 1) >> a.q_shift) * a.q_row;
            // a block's scales are asked for two turns ahead of their use
            float ahead_p[2], ahead_q[2][kMine];
            auto ask = [&](int k, float& p, float (&q)[kMine]) {
                if (k >= k1) return;
                p = ps[k * a.p_block];
#pragma unroll
                for (int j = 0; j < kMine; ++j) q[j] = qs[j][k * a.q_block];
            };
            f32x2 acc[kCols / 2];
#pragma unroll
            for (int i = 0; i < kCols / 2; ++i) acc[i] = 0ull;
            auto add = [&](int k, float& next_p, float (&next_q)[kMine]) {
                const int b = turn % kBufs;
                float scale = next_p;
                if (!COLS) scale *= next_q[0];
                float* cs = col_scales[COLS ? warp : 0][COLS ? turn & 1 : 0];
                if (COLS) {
#pragma unroll
                    for (int j = 0; j < kMine; ++j)
                        if (32 * j + lane < kCols) cs[32 * j + lane] = next_q[j];
                    __syncwarp();
                }
                ask(k + 2, next_p, next_q);
                const f32x2 scale2 = f2_pack(scale, scale);
                if (ok) ok = warp_wait(done + b, (turn / kBufs) & 1, a.limit, a.err);
                ++turn;
                if (!ok) return;
                tc_fence_after();
                // parts of the row: one is on its way while the one before is added
                uint32_t v[2][kPart];
                auto load = [&](int i) {
                    if constexpr (kPart == 32) tmem_ld32(from + b * TN + i * kPart, v[i & 1]);
                    else tmem_ld16(from + b * TN + i * kPart, v[i & 1]);
                };
                load(0);
#pragma unroll
                for (int i = 0; i < kCols / kPart; ++i) {
                    if constexpr (kPart == 32) tmem_wait_ld(v[i & 1]);
                    else tmem_wait_ld16(v[i & 1]);
                    if ((i + 1) * kPart < kCols) {
                        load(i + 1);
                    } else {
                        tc_fence_before();
                        warp_arrive(drained + b);
                    }
#pragma unroll
                    for (int j = 0; j < kPart; j += 4) {
                        const uint32_t* u = v[i & 1] + j;
                        f32x2 lo = f2_pack(__uint_as_float(u[0]), __uint_as_float(u[1])), hi = f2_pack(__uint_as_float(u[2]), __uint_as_float(u[3]));
                        if (COLS) {
                            const float4 w = *reinterpret_cast<const float4*>(cs + i * kPart + j);
                            lo = f2_mul(lo, f2_pack(w.x, w.y));
                            hi = f2_mul(hi, f2_pack(w.z, w.w));
                        }
                        f32x2* to = acc + (i * kPart + j) / 2;
                        to[0] = f2_fma(lo, scale2, to[0]);
                        to[1] = f2_fma(hi, scale2, to[1]);
                    }
                }
            };
            ask(k0, ahead_p[0], ahead_q[0]);
            ask(k0 + 1, ahead_p[1], ahead_q[1]);
            for (int k = k0; k < k1; k += 2) {
                add(k, ahead_p[0], ahead_q[0]);
                if (k + 1 < k1) add(k + 1, ahead_p[1], ahead_q[1]);
            }
            if (a.splits > 1) {
                // the cluster's shares, column by column, in the tiles' place
                float* sums = reinterpret_cast<float*>(dynamic + (tiles - smem_u32(dynamic)));
#pragma unroll
                for (int i = 0; i < kCols / 2; ++i) {
                    const float2 v = f2_unpack(acc[i]);
                    sums[(c0 + 2 * i) * kMmRows + row] = v.x;
                    sums[(c0 + 2 * i + 1) * kMmRows + row] = v.y;
                }
                break;  // one tile for a cluster
            }
            if (p0 + row < a.np) store_row<kCols>(a, acc, (p0 + row) * a.out_p + (long long)q0 * a.out_q, a.nq - q0);
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == S::kWarps + 1) {
        tc_fence_after();
        tmem_free<S::kTmem>(tmem);
    }
    if (a.splits == 1) return;
    // The tensor memory is free before blocks wait for one another: a block that waits for some never holds up one that
    // waits for it.
    cluster_sync();
    const float* sums = reinterpret_cast<const float*>(dynamic + (tiles - smem_u32(dynamic)));
    const int t = blockIdx.x / a.splits, p0 = t % a.tiles_p * kMmRows, q0 = t / a.tiles_p * TN;
    const unsigned me = cluster_rank();
    const int cols = TN / a.splits;  // of the tile, that this block adds and stores
    for (int i = threadIdx.x; i < cols * kMmRows; i += S::kThreads) {
        const int row = i % kMmRows, c = (int)me * cols + i / kMmRows;
        if (p0 + row >= a.np || q0 + c >= a.nq) continue;
        float sum = 0.f;
        for (int r = 0; r < a.splits; ++r) sum += peer_float(sums + c * kMmRows + row, r);
        store_elem(a.out, (p0 + row) * a.out_p + (q0 + c) * a.out_q, a.dtype, sum);
    }
    cluster_sync();  // no block's shared memory goes before the others have read it
}

namespace {

PFN_cuTensorMapEncodeTiled_v12000 encoder() {
    static std::atomic<void*> cache{nullptr};
    void* f = cache.load(std::memory_order_acquire);
    if (!f) {
        cudaDriverEntryPointQueryResult found;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &found) != cudaSuccess ||
            found != cudaDriverEntryPointSuccess)
            return nullptr;
        cache.store(f, std::memory_order_release);
    }
    return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
}

cudaError_t encode(CUtensorMap& map, const void* data, long long k, long long rows, long long stride, int box_rows) {
    auto f = encoder();
    if (!f) return cudaErrorNotSupported;
    const cuuint64_t dims[2] = {(cuuint64_t)k, (cuuint64_t)rows}, strides[1] = {(cuuint64_t)(rows > 1 ? stride : (k + 15) / 16 * 16)};
    const cuuint32_t box[2] = {kMmBlock, (cuuint32_t)box_rows}, step[2] = {1, 1};
    const CUresult r = f(&map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(data), dims, strides, box, step,
                         CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                         CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

template <int TN, bool COLS>
cudaError_t launch(const MmArgs& a, cudaStream_t st) {
    using S = MmShape<TN>;
    auto* kernel = k_matmul_fp8<TN, COLS>;
    static std::atomic<int> cache[256] = {};
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kSmem);
    if (e) return e;
    const int most = resident_blocks(kernel, S::kThreads, S::kSmem, cache);
    if constexpr (S::kShift) {  // registers that the launch does not give would be waited for without end
        static std::atomic<int> given{0};
        int regs = given.load(std::memory_order_relaxed);
        if (regs == 0) {
            cudaFuncAttributes f;
            if ((e = cudaFuncGetAttributes(&f, kernel))) return e;
            given.store(regs = f.numRegs, std::memory_order_relaxed);
        }
        if (regs < S::kLaunch) return cudaErrorLaunchOutOfResources;
    }
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim = {(unsigned)a.splits, 1, 1};
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(a.splits > 1 ? a.tiles * a.splits : std::min(a.tiles, most)));
    cfg.blockDim = dim3(S::kThreads);
    cfg.dynamicSmemBytes = S::kSmem;
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = a.splits > 1 ? 2 : 1;
    count_launches(1);
    return cudaLaunchKernelEx(&cfg, kernel, a);
}

template <bool COLS>
cudaError_t launch(int tn, const MmArgs& a, cudaStream_t st) {
    if constexpr (COLS) {
        if (tn == 16) return launch<16, true>(a, st);
        if (tn == 32) return launch<32, true>(a, st);
        if (tn == 64) return launch<64, true>(a, st);
        if (tn == 256) return launch<256, true>(a, st);
        return launch<128, true>(a, st);
    } else {
        if (tn == 64) return launch<64, false>(a, st);
        if (tn == 128) return launch<128, false>(a, st);
        return launch<256, false>(a, st);
    }
}

}  // namespace

cudaError_t launch_matmul_fp8(const MatmulFp8& x, unsigned* err, cudaStream_t st) {
    MmArgs a{};
    const bool swap = x.m <= 64;  // b's rows along the lanes
    const Fp8Matrix &p = swap ? x.b : x.a, &q = swap ? x.a : x.b;
    const bool cols = q.block == 1;  // scales that differ by column
    a.np = (int)(swap ? x.n : x.m);
    a.nq = (int)(swap ? x.m : x.n);
    a.blocks = (int)((x.k + kMmBlock - 1) / kMmBlock);
    a.p_scale = p.scale;
    a.q_scale = q.scale;
    a.p_row = p.scale_row;
    a.p_block = p.scale_block;
    a.q_row = q.scale_row;
    a.q_block = q.scale_block;
    a.p_shift = p.block == 1 ? 0 : 7;
    a.q_shift = q.block == 1 ? 0 : 7;
    a.out = x.out;
    a.out_p = swap ? 1 : x.out_stride;
    a.out_q = swap ? x.out_stride : 1;
    a.dtype = x.dtype;
    const int size = x.dtype == GS_DTYPE_F32 ? 4 : 2;
    a.wide = !swap && x.out_stride * size % 32 == 0 && reinterpret_cast<uintptr_t>(x.out) % 32 == 0;
    a.limit = 1u << 18;
    a.err = err;
    const int sms = device_sm_count();
    auto over = [](long long n, long long m) { return (n + m - 1) / m; };
    const long long tiles_p = over(a.np, kMmRows);
    int tn;
    if (swap) tn = a.nq <= 16 ? 16 : a.nq <= 32 ? 32 : 64;
    else tn = tiles_p * over(a.nq, 256) >= sms / 2 ? 256 : cols || tiles_p * over(a.nq, 128) >= sms / 2 ? 128 : 64;
    a.tiles_p = (int)tiles_p;
    const long long tiles = tiles_p * over(a.nq, tn);
    if (tiles > 0x0fffffffll) return cudaErrorInvalidConfiguration;
    a.tiles = (int)tiles;
    a.splits = 1;
    const int slots = tn >= 128 ? sms : 2 * sms;
    while (a.splits < 8 && 2 * a.splits * tiles <= slots && 2 * a.splits <= a.blocks) a.splits *= 2;
    if (x.k > 0) {
        cudaError_t e;
        if ((e = encode(a.p, p.data, x.k, a.np, p.stride, kMmRows)) || (e = encode(a.q, q.data, x.k, a.nq, q.stride, tn))) return e;
    }
    return cols ? launch<true>(tn, a, st) : launch<false>(tn, a, st);
}

}  // namespace gs
