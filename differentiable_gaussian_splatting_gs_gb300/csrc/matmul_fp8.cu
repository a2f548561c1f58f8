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
// A warp copies tiles (128 bytes of inner dimension, 128-byte swizzle), two copy scales, one issues the products, the
// others multiply and add; accumulators alternate between places, so that a block's products run beside the additions of the one before.
// Blocks of threads take tiles in turn, and go on copying and multiplying while the result of the last one is stored.
// Large products take tiles of 256 x 256 by pairs of blocks on two SMs, whose products each read both blocks' shared memory
// (every block copies its 128 rows of P and half of Q): one block's 128 x 256 would move 96 KB through its shared memory for
// 512 cycles of products (750 cycles' worth), a pair's moves 64 KB.
// Where tiles are few, a cluster of up to 8 blocks shares the inner dimension of one, joined through their shared
// memory in a fixed order.
//
// Bound by the elementwise warps: a block of 256 x 256 x 128 takes its SMs 512 cycles of products and some 900 of additions (1,380
// where scales differ by column): half of these wait for tensor memory and for one another, each packed multiply-add adds three
// (the registers' ports; scalar ones four). Times in a graph: 16384 x 4096 x 4096 bfloat16 209 us (2.6 PFLOP/s, 69% of twice the measured
// bf16 rate; called back to back 236, at the power limit), 17384 x 4096 x 1024 75 us, 4096 x 1024 x 17,384 with scales by column 100 to 117 us
// (by box); few rows are bound by b's bytes and a launch's latency (1 x 4096 x 1024 4.8 us, 16 x 8192 x 4096 8.3 us, 4.1 TB/s). Sixteen warps of 64 columns instead of eight of
// 128 (234 us), the next block's values asked for before the last of this one are added (240 us), products of 128 columns with
// four accumulators and tiles of 256 x 160 with three (298 us) were slower; so were, with scales by column, loads that give a
// thread two columns of each eight, which read a quarter of the scales (104 to 107 us against 98).
#include <cudaTypedefs.h>

#include <algorithm>

#include "elem.cuh"
#include "fp8.cuh"
#include "gs_internal.h"
#include "pair_ring.h"
#include "tcgen05.cuh"

namespace gs {

constexpr int kMmRows = 128;   // lanes: rows of P in a tile
constexpr int kMmBlock = 128;  // inner dimension of a block, bytes
constexpr int kMmSplits = 8;   // blocks of a cluster that share a tile's inner dimension, at most

struct MmArgs {
    CUtensorMap p, q, to;
    const uint8_t *p_data, *q_data;
    long long p_stride, q_stride;
    const float *p_scale, *q_scale;
    long long p_row, p_block, q_row, q_block;  // strides of the scales
    int p_shift, q_shift;                      // 2^shift rows share a scale
    void* out;
    long long out_p, out_q;  // strides of the result, one of them 1
    int dtype, wide, boxes, np, nq, k, blocks, tiles_p, tiles, splits;  // wide: rows of the result lie on 16 bytes; boxes: columns that `to` has
    unsigned limit, *err;
};

// One product over 32 of the inner dimension; PAIR: of both blocks' rows, issued by the first.
template <bool PAIR>
__device__ __forceinline__ void mma8_ss(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, bool add) {
    if constexpr (PAIR)
        asm volatile(
            "{\n\t.reg .pred p;\n\t.reg .b64 da, db;\n\tsetp.ne.b32 p, %4, 0;\n\tmov.b64 da, {%1, %5};\n\tmov.b64 db, {%2, %5};\n\t"
            "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], da, db, %3, p;\n\t}" ::"r"(d),
            "r"(a), "r"(b), "r"(idesc), "r"((uint32_t)add), "r"(kTileDescHi)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\t.reg .b64 da, db;\n\tsetp.ne.b32 p, %4, 0;\n\tmov.b64 da, {%1, %5};\n\tmov.b64 db, {%2, %5};\n\t"
            "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], da, db, %3, p;\n\t}" ::"r"(d),
            "r"(a), "r"(b), "r"(idesc), "r"((uint32_t)add), "r"(kTileDescHi)
            : "memory");
}
// mma_commit; PAIR: on the barrier at this place in each of the blocks of `mask`.
template <bool PAIR>
__device__ __forceinline__ void mma8_commit(uint64_t* bar, uint16_t mask) {
    if constexpr (PAIR)
        asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(smem_u32(bar)), "h"(mask)
                     : "memory");
    else
        mma_commit(bar);
}
template <int COLS>
__device__ __forceinline__ void tmem_alloc_pair(uint32_t* dst) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(dst)), "n"(COLS) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
}
template <int COLS>
__device__ __forceinline__ void tmem_free_pair(uint32_t addr) {
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(addr), "n"(COLS));
}

// The address of block `rank`'s shared memory at this block's p.
__device__ __forceinline__ uint32_t peer_address(const void* p, unsigned rank) {
    uint32_t a;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
    return a;
}
// One arrival for the whole warp on a barrier of the cluster. Relaxed: it tells of tensor memory that was read, which
// tc_fence_before orders; to release what the thread wrote besides took 1,600 cycles.
__device__ __forceinline__ void warp_arrive_at(uint32_t bar) {
    __syncwarp();
    if (elect_one()) asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}

// The second block's copies are all under way: their turns to the first block's shared memory, and an arrival there.
__device__ __forceinline__ void tell_turns(uint32_t at, uint32_t bar, int turns) {
    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(at), "r"(turns) : "memory");
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ bool mbar_try_wait_cluster(uint64_t* bar, unsigned parity) {
    unsigned ok;
    asm volatile("{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
                 : "=r"(ok)
                 : "r"(smem_u32(bar)), "r"(parity)
                 : "memory");
    return ok != 0;
}
// What end_copies does to the stages' barriers.
struct RingEnd {
    uint64_t* full;
    unsigned *err, bytes;  // bytes: of one block's half
    __device__ __forceinline__ void expect(int s) const { mbar_arrive_expect_tx(full + s, bytes); }
    __device__ __forceinline__ void complete(int s) const {
        asm volatile("mbarrier.complete_tx.relaxed.cta.shared::cta.b64 [%0], %1;" ::"r"(smem_u32(full + s)), "r"(bytes) : "memory");
    }
    __device__ __forceinline__ void drain(int s, unsigned parity) const { mbar_drain(full + s, parity, err); }
};

// A box of a matrix -> this block's shared memory, counted on `bar`: this block's, or (PAIR) one of the pair's.
template <bool PAIR>
__device__ __forceinline__ void tile_load2(uint32_t dst, const CUtensorMap* map, int c0, int c1, uint32_t bar) {
    if constexpr (PAIR)
        asm volatile(
            "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4}], [%2];" ::"r"(dst),
            "l"(map), "r"(bar), "r"(c0), "r"(c1)
            : "memory");
    else
        asm volatile("cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4}], [%2];" ::"r"(dst),
                     "l"(map), "r"(bar), "r"(c0), "r"(c1)
                     : "memory");
}

__device__ __forceinline__ void tmem_ld16(uint32_t addr, uint32_t (&v)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]),
          "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
        : "r"(addr));
}
// Completes the thread's loads (`wait`, once for several); v's values pass through, as in tmem_wait_ld.
__device__ __forceinline__ void tmem_landed(uint32_t (&v)[16], bool wait) {
    if (wait) asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
    asm volatile(""
                 : "+r"(v[0]), "+r"(v[1]), "+r"(v[2]), "+r"(v[3]), "+r"(v[4]), "+r"(v[5]), "+r"(v[6]), "+r"(v[7]), "+r"(v[8]),
                   "+r"(v[9]), "+r"(v[10]), "+r"(v[11]), "+r"(v[12]), "+r"(v[13]), "+r"(v[14]), "+r"(v[15])::"memory");
}

// All threads of the cluster's blocks: what they wrote before to shared memory is seen by the others after.
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// Four floats of block `rank`'s shared memory at this block's address p.
__device__ __forceinline__ float4 peer_floats(const float* p, unsigned rank) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(peer_address(p, rank)) : "memory");
    return v;
}

// What the sizes of a tile decide.
template <int TN>
struct MmShape {
    static constexpr bool kPair = TN == 256;                     // two blocks on two SMs, each with half of Q's tile
    static constexpr int kCols = kPair ? 128 : TN < 64 ? TN : 64;  // columns of an elementwise warp
    static constexpr int kWarps = 4 * (TN / kCols);              // elementwise
    static constexpr int kThreads = 32 * (kWarps + 4);           // and a warpgroup for the copies and the products
    // Registers of the pair's 384 threads: of the 168 that the launch gives each, the last warpgroup leaves all but 40,
    // and the elementwise two take 232: 128 x 40 + 256 x 232 = 384 x 168.
    static constexpr int kLaunch = 168, kFew = 40, kMany = 232;
    static_assert(!kPair || 128 * kFew + (kThreads - 128) * kMany <= kThreads * kLaunch);
    static constexpr int kTileQ = kPair ? TN / 2 : TN;           // rows of Q that a block copies
    static constexpr int kBytes = (kMmRows + kTileQ) * kMmBlock; // a stage: both operands' tiles
    // Results' rows leave by boxes of 32 rows x 128 bytes, so many of each warp's (none with b's rows along the lanes).
    template <bool COLS>
    static constexpr int kBoxes = kPair ? 2 : !COLS || TN >= 128 ? 1 : 0;
    static constexpr int kResident = TN >= 128 ? 1 : 2;          // blocks of threads on an SM
    template <bool COLS>
    static constexpr int kStages = kPair ? 4 : TN == 64 && !COLS ? 3 : TN == 64 ? 4 : 5;
    static constexpr int kBufs = TN == 128 ? 4 : 2;              // accumulators
    static constexpr int kTmem = kBufs * TN;
    template <bool COLS>
    static constexpr int kSmem = 1024 + kStages<COLS> * kBytes + kWarps * kBoxes<COLS> * 4096;
    static_assert(kTmem >= 32 && kResident * kTmem <= 512 && (kTmem & (kTmem - 1)) == 0);
    static_assert(kPair || kStages<false> * kBytes >= kMmRows * (TN + 4) * 4, "a cluster's sums take the tiles' place");
};

// Scales of so many blocks of the inner dimension are copied at a time, to so many places: 8 to 12 blocks ahead of their use.
// (Loaded into registers two blocks ahead, their latency under the tiles' traffic decided the pace of 256 x 256 tiles: 16384 x 4096
// x 4096 bf16 took 707 us where it took 220 so.)
constexpr int kMmBatch = 4, kMmPlaces = 3;
template <int TN, bool COLS>
struct MmScales {
    float p[kMmPlaces][kMmRows][kMmBatch];
    float q[kMmPlaces][COLS ? kMmBatch * TN : (TN + kQBlock - 1) / kQBlock * kMmBatch];  // COLS: [batch][column], else [column / 128][batch]
};

// ---- scales at the ends of float32's range ----
// The hot loop multiplies in float32: by the product of both scales, or (COLS) by the column's and then the row's. That holds
// where the product is a normal number, or a value times the column's scale is (values are 0 or lie between 2^-18, the product of
// two subnormals, and 128 x 448^2 < 2^25). The warps that copy the scales, which have the time, note the smallest and the largest;
// a block whose scales can leave that range looks at its tiles again when they are stored, and forms the elements that have such
// scales once more, with the scales' powers apart. (The test and another form within the hot loop took a quarter to a half of its
// time, 16384 x 4096 x 4096 bf16 265 us instead of 210, whatever the scales.)
struct ScaleRange {
    unsigned least, most;  // magnitudes; the least less one, so that 0 counts as the largest; the most without infinities and NaN
    __device__ __forceinline__ void add(float s) {
        const unsigned m = magnitude(s);
        least = min(least, m - 1);
        if (m < 0x7f800000u) most = max(most, m);
    }
};
constexpr float kLeastColumn = 0x1p-108f, kMostColumn = 0x1p102f;
__device__ __forceinline__ bool leaves_range(float row, float column, bool cols) {
    const float s = fabsf(cols ? column : row * column);
    const bool in = cols ? s >= kLeastColumn && s <= kMostColumn : s >= 0x1p-126f && s < INFINITY;
    return !in && row != 0.f && column != 0.f && isfinite(row) && isfinite(column);
}
// Whether any of the block's scales may.
__device__ __forceinline__ bool may_leave_range(const ScaleRange& p, const ScaleRange& q, bool cols) {
    return leaves_range(__uint_as_float(p.least + 1), __uint_as_float(q.least + 1), cols) ||
           leaves_range(__uint_as_float(p.most), __uint_as_float(q.most), cols);
}

// A scale as m 2^e, 1 <= |m| < 2 (zeros, infinities and NaN: e = 0), so that two of them multiply without leaving float32.
struct SplitScale {
    float m;
    int e;
    __device__ __forceinline__ explicit SplitScale(float s) : m(s), e(0) {
        if (s == 0.f || !isfinite(s)) return;
        if (magnitude(s) < 0x00800000u) m = s * 0x1p64f, e = -64;
        const unsigned u = __float_as_uint(m);
        e += (int)(u >> 23 & 255u) - 127;
        m = __uint_as_float((u & 0x807fffffu) | 0x3f800000u);
    }
};
__device__ __forceinline__ float power_of_2(int e) { return __uint_as_float((unsigned)(e + 127) << 23); }  // -126 <= e <= 127
// sum + v a b: the scales' power in two parts, the one within the multiply-add a normal number, the other before it, where v 2^e a and
// b's significands stay in range or what they give does not (|v| >= 2^-18 with 2^100 before 2^126 is an infinity, 2^27 with 2^-126 twice 0).
__device__ __forceinline__ float add_split(float v, const SplitScale& a, const SplitScale& b, float sum) {
    const int e = a.e + b.e, last = min(max(e, -126), 126), before = min(max(e - last, -126), 100);
    return fmaf(v * (a.m * b.m * power_of_2(before)), power_of_2(last), sum);
}

// 16 bytes of a row from byte `at` on, zeros behind its k.
__device__ __forceinline__ uint4 row16(const uint8_t* row, int at, int k) {
    if (at + 16 <= k) return *reinterpret_cast<const uint4*>(row + at);
    unsigned long long low = 0, high = 0;
#pragma unroll 1
    for (int i = 0; at + i < k; ++i) (i < 8 ? low : high) |= (unsigned long long)row[at + i] << 8 * (i % 8);
    return make_uint4((uint32_t)low, (uint32_t)(low >> 32), (uint32_t)high, (uint32_t)(high >> 32));
}
// Two e4m3 values (of the word's lower or upper half) as float16, which holds all of them.
__device__ __forceinline__ uint32_t halves(uint32_t w, int upper) {
    uint32_t r;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"((uint16_t)(w >> 16 * upper)));
    return r;
}
// c [16 x 8] += a [16 x 16] b [16 x 8] of float16 in float32, by the warp.
__device__ __forceinline__ void warp_mma(float (&c)[4], const uint32_t (&a)[4], const uint32_t (&b)[2]) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]));
}
// The elements of a tile of `rows` x `cols` at (p0, q0) once more that have a scale which leaves the range, in a block of the inner dimension
// of k0 .. k1 first (the blocks of a cluster share a tile's). A warp forms 16 x 16 elements where any of them does, with the warp's own
// tensor-core products, which need neither tensor memory nor another warp: the tile's way of forming them is over. A lane has 16
// bytes in a row of each operand's rows g and g + 8 (g = lane / 4), and the products take these in the same order in both.
__device__ __forceinline__ void form_again(const MmArgs& a, int p0, int rows, int q0, int cols, int k0, int k1, int warp, int warps) {
    const int lane = threadIdx.x & 31, g = lane / 4, t = lane % 4;
    const bool by_col = a.q_shift == 0;
    rows = min(rows, a.np - p0);
    cols = min(cols, a.nq - q0);
    auto p_scale = [&](int p) { return a.p_scale + (long long)(min(p, a.np - 1) >> a.p_shift) * a.p_row; };
    auto q_scale = [&](int q) { return a.q_scale + (long long)(min(q, a.nq - 1) >> a.q_shift) * a.q_row; };
    for (int r0 = warp * 16; r0 < rows; r0 += warps * 16) {
        bool any = false;
        for (int c0 = 0; c0 < cols; c0 += 16) {
            if (by_col || c0 % kQBlock == 0) {  // (tiles start where their columns' common scales do, or hold no others)
                any = false;
                const float *sp = p_scale(p0 + r0 + lane % 16), *sq = q_scale(q0 + c0 + (by_col ? lane % 16 : 0));
                for (int k = lane / 16; k < a.blocks; k += 2) any |= leaves_range(by_col ? 1.f : sp[k * a.p_block], sq[k * a.q_block], by_col);
                any = __any_sync(0xffffffffu, any);
            }
            if (!any) continue;
            const int p = p0 + r0 + g, q = q0 + c0 + g;
            const uint8_t* x[2] = {a.p_data + min(p, a.np - 1) * a.p_stride, a.p_data + min(p + 8, a.np - 1) * a.p_stride};
            const uint8_t* y[2] = {a.q_data + min(q, a.nq - 1) * a.q_stride, a.q_data + min(q + 8, a.nq - 1) * a.q_stride};
            float sum[2][4] = {};
            unsigned left = 0, mine = 0;  // elements that have left the range, and those that did within k0 .. k1
            for (int k = 0; k < a.blocks; ++k) {
                float c[2][4] = {};
#pragma unroll 1
                for (int h = 0; h < 2; ++h) {
                    const int at = k * kMmBlock + 64 * h + 16 * t;
                    const uint4 u0 = row16(x[0], at, a.k), u1 = row16(x[1], at, a.k), v0 = row16(y[0], at, a.k), v1 = row16(y[1], at, a.k);
                    const uint32_t u[2][4] = {{u0.x, u0.y, u0.z, u0.w}, {u1.x, u1.y, u1.z, u1.w}}, v[2][4] = {{v0.x, v0.y, v0.z, v0.w}, {v1.x, v1.y, v1.z, v1.w}};
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const uint32_t ma[4] = {halves(u[0][i], 0), halves(u[1][i], 0), halves(u[0][i], 1), halves(u[1][i], 1)};
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            const uint32_t mb[2] = {halves(v[j][i], 0), halves(v[j][i], 1)};
                            warp_mma(c[j], ma, mb);
                        }
                    }
                }
#pragma unroll
                for (int j = 0; j < 2; ++j)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float sp = p_scale(p + i / 2 * 8)[k * a.p_block], sq = q_scale(q0 + c0 + 8 * j + 2 * t + i % 2)[k * a.q_block];
                        sum[j][i] = add_split(c[j][i], SplitScale(sp), SplitScale(sq), sum[j][i]);
                        const unsigned bit = 1u << (4 * j + i);
                        if (!(left & bit) && leaves_range(sp, sq, by_col)) {
                            left |= bit;
                            if (k >= k0 && k < k1) mine |= bit;
                        }
                    }
            }
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int row = r0 + g + i / 2 * 8, col = c0 + 8 * j + 2 * t + i % 2;
                    if ((mine >> (4 * j + i) & 1u) && row < rows && col < cols) store_elem(a.out, (p0 + row) * a.out_p + (q0 + col) * a.out_q, a.dtype, sum[j][i]);
                }
        }
    }
}
// ... all of the block's tiles, by `warps` of its warps, this the `warp`-th.
__device__ __forceinline__ void form_tiles_again(const MmArgs& a, int tn, int warp, int warps) {
    const bool pair = tn == 256;
    const int group = pair ? 2 : a.splits, rank = blockIdx.x % group;
    const int k0 = pair ? 0 : (int)((long long)a.blocks * rank / group), k1 = pair ? a.blocks : (int)((long long)a.blocks * (rank + 1) / group);
    for (int t = blockIdx.x / group; t < a.tiles; t += gridDim.x / group)
        form_again(a, t % a.tiles_p * (pair ? 2 * kMmRows : kMmRows) + (pair ? rank * kMmRows : 0), kMmRows, t / a.tiles_p * tn, tn, k0, k1, warp, warps);
}
// The same apart from the caller's code. (In the pair's kernel, or anywhere but at the end of its elementwise warps' part, it cost their
// loop, which has no register left, a fifth of its time: 16384 x 4096 x 4096 bf16 247 us.)
__device__ __noinline__ void call_form_tiles_again(const MmArgs& a, int tn, int warp, int warps) { form_tiles_again(a, tn, warp, warps); }

// Barrier ID of the block, for THREADS threads: its arrivals, and those that wait for them.
template <int ID, int THREADS>
__device__ __forceinline__ void named_arrive() { asm volatile("bar.arrive %0, %1;" ::"n"(ID), "n"(THREADS) : "memory"); }
template <int ID, int THREADS>
__device__ __forceinline__ void named_sync() { asm volatile("bar.sync %0, %1;" ::"n"(ID), "n"(THREADS) : "memory"); }

// Counts an arrival of the thread once its asynchronous copies so far have landed.
__device__ __forceinline__ void cp_async_arrive(uint64_t* bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}

// A box of this block's shared memory -> a matrix; what lies outside is left out. Counts to the thread's bulk group.
__device__ __forceinline__ void tile_store2(const CUtensorMap* map, int c0, int c1, uint32_t src) {
    asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%2, %3}], [%1];\n\tcp.async.bulk.commit_group;" ::"l"(map), "r"(src),
                 "r"(c0), "r"(c1)
                 : "memory");
}

// A warp's 32 rows of a tile, COLS columns of them in every thread's sums, the first at (q0, p0) of the result. Where its rows lie
// on 16 bytes: by tiled copies of 128 bytes of each row, laid out (with the copies' swizzle) in BOXES times 4 KB of the warp's, which
// the warp leaves under way. (Until they are stored the products can only go two blocks ahead. Stored by each thread from its
// row a tile of 256 x 256 took 2.2 us, coalesced through 2 KB of shared memory 1.9 us, so 1.2.) Else element by element.
template <int COLS, int BOXES>
__device__ __forceinline__ void store_rows(const MmArgs& a, const f32x2 (&acc)[COLS / 2], unsigned char* stage, int p0, int q0) {
    const int lane = threadIdx.x & 31, rows = a.np - p0, left = a.nq - q0;
    if (rows <= 0 || left <= 0) return;
    // a tiled copy writes whole 16 bytes: what the result has behind its last is stored by the threads
    const int whole = a.boxes - q0;
    if (whole < min(left, COLS) && lane < rows) {
        const long long at = (p0 + lane) * a.out_p + q0 * a.out_q;
#pragma unroll
        for (int i = 0; i < COLS / 2; ++i) {
            const float2 v = f2_unpack(acc[i]);
            if (2 * i >= whole && 2 * i < left) store_elem(a.out, at + 2 * i * a.out_q, a.dtype, v.x);
            if (2 * i + 1 >= whole && 2 * i + 1 < left) store_elem(a.out, at + (2 * i + 1) * a.out_q, a.dtype, v.y);
        }
    }
    __syncwarp();
    if constexpr (BOXES > 0) {
        auto boxes = [&](auto per, auto word) {  // word(i): the 16 bytes of the thread's row from column i on, `per` columns
            constexpr int kPer = decltype(per)::value, kBox = 8 * kPer;
#pragma unroll
            for (int c0 = 0; c0 < COLS; c0 += BOXES * kBox) {
                if (whole <= c0) break;
                if (elect_one()) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");  // the copies before have read the boxes
                __syncwarp();
#pragma unroll
                for (int x = 0; x < BOXES; ++x) {
                    if (c0 + x * kBox >= COLS) break;
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        if (c0 + x * kBox + i * kPer < COLS)
                            *reinterpret_cast<uint4*>(stage + x * 4096 + lane * 128 + ((i ^ lane) & 7) * 16) = word(c0 + x * kBox + i * kPer);
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (elect_one())
#pragma unroll
                    for (int x = 0; x < BOXES; ++x)
                        if (c0 + x * kBox < COLS && c0 + x * kBox < whole) tile_store2(&a.to, q0 + c0 + x * kBox, p0, smem_u32(stage) + x * 4096);
                __syncwarp();
            }
        };
        if (a.dtype == GS_DTYPE_F32)
            boxes(std::integral_constant<int, 4>(), [&](int c) {
                const float2 x = f2_unpack(acc[c / 2]), y = f2_unpack(acc[c / 2 + 1]);
                return make_uint4(__float_as_uint(x.x), __float_as_uint(x.y), __float_as_uint(y.x), __float_as_uint(y.y));
            });
        else
            boxes(std::integral_constant<int, 8>(), [&](int c) {
                uint32_t w[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float2 x = f2_unpack(acc[c / 2 + i]);
                    w[i] = a.dtype == GS_DTYPE_F16 ? pack2<__half>(x.x, x.y) : pack2<__nv_bfloat16>(x.x, x.y);
                }
                return make_uint4(w[0], w[1], w[2], w[3]);
            });
    }
}

template <int TN, bool COLS>
__global__ void __launch_bounds__(MmShape<TN>::kThreads, MmShape<TN>::kResident) k_matmul_fp8(const __grid_constant__ MmArgs a) {
    using S = MmShape<TN>;
    constexpr bool kPair = S::kPair, kAlone = !COLS && TN >= 128;
    constexpr int kStages = S::template kStages<COLS>, kBufs = S::kBufs, kCols = S::kCols, kGroup = kAlone ? 64 : 16;
    extern __shared__ unsigned char dynamic[];
    __shared__ uint64_t full[kStages], empty[kStages], done[kBufs], drained[kBufs], last;
    __shared__ uint32_t tmem_at;
    __shared__ uint64_t scaled[kMmPlaces], used[kMmPlaces], told;
    __shared__ int others_turns;  // of a pair's second block, in the first
    __shared__ __align__(16) MmScales<TN, COLS> scales;
    __shared__ ScaleRange ranges[2];  // of P's scales and of Q's
    const uint32_t tiles = (smem_u32(dynamic) + 1023) & ~1023u;
    const int warp = threadIdx.x / 32, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int i = 0; i < kStages; ++i) {
            mbar_init(full + i, 1);
            mbar_init(empty + i, 1);
        }
        for (int i = 0; i < kBufs; ++i) {
            mbar_init(done + i, 1);
            mbar_init(drained + i, kPair ? 2 * S::kWarps : S::kWarps);
        }
        for (int i = 0; i < kMmPlaces; ++i) {
            mbar_init(scaled + i, 64);
            mbar_init(used + i, S::kWarps);
        }
        mbar_init(&last, 1);
        if (kPair) mbar_init(&told, 1);
        fence_mbar_init();
    }
    // Tensor memory is taken once the kernel before has given up its own, and before the next one's blocks may come, which
    // would otherwise hold what a block of this or of that one waits for.
    pdl_wait();
    if (warp == S::kWarps + 1) {
        if constexpr (kPair) tmem_alloc_pair<S::kTmem>(&tmem_at);
        else tmem_alloc<S::kTmem>(&tmem_at);
    }
    tc_fence_before();
    __syncthreads();
    if constexpr (kPair) cluster_sync();  // the barriers of both are ready
    tc_fence_after();
    pdl_launch_dependents();
    const uint32_t tmem = tmem_at;
    // The blocks that share a tile: a pair with 128 of its rows each, or a cluster with shares of the inner dimension.
    const int group = kPair ? 2 : a.splits, rank = blockIdx.x % group, first = blockIdx.x / group, step = gridDim.x / group;
    const int k0 = kPair ? 0 : (int)((long long)a.blocks * rank / group), k1 = kPair ? a.blocks : (int)((long long)a.blocks * (rank + 1) / group);
    constexpr int kRows = kPair ? 2 * kMmRows : kMmRows;  // of P in a tile
    const int row_of = kPair ? rank * kMmRows : 0;
    if (warp >= S::kWarps) {
        if constexpr (kPair) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(S::kFew));
        if (warp == S::kWarps) {
            // ---- copies ----
            if (elect_one()) {
                const uint32_t bars = kPair ? peer_address(full, 0) : smem_u32(full);
                int s = 0, turns = 0;
                unsigned phase = 1;  // of the stage's products before: a new barrier's is over
                bool ok = true;
                for (int t = first; t < a.tiles && ok; t += step) {
                    const int p0 = t % a.tiles_p * kRows + row_of, q0 = t / a.tiles_p * TN + (kPair ? rank * S::kTileQ : 0);
                    for (int k = k0; k < k1; ++k) {
                        if (!(ok = mbar_wait_bounded(empty + s, phase, a.limit, a.err))) break;
                        const uint32_t at = tiles + s * S::kBytes;
                        // (a pair's bytes are all counted by its first block, which issues the products)
                        if (row_of == 0) mbar_arrive_expect_tx(full + s, kPair ? 2 * S::kBytes : S::kBytes);
                        tile_load2<kPair>(at, &a.p, k * kMmBlock, p0, bars + 8 * s);
                        tile_load2<kPair>(at + kMmRows * kMmBlock, &a.q, k * kMmBlock, q0, bars + 8 * s);
                        ++turns;
                        if (++s == kStages) s = 0, phase ^= 1;
                    }
                }
                // every copy has landed before the blocks end, in a pair those of both (which stop apart where a wait gave up)
                if (kPair && rank == 1) {
                    tell_turns(peer_address(&others_turns, 0), peer_address(&told, 0), turns);
                } else {
                    int others = turns;
                    if (kPair && poll_drain([&] { return mbar_try_wait_cluster(&told, 0); })) others = others_turns;
                    end_copies<kStages>(turns, others, RingEnd{full, a.err, (unsigned)S::kBytes});
                }
            }
            __syncwarp();
        } else if (warp == S::kWarps + 1) {
            // ---- products ----
            constexpr uint32_t idesc = (1u << 4) | ((uint32_t)(TN >> 3) << 17) | ((uint32_t)(kRows >> 4) << 24);  // e4m3 x e4m3, float32
            int s = 0, b = 0;
            unsigned s_phase = 0, b_phase = 1;  // (a new accumulator's reading is over)
            bool ok = row_of == 0;
            for (int t = first; t < a.tiles && ok; t += step)
                for (int k = k0; k < k1; ++k) {
                    // lanes wait for the tiles or for the accumulator
                    if (!(ok = warp_wait_all(full + s, s_phase, drained + b, b_phase, a.limit, a.err))) break;
                    tc_fence_after();
                    if (elect_one()) {
                        const uint32_t at = tiles + s * S::kBytes, p = tile_desc(at), q = tile_desc(at + kMmRows * kMmBlock);
#pragma unroll
                        for (int j = 0; j < 4; ++j) mma8_ss<kPair>(tmem + b * TN, p + 2 * j, q + 2 * j, idesc, j > 0);
                        mma8_commit<kPair>(done + b, 3);
                        mma8_commit<kPair>(empty + s, 3);
                    }
                    __syncwarp();
                    if (++s == kStages) s = 0, s_phase ^= 1;
                    if (++b == kBufs) b = 0, b_phase ^= 1;
                }
            // every product is complete before the tensor memory is freed
            if (row_of == 0 && elect_one()) {
                mma8_commit<kPair>(&last, 1);
                mbar_drain(&last, 0, a.err);
            }
            __syncwarp();
        } else {
            // ---- scales: one warp P's, one Q's, each lane its rows (or columns) ----
            const bool of_q = warp == S::kWarps + 3;
            constexpr int kOfQ = COLS ? (TN + 31) / 32 : 1, kMost = kOfQ > kMmRows / 32 ? kOfQ : kMmRows / 32;
            const long long next = of_q ? a.q_block : a.p_block;
            int batch = 0, sizes = 0;  // sizes: of the last three batches, the last one's in the lowest four bits
            ScaleRange range{~0u, 0u};
            auto note = [&](int at, int n) {  // what the lane copied to a place, which has landed
                if (COLS && !of_q) {  // the columns' decide
                    range.add(1.f);
                } else if (of_q) {
                    for (int j = 0; j < n; ++j)
#pragma unroll
                        for (int i = 0; i < kOfQ; ++i)
                            if (COLS ? 32 * i + lane < TN : lane * kQBlock < TN) range.add(scales.q[at][COLS ? j * TN + 32 * i + lane : lane * kMmBatch + j]);
                } else {
#pragma unroll
                    for (int i = 0; i < kMmRows / 32; ++i) {
                        const float4 s = *reinterpret_cast<const float4*>(scales.p[at][32 * i + lane]);
                        range.add(s.x);
                        if (n > 1) range.add(s.y);
                        if (n > 2) range.add(s.z);
                        if (n > 3) range.add(s.w);
                    }
                }
            };
            bool ok = true;
            for (int t = first; t < a.tiles && ok; t += step) {
                const int p0 = t % a.tiles_p * kRows + row_of, q0 = t / a.tiles_p * TN;
                const float* from[kMost];
#pragma unroll
                for (int i = 0; i < kMost; ++i) {
                    const int p = min(p0 + 32 * i + lane, a.np - 1), q = min(q0 + (COLS ? 32 * i + lane : lane * kQBlock), a.nq - 1);
                    from[i] = of_q ? a.q_scale + (long long)(q >> a.q_shift) * a.q_row : a.p_scale + (long long)(p >> a.p_shift) * a.p_row;
                    from[i] += k0 * next;
                }
                for (int k = k0; k < k1; k += kMmBatch, ++batch) {
                    const int at = batch % kMmPlaces;
                    if (batch >= kMmPlaces) {
                        if (!(ok = warp_wait(used + at, (batch / kMmPlaces - 1) & 1, a.limit, a.err))) break;
                        note(at, sizes >> 4 * (kMmPlaces - 1) & 15);
                    }
                    sizes = sizes << 4 | min(kMmBatch, k1 - k);
#pragma unroll
                    for (int j = 0; j < kMmBatch; ++j) {
                        if (k + j >= k1) break;
                        if (of_q) {
#pragma unroll
                            for (int i = 0; i < kOfQ; ++i)
                                if (COLS ? 32 * i + lane < TN : lane * kQBlock < TN) cp_async4(&scales.q[at][COLS ? j * TN + 32 * i + lane : lane * kMmBatch + j], from[i]);
                        } else {
#pragma unroll
                            for (int i = 0; i < kMmRows / 32; ++i) cp_async4(&scales.p[at][32 * i + lane][j], from[i]);
                        }
#pragma unroll
                        for (int i = 0; i < kMost; ++i) from[i] += next;
                    }
                    cp_async_arrive(scaled + at);
                }
            }
            cp_async_wait_all();
            for (int i = 0; i < min(batch, kMmPlaces); ++i) note((batch - 1 - i) % kMmPlaces, sizes >> 4 * i & 15);
            range.least = __reduce_min_sync(0xffffffffu, range.least);
            range.most = __reduce_max_sync(0xffffffffu, range.most);
            if (lane == 0) ranges[of_q] = range;
        }
        if constexpr (kPair) named_arrive<1, S::kThreads>();  // the ranges are there
    } else {
        if constexpr (kPair) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(S::kMany));
        // ---- scales and sums ----
        const int row = warp % 4 * 32 + lane, c0 = warp / 4 * kCols;
        const uint32_t from = tmem + ((uint32_t)(warp % 4 * 32) << 16) + c0;
        int b = 0, at = 0;  // the next block's accumulators, its batch's place of scales
        unsigned b_phase = 0, at_phase = 0;
        bool ok = true;
        const uint32_t drained_at = kPair ? peer_address(drained, 0) : 0;
        bool mine = true;
        for (int t = first; t < a.tiles; t += step) {
            const int p0 = t % a.tiles_p * kRows + row_of, q0 = t / a.tiles_p * TN + c0;
            f32x2 acc[kCols / 2];
#pragma unroll
            for (int i = 0; i < kCols / 2; ++i) acc[i] = 0ull;
            for (int k = k0; k < k1 && ok; k += kMmBatch) {
                if (!(ok = warp_wait(scaled + at, at_phase, a.limit, a.err) && (!kAlone || __all_sync(0xffffffffu, mine)))) break;
                // (unrolled, with the batch's scales of the rows in registers: 98 instead of 101 us for 4096 x 1024 x 17,384 with scales by column,
                // but 307 instead of 205 for 16384 x 4096 x 4096 without, for want of registers)
                float4 of_p = make_float4(0.f, 0.f, 0.f, 0.f);
                if (COLS) of_p = *reinterpret_cast<const float4*>(scales.p[at][row]);
                const float each[kMmBatch] = {of_p.x, of_p.y, of_p.z, of_p.w};
#pragma unroll(COLS ? kMmBatch : 1)
                for (int j = 0; j < kMmBatch; ++j) {
                    if (k + j >= k1) break;
                    float scale;
                    if constexpr (COLS) scale = each[j];
                    else scale = scales.p[at][row][j] * scales.q[at][c0 / kQBlock * kMmBatch + j];
                    const f32x2 scale2 = f2_pack(scale, scale);
                    // (kAlone: each lane waits for itself, 205 us instead of 219 for 16384 x 4096 x 4096, with 64 columns loaded at a time: a lane that gave
                    // up goes on with its warp to the next batch, where all learn of it)
                    if constexpr (kAlone) {
                        mine &= __builtin_expect(mbar_try_wait(done + b, b_phase), 1) || mbar_wait_bounded(done + b, b_phase, a.limit, a.err);
                        __syncwarp();
                    } else if (!(ok = warp_wait(done + b, b_phase, a.limit, a.err))) {
                        break;
                    }
                    tc_fence_after();
                    const float* cs = scales.q[at] + (COLS ? j * TN + c0 : 0);
#pragma unroll
                    for (int g = 0; g < kCols; g += kGroup) {
                        uint32_t v[kGroup / 16][16];
#pragma unroll
                        for (int i = 0; i < kGroup / 16; ++i) tmem_ld16(from + b * TN + g + 16 * i, v[i]);
#pragma unroll
                        for (int i = 0; i < kGroup / 16; ++i) tmem_landed(v[i], i == 0);
                        if (g + kGroup == kCols) {
                            tc_fence_before();
                            if constexpr (kPair) warp_arrive_at(drained_at + 8 * b);
                            else warp_arrive(drained + b);
                        }
#pragma unroll
                        for (int c = 0; c < kGroup; c += 4) {
                            const uint32_t* u = v[c / 16] + c % 16;
                            f32x2 lo = f2_pack(__uint_as_float(u[0]), __uint_as_float(u[1])), hi = f2_pack(__uint_as_float(u[2]), __uint_as_float(u[3]));
                            if (COLS) {
                                const float4 w = *reinterpret_cast<const float4*>(cs + g + c);
                                lo = f2_mul(lo, f2_pack(w.x, w.y));
                                hi = f2_mul(hi, f2_pack(w.z, w.w));
                            }
                            f32x2* to = acc + (g + c) / 2;
                            to[0] = f2_fma(lo, scale2, to[0]);
                            to[1] = f2_fma(hi, scale2, to[1]);
                        }
                    }
                    if (++b == kBufs) b = 0, b_phase ^= 1;
                }
                warp_arrive(used + at);
                if (++at == kMmPlaces) at = 0, at_phase ^= 1;
            }
            if (!kPair && group > 1) {
                // the cluster's shares, in the tiles' place: rows where the result's rows are the lanes', else columns
                float* sums = reinterpret_cast<float*>(dynamic + (tiles - smem_u32(dynamic)));
#pragma unroll
                for (int i = 0; i < kCols / 2; i += 2) {
                    const float2 x = f2_unpack(acc[i]), y = f2_unpack(acc[i + 1]);
                    if (a.out_q == 1) {
                        *reinterpret_cast<float4*>(sums + row * (TN + 4) + c0 + 2 * i) = make_float4(x.x, x.y, y.x, y.y);
                    } else {
                        float* to = sums + (c0 + 2 * i) * kMmRows + row;
                        to[0] = x.x, to[kMmRows] = x.y, to[2 * kMmRows] = y.x, to[3 * kMmRows] = y.y;
                    }
                }
                break;  // one tile for a cluster
            }
            store_rows<kCols, S::template kBoxes<COLS>>(a, acc, dynamic + (tiles - smem_u32(dynamic)) + kStages * S::kBytes + warp * (S::template kBoxes<COLS> * 4096),
                                                        p0 + warp % 4 * 32, q0);
            __syncwarp();  // the instructions on tensor memory and the cluster's barriers take whole warps
        }
        if (S::template kBoxes<COLS> && elect_one()) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");  // the result is written
        __syncwarp();
        if constexpr (kPair) {
            named_sync<1, S::kThreads>();  // all results are stored
            if (may_leave_range(ranges[0], ranges[1], COLS)) form_tiles_again(a, TN, warp, S::kWarps);
        }
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if constexpr (kPair) {
        cluster_sync();  // the first block's products and copies are over, which use the second's memory too
        if (warp == S::kWarps + 1) {
            tc_fence_after();
            tmem_free_pair<S::kTmem>(tmem);
        }
    } else {
        if (warp == S::kWarps + 1) {
            tc_fence_after();
            tmem_free<S::kTmem>(tmem);
        }
        if (group > 1) {
            // The tensor memory is free before blocks wait for one another: a block that waits for some never holds up one that
            // waits for it.
            cluster_sync();
            const float* sums = reinterpret_cast<const float*>(dynamic + (tiles - smem_u32(dynamic)));
            const int p0 = first % a.tiles_p * kMmRows, q0 = first / a.tiles_p * TN;
            const bool by_row = a.out_q == 1;  // four elements that lie together in the result to a thread
            const int lines = by_row ? kMmRows : TN, fours = (by_row ? TN : kMmRows) / 4, pitch = by_row ? TN + 4 : kMmRows;
            const int l0 = lines * rank / group, l1 = lines * (rank + 1) / group;
            for (int i = l0 * fours + threadIdx.x; i < l1 * fours; i += S::kThreads) {
                const int line = i / fours, at = i % fours * 4;
                const int p = p0 + (by_row ? line : at), q = q0 + (by_row ? at : line), left = by_row ? a.nq - q : a.np - p;
                if (p >= a.np || q >= a.nq) continue;
                float4 v[kMmSplits];
#pragma unroll
                for (int r = 0; r < kMmSplits; ++r)
                    if (r < group) v[r] = peer_floats(sums + line * pitch + at, r);
                float4 t = v[0];
#pragma unroll
                for (int r = 1; r < kMmSplits; ++r)
                    if (r < group) t.x += v[r].x, t.y += v[r].y, t.z += v[r].z, t.w += v[r].w;
                const long long to = p * a.out_p + q * a.out_q;
                if (a.wide && left >= 4) {
                    if (a.dtype == GS_DTYPE_F32) *reinterpret_cast<float4*>(static_cast<float*>(a.out) + to) = t;
                    else if (a.dtype == GS_DTYPE_F16) *reinterpret_cast<uint2*>(static_cast<__half*>(a.out) + to) = make_uint2(pack2<__half>(t.x, t.y), pack2<__half>(t.z, t.w));
                    else *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.out) + to) = make_uint2(pack2<__nv_bfloat16>(t.x, t.y), pack2<__nv_bfloat16>(t.z, t.w));
                } else {
                    const float each[4] = {t.x, t.y, t.z, t.w};
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (e < left) store_elem(a.out, to + e, a.dtype, each[e]);
                }
            }
            __syncwarp();
            cluster_sync();  // no block's shared memory goes before the others have read it
        }
    }
    if (!kPair && may_leave_range(ranges[0], ranges[1], COLS)) call_form_tiles_again(a, TN, warp, S::kThreads / 32);
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

// Boxes of 128 bytes x box_rows of `rows` rows of `cols` elements, `stride` elements apart.
cudaError_t encode(CUtensorMap& map, CUtensorMapDataType type, int size, const void* data, long long cols, long long rows, long long stride, int box_rows) {
    auto f = encoder();
    if (!f) return cudaErrorNotSupported;
    const cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows}, strides[1] = {(cuuint64_t)(rows > 1 ? stride * size : (cols * size + 15) / 16 * 16)};
    const cuuint32_t box[2] = {(cuuint32_t)(kMmBlock / size), (cuuint32_t)box_rows}, step[2] = {1, 1};
    const CUresult r = f(&map, type, 2, const_cast<void*>(data), dims, strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                         CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

// Pairs of blocks that run at once on the current device (an SM may have no partner), looked up once.
template <class Kernel>
int resident_pairs(Kernel kernel, const cudaLaunchConfig_t& cfg, std::atomic<int> (&cache)[256]) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 256) return 0;
    int v = cache[dev].load(std::memory_order_relaxed);
    if (v == 0) {
        if (cudaOccupancyMaxActiveClusters(&v, kernel, &cfg) != cudaSuccess) return 0;
        cache[dev].store(v, std::memory_order_relaxed);
    }
    return v;
}

template <int TN, bool COLS>
cudaError_t launch(const MmArgs& a, cudaStream_t st) {
    using S = MmShape<TN>;
    auto* kernel = k_matmul_fp8<TN, COLS>;
    static std::atomic<int> cache[256] = {}, given{0};
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, S::template kSmem<COLS>);
    if (e) return e;
    if constexpr (S::kPair) {  // registers that the launch does not give would be waited for without end
        int regs = given.load(std::memory_order_relaxed);
        if (regs == 0) {
            cudaFuncAttributes f;
            if ((e = cudaFuncGetAttributes(&f, kernel))) return e;
            given.store(regs = f.numRegs, std::memory_order_relaxed);
        }
        if (regs < S::kLaunch) return cudaErrorLaunchOutOfResources;
    }
    const int group = S::kPair ? 2 : a.splits;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim = {(unsigned)group, 1, 1};
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)group);
    cfg.blockDim = dim3(S::kThreads);
    cfg.dynamicSmemBytes = S::template kSmem<COLS>;
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = group > 1 ? 2 : 1;
    int most;  // groups that run at once; clusters with shares of the inner dimension take a tile each
    if constexpr (S::kPair) most = resident_pairs(kernel, cfg, cache);
    else most = group > 1 ? a.tiles : resident_blocks(kernel, S::kThreads, S::template kSmem<COLS>, cache);
    cfg.gridDim = dim3((unsigned)(group * std::min(a.tiles, most > 0 ? most : 1)));
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
    a.k = (int)x.k;
    a.p_data = static_cast<const uint8_t*>(p.data);
    a.q_data = static_cast<const uint8_t*>(q.data);
    a.p_stride = p.stride;
    a.q_stride = q.stride;
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
    a.wide = x.out_stride * size % 16 == 0 && reinterpret_cast<uintptr_t>(x.out) % 16 == 0;
    a.limit = 1u << 18;
    a.err = err;
    const int sms = device_sm_count();
    auto over = [](long long n, long long m) { return (n + m - 1) / m; };
    long long tiles_p = over(a.np, kMmRows);
    int tn;
    // Pairs' tiles of 256 x 256 from as many columns on as 128-row tiles of 256 fill half the SMs with, else 128 (or 64) columns to a
    // block. Microseconds so and with 128 columns: 1300 x 2048 x 1024 8.9, 10.2; 4346 x 1024 x 1024 8.9, 10.3; 8692 x 1024 x 1024 13.7, 16.9;
    // 4096 x 1024 x 17,384 by column 100, 123. Where pairs' tiles fill about half of the pairs, or results have few columns, smaller
    // ones would be faster: 2432 x 1024 x 4096 19.1, 15.1 (by column 29.7, 17.6); 4864 x 512 x 4096 18.2, 15.2; 17,384 x 14 x 8192 44.6, 41.5, and
    // 30.2 with 64 columns; 100 x 20,000 x 1024 13.5, 9.8. Below: 2000 x 1024 x 1024 6.9 with 128 columns, 8.6 with 64; 300 x 1024 x 1024 7.0, 6.9.
    if (swap) tn = a.nq <= 16 ? 16 : a.nq <= 32 ? 32 : 64;
    else tn = tiles_p * over(a.nq, 256) >= sms / 2 ? 256 : cols || tiles_p * over(a.nq, 128) >= sms / 2 ? 128 : 64;
    if (tn == 256) tiles_p = over(a.np, 2 * kMmRows);
    a.tiles_p = (int)tiles_p;
    const long long tiles = tiles_p * over(a.nq, tn);
    if (tiles > 0x0fffffffll) return cudaErrorInvalidConfiguration;
    a.tiles = (int)tiles;
    a.splits = 1;
    const int slots = tn >= 128 ? sms : 2 * sms;
    while (tn < 256 && a.splits < kMmSplits && 2 * a.splits * tiles <= slots && 2 * a.splits <= a.blocks) a.splits *= 2;
    cudaError_t e;
    constexpr auto kBytes = CU_TENSOR_MAP_DATA_TYPE_UINT8;
    if (x.k > 0 && ((e = encode(a.p, kBytes, 1, p.data, x.k, a.np, p.stride, kMmRows)) ||
                    (e = encode(a.q, kBytes, 1, q.data, x.k, a.nq, q.stride, tn == 256 ? 128 : tn))))
        return e;
    a.boxes = a.wide && !swap && a.splits == 1 ? (int)(x.n / (16 / size) * (16 / size)) : 0;
    if (a.boxes && (e = encode(a.to, size == 4 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, size, x.out, a.boxes, x.m, x.out_stride, 32)))
        return e;
    return cols ? launch<true>(tn, a, st) : launch<false>(tn, a, st);
}

}  // namespace gs
