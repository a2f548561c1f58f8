// Inline PTX of the fifth-generation tensor cores (tcgen05, sm_103a) and of tiled bulk copies, as the
// cross attention kernels use them: 16-bit operands, float32 accumulators in tensor memory, one CTA.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include "gs_common.cuh"

namespace gs {

// ---- tensor memory --------------------------------------------------------------------------------
// 128 lanes x 512 columns of 32 bits; an address holds the lane in its upper and the column in its
// lower half. A warp reads and writes the 32 lanes 32 (warp index % 4) ...

// Allocates COLS columns (a power of two of at least 32); the address is left in *dst (shared memory).
// Executed by one whole warp; the same warp frees them.
template <int COLS>
__device__ __forceinline__ void tmem_alloc(uint32_t* dst) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(dst)), "n"(COLS) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
}
template <int COLS>
__device__ __forceinline__ void tmem_free(uint32_t addr) {
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(addr), "n"(COLS));
}

// 32 columns of the warp's lanes: v[i] is column i of the thread's lane. Loads are complete after
// tmem_wait_ld, stores after tmem_wait_st.
__device__ __forceinline__ void tmem_ld32(uint32_t addr, uint32_t (&v)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]),
          "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15]), "=r"(v[16]),
          "=r"(v[17]), "=r"(v[18]), "=r"(v[19]), "=r"(v[20]), "=r"(v[21]), "=r"(v[22]), "=r"(v[23]), "=r"(v[24]),
          "=r"(v[25]), "=r"(v[26]), "=r"(v[27]), "=r"(v[28]), "=r"(v[29]), "=r"(v[30]), "=r"(v[31])
        : "r"(addr));
}
__device__ __forceinline__ void tmem_st32(uint32_t addr, const uint32_t (&v)[32]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(addr),
        "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
        "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15]), "r"(v[16]), "r"(v[17]), "r"(v[18]),
        "r"(v[19]), "r"(v[20]), "r"(v[21]), "r"(v[22]), "r"(v[23]), "r"(v[24]), "r"(v[25]), "r"(v[26]), "r"(v[27]),
        "r"(v[28]), "r"(v[29]), "r"(v[30]), "r"(v[31])
        : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t addr, const uint32_t (&v)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16};" ::"r"(addr),
        "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
        "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
        : "memory");
}
// Completes the thread's loads; v's values pass through, so that nothing which reads them can be moved before it.
__device__ __forceinline__ void tmem_wait_ld(uint32_t (&v)[32]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(v[0]), "+r"(v[1]), "+r"(v[2]), "+r"(v[3]), "+r"(v[4]), "+r"(v[5]), "+r"(v[6]), "+r"(v[7]), "+r"(v[8]),
                   "+r"(v[9]), "+r"(v[10]), "+r"(v[11]), "+r"(v[12]), "+r"(v[13]), "+r"(v[14]), "+r"(v[15]), "+r"(v[16]),
                   "+r"(v[17]), "+r"(v[18]), "+r"(v[19]), "+r"(v[20]), "+r"(v[21]), "+r"(v[22]), "+r"(v[23]), "+r"(v[24]),
                   "+r"(v[25]), "+r"(v[26]), "+r"(v[27]), "+r"(v[28]), "+r"(v[29]), "+r"(v[30]), "+r"(v[31])::"memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Orders tensor-memory accesses across a barrier: before its arrival, after its wait.
__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// ---- matrix products ---------------------------------------------------------------------------------

// Operand tiles in shared memory are rows of 64 16-bit elements (128 bytes) with the 128-byte swizzle, as
// a tiled copy with that swizzle leaves them: 8 rows are 1024 bytes, and the tile starts on 1024 bytes.
// Descriptor of such a tile at `addr`:
//   K-major (the products' inner dimension along a row): 16 elements of it are 32 bytes further on;
//   MN-major (the inner dimension down the rows): 16 of them are 2048 bytes further on, and `lead` is the
//   distance of the tiles that hold the next 64 of the outer dimension.
// The lower word, to which a byte offset / 16 within the tile is added; the upper word is the same for all.
__device__ __forceinline__ uint32_t tile_desc(uint32_t addr, uint32_t lead = 16) { return (addr >> 4) | ((lead >> 4) << 16); }
constexpr uint32_t kTileDescHi = (1024u >> 4) | (1u << 14) | (2u << 29);

// True in one thread of a converged warp, always the same one. Products are issued under it rather than under
// a comparison of the lane: the compiler then knows that their operands are uniform, and an issue takes a
// few instead of about 60 to 100 cycles.
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
    return p != 0;
}

template <class T>
struct TcType;  // the operand type's code in the instruction descriptor
template <>
struct TcType<__half> {
    static constexpr uint32_t code = 0;
};
template <>
struct TcType<__nv_bfloat16> {
    static constexpr uint32_t code = 1;
};

// Instruction descriptor: D[128 x n] float32 (+)= A B, A K-major, B K-major or (b_mn) MN-major.
template <class T>
__device__ __forceinline__ uint32_t mma_desc(int n, bool b_mn) {
    return (1u << 4) | (TcType<T>::code << 7) | (TcType<T>::code << 10) | (b_mn ? 1u << 16 : 0u) |
           ((uint32_t)(n >> 3) << 17) | ((128u >> 4) << 24);
}

// One product over 16 of the inner dimension, issued by one thread; asynchronous, in issue order. A and B by
// the lower words of their descriptors.
__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, bool add) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 da, db;\n\tsetp.ne.b32 p, %4, 0;\n\tmov.b64 da, {%1, %5};\n\tmov.b64 db, {%2, %5};\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %3, p;\n\t}" ::"r"(d),
        "r"(a), "r"(b), "r"(idesc), "r"((uint32_t)add), "r"(kTileDescHi)
        : "memory");
}
// ... with A in tensor memory: lane = row, two elements of the inner dimension per column.
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, bool add) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 db;\n\tsetp.ne.b32 p, %4, 0;\n\tmov.b64 db, {%2, %5};\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], db, %3, p;\n\t}" ::"r"(d),
        "r"(a), "r"(b), "r"(idesc), "r"((uint32_t)add), "r"(kTileDescHi)
        : "memory");
}
// Arrives on `bar` once every product that this thread issued so far is complete.
__device__ __forceinline__ void mma_commit(uint64_t* bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}

__device__ __forceinline__ void mbar_arrive(uint64_t* bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}

// One arrival for the whole warp, after all its lanes got here (128 arrivals on one word would take turns).
__device__ __forceinline__ void warp_arrive(uint64_t* bar) {
    __syncwarp();
    if (elect_one()) mbar_arrive(bar);
}

// mbar_wait_bounded by a whole warp: one answer, so that a warp whose wait gave up stays together for the warp-wide
// tensor-memory instructions that follow. Lanes may name different barriers: all of them are waited for, at the price
// of one (about 100 cycles where they are over, which a thread that issues products cannot spend on each).
__device__ __forceinline__ bool warp_wait(uint64_t* bar, unsigned parity, unsigned limit, unsigned* err) {
    if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
    return __all_sync(0xffffffffu, mbar_wait_bounded(bar, parity, limit, err));
}
__device__ __forceinline__ bool warp_wait_all(uint64_t* a, unsigned pa, uint64_t* b, unsigned pb, unsigned limit, unsigned* err) {
    const bool odd = threadIdx.x & 1;
    return warp_wait(odd ? b : a, (odd ? pb : pa) & 1, limit, err);
}
__device__ __forceinline__ bool warp_wait_all(uint64_t* a, unsigned pa, uint64_t* b, unsigned pb, uint64_t* c, unsigned pc, unsigned limit,
                                              unsigned* err) {
    const bool odd = threadIdx.x & 1, two = threadIdx.x & 2;
    return warp_wait(two ? c : odd ? b : a, (two ? pc : odd ? pb : pa) & 1, limit, err);
}

// ---- tiled bulk copies -------------------------------------------------------------------------------

// A box of a four-dimensional tensor map -> shared memory; what lies outside the tensor is 0. c0 * element
// size is a multiple of 16 bytes.
__device__ __forceinline__ void tile_load(uint32_t dst, const CUtensorMap* map, int c0, int c1, int c2, int c3, uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(dst),
        "l"(map), "r"(smem_u32(bar)), "r"(c0), "r"(c1), "r"(c2), "r"(c3)
        : "memory");
}

// The largest of three.
__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

// Two floats -> two 16-bit values in one word, the first in the lower half.
template <class T>
__device__ __forceinline__ uint32_t pack2(float lo, float hi);
template <>
__device__ __forceinline__ uint32_t pack2<__half>(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
template <>
__device__ __forceinline__ uint32_t pack2<__nv_bfloat16>(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

}  // namespace gs
