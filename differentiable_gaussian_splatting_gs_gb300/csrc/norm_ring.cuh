// The layer norm kernels' rows on their way into shared memory. Uses the barrier and copy functions of gs_common.cuh, which is
// included before it (a host program may bring its own).
#pragma once

namespace gs {

constexpr int kNormBlock = 256;  // threads per block of the row kernels

// Rows on their way: of each of ARRAYS arrays the row of the next STAGES turns, copied into shared memory with bulk
// copies by the first thread of the row's threads (a warp or the block). So many bytes are in flight
// whatever registers the row takes, which decides how many warps there are.
template <int NV, int LPR>
constexpr int norm_stages = LPR > 128 && NV >= 8 ? 2 : 3;  // two of the longest rows' 64 KB beside their weights
template <int ARRAYS, int LPR, int kNormStages>
struct NormRing {
    static_assert(LPR >= 32);
    unsigned char* data;  // [STAGES][ARRAYS][bytes]
    uint64_t* full;
    const char* src[ARRAYS];
    long long stride[ARRAYS], row, rows, step;  // row: the next to ask for
    unsigned bytes, limit, *err;
    int turn = 0, asked = 0;
    bool ok = true;

    static __host__ __device__ size_t smem(int cols, size_t elem) { return (size_t)(kNormBlock / LPR) * kNormStages * ARRAYS * cols * elem; }

    __device__ __forceinline__ void ask() {
        // (after a wait that gave up, the copy before this one in the same place may still be on its way: nothing more is
        // asked for, or its barrier would count an arrival too many)
        if (row < rows && ok) {
            if (threadIdx.x % LPR == 0) {
                const int s = asked % kNormStages;
                mbar_arrive_expect_tx(full + s, ARRAYS * bytes);
#pragma unroll
                for (int a = 0; a < ARRAYS; ++a)
                    bulk_copy_g2s(data + (size_t)(s * ARRAYS + a) * bytes, src[a] + row * stride[a], bytes, full + s);
            }
            ++asked;
        }
        row += step;
    }
    // After the block's barriers were initialised (bars: kNormStages of them for each row of the block).
    __device__ __forceinline__ void start(unsigned char* smem, uint64_t* bars, int cols, int elem, long long first, long long rows_, long long step_,
                                          unsigned limit_, unsigned* err_) {
        const int g = threadIdx.x / LPR;
        bytes = (unsigned)(cols * elem);
        data = smem + (size_t)g * kNormStages * ARRAYS * bytes;
        full = bars + g * kNormStages;
        row = first, rows = rows_, step = step_, limit = limit_, err = err_;
        for (int s = 0; s < kNormStages; ++s) ask();
    }
    // The present turn's row of array a; a wait that gave up leaves garbage and goes on, since others wait at barriers.
    __device__ __forceinline__ void wait() {
        if (ok) ok = mbar_wait_bounded(full + turn % kNormStages, (turn / kNormStages) & 1, limit, err);
    }
    __device__ __forceinline__ const unsigned char* at(int a) const { return data + (size_t)((turn % kNormStages) * ARRAYS + a) * bytes; }
    // Once all threads of the row have read it.
    __device__ __forceinline__ void next() {
        ++turn;
        ask();
    }
    // Every copy has landed before the block ends.
    __device__ __forceinline__ void finish() {
        if (!ok && threadIdx.x % LPR == 0)
            for (int t = asked > kNormStages ? asked - kNormStages : 0; t < asked; ++t)
                mbar_drain(full + t % kNormStages, (t / kNormStages) & 1, err);
    }
};

}  // namespace gs
