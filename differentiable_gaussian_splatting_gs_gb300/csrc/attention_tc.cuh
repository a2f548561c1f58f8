// Cross attention on the tensor cores: what the forward and the backward kernels share.
//
// Operands are 16-bit. float32 tensors are split into three bfloat16 planes, x = x0 + x1 + x2 with 8 bits of
// the significand each; a product keeps the six pairs whose size is at least 2^-16 of the leading one (the
// dropped ones are 2^-24 of it), accumulated in float32 like the rest.
//
// The kernels read Q, K, V and dout with tiled bulk copies, straight from the caller's tensors when these are
// 16-bit with 16-byte aligned rows and every key takes part. Otherwise a copy kernel first lays a tensor out
// in the workspace ("packed"): split into planes, padded to a row of 64, 128 or 256 elements and, for K and V, with
// only the keys that take part, in their order, and zeros up to the next multiple of 128 keys. A masked
// key then costs nothing, and what it holds (NaN) never meets a product.
#pragma once

#include "attention.cuh"
#include "tcgen05.cuh"

namespace gs {

constexpr int kTileRows = 128;  // rows of an operand tile's copy, and of an accumulator

// The pairs of planes whose products are summed, small ones first: (1, 1), (0, 2), (2, 0), (0, 1), (1, 0), (0, 0).
template <int PL>
struct Pairs {
    static constexpr int n = PL == 1 ? 1 : 6;
    __host__ __device__ static constexpr int a(int c) { return PL == 1 ? 0 : c == 2 ? 2 : (c == 0 || c == 4); }
    __host__ __device__ static constexpr int b(int c) { return PL == 1 ? 0 : c == 1 ? 2 : (c == 0 || c == 3); }
};

// A tensor that the tiled copies read: as the caller's (coordinates: element, row, head, batch entry) or packed
// (element, row, plane, batch entry x head).
struct TcTensor {
    CUtensorMap map;
    int packed;
};

struct TcArgs {
    AttnArgs a;
    const int* count;  // keys per batch entry that the key mask leaves, or NULL without one
    float* part;       // a split's share of the output or of a gradient, float32, or NULL
    float* part_lse;
    int tiles, splits;
    int whole, tail;   // forward: the first `whole` blocks of (head, tile) walk all keys, `tail` more share their walk
    int fold, fold_rows;  // forward: a tile's 128 rows are `fold` heads that share a key head, of fold_rows queries each
};

__device__ __forceinline__ int keys_of(const TcArgs& t, int b) { return t.count ? t.count[b] : key_count(t.a, b); }

// Loads rows row0 .. row0 + ROWS - 1 of a head, all planes: PL x DP/64 tiles of ROWS x 64 elements.
template <int DP, int PL, int ROWS>
__device__ __forceinline__ void load_rows(uint32_t dst, const TcTensor& t, int row0, int b, int h, int heads, uint64_t* bar) {
#pragma unroll
    for (int p = 0; p < PL; ++p)
#pragma unroll
        for (int c = 0; c < DP / 64; ++c)
            tile_load(dst + (p * (DP / 64) + c) * ROWS * 128, &t.map, c * 64, row0, t.packed ? p : h,
                      t.packed ? b * heads + h : b, bar);
}

// count[b] and index[b][0 .. count[b]): the keys that take part, in order.
cudaError_t launch_attn_index(const AttnArgs& a, int* count, int* index, cudaStream_t st);
// A tensor (heads heads; K or V when keys) to be laid out at dst as [batch x heads][planes][rows][dp] 16-bit values.
struct PackJob {
    AttnTensor t;
    int heads, len, keys;
    long long rows;
    void* dst;
};
cudaError_t launch_attn_pack(const AttnArgs& a, const PackJob* jobs, int n, const int* count, const int* index, int planes, int dp,
                             cudaStream_t st);
// out and lse of t.tail blocks of `rows` rows (tiles of 128, or one row) from the splits' shares [t.splits][t.tail][rows][dp].
cudaError_t launch_attn_combine(const TcArgs& t, int rows, int dp, cudaStream_t st);
// One query, no shared heads; part, part_lse: the splits' shares, or NULL.
cudaError_t launch_attn_decode(const AttnArgs& a, int splits, int dp, float* part, float* part_lse, cudaStream_t st);
// nq: query tiles per block, 1 or 2.
cudaError_t launch_attn_fwd_tc(const TcArgs& t, const TcTensor& q, const TcTensor& k, const TcTensor& v, int planes, int dp,
                               int nq, cudaStream_t st);


constexpr int kBN = 64;  // rows per tile that the backward walks
struct BwdArgs {
    TcArgs t;              // t.part: float32 shares of dq, or of dk and then dv, or NULL; t.tiles: row blocks of a head
    const float* nlse;     // [batch x heads][len_q padded]: the exponent's offset of each query (k_attn_stats)
    const float* ndelta;   // likewise: -delta
    long long qpad;
    const unsigned* norms; // float16: the largest squared norms of each batch entry's and key head's dout and v, or NULL
    const int* index;      // packed key -> key, or NULL
    long long rows_k;
    int blocks;            // of the role
};
struct BwdTensors {
    TcTensor q, dout, k, v, q_walk, dout_walk, k_walk, v_walk;  // as row tiles; as walked tiles
};
// The backward of three planes, heads of up to 64: the roles of queries and of keys.
cudaError_t launch_attn_bwd_wide(const BwdArgs& gq, const BwdArgs& gk, const BwdTensors& x, bool keys_first, cudaStream_t st);

struct TcBwd {
    AttnArgs a;
    const int *count, *index;    // of the key mask, or NULL
    float *nlse, *ndelta;        // [batch x heads][qpad], written first
    unsigned* norms;             // float16: [batch x kv_heads][2], zero
    float *part_q, *part_k;      // shares of dq and of dk and dv, or NULL
    long long qpad, rows_k;
    int dp, splits_q, splits_k;  // of the walk for dq, and for dk and dv
    bool keys_first;
};
// dq, dk and dv.
cudaError_t launch_attn_bwd_tc(const TcBwd& w, const BwdTensors& x, cudaStream_t st);

}  // namespace gs
