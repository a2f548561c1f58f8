// Cross attention, backward, on the tensor cores: float32 tensors in three bfloat16 planes, heads of up to 64.
//
// The two roles, rows and walked tiles are those of the 16-bit kernel (attention_bwd.cu), with 128 rows per block. Six
// products take the place of one, so the products bound the kernel (S, dP, dk and dv of 128 x 64 elements: 3900 cycles,
// their elementwise part about 1500 beside them). P and dS are split into planes too. The tensor cores add by
// truncation, 2^-25 of the accumulator each time, which hundreds of walked tiles would make a drift of 10^-5: every
// tile's product starts from zero, and a third warpgroup adds it in registers, rounded to nearest.
//
// Shared memory holds two walked tiles, so the order of the products hides their copies: both tiles' gradients, then
// both next tiles' S and dP.
#include "attention_tc.cuh"

namespace gs {

namespace {

constexpr int kDP = 64, kPL = 3;
constexpr int kRowBytes = kPL * kDP * kTileRows * 2;      // a row operand
constexpr int kWalkBytes = kPL * kDP * kBN * 2;           // a walked tile's operand
constexpr int kStage = 2 * kWalkBytes + 1024;             // with the tile's exponent offsets and deltas (KEYS)
constexpr int kSmem = 2 * kRowBytes + 2 * kStage + 1024;
constexpr int kBuffer = 192;                              // columns of a walked tile's S, dP and then P, dS
constexpr int kProduct = 2 * kBuffer;

// Column of plane q of the 16 walked rows from 16 x on; of P (which = 0) or dS (1). 32 walked rows' first two planes
// take the columns of their S or dP, the third ones lie behind.
__device__ __forceinline__ int plane_column(int which, int q, int x) {
    return q < 2 ? which * 64 + (x / 2) * 32 + q * 16 + (x % 2) * 8 : 128 + (x / 2) * 32 + which * 16 + (x % 2) * 8;
}

// The planes of 32 values as 16-bit pairs in their columns.
__device__ __forceinline__ void store_planes(uint32_t buffer, int which, int y, float (&v)[32]) {
#pragma unroll
    for (int q = 0; q < kPL; ++q) {
        uint32_t p[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) {
            p[e] = pack2<__nv_bfloat16>(v[2 * e], v[2 * e + 1]);
            v[2 * e] -= __uint_as_float(p[e] << 16);
            v[2 * e + 1] -= __uint_as_float(p[e] & 0xffff0000u);
        }
        tmem_st16(buffer + plane_column(which, q, 2 * y), p);
    }
}

}  // namespace

template <bool KEYS>
__device__ __forceinline__ void wide_block(const BwdArgs& g, int at, const TcTensor& ta1, const TcTensor& ta2, const TcTensor& tb1,
                                           const TcTensor& tb2) {
    using C = Pairs<kPL>;
    constexpr int kProducts = KEYS ? 1 : 2;              // places of a tile's product: dk and dv, or dq in turn
    constexpr int kCols = KEYS ? 2 * kDP : kDP;          // columns of one
    extern __shared__ unsigned char raw[];
    __shared__ uint64_t a_full, full[2], empty[2], s_full[2], p_full[2], x_full[2], x_free[2], drain;
    __shared__ uint32_t tmem_base;
    const TcArgs& t = g.t;
    const AttnArgs& a = t.a;
    unsigned char* base = raw + (((smem_u32(raw) + 1023u) & ~1023u) - smem_u32(raw));
    const uint32_t sa1 = smem_u32(base), sa2 = sa1 + kRowBytes, sb = sa2 + kRowBytes;
    auto stats = [&](int s) { return reinterpret_cast<float*>(base + 2 * kRowBytes + s * kStage + 2 * kWalkBytes); };

    const int block = at % t.tiles;
    at /= t.tiles;
    const int split = at % t.splits;
    at /= t.splits;
    const int share = a.heads / a.kv_heads, row_heads = KEYS ? a.kv_heads : a.heads;
    const int h = at % row_heads, b = at / row_heads;
    const int keys = keys_of(t, b), row0 = block * kTileRows;
    const int rows = KEYS ? keys : a.len_q;
    // walked tiles: of the keys, or of the queries of `share` heads one after the other
    const int per_head = KEYS ? (a.len_q + kBN - 1) / kBN : (keys + kBN - 1) / kBN;
    const int all = KEYS ? per_head * share : per_head, per = (all + t.splits - 1) / t.splits;
    const int first = min(split * per, all), n = row0 < rows ? min(per, all - first) : 0;
    const int warp = threadIdx.x >> 5;
    const unsigned limit = a.spin_limit;

    if (threadIdx.x == 0) {
        mbar_init(&a_full, 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], 1);
            mbar_init(&s_full[i], 1);
            mbar_init(&p_full[i], 4);
            mbar_init(&x_full[i], 1);
            mbar_init(&x_free[i], 4);
        }
        mbar_init(&drain, 1);
        fence_mbar_init();
    }
    if (warp == 12) tmem_alloc<512>(&tmem_base);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tm = tmem_base;
    const uint32_t lanes = (uint32_t)(warp & 3) << 21;

    // 512 threads x 128 registers at launch = 256 x 136 + 128 x 184 + 128 x 56
    if (warp >= 12) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
        if (warp == 12 && n > 0 && elect_one()) {  // copies
            mbar_arrive_expect_tx(&a_full, 2 * kRowBytes);
            load_rows<kDP, kPL, kTileRows>(sa1, ta1, row0, b, h, row_heads, &a_full);
            load_rows<kDP, kPL, kTileRows>(sa2, ta2, row0, b, h, row_heads, &a_full);
            int sent = 0;
            for (int j = 0; j < n; ++j) {
                const int s = j & 1, x = first + j;
                if (j >= 2 && !mbar_wait_bounded(&empty[s], (j / 2 + 1) & 1, limit, a.err)) break;
                const int wh = KEYS ? h * share + x / per_head : h / share, w0 = (KEYS ? x % per_head : x) * kBN;
                mbar_arrive_expect_tx(&full[s], 2 * kWalkBytes + (KEYS ? 2 * kBN * 4 : 0));
                load_rows<kDP, kPL, kBN>(sb + s * kStage, tb1, w0, b, wh, KEYS ? a.heads : a.kv_heads, &full[s]);
                load_rows<kDP, kPL, kBN>(sb + s * kStage + kWalkBytes, tb2, w0, b, wh, KEYS ? a.heads : a.kv_heads, &full[s]);
                if (KEYS) {
                    const long long q = ((long long)b * a.heads + wh) * g.qpad + w0;
                    bulk_copy_g2s(stats(s), g.nlse + q, kBN * 4, &full[s]);
                    bulk_copy_g2s(stats(s) + kBN, g.ndelta + q, kBN * 4, &full[s]);
                }
                sent = j + 1;
            }
            // every copy lands before the block ends, whatever became of its reader
            mbar_drain(&a_full, 0, a.err);
            for (int j = max(0, sent - 2); j < sent; ++j) mbar_drain(&full[j & 1], (j / 2) & 1, a.err);
        } else if (warp == 13 && n > 0 && elect_one()) {  // products
            const int steps = (a.d + 15) / 16;
            const uint32_t s_desc = mma_desc<__nv_bfloat16>(kBN, false), g_desc = mma_desc<__nv_bfloat16>(steps * 16, true);
            auto wait = [&](uint64_t* bar, int k) { return mbar_wait_bounded(bar, k & 1, limit, a.err); };
            bool ok = wait(&a_full, 0);
            auto scores = [&](int j) {
                const int w = j & 1;
                if (!(ok = ok && wait(&full[w], j / 2))) return;
                tc_fence_after();
                const uint32_t tile = sb + w * kStage;
#pragma unroll 1
                for (int which = 0; which < 2; ++which) {
#pragma unroll
                    for (int c = 0; c < C::n; ++c) {
                        const uint32_t x = tile_desc((which ? sa2 : sa1) + C::a(c) * kDP * kTileRows * 2);
                        const uint32_t y = tile_desc(tile + which * kWalkBytes + C::b(c) * kDP * kBN * 2);
#pragma unroll
                        for (int k = 0; k < kDP / 16; ++k)
                            if (k < steps) mma_ss(tm + w * kBuffer + which * 64, x + k * 2, y + k * 2, s_desc, c > 0 || k > 0);
                    }
                }
                mma_commit(&s_full[w]);
            };
            auto gradients = [&](int j) {
                const int w = j & 1, p = kProducts == 2 ? j & 1 : 0, use = kProducts == 2 ? j / 2 : j;
                if (!(ok = ok && wait(&p_full[w], j / 2) && (use == 0 || wait(&x_free[p], use - 1)))) return;
                tc_fence_after();
                const uint32_t tile = sb + w * kStage, acc = tm + kProduct + p * kDP;
#pragma unroll 1
                for (int which = 1; which >= (KEYS ? 0 : 1); --which) {  // dS B1, then P B2
#pragma unroll
                    for (int c = 0; c < C::n; ++c) {
                        const uint32_t y = tile_desc(tile + (1 - which) * kWalkBytes + C::b(c) * kDP * kBN * 2, kBN * 128);
#pragma unroll
                        for (int x = 0; x < kBN / 16; ++x)
                            mma_ts(acc + (1 - which) * kDP, tm + w * kBuffer + plane_column(which, C::a(c), x), y + x * 128, g_desc,
                                   c > 0 || x > 0);
                    }
                }
                mma_commit(&x_full[p]);
                mma_commit(&empty[w]);
            };
            for (int j = 0; j < 2 && j < n; ++j) scores(j);
            for (int j0 = 0; j0 < n && ok; j0 += 2) {
                for (int j = j0; j < j0 + 2 && j < n; ++j) gradients(j);
                for (int j = j0 + 2; j < j0 + 4 && j < n; ++j) scores(j);
            }
            // no product is in flight when the tensor memory is freed
            mma_commit(&drain);
            mbar_drain(&drain, 0, a.err);
        }
    } else if (warp >= 8) {  // sums of the tiles' products, and the results: thread = row
        asm volatile("setmaxnreg.inc.sync.aligned.u32 184;");
        const int row = row0 + (threadIdx.x & 127);
        float sum[kCols];
#pragma unroll
        for (int e = 0; e < kCols; ++e) sum[e] = 0.f;
        bool ok = true;
        for (int j = 0; j < n; ++j) {
            const int p = kProducts == 2 ? j & 1 : 0, use = kProducts == 2 ? j / 2 : j;
            if (!(ok = warp_wait(&x_full[p], use & 1, limit, a.err))) break;  // the same in all lanes
            tc_fence_after();
#pragma unroll
            for (int y = 0; y < kCols / 32; ++y) {
                uint32_t o[32];
                tmem_ld32(tm + kProduct + p * kDP + lanes + y * 32, o);
                tmem_wait_ld(o);
#pragma unroll
                for (int e = 0; e < 32; ++e) sum[y * 32 + e] += __uint_as_float(o[e]);
            }
            tc_fence_before();
            warp_arrive(&x_free[p]);
        }
        const bool live = row < rows && ok;
#pragma unroll
        for (int e = 0; e < kDP; ++e) sum[e] *= a.scale;  // dS was formed without it
#pragma unroll
        for (int which = 0; which < (KEYS ? 2 : 1); ++which) {  // 0: of dS B1, 1: of P B2
            const AttnTensor& out = KEYS ? (which == 0 ? a.dk : a.dv) : a.dq;
            const long long to = KEYS && g.index && live ? g.index[(long long)b * a.len_k + row] : row;
            float* dst = static_cast<float*>(out.data) + b * out.batch_stride + h * out.head_stride + to * out.len_stride;
            const long long part_rows = KEYS ? g.rows_k : a.len_q, heads_all = (long long)a.batch * row_heads;
            float* part = t.part ? t.part + ((((long long)split * (KEYS ? 2 : 1) + which) * heads_all + (long long)b * row_heads + h) * part_rows + row) * kDP
                                 : nullptr;
            const bool vec = part || (a.d % 4 == 0 && out.batch_stride % 4 == 0 && out.head_stride % 4 == 0 && out.len_stride % 4 == 0 &&
                                      reinterpret_cast<uintptr_t>(out.data) % 16 == 0);
            float* to_row = part ? part : dst;
            if (!live) continue;
#pragma unroll
            for (int e = 0; e < kDP; e += 4) {
                const float* v = sum + which * kDP + e;
                if (vec) {
                    if (e < a.d) *reinterpret_cast<float4*>(to_row + e) = make_float4(v[0], v[1], v[2], v[3]);
                } else {
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        if (e + k < a.d) to_row[e + k] = v[k];
                }
            }
        }
    } else {  // elementwise: thread = row, a warpgroup per walked tile in turn
        asm volatile("setmaxnreg.inc.sync.aligned.u32 136;");
        const int w = warp / 4, row = row0 + (threadIdx.x & 127);
        const uint32_t buffer = tm + w * kBuffer + lanes;
        const float c = a.scale * 1.4426950408889634f;
        float l = -INFINITY, d = 0.f;  // the row's own, where rows are queries
        if (!KEYS && row < a.len_q) {
            const long long q = ((long long)b * a.heads + h) * g.qpad + row;
            l = g.nlse[q];
            d = g.ndelta[q];
        }
        for (int j = w; j < n; j += 2) {
            if (!warp_wait(&s_full[w], (j / 2) & 1, limit, a.err)) break;  // the same in all lanes
            tc_fence_after();
            const float* st = stats(w);
#pragma unroll 1
            for (int y = 0; y < 2; ++y) {
                uint32_t s[32], dp[32];
                tmem_ld32(buffer + y * 32, s);
                tmem_ld32(buffer + 64 + y * 32, dp);
                tmem_wait_ld(s);
                tmem_wait_ld(dp);
                float p[32], ds[32];
                const int left = keys - (first + j) * kBN - y * 32;
#pragma unroll
                for (int e = 0; e < 32; ++e) {
                    if (KEYS) {  // columns are queries
                        l = st[y * 32 + e];
                        d = st[kBN + y * 32 + e];
                    }
                    p[e] = ex2_approx(fmaf(__uint_as_float(s[e]), c, l));
                    ds[e] = p[e] * (__uint_as_float(dp[e]) + d);
                }
                if (!KEYS && left < 32) {
                    asm volatile("");  // a branch
                    // a key beyond the last one: exp of an unbounded number came of its score of 0
#pragma unroll
                    for (int e = 0; e < 32; ++e)
                        if (e >= left) ds[e] = 0.f;
                }
                store_planes(buffer, 1, y, ds);
                if (KEYS) store_planes(buffer, 0, y, p);
            }
            tmem_wait_st();
            tc_fence_before();
            warp_arrive(&p_full[w]);
        }
    }
    __syncwarp();
    __syncthreads();
    tc_fence_after();
    if (warp == 12) tmem_free<512>(tm);
}

// Both roles in one launch (attention_bwd.cu).
__global__ void __launch_bounds__(512, 1)
    k_attn_bwd_wide(const __grid_constant__ BwdArgs gq, const __grid_constant__ BwdArgs gk, const __grid_constant__ BwdTensors x,
                    int keys_first) {
    pdl_entry();
    const int at = blockIdx.x, n = keys_first ? gk.blocks : gq.blocks;
    if ((at < n) == (keys_first != 0))
        wide_block<true>(gk, keys_first ? at : at - n, x.k, x.v, x.q_walk, x.dout_walk);
    else
        wide_block<false>(gq, keys_first ? at - n : at, x.q, x.dout, x.k_walk, x.v_walk);
}

cudaError_t launch_attn_bwd_wide(const BwdArgs& gq, const BwdArgs& gk, const BwdTensors& x, bool keys_first, cudaStream_t st) {
    const cudaError_t e = cudaFuncSetAttribute(k_attn_bwd_wide, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (e) return e;
    return launch_pdl(k_attn_bwd_wide, dim3((unsigned)(gq.blocks + gk.blocks)), dim3(512), kSmem, st, gq, gk, x, (int)keys_first);
}

}  // namespace gs
