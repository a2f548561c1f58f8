// Cross attention, backward, on the tensor cores (16-bit types).
//
// One kernel in two roles. In both a block holds 128 rows and walks the other side in tiles of 64, forming
//   S = A1 B1^T,  dP = A2 B2^T,  P = exp(scale S - lse),  dS = P (dP - delta):
//   queries: rows are queries, A1 = Q, A2 = dout, B1 = K, B2 = V:   dq = scale sum dS B1;
//   keys:    rows are keys,    A1 = K, A2 = V, B1 = Q, B2 = dout:   dk = scale sum dS B1,  dv = sum P B2,
//            over the queries of every head that shares the key head.
// So each result is summed by one block in a fixed order, without atomics or a float32 copy in memory, at the
// price of forming S and dP twice (7 products instead of 5); atomics would add 32 KB to every tile's work. lse and delta
// are known, so nothing is rescaled and a tile's elements are independent of the others'.
//
// float16: P is formed 2^15 times as large, and dS as many times (a power of two for each key head) as its bound
// |dS| <= 2 scale max|dout| max|v| allows below the type's largest value; the sums are scaled back. Unscaled, the
// small probabilities of long or peaked rows fell into the type's subnormal range (or, with large dout, out of it).
//
// Thread = row: a warpgroup turns a 128 x 64 tile of S and dP from tensor memory into dS and P, 16-bit in the
// same columns, which feed the next products as their A operand there. A tile's way (products, load, elementwise part,
// store, products) takes about 2200 cycles and its products 400 to 1300, so tensor memory holds as many tiles as fit
// beside the sums, three (two for dk and dv of heads above 64), each with a warpgroup of its own. A thread each
// issues S, dP and the sums, in the tiles' order (an issue takes 20 to 45 cycles, a commit 75); with two tiles one thread
// issues all, since the next S follows the sums at once.
//
// A product of 64 columns with both operands in shared memory takes 49 cycles, with A in tensor memory 33 (the
// products' reads of shared memory bound it). Where columns are left (queries, heads of up to 64) Q and dout are moved there
// first.
//
// Sums over few rows (FINE) keep what the rounding of P and dS to 16 bits left beside them and multiply it too.
#include "attention_tc.cuh"

namespace gs {

constexpr int kBoost = 15;  // float16: P times 2^kBoost

// float16: the power of two that leaves the bound of dS / scale, 2 max|dout| max|v|, below 2^15; 0 where there is none.
// norms: their squares, as bits.
__device__ __forceinline__ int ds_exponent(const unsigned* norms) {
    const float bound = 2.f * sqrtf(__uint_as_float(norms[0])) * sqrtf(__uint_as_float(norms[1]));
    if (!(bound < 3e38f) || bound <= 0.f) return 0;
    int e;
    frexpf(bound, &e);  // bound < 2^e
    return min(max(15 - e, -24), 24);
}

// Column of P or dS of 16 walked rows from 16 x on; what their rounding left of them (FINE) lies 16 columns behind.
__device__ __forceinline__ constexpr int part_column(int x) { return x / 2 * 32 + x % 2 * 8; }

// Two floats less their rounded values, rounded.
template <class T>
__device__ __forceinline__ uint32_t rest2(uint32_t rounded, float x, float y) {
    Pack<T, 2> r;
    memcpy(&r, &rounded, 4);
    return pack2<T>(x - to_float(r.v[0]), y - to_float(r.v[1]));
}

template <int DP, bool KEYS>
struct BwdShape {
    static constexpr int kA = DP * kTileRows * 2;       // bytes of one operand's rows
    static constexpr int kB = DP * kBN * 2;             // bytes of one operand's walked tile
    static constexpr int kStage = 2 * kB + 1024;        // with the tile's exponent offsets and deltas (KEYS)
    static constexpr int kRoom = (225 * 1024 - 1024 - 2 * kA) / kStage;
    static constexpr int kStages = kRoom > 6 ? 6 : kRoom;
    static constexpr int kSmem = 2 * kA + kStages * kStage + 1024;
    static constexpr int kAccs = KEYS ? 2 : 1;
    static constexpr int kBuffers = KEYS && DP == 128 ? 2 : 3;  // walked tiles in tensor memory, 128 columns each
    static constexpr bool kOneIssuer = kBuffers == 2;
    // a warpgroup per buffer, one that copies and issues, and with two buffers one that rests. Registers are moved
    // between them (setmaxnreg): 512 threads x 128 at launch = 384 x 144 + 128 x 80 = 256 x 208 + 128 x 72 + 128 x 24
    static constexpr int kElem = kBuffers * 4;  // elementwise warps
    static constexpr int kAcc = kBuffers * 128;                 // first accumulator column
    static constexpr bool kInTmem = !KEYS && DP == 64;          // the row operands, 32 columns each
    static constexpr int kRowCol = kAcc + kAccs * DP;
    static_assert(kRowCol + (kInTmem ? 64 : 0) <= 512 && kStages > kBuffers);
};

// One block in its role; at: its number among the role's blocks. ta1, ta2: A1 and A2; tb1, tb2: B1 and B2.
template <class T, int DP, bool KEYS, bool FINE>
__device__ __forceinline__ void bwd_block(const BwdArgs& g, int at, const TcTensor& ta1, const TcTensor& ta2, const TcTensor& tb1,
                                          const TcTensor& tb2) {
    using S = BwdShape<DP, KEYS>;
    constexpr int kSt = S::kStages, kNB = S::kBuffers;
    constexpr bool kHalf = std::is_same<T, __half>::value;
    extern __shared__ unsigned char raw[];
    __shared__ uint64_t a_full, a_moved, full[kSt], empty[kSt], s_full[kNB], p_full[kNB], b_free[kNB], done, drain[3];
    __shared__ uint32_t tmem_base;
    const TcArgs& t = g.t;
    const AttnArgs& a = t.a;
    unsigned char* base = raw + (((smem_u32(raw) + 1023u) & ~1023u) - smem_u32(raw));
    const uint32_t sa1 = smem_u32(base), sa2 = sa1 + S::kA, sb = sa2 + S::kA;
    auto stats = [&](int s) { return reinterpret_cast<float*>(base + 2 * S::kA + s * S::kStage + 2 * S::kB); };

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
        mbar_init(&a_moved, 8);
        for (int i = 0; i < kSt; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], 1);
        }
        for (int i = 0; i < kNB; ++i) {
            mbar_init(&s_full[i], S::kOneIssuer ? 1 : 2);
            mbar_init(&p_full[i], 4);
            mbar_init(&b_free[i], 1);
        }
        mbar_init(&done, 1);
        mbar_init(&drain[0], 1);
        mbar_init(&drain[1], 1);
        mbar_init(&drain[2], 1);
        fence_mbar_init();
    }
    if (warp == S::kElem) tmem_alloc<512>(&tmem_base);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tm = tmem_base;

    if (warp >= S::kElem + 4) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 24;");
    } else if (warp >= S::kElem) {
        if (kNB == 3) asm volatile("setmaxnreg.dec.sync.aligned.u32 80;");
        else asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
        const int steps = (a.d + 15) / 16;
        if (warp == S::kElem && n > 0 && elect_one()) {  // copies
            mbar_arrive_expect_tx(&a_full, 2 * S::kA);
            load_rows<DP, 1, kTileRows>(sa1, ta1, row0, b, h, row_heads, &a_full);
            load_rows<DP, 1, kTileRows>(sa2, ta2, row0, b, h, row_heads, &a_full);
            int sent = 0;
            for (int j = 0; j < n; ++j) {
                const int s = j % kSt, x = first + j;
                if (j >= kSt && !mbar_wait_bounded(&empty[s], (j / kSt + 1) & 1, limit, a.err)) break;
                const int wh = KEYS ? h * share + x / per_head : h / share, w0 = (KEYS ? x % per_head : x) * kBN;
                mbar_arrive_expect_tx(&full[s], 2 * S::kB + (KEYS ? 2 * kBN * 4 : 0));
                load_rows<DP, 1, kBN>(sb + s * S::kStage, tb1, w0, b, wh, KEYS ? a.heads : a.kv_heads, &full[s]);
                load_rows<DP, 1, kBN>(sb + s * S::kStage + S::kB, tb2, w0, b, wh, KEYS ? a.heads : a.kv_heads, &full[s]);
                if (KEYS) {
                    const long long q = ((long long)b * a.heads + wh) * g.qpad + w0;
                    bulk_copy_g2s(stats(s), g.nlse + q, kBN * 4, &full[s]);
                    bulk_copy_g2s(stats(s) + kBN, g.ndelta + q, kBN * 4, &full[s]);
                }
                sent = j + 1;
            }
            // every copy lands before the block ends, whatever became of its reader
            mbar_drain(&a_full, 0, a.err);
            for (int j = max(0, sent - kSt); j < sent; ++j) mbar_drain(&full[j % kSt], (j / kSt) & 1, a.err);
        } else if (warp > S::kElem && (!S::kOneIssuer || warp == S::kElem + 1) && n > 0) {  // products: the warp waits, one thread issues
            const uint32_t s_desc = mma_desc<T>(kBN, false), g_desc = mma_desc<T>(steps * 16, true);
            const int me = warp - S::kElem - 1;  // 0: S (and all with one issuer), 1: dP, 2: the sums
            // S or dP of walked tile j
            auto product = [&](int j, int which) {
                const uint32_t tile = sb + j % kSt * S::kStage, d = tm + j % kNB * 128 + which * 64;
                const uint32_t r = tile_desc(which ? sa2 : sa1), y = tile_desc(tile + which * S::kB);
#pragma unroll
                for (int x = 0; x < DP / 16; ++x) {
                    if (x >= steps) continue;
                    const uint32_t yx = y + (x / 4) * kBN * 8 + (x % 4) * 2;
                    if (S::kInTmem) mma_ts(d, tm + S::kRowCol + which * 32 + x * 8, yx, s_desc, x > 0);
                    else mma_ss(d, r + (x / 4) * kTileRows * 8 + (x % 4) * 2, yx, s_desc, x > 0);
                }
            };
            auto scores = [&](int j) {
                if (!elect_one()) return;
                if (S::kOneIssuer) {
                    product(j, 0);
                    product(j, 1);
                } else {
                    product(j, me);
                }
                mma_commit(&s_full[j % kNB]);
            };
            auto sums = [&](int j) {
                if (!elect_one()) return;
                const uint32_t acc = tm + S::kAcc, tile = sb + j % kSt * S::kStage, buffer = tm + j % kNB * 128;
                const uint32_t y1 = tile_desc(tile, kBN * 128), y2 = tile_desc(tile + S::kB, kBN * 128);
#pragma unroll
                for (int x = 0; x < kBN / 16; ++x) mma_ts(acc, buffer + 64 + part_column(x), y1 + x * 128, g_desc, j > 0 || x > 0);
                if (KEYS)
#pragma unroll
                    for (int x = 0; x < kBN / 16; ++x) mma_ts(acc + DP, buffer + part_column(x), y2 + x * 128, g_desc, j > 0 || x > 0);
                if (FINE) {
#pragma unroll
                    for (int x = 0; x < kBN / 16; ++x) mma_ts(acc, buffer + 64 + 16 + part_column(x), y1 + x * 128, g_desc, true);
                    if (KEYS)
#pragma unroll
                        for (int x = 0; x < kBN / 16; ++x) mma_ts(acc + DP, buffer + 16 + part_column(x), y2 + x * 128, g_desc, true);
                }
                if (!S::kOneIssuer) mma_commit(&b_free[j % kNB]);
                mma_commit(&empty[j % kSt]);
            };
            const bool does_s = me < 2, does_g = S::kOneIssuer || me == 2;
            bool ok = !does_s || warp_wait(S::kInTmem ? &a_moved : &a_full, 0, limit, a.err);
            if (does_s)
                for (int j = 0; j < (S::kOneIssuer ? min(kNB, n) : n) && ok; ++j) {
                    if (!(ok = j < kNB ? warp_wait(&full[j % kSt], (j / kSt) & 1, limit, a.err)
                                       : warp_wait_all(&full[j % kSt], j / kSt, &b_free[j % kNB], j / kNB - 1, limit, a.err)))
                        break;
                    tc_fence_after();
                    scores(j);
                }
            if (does_g) {
                for (int j = 0; j < n && ok; ++j) {
                    const int next = j + kNB;
                    const bool more = S::kOneIssuer && next < n;
                    if (!(ok = more ? warp_wait_all(&p_full[j % kNB], j / kNB, &full[next % kSt], next / kSt, limit, a.err)
                                    : warp_wait(&p_full[j % kNB], (j / kNB) & 1, limit, a.err)))
                        break;
                    tc_fence_after();
                    sums(j);
                    if (more) scores(next);
                }
                if (elect_one()) mma_commit(&done);
            }
            // no product is in flight when the tensor memory is freed
            if (elect_one()) {
                mma_commit(&drain[me]);
                mbar_drain(&drain[me], 0, a.err);
            }
        }
    } else {  // elementwise: thread = row
        if (kNB == 3) asm volatile("setmaxnreg.inc.sync.aligned.u32 144;");
        else asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
        const int w = warp / 4;
        const uint32_t lanes = (uint32_t)(warp & 3) << 21;
        const int row = row0 + (threadIdx.x & 127);
        const float c = a.scale * 1.4426950408889634f;
        // of dS / scale as it is stored, over P's times dP - delta; and of the sum of dS B1
        float ds_in = 1.f, ds_out = a.scale;
        if (kHalf) {
            const int e = ds_exponent(g.norms + (b * a.kv_heads + (KEYS ? h : h / share)) * 2);
            ds_in = exp2f((float)(e - kBoost));
            ds_out *= exp2f((float)-e);
        }
        const f32x2 c2 = f2_pack(c, c), i2 = f2_pack(ds_in, ds_in);
        f32x2 l2 = 0, d2 = 0;  // the row's own, where rows are queries
        if (!KEYS) {
            const long long q = ((long long)b * a.heads + h) * g.qpad + row;
            const float l = row < a.len_q ? g.nlse[q] : -INFINITY, d = row < a.len_q ? g.ndelta[q] : 0.f;
            l2 = f2_pack(l, l);
            d2 = f2_pack(d * ds_in, d * ds_in);
        }
        bool ok = true;
        if (S::kInTmem && n > 0 && w < 2) {
            // a warpgroup per operand, the thread's row of it: 128 bytes, whose 16-byte pieces the copy's swizzle has exchanged
            ok = warp_wait(&a_full, 0, limit, a.err);
            const int r = threadIdx.x & 127;
            const unsigned char* from = base + w * S::kA + r * 128;
            uint32_t v[32];
#pragma unroll
            for (int x = 0; x < 8; ++x) {
                const uint4 q = *reinterpret_cast<const uint4*>(from + ((x ^ (r & 7)) * 16));
                v[4 * x] = q.x, v[4 * x + 1] = q.y, v[4 * x + 2] = q.z, v[4 * x + 3] = q.w;
            }
            tmem_st32(tm + S::kRowCol + w * 32 + lanes, v);
            tmem_wait_st();
            tc_fence_before();
            warp_arrive(&a_moved);
        }
        for (int j = w; j < n; j += kNB) {
            const uint32_t ts = tm + w * 128 + lanes;
            ok = ok && warp_wait(&s_full[w], (j / kNB) & 1, limit, a.err);
            if (!ok) break;  // the same in all lanes; nothing below waits for this warp without a limit
            tc_fence_after();
            const float* st = stats(j % kSt);
#pragma unroll
            for (int y = 0; y < 2; ++y) {
                uint32_t s[32], dp[32], p[16], ds[16], p_rest[FINE ? 16 : 1], ds_rest[FINE ? 16 : 1];
                tmem_ld32(ts + y * 32, s);
                tmem_ld32(ts + 64 + y * 32, dp);
                tmem_wait_ld(s);
                tmem_wait_ld(dp);
                float4 l4, d4;
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    if (KEYS) {  // columns are queries
                        if (e % 2 == 0) {
                            l4 = *reinterpret_cast<const float4*>(st + y * 32 + 2 * e);
                            d4 = *reinterpret_cast<const float4*>(st + kBN + y * 32 + 2 * e);
                        }
                        l2 = e % 2 ? f2_pack(l4.z, l4.w) : f2_pack(l4.x, l4.y);
                        d2 = e % 2 ? f2_pack(d4.z, d4.w) : f2_pack(d4.x, d4.y);
                    }
                    const float2 z = f2_unpack(f2_fma(f2_pack(__uint_as_float(s[2 * e]), __uint_as_float(s[2 * e + 1])), c2, l2));
                    const float u0 = ex2_approx(z.x), u1 = ex2_approx(z.y);
                    f32x2 x = f2_pack(__uint_as_float(dp[2 * e]), __uint_as_float(dp[2 * e + 1]));
                    x = KEYS || !kHalf ? f2_add(x, d2) : f2_fma(x, i2, d2);
                    if (KEYS && kHalf) x = f2_mul(x, i2);
                    const float2 v = f2_unpack(f2_mul(f2_pack(u0, u1), x));
                    if (KEYS) p[e] = pack2<T>(u0, u1);
                    ds[e] = pack2<T>(v.x, v.y);
                    if (FINE) {
                        if (KEYS) p_rest[e] = rest2<T>(p[e], u0, u1);
                        ds_rest[e] = rest2<T>(ds[e], v.x, v.y);
                    }
                }
                if (!KEYS) {
                    const int left = keys - (first + j) * kBN - y * 32;
                    if (left < 32) {
                        asm volatile("");  // a branch
                        // a key beyond the last one: exp of an unbounded number came of its score of 0
#pragma unroll
                        for (int e = 0; e < 16; ++e) {
                            if (2 * e >= left) ds[e] = 0u;
                            else if (2 * e + 1 >= left) ds[e] &= 0xffffu;
                            if (!FINE) continue;
                            if (2 * e >= left) ds_rest[e] = 0u;
                            else if (2 * e + 1 >= left) ds_rest[e] &= 0xffffu;
                        }
                    }
                }
                // over the scores of their own half
                tmem_st16(ts + 64 + y * 32, ds);
                if (KEYS) tmem_st16(ts + y * 32, p);
                if constexpr (FINE) {
                    tmem_st16(ts + 64 + 16 + y * 32, ds_rest);
                    if (KEYS) tmem_st16(ts + 16 + y * 32, p_rest);
                }
            }
            tmem_wait_st();
            tc_fence_before();
            warp_arrive(&p_full[w]);
        }
        if (n > 0) ok = warp_wait(&done, 0, limit, a.err) && ok;
        tc_fence_after();
        // of the first two warpgroups: a sum each for keys, half of its columns for queries
        const int which = KEYS ? w & 1 : 0;  // 0: of dS B1, 1: of P B2
        constexpr int kOut = KEYS ? DP : DP / 2;
        const int col0 = KEYS ? 0 : (w & 1) * kOut;
        const uint32_t acc = tm + S::kAcc + lanes + which * DP + col0;
        const float f = which == 0 ? ds_out : kHalf ? 1.f / (1 << kBoost) : 1.f;
        const bool live = row < rows && ok && w < 2;
        const AttnTensor& out = KEYS ? (which == 0 ? a.dk : a.dv) : a.dq;
        const long long to = KEYS && g.index && live ? g.index[(long long)b * a.len_k + row] : row;
        T* dst = static_cast<T*>(out.data) + b * out.batch_stride + h * out.head_stride + to * out.len_stride;
        const long long part_rows = KEYS ? g.rows_k : a.len_q, heads_all = (long long)a.batch * row_heads;
        float* part = t.part ? t.part + ((((long long)split * S::kAccs + which) * heads_all + (long long)b * row_heads + h) * part_rows + row) * DP
                             : nullptr;
        const bool vec = a.d % 8 == 0 && out.batch_stride % 8 == 0 && out.head_stride % 8 == 0 && out.len_stride % 8 == 0 &&
                         reinterpret_cast<uintptr_t>(out.data) % 16 == 0;
#pragma unroll
        for (int y = 0; y < kOut / 32; ++y) {
            uint32_t o[32];
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = 0u;
            if (n > 0) {
                tmem_ld32(acc + y * 32, o);
                tmem_wait_ld(o);
            }
            if (live) {
#pragma unroll
                for (int e = 0; e < 32; e += 8) {
                    const int col = col0 + y * 32 + e;
                    if (part) {
                        *reinterpret_cast<float4*>(part + col) = make_float4(__uint_as_float(o[e]) * f, __uint_as_float(o[e + 1]) * f,
                                                                             __uint_as_float(o[e + 2]) * f, __uint_as_float(o[e + 3]) * f);
                        *reinterpret_cast<float4*>(part + col + 4) = make_float4(__uint_as_float(o[e + 4]) * f, __uint_as_float(o[e + 5]) * f,
                                                                                 __uint_as_float(o[e + 6]) * f, __uint_as_float(o[e + 7]) * f);
                        continue;
                    }
                    Pack<T, 8> v;
#pragma unroll
                    for (int k = 0; k < 8; ++k) v.v[k] = from_float<T>(__uint_as_float(o[e + k]) * f);
                    if (vec) {
                        if (col < a.d) *reinterpret_cast<Pack<T, 8>*>(dst + col) = v;
                    } else {
#pragma unroll
                        for (int k = 0; k < 8; ++k)
                            if (col + k < a.d) dst[col + k] = v.v[k];
                    }
                }
            }
            __syncwarp();
        }
        tc_fence_before();
    }
    __syncwarp();
    __syncthreads();
    tc_fence_after();
    if (warp == S::kElem) tmem_free<512>(tm);
}

// Both roles in one launch, so that the blocks of the second fill the SMs that the first's last round leaves: keys
// first where their walks are longer.
template <class T, int DP, bool FINE>
__global__ void __launch_bounds__(512, 1)
    k_attn_bwd(const __grid_constant__ BwdArgs gq, const __grid_constant__ BwdArgs gk, const __grid_constant__ BwdTensors x,
               int keys_first) {
    pdl_entry();
    const int at = blockIdx.x, n = keys_first ? gk.blocks : gq.blocks;
    if ((at < n) == (keys_first != 0))
        bwd_block<T, DP, true, FINE>(gk, keys_first ? at : at - n, x.k, x.v, x.q_walk, x.dout_walk);
    else
        bwd_block<T, DP, false, FINE>(gq, keys_first ? at - n : at, x.q, x.dout, x.k_walk, x.v_walk);
}

// What the walks need of every row, eight lanes each. blockIdx.y = 0: of every query, padded: boost - lse log2(e), so
// that P times 2^boost = exp2(scale log2(e) S + that), and -delta; -inf and 0 where there is no query, -inf where it
// has no key. 1: zero gradients of the keys that take no part. With norms, the largest squared norms of dout's (0) and
// of v's rows (1) of each batch entry and key head too, as bits of floats (zero before; maxima do not depend on
// their order).
template <class T>
__global__ void __launch_bounds__(256) k_attn_stats(const AttnArgs a, long long qpad, long long rows_k, int boost, unsigned* norms,
                                                    float* nlse, float* ndelta) {
    pdl_entry();
    constexpr int V = 16 / (int)sizeof(T);
    const bool keys = blockIdx.y;
    const unsigned blocks = (unsigned)((keys ? rows_k : qpad) / 32);  // of a head: a block's 32 rows are of one head
    const int bh = (int)(blockIdx.x / blocks), i = (int)(blockIdx.x % blocks) * 32 + threadIdx.x / 8, lane = threadIdx.x & 7;
    const int heads = keys ? a.kv_heads : a.heads, b = bh / heads, h = bh % heads;
    const long long at = (long long)bh * qpad + i;
    if (b >= a.batch) return;  // the whole block
    __shared__ unsigned most;
    if (norms && threadIdx.x == 0) most = 0u;
    const bool in = i < (keys ? a.len_k : a.len_q), valid = in && (!keys || key_valid(a, b, i, key_count(a, b)));
    const float l = !keys && in ? a.lse[(long long)bh * a.len_q + i] : -INFINITY;
    float s = 0.f, n2 = 0.f;  // of out and dout; of dout or v with itself
    if (valid && (!keys || norms)) {
        const AttnTensor& t = keys ? a.v : a.dout;
        const T* d = head_base<T>(t, b, h) + (long long)i * t.len_stride;
        const T* o = keys ? d : head_base<T>(a.out, b, h) + (long long)i * a.out.len_stride;
        const bool vec = a.d % V == 0 && (reinterpret_cast<uintptr_t>(o) | reinterpret_cast<uintptr_t>(d)) % 16 == 0;
        constexpr int kTurns = (sizeof(T) == 2 ? 128 : 64) / (8 * V);  // heads of up to 128, float32 of up to 64
        Pack<T, V> x[kTurns], y[kTurns];
        const T zero = from_float<T>(0.f);
#pragma unroll
        for (int u = 0; u < kTurns; ++u) {
            const int c = (u * 8 + lane) * V;
            if (vec && c < a.d) {
                x[u] = *reinterpret_cast<const Pack<T, V>*>(o + c), y[u] = *reinterpret_cast<const Pack<T, V>*>(d + c);
            } else {  // the same elements per lane, so that a layout changes no sum
#pragma unroll
                for (int k = 0; k < V; ++k) x[u].v[k] = c + k < a.d ? o[c + k] : zero, y[u].v[k] = c + k < a.d ? d[c + k] : zero;
            }
        }
#pragma unroll
        for (int u = 0; u < kTurns; ++u)
#pragma unroll
            for (int k = 0; k < V; ++k) {
                s = fmaf(to_float(x[u].v[k]), to_float(y[u].v[k]), s);
                if (norms) n2 = fmaf(to_float(y[u].v[k]), to_float(y[u].v[k]), n2);
            }
    }
#pragma unroll
    for (int k = 4; k > 0; k >>= 1) s += __shfl_xor_sync(0xffffffffu, s, k);
    if (!keys && lane == 0) {
        nlse[at] = l == -INFINITY ? -INFINITY : (float)boost - l * 1.4426950408889634f;
        ndelta[at] = -s;
    }
    if (keys && in && !valid) {
        T* dk = static_cast<T*>(a.dk.data) + b * a.dk.batch_stride + h * a.dk.head_stride + i * a.dk.len_stride;
        T* dv = static_cast<T*>(a.dv.data) + b * a.dv.batch_stride + h * a.dv.head_stride + i * a.dv.len_stride;
        for (int c = lane; c < a.d; c += 8) dk[c] = dv[c] = from_float<T>(0.f);
    }
    if (norms) {
#pragma unroll
        for (int k = 4; k > 0; k >>= 1) n2 += __shfl_xor_sync(0xffffffffu, n2, k);
        const unsigned w = __reduce_max_sync(0xffffffffu, __float_as_uint(fabsf(n2)));  // NaN compares above every number
        __syncthreads();
        if ((threadIdx.x & 31) == 0) atomicMax(&most, w);
        __syncthreads();
        if (threadIdx.x == 0) {
            // (thousands of blocks' atomics on a few words follow one another: only those that raise the maximum)
            unsigned* to = norms + (b * a.kv_heads + (keys ? h : h / (a.heads / a.kv_heads))) * 2 + keys;
            if (most > *static_cast<volatile unsigned*>(to)) atomicMax(to, most);
        }
    }
}

// What a walk that was split left: the shares added up in order, a thread per eight elements of a row; dq, or dk and dv
// (blockIdx.y). rows: of a head in the shares, of which the first `live` of a batch entry were written.
template <class T>
__global__ void __launch_bounds__(256) k_attn_sum(const BwdArgs g, int heads, int keys, const float* part, int splits, int dp, long long rows) {
    pdl_entry();
    const AttnArgs& a = g.t.a;
    const AttnTensor& t = !keys ? a.dq : blockIdx.y == 0 ? a.dk : a.dv;
    const long long share = (long long)a.batch * heads * rows * dp, split_stride = share * gridDim.y;
    part += blockIdx.y * share;
    const long long at = (long long)blockIdx.x * 256 + threadIdx.x;
    const int per = dp / 8, c = (int)(at % per) * 8;
    const long long r = at / per, bh = r / rows;
    const int row = (int)(r % rows), b = (int)(bh / heads), h = (int)(bh % heads);
    if (b >= a.batch || c >= a.d || row >= (keys ? keys_of(g.t, b) : a.len_q)) return;
    float x[8] = {};
    for (int s = 0; s < splits; ++s) {
        const float4* p = reinterpret_cast<const float4*>(part + s * split_stride + r * dp + c);
        const float4 u = p[0], v = p[1];
        x[0] += u.x, x[1] += u.y, x[2] += u.z, x[3] += u.w, x[4] += v.x, x[5] += v.y, x[6] += v.z, x[7] += v.w;
    }
    const long long to = keys && g.index ? g.index[(long long)b * a.len_k + row] : row;
    T* dst = static_cast<T*>(t.data) + b * t.batch_stride + h * t.head_stride + to * t.len_stride + c;
#pragma unroll
    for (int k = 0; k < 8; ++k)
        if (c + k < a.d) dst[k] = from_float<T>(x[k]);
}

namespace {

template <class T, int DP, bool FINE>
cudaError_t run(const BwdArgs& gq, const BwdArgs& gk, const BwdTensors& x, bool keys_first, cudaStream_t st) {
    constexpr int smem = BwdShape<DP, false>::kSmem > BwdShape<DP, true>::kSmem ? BwdShape<DP, false>::kSmem : BwdShape<DP, true>::kSmem;
    auto* kernel = k_attn_bwd<T, DP, FINE>;
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e) return e;
    return launch_pdl(kernel, dim3((unsigned)(gq.blocks + gk.blocks)), dim3(512), smem, st, gq, gk, x, (int)keys_first);
}

template <class T>
cudaError_t typed(const BwdArgs& gq, const BwdArgs& gk, const BwdTensors& x, bool keys_first, int dp, bool fine, cudaStream_t st) {
    if (dp == 64) return fine ? run<T, 64, true>(gq, gk, x, keys_first, st) : run<T, 64, false>(gq, gk, x, keys_first, st);
    return fine ? run<T, 128, true>(gq, gk, x, keys_first, st) : run<T, 128, false>(gq, gk, x, keys_first, st);
}

template <class F>
cudaError_t by_type(int dtype, F&& f) {
    return dtype == GS_DTYPE_F32 ? f(float()) : dtype == GS_DTYPE_F16 ? f(__half()) : f(__nv_bfloat16());
}

unsigned blocks_of(long long threads) { return (unsigned)((threads + 255) / 256); }

}  // namespace

cudaError_t launch_attn_bwd_tc(const TcBwd& w, const BwdTensors& x, cudaStream_t st) {
    const AttnArgs& a = w.a;
    const bool half = a.dtype == GS_DTYPE_F16, by_key = half || a.key_mask || a.k_len;
    const long long q = (long long)a.batch * a.heads * w.qpad * 8, k = by_key ? (long long)a.batch * a.kv_heads * w.rows_k * 8 : 0;
    count_launches(1);
    cudaError_t e = by_type(a.dtype, [&](auto t) {
        return launch_pdl(k_attn_stats<decltype(t)>, dim3(blocks_of(q > k ? q : k), by_key ? 2 : 1), dim3(256), 0, st, a, w.qpad,
                          w.rows_k, half ? kBoost : 0, half ? w.norms : nullptr, w.nlse, w.ndelta);
    });
    if (e) return e;
    const int tiles_q = (a.len_q + kTileRows - 1) / kTileRows, tiles_k = (a.len_k + kTileRows - 1) / kTileRows;
    const long long blocks_q = (long long)tiles_q * w.splits_q * a.heads * a.batch,
                    blocks_k = (long long)tiles_k * w.splits_k * a.kv_heads * a.batch;
    if (blocks_q + blocks_k > 0x7fffffffll) return cudaErrorInvalidConfiguration;
    const BwdArgs gq{{a, w.count, w.part_q, nullptr, tiles_q, w.splits_q}, w.nlse, w.ndelta, w.qpad, half ? w.norms : nullptr,
                     w.index, w.rows_k, (int)blocks_q};
    BwdArgs gk = gq;
    gk.t.part = w.part_k;
    gk.t.tiles = tiles_k;
    gk.t.splits = w.splits_k;
    gk.blocks = (int)blocks_k;
    // Rounding P and dS to 16 bits makes errors as large as the results' own rounding: 1.4 times it over a call's gradients
    // whatever its size, but the fewer rows a sum of dk or dv runs over, the more may be rounded the same way. The worst key
    // head of 8 x 16 (bfloat16, dv) is off by 2.3 times that rounding with one row, 2.0 with five, 1.6 with 64 and 1.5 from
    // 128 on. So sums of up to 64 rows (a walked tile) take what the rounding left too, which leaves 1.0 (8 x 16 heads of
    // 64, 5 queries over 400 keys: 27.4 us without, 31.6 with it; 64 over 2000: 87 and 101), and small calls do, whose
    // time is mostly latency (one head of 512 over 2500: 18.0 and 19.4; 2 x 16 heads of 256 over 2500, which stay without: 42 and 51).
    const bool fine = (long long)a.len_q * (a.heads / a.kv_heads) <= kBN || (long long)a.batch * a.heads * a.len_q <= 512;
    count_launches(1);
    if (a.dtype == GS_DTYPE_F32) e = launch_attn_bwd_wide(gq, gk, x, w.keys_first, st);
    else if (half) e = typed<__half>(gq, gk, x, w.keys_first, w.dp, fine, st);
    else e = typed<__nv_bfloat16>(gq, gk, x, w.keys_first, w.dp, fine, st);
    if (e) return e;
    for (int keys = 0; keys < 2; ++keys) {
        const BwdArgs& g = keys ? gk : gq;
        if (g.t.splits == 1) continue;
        const int heads = keys ? a.kv_heads : a.heads;
        const long long rows = keys ? w.rows_k : a.len_q;
        count_launches(1);
        e = by_type(a.dtype, [&](auto t) {
            return launch_pdl(k_attn_sum<decltype(t)>, dim3(blocks_of((long long)a.batch * heads * rows * (w.dp / 8)), 1 + keys), dim3(256), 0,
                              st, g, heads, keys, (const float*)g.t.part, g.t.splits, w.dp, rows);
        });
        if (e) return e;
    }
    return cudaSuccess;
}

}  // namespace gs
