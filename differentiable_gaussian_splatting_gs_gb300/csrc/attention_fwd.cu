// Cross attention, forward, on the tensor cores.
//
// A block takes NQ tiles of 128 queries of one head (or of the heads that share a key head, where queries are few) and
// walks the keys, or its share of them, in tiles of BN. One warp copies K and
// V tiles ahead, a thread issues the products S = Q K^T and O += P V, and a warpgroup per query tile turns S
// into P: thread = query, so the row's maximum and sum need no exchange. S, P and O stay in tensor memory; P
// takes half the columns of its S. With two query tiles the products of one run beside the softmax of the
// other. Where the columns suffice (16-bit, heads of up to 64) a tile has 192 for S, and S takes the first and the
// last 128 of them in turn: the next S is then formed while this one's softmax runs, and the softmax
// never waits for P V. Otherwise the next S waits for P V.
//
// The softmax is bound by what a warp issues one after the other, its exponentials first (4 cycles a warp instruction
// and scheduler: 1024 for two 128 x 128 tiles, as many as their products take with heads of 64). So bfloat16 tiles do not
// look for the row's maximum: P is formed with the one in use, and only when the tile's sum shows that a score passed
// it far (a sum above 2^12) is the maximum found and raised, O rescaled and P formed again. Below that P, its sums and its
// products are as exact as with the maximum itself.
//
// float16 has no such room: P loses bits below 2^-14 and vanishes below 2^-25, and thousands of keys there may carry
// the output, where the few others' values are zero or cancel. P is formed 2^12 times as large, so that a key keeps its
// bits down to 2^-26 of the maximum in use (18 nats below it), and the maximum of every tile is looked for before P is formed
// and raised as soon as P would pass 2^15.9 (16384 x 4346, 32 heads of 64: 544 us, 498 without. Scores of spread 10: 623 us,
// where bfloat16's way takes 822. Forming P first and again where it passed took 557 to 1142).
//
// P is rounded to the tensors' type, the operand's of P V: the output's error against 64 bits is 1.4 times that of its own
// rounding. Multiplying what the rounding leaves too would be half as many products again.
#include "attention_tc.cuh"

namespace gs {

// Tensor-memory column, from the start of S, of the 16 probabilities from key 16 x on, plane q. With three
// planes a group of 32 keys' first two planes take the columns of its scores, so that P can replace S group by
// group; the third lies behind S.
template <int PL, int BN>
__device__ __forceinline__ int p_column(int q, int x) {
    return PL == 1 ? x * 8 : q < 2 ? (x / 2) * 32 + q * 16 + (x % 2) * 8 : BN + x * 8;
}

template <int DP, int PL, int NQ, int BN>
struct FwdShape {
    static constexpr int kQ = PL * DP * kTileRows * 2;  // bytes of a query tile
    static constexpr int kKV = PL * DP * BN * 2;        // bytes of a tile of K or V
    static constexpr int kRoom = 226 * 1024 - 1024 - NQ * kQ;
    static constexpr int kStages = kRoom / (2 * kKV) > 4 ? 4 : kRoom / (2 * kKV);
    static constexpr int kSmem = NQ * kQ + kStages * 2 * kKV + 1024;
    static constexpr bool kTurns = PL == 1 && DP == 64;  // S in two places
    static constexpr int kP = kTurns || PL == 3 ? BN + BN / 2 : BN;  // columns of a query tile's S and P
    // first column of S and of P of key tile j
    __device__ static int s_at(int j) { return kTurns && (j & 1) ? BN / 2 : 0; }
    __device__ static int p_at(int j) { return kTurns && (j & 1) ? BN : 0; }
    static constexpr int kIssuers = kTurns ? NQ : 1;  // threads that issue products
    // Tiles whose softmaxes nothing else keeps apart begin them half a tile apart.
    static constexpr bool kStagger = kTurns && NQ == 2;
    // Barriers that count a query tile's warps whose P is written. Where S takes turns a warp may be a key tile ahead of
    // the other three (one that raises its maximum takes about twice as long): with a barrier for even and one for odd
    // key tiles its arrival cannot be taken for theirs. The stagger's barriers bring a query tile's warps together before
    // each P, so that one suffices there (16384 x 4346 bf16, 32 heads: 495 us, with two 527).
    static constexpr int kPF = kTurns && !kStagger ? 2 : 1;
    // The tensor cores add to the accumulator by truncation: over hundreds of products that is a drift of
    // 2^-25 each, lost in 16-bit results but not in float32 ones (-1.4e-5 at 2,500 keys). With three planes
    // each key tile's product therefore starts from zero and is added to O in registers, rounded (2e-7).
    static constexpr bool kRegO = PL == 3;
    static constexpr int kO = NQ * kP;                              // first column of O
    // two query tiles: a third warpgroup of which two or three warps work, so that registers can be moved between whole
    // warpgroups (setmaxnreg): 384 threads x 168 at launch = 256 x 216 + 128 x 72,
    // or 256 x 200 + 128 x 104 with six products to issue for one
    static constexpr int kThreads = NQ == 2 ? 384 : 224;
    static constexpr int kCols = kO + NQ * DP <= 256 ? 256 : 512;
    static_assert(kO + NQ * DP <= 512 && kStages >= 1);
};

template <class T, int DP, int PL, int NQ, int BN>
__global__ void __launch_bounds__(FwdShape<DP, PL, NQ, BN>::kThreads, 1)
    k_attn_fwd(const __grid_constant__ TcArgs t, const __grid_constant__ TcTensor tq, const __grid_constant__ TcTensor tk,
               const __grid_constant__ TcTensor tv) {
    using S = FwdShape<DP, PL, NQ, BN>;
    using C = Pairs<PL>;
    constexpr int kSt = S::kStages, kPF = S::kPF;
    pdl_entry();
    extern __shared__ unsigned char raw[];
    __shared__ uint64_t q_full, k_full[kSt], v_full[kSt], k_free[kSt], v_free[kSt], s_full[NQ], s_free[NQ],
        p_full[NQ][kPF], o_done[NQ][2], drain[2];
    __shared__ uint32_t tmem_base;
    const AttnArgs& a = t.a;
    const uint32_t sq = (smem_u32(raw) + 1023u) & ~1023u, sk = sq + NQ * S::kQ, sv = sk + kSt * S::kKV;
    const bool whole = (int)blockIdx.x < t.whole;
    const int shared = (int)blockIdx.x - t.whole, split = whole ? 0 : shared % t.splits;
    const int block = whole ? (int)blockIdx.x : t.whole + shared / t.splits, tile = block % t.tiles, bh = block / t.tiles;
    const int groups = a.heads / t.fold, h0 = bh % groups * t.fold, b = bh / groups, hk = h0 / (a.heads / a.kv_heads);
    const int keys = keys_of(t, b), q0 = tile * NQ * t.fold_rows;
    // this block's key tiles
    const int all = (keys + BN - 1) / BN, per = whole ? all : (all + t.splits - 1) / t.splits;
    const int first = min(split * per, all), n = min(per, all - first);
    const int warp = threadIdx.x >> 5;
    const unsigned limit = a.spin_limit;

    if (threadIdx.x == 0) {
        mbar_init(&q_full, 1);
        for (int i = 0; i < kSt; ++i) {
            mbar_init(&k_full[i], 1);
            mbar_init(&v_full[i], 1);
            mbar_init(&k_free[i], S::kIssuers);
            mbar_init(&v_free[i], S::kIssuers);
        }
        for (int i = 0; i < NQ; ++i) {
            mbar_init(&s_full[i], 1);
            mbar_init(&s_free[i], 4);
            for (int e = 0; e < kPF; ++e) mbar_init(&p_full[i][e], 4);
            for (int e = 0; e < 2; ++e) mbar_init(&o_done[i][e], 1);
        }
        mbar_init(&drain[0], 1);
        mbar_init(&drain[1], 1);
        fence_mbar_init();
    }
    if (warp == NQ * 4) tmem_alloc<S::kCols>(&tmem_base);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tm = tmem_base;

    if (warp >= NQ * 4) {
        if (NQ == 2 && PL == 1) asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
        if (NQ == 2 && PL == 3) asm volatile("setmaxnreg.dec.sync.aligned.u32 104;");
        if (warp == NQ * 4) {  // copies
            if (n > 0 && elect_one()) {
                bool ok = true;
                int sent = 0;
                mbar_arrive_expect_tx(&q_full, NQ * S::kQ / kTileRows * t.fold * t.fold_rows);
                for (int i = 0; i < NQ; ++i) load_rows<DP, PL, kTileRows>(sq + i * S::kQ, tq, q0 + i * t.fold_rows, b, h0, a.heads, &q_full);
                for (int j = 0; j < n && ok; ++j) {
                    const int s = j % kSt;
                    const unsigned ph = (j / kSt + 1) & 1;
                    if (j >= kSt && !(ok = mbar_wait_bounded(&k_free[s], ph, limit, a.err))) break;
                    mbar_arrive_expect_tx(&k_full[s], S::kKV);
                    load_rows<DP, PL, BN>(sk + s * S::kKV, tk, (first + j) * BN, b, hk, a.kv_heads, &k_full[s]);
                    sent = 2 * j + 1;
                    if (j >= kSt && !(ok = mbar_wait_bounded(&v_free[s], ph, limit, a.err))) break;
                    mbar_arrive_expect_tx(&v_full[s], S::kKV);
                    load_rows<DP, PL, BN>(sv + s * S::kKV, tv, (first + j) * BN, b, hk, a.kv_heads, &v_full[s]);
                    sent = 2 * j + 2;
                }
                // every copy lands before the block ends, whatever became of its reader
                mbar_drain(&q_full, 0, a.err);
                const int nk = (sent + 1) / 2, nv = sent / 2;
                for (int j = max(0, nk - kSt); j < nk; ++j) mbar_drain(&k_full[j % kSt], (j / kSt) & 1, a.err);
                for (int j = max(0, nv - kSt); j < nv; ++j) mbar_drain(&v_full[j % kSt], (j / kSt) & 1, a.err);
            }
        } else if (warp - NQ * 4 - 1 < S::kIssuers && n > 0) {
            // Products: the warp waits, one thread issues. Where S takes turns, each query tile has a warp that
            // issues them. Otherwise one serves both tiles, and its order (P V and S of one, then of the other) keeps
            // their softmaxes half a turn apart.
            const int i0 = warp - NQ * 4 - 1, i1 = S::kTurns ? i0 + 1 : NQ;
            const uint32_t qk_desc = mma_desc<T>(BN, false), pv_desc = mma_desc<T>((a.d + 15) / 16 * 16, true);
            const int steps = (a.d + 15) / 16;  // of the inner dimension of Q K^T
            auto scores = [&](int i, int j) {
                const int s = j % kSt;
                if (!elect_one()) return;
#pragma unroll
                for (int c = 0; c < C::n; ++c) {
                    const uint32_t qa = tile_desc(sq + i * S::kQ + C::a(c) * DP * kTileRows * 2);
                    const uint32_t kb = tile_desc(sk + s * S::kKV + C::b(c) * DP * BN * 2);
#pragma unroll
                    for (int x = 0; x < DP / 16; ++x)
                        if (x < steps)
                            mma_ss(tm + i * S::kP + S::s_at(j), qa + (x / 4) * kTileRows * 8 + (x % 4) * 2,
                                   kb + (x / 4) * BN * 8 + (x % 4) * 2, qk_desc, c > 0 || x > 0);
                }
                mma_commit(&s_full[i]);
                if (i == i1 - 1) mma_commit(&k_free[s]);
            };
            auto values = [&](int i, int j) {
                const int s = j % kSt;
                if (!elect_one()) return;
#pragma unroll
                for (int c = 0; c < C::n; ++c) {
                    const uint32_t vb = tile_desc(sv + s * S::kKV + C::b(c) * DP * BN * 2, BN * 128);
#pragma unroll
                    for (int x = 0; x < BN / 16; ++x)
                        mma_ts(tm + S::kO + i * DP, tm + i * S::kP + S::p_at(j) + p_column<PL, BN>(C::a(c), x), vb + x * 128, pv_desc,
                               (!S::kRegO && j > 0) || c > 0 || x > 0);
                }
                if (j >= n - 2) mma_commit(&o_done[i][j & 1]);
                if (i == i1 - 1) mma_commit(&v_free[s]);
            };
            bool ok = warp_wait_all(&q_full, 0, &k_full[0], 0, limit, a.err);
            tc_fence_after();
            if (ok)
                for (int i = i0; i < i1; ++i) scores(i, 0);
            for (int j = 0; j < n && ok; ++j) {
                const bool more = j + 1 < n;
                uint64_t *vf = &v_full[j % kSt], *kf = &k_full[(j + 1) % kSt];
                const unsigned vp = j / kSt, kp = (j + 1) / kSt, pp = j / kPF;
                if (S::kTurns) {
                    if (more) {
                        // over the P of tile j - 1, whose P V this thread issued before
                        if (!(ok = warp_wait_all(kf, kp, &s_free[i0], j, limit, a.err))) break;
                        tc_fence_after();
                        scores(i0, j + 1);
                    }
                    if (!(ok = warp_wait_all(vf, vp, &p_full[i0][j % kPF], pp, limit, a.err))) break;
                    tc_fence_after();
                    values(i0, j);
                } else {
                    for (int i = 0; i < NQ; ++i) {
                        // with one stage the next K comes while P V runs
                        if (!(ok = more && kSt > 1 ? warp_wait_all(vf, vp, &p_full[i][j % kPF], pp, kf, kp, limit, a.err)
                                                   : warp_wait_all(vf, vp, &p_full[i][j % kPF], pp, limit, a.err)))
                            break;
                        tc_fence_after();
                        values(i, j);
                        if (!more) continue;
                        if (kSt == 1 && i == 0 && !(ok = warp_wait(kf, kp & 1, limit, a.err))) break;
                        scores(i, j + 1);
                    }
                }
            }
            // no product is in flight when the tensor memory is freed
            if (elect_one()) {
                mma_commit(&drain[i0]);
                mbar_drain(&drain[i0], 0, a.err);
            }
        }
    } else {  // softmax: thread = query
        if (NQ == 2 && PL == 1) asm volatile("setmaxnreg.inc.sync.aligned.u32 216;");
        if (NQ == 2 && PL == 3) asm volatile("setmaxnreg.inc.sync.aligned.u32 200;");
        const int i = warp / 4, r = threadIdx.x & 127, h = h0 + r / t.fold_rows, row = q0 + i * t.fold_rows + r % t.fold_rows;
        const uint32_t lanes = (uint32_t)(warp & 3) << 21, ti = tm + i * S::kP + lanes,
                       to = tm + S::kO + i * DP + lanes;
        const float c = a.scale * 1.4426950408889634f;  // scores in units of log2
        float top = -INFINITY, sum = 0.f;               // top: raw score in use as the maximum
        constexpr bool kHalf = std::is_same<T, __half>::value;
        // how far (log2) a score may pass the maximum in use where every tile's is looked for; the power of P for its range
        constexpr float kRoom = kHalf ? 3.9f : 8.f, kBoost = kHalf ? 12.f : 0.f;
        // the exponent's offset of a maximum in use; float16: rounded down, so that P of the maximum is 2^12 at most
        auto offset = [&](float t) { return t == -INFINITY ? 0.f : kHalf ? __fmaf_rd(-t, c, kBoost) : -t * c; };
        constexpr int kOut = S::kRegO ? DP : 1;
        float out[kOut];
#pragma unroll
        for (int e = 0; e < kOut; ++e) out[e] = 0.f;
        auto add_tile = [&]() {
#pragma unroll
            for (int g = 0; g < kOut / 32; ++g) {
                uint32_t o[32];
                tmem_ld32(to + g * 32, o);
                tmem_wait_ld(o);
#pragma unroll
                for (int e = 0; e < 32; ++e) out[(g * 32 + e) % kOut] += __uint_as_float(o[e]);
            }
        };
        // 32 columns of O
        auto get = [&](int g, uint32_t (&o)[32]) {
            if (S::kRegO) {
#pragma unroll
                for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(out[(g * 32 + e) % kOut]);
            } else {
                tmem_ld32(to + g * 32, o);
                tmem_wait_ld(o);
            }
        };
        // Two tiles whose softmaxes nothing else keeps apart fall into step, and the exponentials stand still while both
        // load: one may begin its tile when the other is half through. Every warp comes through every turn, one
        // whose wait gave up too.
        constexpr bool kStagger = S::kStagger;
        if (kStagger && i == 1 && n > 0) asm volatile("bar.arrive 1, 256;" ::: "memory");
        bool ok = true;
        for (int j = 0; j < n; ++j) {
            ok = ok && warp_wait(&s_full[i], j & 1, limit, a.err);
            tc_fence_after();
            const uint32_t ts = ti + S::s_at(j), tp = ti + S::p_at(j);
            const int left = keys - (first + j) * BN;
            auto mask = [&](uint32_t (&x)[32], int g) {
                if (left < BN) {
                    asm volatile("");  // a branch, not 32 selects in every tile
#pragma unroll
                    for (int e = 0; e < 32; ++e)
                        if (g * 32 + e >= left) x[e] = 0xff800000u;  // -inf
                }
            };
            float m8[8];  // eight chains: a maximum takes about ten cycles
#pragma unroll
            for (int e = 0; e < 8; ++e) m8[e] = -INFINITY;
            auto largest = [&](const uint32_t (&x)[32]) {
#pragma unroll
                for (int e = 0; e < 32; e += 2) m8[e / 2 % 8] = max3(m8[e / 2 % 8], __uint_as_float(x[e]), __uint_as_float(x[e + 1]));
            };
            auto row_max = [&]() { return max3(max3(m8[0], m8[1], m8[2]), max3(m8[3], m8[4], m8[5]), fmaxf(m8[6], m8[7])); };
            // P of 32 keys into its columns; s: the thread's sum
            auto probabilities = [&](const uint32_t (&x)[32], int g, f32x2 b2, f32x2 (&s)[4]) {
                uint32_t p[PL][16];
                const f32x2 c2 = f2_pack(c, c), one = f2_pack(1.f, 1.f);
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    float u[16];
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const int k = h * 16 + 2 * e;
                        const float2 y = f2_unpack(f2_fma(f2_pack(__uint_as_float(x[k]), __uint_as_float(x[k + 1])), c2, b2));
                        u[2 * e] = y.x;
                        u[2 * e + 1] = y.y;
                    }
#pragma unroll
                    for (int e = 0; e < 16; ++e) u[e] = ex2_approx(u[e]);
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        s[e & 3] = f2_fma(f2_pack(u[2 * e], u[2 * e + 1]), one, s[e & 3]);
#pragma unroll
                        for (int q = 0; q < PL; ++q) {
                            uint32_t& w = p[q][h * 8 + e];
                            w = pack2<T>(u[2 * e], u[2 * e + 1]);
                            if (q + 1 < PL) {  // what the plane leaves (bfloat16 is the upper half of a float)
                                u[2 * e] -= __uint_as_float(w << 16);
                                u[2 * e + 1] -= __uint_as_float(w & 0xffff0000u);
                            }
                        }
                    }
                }
#pragma unroll
                for (int q = 0; q < PL; ++q) tmem_st16(tp + p_column<PL, BN>(q, 2 * g), p[q]);
            };
            auto total = [&](const f32x2 (&s)[4]) {
                const f32x2 one = f2_pack(1.f, 1.f);
                const float2 p = f2_unpack(f2_fma(s[0], one, s[2])), q = f2_unpack(f2_fma(s[1], one, s[3]));
                return (p.x + p.y) + (q.x + q.y);
            };
            // whether the row's maximum in use is too far below m; a score of -inf is no error: exp(-inf) = 0
            auto passed = [&](float m) { return (m - top) * c > kRoom || (top == -INFINITY && m > -INFINITY); };
            auto base = [&]() { const float t0 = offset(top); return f2_pack(t0, t0); };
            f32x2 s2[4];
            if constexpr (S::kRegO) {
                // the registers hold O: the scores are read twice, and each group of P takes the columns of its scores
                if (j > 0) add_tile();
                uint32_t x[32];
#pragma unroll
                for (int g = 0; g < BN / 32; ++g) {
                    tmem_ld32(ts + g * 32, x);
                    tmem_wait_ld(x);
                    mask(x, g);
                    largest(x);
                }
                const float m = row_max();
                if (passed(m)) {
                    const float keep = top == -INFINITY ? 0.f : ex2_approx((top - m) * c);
                    top = m;
                    sum *= keep;
#pragma unroll
                    for (int e = 0; e < kOut; ++e) out[e] *= keep;
                }
                __syncwarp();
                s2[0] = s2[1] = s2[2] = s2[3] = f2_pack(0.f, 0.f);
#pragma unroll
                for (int g = 0; g < BN / 32; ++g) {
                    tmem_ld32(ts + g * 32, x);
                    tmem_wait_ld(x);
                    mask(x, g);
                    probabilities(x, g, base(), s2);
                }
            } else {
                constexpr int G = BN / 32;
                uint32_t x[G][32];
                // where S takes no turns, the second half of the scores is on its way while the first becomes P
#pragma unroll
                for (int g = 0; g < G / 2; ++g) tmem_ld32(ts + g * 32, x[g]);
#pragma unroll
                for (int g = 0; g < G / 2; ++g) {
                    tmem_wait_ld(x[g]);
                    mask(x[g], g);
                }
#pragma unroll
                for (int g = G / 2; g < G; ++g) tmem_ld32(ts + g * 32, x[g]);
                auto second_half = [&]() {
#pragma unroll
                    for (int g = G / 2; g < G; ++g) {
                        tmem_wait_ld(x[g]);
                        mask(x[g], g);
                    }
                };
                auto find_max = [&]() {
#pragma unroll
                    for (int g = 0; g < G; ++g) largest(x[g]);
                    return row_max();
                };
                if (S::kTurns) {  // the next S can start
                    second_half();
                    tc_fence_before();
                    warp_arrive(&s_free[i]);
                }
                // O times keep, once P V of tile j - 1 has left it: before this S where that takes no turns, else before the next
                auto rescale = [&](float keep) {
                    if (S::kTurns) {
                        ok = ok && (j + 1 < n ? warp_wait(&s_full[i], (j + 1) & 1, limit, a.err)
                                              : warp_wait(&o_done[i][(j - 1) & 1], 0, limit, a.err));
                        tc_fence_after();
                    }
#pragma unroll
                    for (int g = 0; g < DP / 32; ++g) {
                        uint32_t o[32];
                        tmem_ld32(to + g * 32, o);
                        tmem_wait_ld(o);
#pragma unroll
                        for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * keep);
                        tmem_st32(to + g * 32, o);
                    }
                };
                bool far = false;
                float keep = 1.f;
                if (kHalf || j == 0) {
                    if (!S::kTurns) second_half();
                    const float m = find_max();
                    if (!kHalf) {
                        top = m;
                    } else if ((far = passed(m))) {
                        keep = top == -INFINITY ? 0.f : ex2_approx(offset(m) - offset(top));
                        top = m;
                        sum *= keep;
                    }
                }
                s2[0] = s2[1] = s2[2] = s2[3] = f2_pack(0.f, 0.f);
                f32x2 b2 = base();
                if (kStagger) asm volatile("bar.sync %0, 256;" ::"r"(1 + i) : "memory");
#pragma unroll
                for (int g = 0; g < G / 2; ++g) probabilities(x[g], g, b2, s2);
                if (kStagger && (i == 0 || j + 1 < n)) asm volatile("bar.arrive %0, 256;" ::"r"(2 - i) : "memory");
                if (!kHalf && !S::kTurns) second_half();
#pragma unroll
                for (int g = G / 2; g < G; ++g) probabilities(x[g], g, b2, s2);
                if (kHalf) {
                    if (j > 0 && __any_sync(0xffffffffu, far)) rescale(keep);
                } else if (far = total(s2) > 4096.f || top == -INFINITY; __any_sync(0xffffffffu, far)) {
                    // (a row whose scores were all -inf has no maximum in use: it is looked for too)
                    const float m = find_max();
                    if (far) {
                        keep = top == -INFINITY ? 0.f : ex2_approx((top - m) * c);
                        top = m;
                    }
                    sum *= keep;
                    if (j > 0) rescale(keep);
                    s2[0] = s2[1] = s2[2] = s2[3] = f2_pack(0.f, 0.f);
                    b2 = base();
#pragma unroll
                    for (int g = 0; g < G; ++g) probabilities(x[g], g, b2, s2);
                }
            }
            sum += total(s2);
            tmem_wait_st();
            tc_fence_before();
            warp_arrive(&p_full[i][j % kPF]);
        }
        // committed for the last two tiles, on a barrier each; the last one's commit covers every product before it
        if (n > 0) ok = ok && warp_wait(&o_done[i][(n - 1) & 1], 0, limit, a.err);
        tc_fence_after();
        if (S::kRegO && n > 0) add_tile();
        const bool live = row < a.len_q && h < h0 + t.fold && ok;
        const float f = sum == 0.f ? 0.f : 1.f / sum;
        const float lse = sum == 0.f ? -INFINITY : (kHalf ? log2f(sum) - offset(top) : top * c + log2f(sum)) * 0.6931471805599453f;
        const long long qrow = ((long long)b * a.heads + h) * a.len_q + row;
        if (!whole) {
            const long long prow = ((long long)split * t.tail + block - t.whole) * (NQ * kTileRows) + i * kTileRows + r;
            if (live) t.part_lse[prow] = lse;
            if (n > 0) {
#pragma unroll
                for (int g = 0; g < DP / 32; ++g) {
                    uint32_t o[32];
                    get(g, o);
                    if (live) {
#pragma unroll
                        for (int e = 0; e < 32; e += 4)
                            *reinterpret_cast<float4*>(t.part + prow * DP + g * 32 + e) =
                                make_float4(__uint_as_float(o[e]) * f, __uint_as_float(o[e + 1]) * f,
                                            __uint_as_float(o[e + 2]) * f, __uint_as_float(o[e + 3]) * f);
                    }
                    __syncwarp();
                }
            }
        } else {
            if (live) a.lse[qrow] = lse;
            using E = typename std::conditional<PL == 3, float, T>::type;
            E* dst = static_cast<E*>(a.out.data) + b * a.out.batch_stride + h * a.out.head_stride + row * a.out.len_stride;
            constexpr int V = 16 / (int)sizeof(E);
            const bool vec = a.d % V == 0 && a.out.batch_stride % V == 0 && a.out.head_stride % V == 0 &&
                             a.out.len_stride % V == 0 && reinterpret_cast<uintptr_t>(a.out.data) % 16 == 0;
#pragma unroll
            for (int g = 0; g < DP / 32; ++g) {
                uint32_t o[32];
                if (n > 0) get(g, o);
                if (live) {
#pragma unroll
                    for (int e = 0; e < 32; e += V) {
                        Pack<E, V> w;
#pragma unroll
                        for (int y = 0; y < V; ++y) w.v[y] = from_float<E>(n > 0 ? __uint_as_float(o[e + y]) * f : 0.f);
                        const int col = g * 32 + e;
                        if (vec) {
                            if (col < a.d) *reinterpret_cast<Pack<E, V>*>(dst + col) = w;
                        } else {
#pragma unroll
                            for (int y = 0; y < V; ++y)
                                if (col + y < a.d) dst[col + y] = w.v[y];
                        }
                    }
                }
                __syncwarp();
            }
        }
        tc_fence_before();
    }
    __syncwarp();
    __syncthreads();
    tc_fence_after();
    if (warp == NQ * 4) tmem_free<S::kCols>(tm);
}

namespace {

template <class T, int DP, int PL, int NQ, int BN>
cudaError_t run(TcArgs t, const TcTensor& q, const TcTensor& k, const TcTensor& v, cudaStream_t st) {
    using S = FwdShape<DP, PL, NQ, BN>;
    auto* kernel = k_attn_fwd<T, DP, PL, NQ, BN>;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kSmem);
    if (e) return e;
    const long long blocks = t.whole + (long long)t.tail * t.splits;
    if (blocks > 0x7fffffffll) return cudaErrorInvalidConfiguration;
    count_launches(1);
    return launch_pdl(kernel, dim3((unsigned)blocks), dim3(S::kThreads), S::kSmem, st, t, q, k, v);
}

}  // namespace

cudaError_t launch_attn_fwd_tc(const TcArgs& t, const TcTensor& q, const TcTensor& k, const TcTensor& v, int planes, int dp,
                               int nq, cudaStream_t st) {
    if (planes == 3) {
        if (dp == 128) return run<__nv_bfloat16, 128, 3, 1, 64>(t, q, k, v, st);
        return nq == 1 ? run<__nv_bfloat16, 64, 3, 1, 128>(t, q, k, v, st) : run<__nv_bfloat16, 64, 3, 2, 128>(t, q, k, v, st);
    }
    const bool half = t.a.dtype == GS_DTYPE_F16;
    if (dp == 256) return half ? run<__half, 256, 1, 1, 64>(t, q, k, v, st) : run<__nv_bfloat16, 256, 1, 1, 64>(t, q, k, v, st);
    if (dp == 128) {
        if (nq == 1) return half ? run<__half, 128, 1, 1, 128>(t, q, k, v, st) : run<__nv_bfloat16, 128, 1, 1, 128>(t, q, k, v, st);
        return half ? run<__half, 128, 1, 2, 128>(t, q, k, v, st) : run<__nv_bfloat16, 128, 1, 2, 128>(t, q, k, v, st);
    }
    if (nq == 1) return half ? run<__half, 64, 1, 1, 128>(t, q, k, v, st) : run<__nv_bfloat16, 64, 1, 1, 128>(t, q, k, v, st);
    return half ? run<__half, 64, 1, 2, 128>(t, q, k, v, st) : run<__nv_bfloat16, 64, 1, 2, 128>(t, q, k, v, st);
}

}  // namespace gs
