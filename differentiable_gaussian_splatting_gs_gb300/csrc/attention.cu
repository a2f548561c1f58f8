// Cross attention: which kernels a call runs, its workspace, and the tensor maps of its copies.
#include <cudaTypedefs.h>

#include "attention_tc.cuh"

#include <algorithm>

namespace gs {

namespace {

// The largest head dimension on the tensor cores; the float32 kernels take the others. Three planes of wider float32 rows and of
// two tiles do not fit shared memory, nor do the backward's two accumulators of 256 columns with a walked tile the tensor memory.
int max_tc_dim(int dtype, bool backward) { return dtype == GS_DTYPE_F32 ? (backward ? 64 : 128) : backward ? 128 : 256; }

// What a call packs, how it splits its walks, and where the pieces lie in the workspace (byte offsets).
struct Plan {
    bool tc, decode, pack_q, pack_kv, pack_do, keys_first;
    int planes, dp, nq, splits;
    int fold, fold_rows;     // forward: heads to a tile, queries of each
    int tiles, tail;         // forward: of a (group of) head's queries; blocks whose walk is split
    long long whole;         // blocks that walk all keys
    int splits_q, splits_k;  // backward: of the walks for dq, and for dk and dv
    long long rows_k;        // rows of a packed head of K or V
    long long qpad;          // queries of a head, rounded up to the tiles that the backward walks
    size_t count, index, q, k, v, dout, part, part_k, part_lse, delta, nlse, norms, bytes;
};

bool copyable(const AttnTensor& t, const AttnArgs& a, int len) {
    // a tiled copy wants 16-byte aligned rows and positive strides; the caller's sizes of 1 have no stride
    auto fine = [](long long stride, long long n) { return n <= 1 || (stride > 0 && stride % 8 == 0 && stride < (1ll << 38)); };
    return a.d % 8 == 0 && reinterpret_cast<uintptr_t>(t.data) % 16 == 0 && fine(t.batch_stride, a.batch) &&
           fine(t.len_stride, len) && fine(t.head_stride, 2);
}

// `tensors`: whether a's tensors are known; the size of the workspace counts on every one being packed.
Plan plan(const AttnArgs& a, bool backward, bool tensors) {
    Plan p{};
    size_t at = 0;
    auto take = [&](size_t bytes) {
        const size_t here = at;
        at += (bytes + 255) / 256 * 256;
        return here;
    };
    const size_t bq = (size_t)a.batch * a.heads * a.len_q, bk = (size_t)a.batch * a.kv_heads;
    p.tc = a.d <= max_tc_dim(a.dtype, backward) && a.len_k > 0 && a.len_q > 0;
    if (!backward && a.len_q == 1 && a.len_k > 0 && a.heads == a.kv_heads) {
        // two blocks an SM, with at least 64 keys each
        p.tc = false;
        p.decode = true;
        p.dp = (a.d + 3) / 4 * 4;
        const long long blocks = (long long)bk, most = (a.len_k + 63) / 64;
        long long splits = 2 * device_sm_count() / (blocks > 0 ? blocks : 1);
        if (splits > most) splits = most;
        p.splits = splits < 1 ? 1 : (int)splits;
        if (p.splits > 1) {
            p.part = take((size_t)p.splits * bq * p.dp * sizeof(float));
            p.part_lse = take((size_t)p.splits * bq * sizeof(float));
        }
    }
    if (backward && !p.tc && a.len_k > 0) p.delta = take(bq * sizeof(float));
    if (p.tc) {
        const bool wide = a.dtype == GS_DTYPE_F32, masked = a.key_mask || a.k_len;
        p.planes = wide ? 3 : 1;
        p.dp = a.d <= 64 ? 64 : a.d <= 128 ? 128 : 256;
        p.rows_k = ((long long)a.len_k + kTileRows - 1) / kTileRows * kTileRows;
        p.pack_q = wide || !tensors || !copyable(a.q, a, a.len_q);
        p.pack_do = backward && (wide || !tensors || !copyable(a.dout, a, a.len_q));
        p.pack_kv = wide || masked || !tensors || !copyable(a.k, a, a.len_k) || !copyable(a.v, a, a.len_k);
        const int sms = device_sm_count();
        auto over = [](long long n, long long m) { return (n + m - 1) / m; };
        if (!backward) {
            // Whole rounds of the SMs walk all keys; the blocks of the last round split their walks where that fills it.
            // A split block costs about `extra` tiles' time at its start and end, the shares' joining as much again. 5000 x
            // 2500 float32, 16 heads of 64 (2 rounds and 16 blocks): 293 us whole, 229 us with nine shares; 16384 x 4346
            // bf16, 32 heads (13 rounds and 72 blocks): 501 and 491 us. Two query tiles per block work beside each
            // other; a block of one takes 0.81 (16-bit heads of 64) to 0.89 (128) of their time.
            const long long extra = wide ? 2 : 3, walk = p.rows_k / kTileRows;
            long long best = 0;
            // Heads that share a key head may share tiles too, which leaves fewer rows empty where queries are few: one
            // query of 4 x 32 heads over 8192 keys of 8 heads of 128, float16: 96 us without, 33 us so.
            const int group = a.heads / a.kv_heads;
            for (int way = 0; way < 4; ++way) {
                const int nq = way % 2 ? 1 : 2, fold = way / 2 ? group : 1, fold_rows = kTileRows / fold;
                if ((nq == 2 && (wide ? p.dp == 128 : p.dp == 256)) || (way / 2 && group == 1) || fold > kTileRows) continue;
                const long long tiles = over(a.len_q, fold_rows * nq), blocks = tiles * (a.heads / fold) * a.batch, tail = blocks % sms;
                for (int rounds = 0; rounds <= (tail > 0 ? 4 : 0); ++rounds) {  // that the shares take; 0: no split
                    long long s = rounds == 0 ? 1 : std::min((long long)sms * rounds / tail, walk / 2);
                    if (rounds > 0 && s < 2) continue;
                    s = over(walk, over(walk, s));  // no share without tiles
                    const long long time = (blocks / sms * (walk + extra) + over(tail * s, sms) * (over(walk, s) + extra) +
                                            (s > 1 ? extra : 0)) * (nq == 1 ? 85 : 100);
                    if (p.nq && time >= best) continue;
                    best = time;
                    p.nq = nq;
                    p.fold = fold;
                    p.fold_rows = fold_rows;
                    p.splits = (int)s;
                    p.tiles = (int)tiles;
                    p.tail = s > 1 ? (int)tail : 0;
                    p.whole = blocks - p.tail;
                }
            }
        } else {
            p.qpad = over(a.len_q, kBN) * kBN;
            // A block walks at most one and a half times an SM's share of all walks, at least four tiles: 500 x 2500 bf16, 8
            // heads of 64, splits of 3: 25.4 us, 2: 25.4; 4000 x 500: 1: 43.2, 2: 32.9, 3: 34.4, 8: 44.2 us.
            const long long walk_q = over(a.len_k, kBN), walk_k = p.qpad / kBN * (a.heads / a.kv_heads),
                            all = over(a.len_q, kTileRows) * a.heads * a.batch * walk_q +
                                  over(a.len_k, kTileRows) * a.kv_heads * a.batch * walk_k,
                            share = 3 * all > 8ll * sms ? over(3 * all, 2 * sms) : 4;
            p.splits_q = (int)over(walk_q, share);
            p.splits_k = (int)over(walk_k, share);
            p.keys_first = over(walk_k, p.splits_k) > over(walk_q, p.splits_q);
            p.nlse = take((size_t)a.batch * a.heads * p.qpad * sizeof(float));
            p.delta = take((size_t)a.batch * a.heads * p.qpad * sizeof(float));
            if (a.dtype == GS_DTYPE_F16) p.norms = take(bk * 2 * sizeof(unsigned));
        }
        const size_t row = (size_t)p.planes * p.dp * 2;
        if (a.key_mask) {
            p.count = take(a.batch * sizeof(int));
            p.index = take((size_t)a.batch * a.len_k * sizeof(int));
        }
        if (p.pack_q) p.q = take(bq * row);
        if (p.pack_do) p.dout = take(bq * row);
        if (p.pack_kv) {
            p.k = take(bk * p.rows_k * row);
            p.v = take(bk * p.rows_k * row);
        }
        if (backward) {
            if (p.splits_q > 1) p.part = take((size_t)p.splits_q * bq * p.dp * sizeof(float));
            if (p.splits_k > 1) p.part_k = take((size_t)p.splits_k * 2 * bk * p.rows_k * p.dp * sizeof(float));
        } else if (p.splits > 1) {
            const size_t rows = (size_t)p.splits * p.tail * p.nq * kTileRows;
            p.part = take(rows * p.dp * sizeof(float));
            p.part_lse = take(rows * sizeof(float));
        }
    }
    p.bytes = at;
    return p;
}

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

cudaError_t encode(TcTensor& t, bool half, void* base, const long long (&dim)[4], const long long (&stride)[3], int box_rows,
                   int box_2, int box_3) {
    auto f = encoder();
    if (!f) return cudaErrorNotSupported;
    cuuint64_t dims[4], strides[3];
    for (int i = 0; i < 4; ++i) dims[i] = (cuuint64_t)dim[i];
    for (int i = 0; i < 3; ++i) strides[i] = (cuuint64_t)(dim[i + 1] > 1 ? stride[i] * 2 : 16);
    const cuuint32_t box[4] = {64, (cuuint32_t)box_rows, (cuuint32_t)box_2, (cuuint32_t)box_3}, step[4] = {1, 1, 1, 1};
    const CUresult r = f(&t.map, half ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, base, dims,
                         strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                         CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

// The tensor as the kernels read it: packed at `at`, or the caller's.
cudaError_t operand(TcTensor& t, const Plan& p, const AttnArgs& a, const AttnTensor& src, int heads, int len, bool packed,
                    void* at, long long rows, int box_rows, int box_heads = 1) {
    t.packed = packed;
    const bool half = a.dtype == GS_DTYPE_F16;
    if (packed)
        return encode(t, half, at, {p.dp, rows, p.planes, (long long)a.batch * heads},
                      {p.dp, rows * p.dp, p.planes * rows * p.dp}, box_rows, 1, box_heads);
    return encode(t, half, src.data, {a.d, len, heads, a.batch}, {src.len_stride, src.head_stride, src.batch_stride}, box_rows, box_heads, 1);
}

// The key mask's index, and K, V, Q and dout laid out where the kernels cannot read them as they are.
cudaError_t lay_out(const Plan& p, const AttnArgs& a, char* ws, int*& count, int*& index, cudaStream_t st) {
    cudaError_t e = cudaSuccess;
    count = index = nullptr;
    if (a.key_mask) {
        count = reinterpret_cast<int*>(ws + p.count);
        index = reinterpret_cast<int*>(ws + p.index);
        if ((e = launch_attn_index(a, count, index, st))) return e;
    }
    PackJob jobs[4];
    int n = 0;
    if (p.pack_q) jobs[n++] = {a.q, a.heads, a.len_q, 0, a.len_q, ws + p.q};
    if (p.pack_do) jobs[n++] = {a.dout, a.heads, a.len_q, 0, a.len_q, ws + p.dout};
    if (p.pack_kv) {
        jobs[n++] = {a.k, a.kv_heads, a.len_k, 1, p.rows_k, ws + p.k};
        jobs[n++] = {a.v, a.kv_heads, a.len_k, 1, p.rows_k, ws + p.v};
    }
    return launch_attn_pack(a, jobs, n, count, index, p.planes, p.dp, st);
}

}  // namespace

size_t attn_workspace_bytes(const AttnArgs& a, bool backward) { return plan(a, backward, false).bytes; }

cudaError_t launch_attn_fwd(const AttnArgs& a, void* workspace, cudaStream_t st) {
    const Plan p = plan(a, false, true);
    char* ws = static_cast<char*>(workspace);
    cudaError_t e;
    if (p.decode) {
        float* part = p.splits > 1 ? reinterpret_cast<float*>(ws + p.part) : nullptr;
        float* part_lse = p.splits > 1 ? reinterpret_cast<float*>(ws + p.part_lse) : nullptr;
        e = launch_attn_decode(a, p.splits, p.dp, part, part_lse, st);
        const TcArgs t{a, nullptr, part, part_lse, 1, p.splits, 0, a.batch * a.heads, 1, 1};
        return e || !part ? e : launch_attn_combine(t, 1, p.dp, st);
    }
    if (a.len_k == 0) return launch_attn_zero(a, a.out, a.heads, a.len_q, a.lse, st);
    if (!p.tc) return launch_attn_fwd_simt(a, st);
    if (p.whole > 0x7fffff00ll) return cudaErrorInvalidConfiguration;
    int *count, *index;
    e = lay_out(p, a, ws, count, index, st);
    if (e) return e;
    TcArgs t{a, count, nullptr, nullptr, p.tiles, p.splits, (int)p.whole, p.tail, p.fold, p.fold_rows};
    const int bn = (p.planes == 3 && p.dp == 128) || p.dp == 256 ? 64 : 128;
    TcTensor q, k, v;
    if ((e = operand(q, p, a, a.q, a.heads, a.len_q, p.pack_q, ws + p.q, a.len_q, p.fold_rows, p.fold)) ||
        (e = operand(k, p, a, a.k, a.kv_heads, a.len_k, p.pack_kv, ws + p.k, p.rows_k, bn)) ||
        (e = operand(v, p, a, a.v, a.kv_heads, a.len_k, p.pack_kv, ws + p.v, p.rows_k, bn)))
        return e;
    if (p.splits > 1) {
        t.part = reinterpret_cast<float*>(ws + p.part);
        t.part_lse = reinterpret_cast<float*>(ws + p.part_lse);
    }
    if ((e = launch_attn_fwd_tc(t, q, k, v, p.planes, p.dp, p.nq, st))) return e;
    return p.splits > 1 ? launch_attn_combine(t, p.nq * kTileRows, p.dp, st) : cudaSuccess;
}

cudaError_t launch_attn_bwd(const AttnArgs& args, void* workspace, cudaStream_t st) {
    const Plan p = plan(args, true, true);
    AttnArgs a = args;
    char* ws = static_cast<char*>(workspace);
    cudaError_t e;
    if (a.len_q == 0 || a.len_k == 0) {
        if ((e = launch_attn_zero(a, a.dq, a.heads, a.len_q, nullptr, st)) || (e = launch_attn_zero(a, a.dk, a.kv_heads, a.len_k, nullptr, st))) return e;
        return launch_attn_zero(a, a.dv, a.kv_heads, a.len_k, nullptr, st);
    }
    if (!p.tc) {
        a.delta = reinterpret_cast<float*>(ws + p.delta);
        return (e = launch_attn_delta(a, st)) ? e : launch_attn_bwd_simt(a, st);
    }
    int *count, *index;
    unsigned* norms = reinterpret_cast<unsigned*>(ws + p.norms);
    const size_t norm_bytes = (size_t)a.batch * a.kv_heads * 2 * sizeof(unsigned);
    if (a.dtype == GS_DTYPE_F16 && (e = cudaMemsetAsync(norms, 0, norm_bytes, st))) return e;
    if ((e = lay_out(p, a, ws, count, index, st))) return e;
    auto shares = [&](int splits, size_t at) { return splits > 1 ? reinterpret_cast<float*>(ws + at) : nullptr; };
    const TcBwd w{a, count, index, reinterpret_cast<float*>(ws + p.nlse), reinterpret_cast<float*>(ws + p.delta), norms,
                  shares(p.splits_q, p.part), shares(p.splits_k, p.part_k), p.qpad, p.rows_k, p.dp, p.splits_q, p.splits_k,
                  p.keys_first};
    BwdTensors x;
    TcTensor* to[2][4] = {{&x.q, &x.dout, &x.k, &x.v}, {&x.q_walk, &x.dout_walk, &x.k_walk, &x.v_walk}};
    for (int i = 0; i < 2; ++i) {
        const int box = i == 0 ? kTileRows : kBN;
        if ((e = operand(*to[i][0], p, a, a.q, a.heads, a.len_q, p.pack_q, ws + p.q, a.len_q, box)) ||
            (e = operand(*to[i][1], p, a, a.dout, a.heads, a.len_q, p.pack_do, ws + p.dout, a.len_q, box)) ||
            (e = operand(*to[i][2], p, a, a.k, a.kv_heads, a.len_k, p.pack_kv, ws + p.k, p.rows_k, box)) ||
            (e = operand(*to[i][3], p, a, a.v, a.kv_heads, a.len_k, p.pack_kv, ws + p.v, p.rows_k, box)))
            return e;
    }
    return launch_attn_bwd_tc(w, x, st);
}

}  // namespace gs
