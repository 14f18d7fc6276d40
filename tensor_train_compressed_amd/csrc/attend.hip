// Attention over packed whole prompts, forward and backward.
//
//   s_ij = scale q_i . k_j  (j of i's sequence; causal: j <= i),  p_ij = e^(s_ij - lse_i)
//   lse_i = log sum_j e^(s_ij),  o_i = sum_j p_ij v_j
//   delta_i = do_i . o_i,  ds_ij = p_ij (do_i . v_j - delta_i)
//   dq_i = scale sum_j ds_ij k_j,  dk_j = scale sum_i ds_ij q_i,  dv_j = sum_i p_ij do_i
// with dk and dv summed over the query heads that share a key head.
//
// One pass over keys and values: a wave keeps 32 queries of one head and goes over the
// sequence's tiles of keys in LDS with the running maximum and sum of a softmax; scores and
// weights never leave registers. Products are formed transposed, scores as K Q^T and
// outputs as V^T P^T, so that a lane has one query: its maximum and sum are its own (and
// one other lane's), and the weights it holds are the next product's operand as they are.
//
// The backward forms scores twice, once by queries (dq) and once by keys (dk and dv): seven
// products instead of five, but each result is summed by one wave in a fixed order, without
// atomics, and no partial sum goes through memory.
//
// Workgroups: heads that share keys are launched together and, where 8 divides the key
// heads, on one XCD, whose L2 then holds their keys; of a sequence the tiles with the most
// work come first.
#include "tt_attend.h"

namespace tt {
namespace {

struct AttendArgs {
    const void *q, *k, *v, *out, *dout;
    int64_t ldq, ldk, ldv, ldo, lddo;
    void *o, *dq, *dk, *dv;
    int64_t lddq, lddk, lddv;
    const int64_t* offsets;
    int64_t seqs, rows;
    int heads, kv, D, causal;
    float scale;
    float *lse, *delta;   // [heads][rows]
    hipStream_t s;
};

constexpr int kQueries = 32;   // a wave's

// Rows of a tile that goes through LDS, and waves of a workgroup.
template <class T, int DP>
constexpr int tile_rows() {
    return Tile<T, DP>::ROW <= 256 ? 64 : 32;
}
constexpr int kWaves = 4;

// The workgroup's head (its key head): those of one key head next to each other.
struct Job {
    int64_t tile;
    int kv, head;
};
__device__ __forceinline__ Job job_of(const AttendArgs& a) {
    const int i = blockIdx.x % a.heads, kv = i % a.kv;
    return {(int64_t)(blockIdx.x / a.heads), kv, kv * (a.heads / a.kv) + i / a.kv};
}

template <class T, int DP>
__global__ __launch_bounds__(kWaves * 64) void k_attend(const AttendArgs a) {
    typedef Tile<T, DP> L;
    constexpr int BN = tile_rows<T, DP>(), BLOCKS = BN / 32, BM = kWaves * kQueries;
    __shared__ __align__(16) char sk[BN * L::ROW], sv[BN * L::ROW];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const Job job = job_of(a);
    Span sp;
    if (!find_tile(a.offsets, a.seqs, a.rows, BM, job.tile, sp)) return;
    const int first = (sp.tiles - 1 - sp.tile) * BM, q0 = first + wave * kQueries, qi = q0 + (lane & 31);
    const bool there = qi < sp.len;
    const int64_t row = sp.first + qi;
    Piece fq[L::STEPS];
    load_row<T, DP>(fq, (const T*)a.q + row * a.ldq + (int64_t)job.head * a.D, there, a.D);
    const T* pk = (const T*)a.k + sp.first * a.ldk + (int64_t)job.kv * a.D;
    const T* pv = (const T*)a.v + sp.first * a.ldv + (int64_t)job.kv * a.D;
    const int last = a.causal ? min(sp.len, first + BM) : sp.len;              // of the workgroup's keys
    const int mine = a.causal ? min(sp.len, q0 + kQueries) : sp.len;           // of this wave's
    const int whole = a.causal ? min(sp.len, q0 + 1) : sp.len;                 // seen by all of its queries
    const int limit = a.causal ? min(sp.len, qi + 1) : sp.len;                 // seen by this lane's
    const float c = a.scale * kLog2e;
    floatx16 o[DP / 32] = {};
    Softmax<T> sm;
    sm.init();
    TileLoad<T, DP, BN, kWaves * 64> lk, lv;
    lk.load(pk, a.ldk, sp.len, a.D);
    lv.load(pv, a.ldv, sp.len, a.D);
    for (int k0 = 0; k0 < last; k0 += BN) {
        __syncthreads();
        lk.store(sk);
        lv.store(sv);
        __syncthreads();
        if (k0 + BN < last) {
            lk.load(pk + (k0 + BN) * a.ldk, a.ldk, sp.len - k0 - BN, a.D);
            lv.load(pv + (k0 + BN) * a.ldv, a.ldv, sp.len - k0 - BN, a.D);
        }
        if (k0 >= mine) continue;
        floatx16 s[BLOCKS] = {};
#pragma unroll
        for (int x = 0; x < L::STEPS; ++x)
#pragma unroll
            for (int b = 0; b < BLOCKS; ++b) s[b] = mma_rows<T>(L::row_piece(sk, 32 * b, x), fq[x], s[b]);
        if (k0 + BN > whole) {
#pragma unroll
            for (int b = 0; b < BLOCKS; ++b)
#pragma unroll
                for (int r = 0; r < 16; ++r)
                    if (k0 + 32 * b + block_row(r) >= limit) s[b][r] = -INFINITY;
        }
        sm.step(s, c, [&](float f) {
#pragma unroll
            for (int j = 0; j < DP / 32; ++j) o[j] *= f;
        });
#pragma unroll
        for (int b = 0; b < BLOCKS; ++b) {
            Weights<T> w;
            w.set(s[b]);
#pragma unroll
            for (int j = 0; j < DP / 32; ++j) o[j] = mma_columns<T, DP>(sv, 32 * b, j, w, o[j]);
        }
    }
    const float total = sm.total();
    if (!there) return;
    store_columns<T, DP>((T*)a.o + row * a.ldo + (int64_t)job.head * a.D, o, total == 0.f ? 0.f : 1.f / total, a.D);
    if (a.lse && lane < 32) a.lse[(int64_t)job.head * a.rows + row] = sm.log_sum(total);
}

// What weights are relative to, in powers of two: 2^(c s - it). Rows that see nothing have
// none.
__device__ __forceinline__ float log2_sum(float lse) { return lse == -INFINITY ? INFINITY : lse * kLog2e; }

// dq, and delta for the kernel below: by queries, as the forward.
template <class T, int DP>
__global__ __launch_bounds__(kWaves * 64) void k_attend_dq(const AttendArgs a) {
    typedef Tile<T, DP> L;
    constexpr int BN = tile_rows<T, DP>(), BLOCKS = BN / 32, BM = kWaves * kQueries;
    __shared__ __align__(16) char sk[BN * L::ROW], sv[BN * L::ROW];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const Job job = job_of(a);
    Span sp;
    if (!find_tile(a.offsets, a.seqs, a.rows, BM, job.tile, sp)) return;
    const int first = (sp.tiles - 1 - sp.tile) * BM, q0 = first + wave * kQueries, qi = q0 + (lane & 31);
    const bool there = qi < sp.len;
    const int64_t row = sp.first + qi;
    const int64_t at = (int64_t)job.head * a.D;
    Piece fq[L::STEPS], fd[L::STEPS];
    load_row<T, DP>(fq, (const T*)a.q + row * a.ldq + at, there, a.D);
    load_row<T, DP>(fd, (const T*)a.dout + row * a.lddo + at, there, a.D);
    float delta = 0.f;
    {
        Piece fo[L::STEPS];
        load_row<T, DP>(fo, (const T*)a.out + row * a.ldo + at, there, a.D);
#pragma unroll
        for (int x = 0; x < L::STEPS; ++x) {
            Raw8<T> u{}, w{};   // (fp32: the first four)
            __builtin_memcpy(&u, &fd[x], 16);
            __builtin_memcpy(&w, &fo[x], 16);
#pragma unroll
            for (int e = 0; e < L::P; ++e) delta = fmaf(u.at(e), w.at(e), delta);
        }
        delta = halves_sum(delta);
    }
    float lse2 = INFINITY;
    if (there) {
        lse2 = log2_sum(a.lse[(int64_t)job.head * a.rows + row]);
        if (lane < 32) a.delta[(int64_t)job.head * a.rows + row] = delta;
    }
    const T* pk = (const T*)a.k + sp.first * a.ldk + (int64_t)job.kv * a.D;
    const T* pv = (const T*)a.v + sp.first * a.ldv + (int64_t)job.kv * a.D;
    const int last = a.causal ? min(sp.len, first + BM) : sp.len;
    const int mine = a.causal ? min(sp.len, q0 + kQueries) : sp.len;
    const int whole = a.causal ? min(sp.len, q0 + 1) : sp.len;
    const int limit = a.causal ? min(sp.len, qi + 1) : sp.len;
    const float c = a.scale * kLog2e;
    floatx16 dq[DP / 32] = {};
    TileLoad<T, DP, BN, kWaves * 64> lk, lv;
    lk.load(pk, a.ldk, sp.len, a.D);
    lv.load(pv, a.ldv, sp.len, a.D);
    for (int k0 = 0; k0 < last; k0 += BN) {
        __syncthreads();
        lk.store(sk);
        lv.store(sv);
        __syncthreads();
        if (k0 + BN < last) {
            lk.load(pk + (k0 + BN) * a.ldk, a.ldk, sp.len - k0 - BN, a.D);
            lv.load(pv + (k0 + BN) * a.ldv, a.ldv, sp.len - k0 - BN, a.D);
        }
        if (k0 >= mine) continue;
#pragma unroll
        for (int b = 0; b < BLOCKS; ++b) {
            floatx16 s = {}, dp = {};
#pragma unroll
            for (int x = 0; x < L::STEPS; ++x) {
                s = mma_rows<T>(L::row_piece(sk, 32 * b, x), fq[x], s);
                dp = mma_rows<T>(L::row_piece(sv, 32 * b, x), fd[x], dp);
            }
#pragma unroll
            for (int r = 0; r < 16; ++r) s[r] = exp2_hw(fmaf(s[r], c, -lse2)) * (dp[r] - delta);
            if (k0 + 32 * (b + 1) > whole) {
#pragma unroll
                for (int r = 0; r < 16; ++r)
                    if (k0 + 32 * b + block_row(r) >= limit) s[r] = 0.f;
            }
            Weights<T> w;
            w.set(s);
#pragma unroll
            for (int j = 0; j < DP / 32; ++j) dq[j] = mma_columns<T, DP>(sk, 32 * b, j, w, dq[j]);
        }
    }
    if (there) store_columns<T, DP>((T*)a.dq + row * a.lddq + at, dq, a.scale, a.D);
}

// dk and dv: a wave keeps 32 keys and goes over the queries of every head that reads them.
template <class T, int DP>
__global__ __launch_bounds__(kWaves * 64) void k_attend_dkv(const AttendArgs a) {
    typedef Tile<T, DP> L;
    constexpr int BM = tile_rows<T, DP>(), BLOCKS = BM / 32, BN = kWaves * kQueries;
    __shared__ __align__(16) char sq[BM * L::ROW], sd[BM * L::ROW];
    __shared__ __align__(16) float slse[BM], sdelta[BM];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int kv = blockIdx.x % a.kv, group = a.heads / a.kv;
    Span sp;
    if (!find_tile(a.offsets, a.seqs, a.rows, BN, blockIdx.x / a.kv, sp)) return;
    const int first = sp.tile * BN, k0 = first + wave * kQueries, ki = k0 + (lane & 31);
    const bool there = ki < sp.len;
    const int64_t row = sp.first + ki, at = (int64_t)kv * a.D;
    Piece fk[L::STEPS], fv[L::STEPS];
    load_row<T, DP>(fk, (const T*)a.k + row * a.ldk + at, there, a.D);
    load_row<T, DP>(fv, (const T*)a.v + row * a.ldv + at, there, a.D);
    const float c = a.scale * kLog2e;
    floatx16 dk[DP / 32] = {}, dv[DP / 32] = {};
    const int begin = a.causal ? first / BM : 0, per = (sp.len + BM - 1) / BM - begin;   // tiles of queries a head
    const int all = per * group;
    TileLoad<T, DP, BM, kWaves * 64> lq, ld;
    float l = INFINITY, d = 0.f;   // of query threadIdx.x of the tile
    auto load = [&](int i) {
        const int head = kv * group + i / per, q0 = (begin + i % per) * BM, left = sp.len - q0;
        const int64_t r = sp.first + q0;
        lq.load((const T*)a.q + r * a.ldq + (int64_t)head * a.D, a.ldq, left, a.D);
        ld.load((const T*)a.dout + r * a.lddo + (int64_t)head * a.D, a.lddo, left, a.D);
        l = INFINITY;
        d = 0.f;
        if ((int)threadIdx.x < BM && (int)threadIdx.x < left) {
            l = log2_sum(a.lse[(int64_t)head * a.rows + r + threadIdx.x]);
            d = a.delta[(int64_t)head * a.rows + r + threadIdx.x];
        }
    };
    load(0);
    for (int i = 0; i < all; ++i) {
        __syncthreads();
        lq.store(sq);
        ld.store(sd);
        if (threadIdx.x < BM) {
            slse[threadIdx.x] = l;
            sdelta[threadIdx.x] = d;
        }
        __syncthreads();
        if (i + 1 < all) load(i + 1);
        const int q0 = (begin + i % per) * BM;
#pragma unroll
        for (int b = 0; b < BLOCKS; ++b) {
            const int first_q = q0 + 32 * b;
            if (first_q >= sp.len || (a.causal && first_q + 31 < k0)) continue;
            floatx16 s = {}, dp = {};
#pragma unroll
            for (int x = 0; x < L::STEPS; ++x) {
                s = mma_rows<T>(L::row_piece(sq, 32 * b, x), fk[x], s);
                dp = mma_rows<T>(L::row_piece(sd, 32 * b, x), fv[x], dp);
            }
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                float lg[4], dg[4];
                const int q = 32 * b + block_row(4 * g);
                __builtin_memcpy(lg, slse + q, 16);
                __builtin_memcpy(dg, sdelta + q, 16);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int r = 4 * g + e;
                    s[r] = exp2_hw(fmaf(s[r], c, -lg[e]));
                    dp[r] = s[r] * (dp[r] - dg[e]);
                }
            }
            if (first_q + 32 > sp.len || (a.causal && first_q < k0 + 31)) {
#pragma unroll
                for (int r = 0; r < 16; ++r) {
                    const int q = first_q + block_row(r);
                    if (q >= sp.len || (a.causal && q < ki)) s[r] = dp[r] = 0.f;
                }
            }
            Weights<T> w;
            w.set(s);
#pragma unroll
            for (int j = 0; j < DP / 32; ++j) dv[j] = mma_columns<T, DP>(sd, 32 * b, j, w, dv[j]);
            w.set(dp);
#pragma unroll
            for (int j = 0; j < DP / 32; ++j) dk[j] = mma_columns<T, DP>(sq, 32 * b, j, w, dk[j]);
        }
    }
    if (!there) return;
    store_columns<T, DP>((T*)a.dk + row * a.lddk + at, dk, a.scale, a.D);
    store_columns<T, DP>((T*)a.dv + row * a.lddv + at, dv, 1.f, a.D);
}

template <class T, int DP>
tt_status attend_launch(const AttendArgs& a, bool backward) {
    const int64_t tiles = a.rows / (kWaves * kQueries) + a.seqs;
    const dim3 grid((unsigned)(tiles * a.heads)), block(kWaves * 64);
    if (!backward) {
        TT_LAUNCH(nullptr, "k_attend", a.s, (k_attend<T, DP>), grid, block, 0, a.s, a);
        TT_LAUNCH_CHECK();
        return TT_OK;
    }
    TT_LAUNCH(nullptr, "k_attend_dq", a.s, (k_attend_dq<T, DP>), grid, block, 0, a.s, a);
    TT_LAUNCH_CHECK();
    TT_LAUNCH(nullptr, "k_attend_dkv", a.s, (k_attend_dkv<T, DP>), dim3((unsigned)(tiles * a.kv)), block, 0, a.s, a);
    TT_LAUNCH_CHECK();
    return TT_OK;
}

template <class T>
tt_status attend_by_dim(const AttendArgs& a, bool backward) {
    if (a.rows == 0 || a.seqs == 0) return TT_OK;
    if (a.D <= 32) return attend_launch<T, 32>(a, backward);
    if (a.D <= 64) return attend_launch<T, 64>(a, backward);
    if (a.D <= 96) return attend_launch<T, 96>(a, backward);
    return attend_launch<T, 128>(a, backward);
}

tt_status attend_by_type(int32_t dtype, const AttendArgs& a, bool backward) {
    if (dtype == TT_F32) return attend_by_dim<float>(a, backward);
    if (dtype == TT_BF16) return attend_by_dim<bf16>(a, backward);
    return attend_by_dim<f16>(a, backward);
}

constexpr int64_t kMaxLd = (int64_t(1) << 22) - 1;

tt_status attend_sizes(int32_t dtype, int64_t rows, int64_t heads, int64_t kv, int64_t dim) {
    if (!dtype_ok(dtype) || rows < 0 || heads < 1 || kv < 1 || dim < 1 || heads % kv != 0) return TT_ERR_INVALID_ARG;
    if (dim > 128 || rows > INT32_MAX || heads > (int64_t(1) << 22)) return TT_ERR_UNSUPPORTED;
    return TT_OK;
}

// The arguments that every call takes.
tt_status attend_args(AttendArgs& a, int32_t dtype, const void* q, int64_t ldq, const void* k, int64_t ldk,
                      const void* v, int64_t ldv, const int64_t* offsets, int64_t seqs, int64_t rows, int64_t heads,
                      int64_t kv, int64_t dim, int32_t causal, float scale, void* stream) {
    const tt_status st = attend_sizes(dtype, rows, heads, kv, dim);
    if (st != TT_OK) return st;
    if (seqs < 0 || !(scale > 0.f && scale < INFINITY)) return TT_ERR_INVALID_ARG;
    if (ldq < heads * dim || ldk < kv * dim || ldv < kv * dim) return TT_ERR_INVALID_ARG;
    if (rows > 0 && seqs > 0 && (!q || !k || !v || !offsets)) return TT_ERR_INVALID_ARG;
    if (ldq > kMaxLd || ldk > kMaxLd || ldv > kMaxLd || seqs > INT32_MAX) return TT_ERR_UNSUPPORTED;
    if ((rows / kQueries + seqs) * heads > int64_t(1) << 24) return TT_ERR_UNSUPPORTED;
    a = AttendArgs{};
    a.q = q; a.k = k; a.v = v;
    a.ldq = ldq; a.ldk = ldk; a.ldv = ldv;
    a.offsets = offsets; a.seqs = seqs; a.rows = rows;
    a.heads = (int)heads; a.kv = (int)kv; a.D = (int)dim; a.causal = causal;
    a.scale = scale;
    a.s = (hipStream_t)stream;
    return TT_OK;
}

}  // namespace
}  // namespace tt

using namespace tt;

extern "C" size_t tt_emb_attend_workspace_bytes(int32_t dtype, int64_t rows, int64_t heads, int64_t kv_heads,
                                                int64_t dim) {
    if (attend_sizes(dtype, rows, heads, kv_heads, dim) != TT_OK) return 0;
    return std::max<size_t>(256, ((size_t)rows * heads * sizeof(float) + 255) & ~size_t(255));
}

extern "C" tt_status tt_emb_attend_forward(int32_t dtype, const void* q, int64_t ldq, const void* k, int64_t ldk,
                                           const void* v, int64_t ldv, const int64_t* offsets, int64_t seqs, void* out,
                                           int64_t ldo, float* lse, int64_t rows, int64_t heads, int64_t kv_heads,
                                           int64_t dim, int32_t causal, float scale, void* stream) {
    AttendArgs a;
    const tt_status st = attend_args(a, dtype, q, ldq, k, ldk, v, ldv, offsets, seqs, rows, heads, kv_heads, dim, causal,
                                     scale, stream);
    if (st != TT_OK) return st;
    if (ldo < heads * dim || (rows > 0 && seqs > 0 && !out)) return TT_ERR_INVALID_ARG;
    a.o = out; a.ldo = ldo;
    a.lse = lse;
    return attend_by_type(dtype, a, false);
}

extern "C" tt_status tt_emb_attend_backward(int32_t dtype, const void* q, int64_t ldq, const void* k, int64_t ldk,
                                            const void* v, int64_t ldv, const int64_t* offsets, int64_t seqs,
                                            const void* out, int64_t ldo, const float* lse, const void* dout,
                                            int64_t lddo, void* dq, int64_t lddq, void* dk, int64_t lddk, void* dv,
                                            int64_t lddv, int64_t rows, int64_t heads, int64_t kv_heads, int64_t dim,
                                            int32_t causal, float scale, void* workspace, size_t workspace_bytes,
                                            void* stream) {
    AttendArgs a;
    const tt_status st = attend_args(a, dtype, q, ldq, k, ldk, v, ldv, offsets, seqs, rows, heads, kv_heads, dim, causal,
                                     scale, stream);
    if (st != TT_OK) return st;
    if (ldo < heads * dim || lddo < heads * dim || lddq < heads * dim || lddk < kv_heads * dim || lddv < kv_heads * dim)
        return TT_ERR_INVALID_ARG;
    if (rows > 0 && seqs > 0 && (!out || !lse || !dout || !dq || !dk || !dv)) return TT_ERR_INVALID_ARG;
    if (lddo > kMaxLd) return TT_ERR_UNSUPPORTED;
    if (!workspace || ((uintptr_t)workspace & 255) != 0) return TT_ERR_INVALID_ARG;
    if (workspace_bytes < tt_emb_attend_workspace_bytes(dtype, rows, heads, kv_heads, dim)) return TT_ERR_WORKSPACE;
    a.out = out; a.ldo = ldo;
    a.lse = const_cast<float*>(lse);
    a.dout = dout; a.lddo = lddo;
    a.dq = dq; a.dk = dk; a.dv = dv;
    a.lddq = lddq; a.lddk = lddk; a.lddv = lddv;
    a.delta = (float*)workspace;
    return attend_by_type(dtype, a, true);
}
