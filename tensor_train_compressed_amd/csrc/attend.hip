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
    float* part;          // dk's, then dv's sums [splits][rows][kv * D]
    int splits;
    hipStream_t s;
};

// Lambdas of a kernel's loop are part of it, whatever their size.
#define TT_INLINE __attribute__((always_inline))

constexpr int kQueries = 32;   // a wave's

// Rows of a tile that goes through LDS, and waves of a workgroup.
template <class T, int DP>
constexpr int tile_rows() {
    return Tile<T, DP>::ROW <= 256 ? 64 : 32;
}
constexpr int kWaves = 4;

// Waves a SIMD is to hold: two where their registers allow it without spilling.
enum Pass { FWD, DQ, DKV };
template <class T, int DP, bool DMA, Pass PASS>
constexpr int waves_of() {
    if (sizeof(T) == 4) return DP == 32 || (DP == 64 && DMA && PASS != DKV) ? 2 : 1;
    if (PASS == DKV) return DP <= 64 || DMA ? 2 : 1;
    return DP <= 96 || DMA ? 2 : 1;
}

// The workgroup's head (its key head): those of one key head next to each other.
struct Job {
    int64_t tile;
    int kv, head;
};
__device__ __forceinline__ Job job_of(const AttendArgs& a) {
    const int i = blockIdx.x % a.heads, kv = i % a.kv;
    return {(int64_t)(blockIdx.x / a.heads), kv, kv * (a.heads / a.kv) + i / a.kv};
}

template <class T, int DP, bool DMA>
__global__ __launch_bounds__(kWaves * 64, (waves_of<T, DP, DMA, FWD>())) void k_attend(const AttendArgs a) {
    typedef Tile<T, DP> L;
    constexpr int BN = tile_rows<T, DP>(), BLOCKS = BN / 32, BM = kWaves * kQueries;
    __shared__ __align__(16) char sk0[BN * L::ROW], sv0[BN * L::ROW], sk1[BN * L::ROW], sv1[BN * L::ROW];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const Job job = job_of(a);
    Span sp;
    if (!find_tile(a.offsets, a.seqs, a.rows, BM, job.tile, sp)) return;
    const int first = (sp.tiles - 1 - sp.tile) * BM, q0 = first + wave * kQueries, qi = q0 + (lane & 31);
    const bool there = qi < sp.len;
    const int64_t row = sp.first + qi;
    const T* pk = (const T*)a.k + sp.first * a.ldk + (int64_t)job.kv * a.D;
    const T* pv = (const T*)a.v + sp.first * a.ldv + (int64_t)job.kv * a.D;
    const int last = a.causal ? min(sp.len, first + BM) : sp.len;              // of the workgroup's keys
    const int mine = a.causal ? min(sp.len, q0 + kQueries) : sp.len;           // of this wave's
    const int whole = a.causal ? min(sp.len, q0 + 1) : sp.len;                 // seen by all of its queries
    const int limit = a.causal ? min(sp.len, qi + 1) : sp.len;                 // seen by this lane's
    TileLoad<T, DP, BN, kWaves, DMA> lk, lv;
    lk.init(a.ldk, a.D, wave);
    lv.init(a.ldv, a.D, wave);
    lk.issue(sk0, pk, sp.len);
    lv.issue(sv0, pv, sp.len);
    Piece fq[L::STEPS];
    load_row<T, DP>(fq, (const T*)a.q + row * a.ldq + (int64_t)job.head * a.D, there, a.D);
    const float c = a.scale * kLog2e;
    floatx16 o[DP / 32] = {};
    Softmax<T> sm;
    sm.init();
    lk.store(sk0);
    lv.store(sv0);
    // the tile of keys from k0 on, in (sk, sv); the next one's loads to (tk, tv)
    auto step = [&](int k0, const char* sk, const char* sv, char* tk, char* tv) TT_INLINE {
        landed_barrier();
        const int next = k0 + BN;
        if (next < last) {
            lk.issue(tk, pk + next * a.ldk, sp.len - next);
            lv.issue(tv, pv + next * a.ldv, sp.len - next);
        }
        if (k0 < mine) {
            floatx16 s[BLOCKS] = {};
#pragma unroll
            for (int x = 0; x < L::STEPS; ++x)
#pragma unroll
                for (int b = 0; b < BLOCKS; ++b) s[b] = mma_rows<T>(L::row_piece(sk, 32 * b, x), fq[x], s[b]);
            if (next > whole) {
#pragma unroll
                for (int b = 0; b < BLOCKS; ++b)
#pragma unroll
                    for (int r = 0; r < 16; ++r)
                        if (k0 + 32 * b + block_row(r) >= limit) s[b][r] = -INFINITY;
            }
            sm.step(s, c, [&](float f) TT_INLINE {
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
        if (next < last) {
            lk.store(tk);
            lv.store(tv);
        }
    };
    for (int k0 = 0; k0 < last; k0 += 2 * BN) {
        step(k0, sk0, sv0, sk1, sv1);
        if (k0 + BN < last) step(k0 + BN, sk1, sv1, sk0, sv0);
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
template <class T, int DP, bool DMA>
__global__ __launch_bounds__(kWaves * 64, (waves_of<T, DP, DMA, DQ>())) void k_attend_dq(const AttendArgs a) {
    typedef Tile<T, DP> L;
    constexpr int BN = tile_rows<T, DP>(), BLOCKS = BN / 32, BM = kWaves * kQueries;
    __shared__ __align__(16) char sk0[BN * L::ROW], sv0[BN * L::ROW], sk1[BN * L::ROW], sv1[BN * L::ROW];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const Job job = job_of(a);
    Span sp;
    if (!find_tile(a.offsets, a.seqs, a.rows, BM, job.tile, sp)) return;
    const int first = (sp.tiles - 1 - sp.tile) * BM, q0 = first + wave * kQueries, qi = q0 + (lane & 31);
    const bool there = qi < sp.len;
    const int64_t row = sp.first + qi, at = (int64_t)job.head * a.D;
    const T* pk = (const T*)a.k + sp.first * a.ldk + (int64_t)job.kv * a.D;
    const T* pv = (const T*)a.v + sp.first * a.ldv + (int64_t)job.kv * a.D;
    const int last = a.causal ? min(sp.len, first + BM) : sp.len;
    const int mine = a.causal ? min(sp.len, q0 + kQueries) : sp.len;
    const int whole = a.causal ? min(sp.len, q0 + 1) : sp.len;
    const int limit = a.causal ? min(sp.len, qi + 1) : sp.len;
    TileLoad<T, DP, BN, kWaves, DMA> lk, lv;
    lk.init(a.ldk, a.D, wave);
    lv.init(a.ldv, a.D, wave);
    lk.issue(sk0, pk, sp.len);
    lv.issue(sv0, pv, sp.len);
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
    const float c = a.scale * kLog2e;
    floatx16 dq[DP / 32] = {};
    lk.store(sk0);
    lv.store(sv0);
    auto step = [&](int k0, const char* sk, const char* sv, char* tk, char* tv) TT_INLINE {
        landed_barrier();
        const int next = k0 + BN;
        if (next < last) {
            lk.issue(tk, pk + next * a.ldk, sp.len - next);
            lv.issue(tv, pv + next * a.ldv, sp.len - next);
        }
        if (k0 < mine) {
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
        if (next < last) {
            lk.store(tk);
            lv.store(tv);
        }
    };
    for (int k0 = 0; k0 < last; k0 += 2 * BN) {
        step(k0, sk0, sv0, sk1, sv1);
        if (k0 + BN < last) step(k0 + BN, sk1, sv1, sk0, sv0);
    }
    if (there) store_columns<T, DP>((T*)a.dq + row * a.lddq + at, dq, a.scale, a.D);
}

// dk and dv: a wave keeps 32 keys and goes over the queries of every head that reads them.
//
// GROUPS = 2: two waves a SIMD, where the registers for keys, values and both sums are too
// many for two (heads of more than 64): the second four waves have the first's keys and take
// the other half of each tile of queries, keys and values are read from LDS, and the halves' sums
// meet at the end.
//
// The (head, tile of queries) pairs of a tile of keys are split over a.splits workgroups where
// there are too few of these to fill the chip; sums then go to the workspace and are joined by
// k_attend_join.
template <class T, int DP, bool DMA, int GROUPS>
__global__ __launch_bounds__(GROUPS * kWaves * 64, (waves_of<T, DP, DMA, DKV>())) void k_attend_dkv(const AttendArgs a) {
    typedef Tile<T, DP> L;
    constexpr int BM = tile_rows<T, DP>(), BLOCKS = BM / 32, BN = kWaves * kQueries, WAVES = GROUPS * kWaves;
    static_assert(BLOCKS % GROUPS == 0, "a group takes whole blocks");
    __shared__ __align__(16) char sq0[BM * L::ROW], sd0[BM * L::ROW], sq1[BM * L::ROW], sd1[BM * L::ROW];
    __shared__ __align__(16) float st0[2 * BM], st1[2 * BM];   // a tile's lse (in powers of two), then its delta
    __shared__ __align__(16) char sk[GROUPS == 2 ? BN * L::ROW : 16], sv[GROUPS == 2 ? BN * L::ROW : 16];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int group = wave / kWaves, mine = wave % kWaves;   // of keys
    int job = blockIdx.x;
    const int kv = job % a.kv, heads = a.heads / a.kv;
    job /= a.kv;
    const int split = job % a.splits;
    Span sp;
    if (!find_tile(a.offsets, a.seqs, a.rows, BN, job / a.splits, sp)) return;
    const int first = sp.tile * BN, k0 = first + mine * kQueries, ki = k0 + (lane & 31);
    const bool there = ki < sp.len;
    const int64_t row = sp.first + ki, at = (int64_t)kv * a.D;
    const int begin = a.causal ? first / BM : 0, per = (sp.len + BM - 1) / BM - begin;   // tiles of queries a head
    const int all = per * heads, each = (all + a.splits - 1) / a.splits;
    const int i0 = min(all, split * each), i1 = min(all, i0 + each);
    TileLoad<T, DP, BM, WAVES, DMA> lq, ld;
    lq.init(a.ldq, a.D, wave);
    ld.init(a.lddo, a.D, wave);
    float stat = 0.f;   // of query threadIdx.x % BM of the tile
    auto issue = [&](int i, char* tq, char* td) TT_INLINE {
        const int head = kv * heads + i / per, q0 = (begin + i % per) * BM, left = sp.len - q0;
        const int64_t r = sp.first + q0;
        lq.issue(tq, (const T*)a.q + r * a.ldq + (int64_t)head * a.D, left);
        ld.issue(td, (const T*)a.dout + r * a.lddo + (int64_t)head * a.D, left);
        const int x = threadIdx.x % BM;
        const bool is_delta = threadIdx.x >= BM;
        stat = is_delta ? 0.f : INFINITY;
        if (threadIdx.x < 2 * BM && x < left) {
            const float f = (is_delta ? a.delta : a.lse)[(int64_t)head * a.rows + r + x];
            stat = is_delta ? f : log2_sum(f);
        }
    };
    auto store = [&](char* tq, char* td, float* ts) TT_INLINE {
        lq.store(tq);
        ld.store(td);
        if (threadIdx.x < 2 * BM) ts[threadIdx.x] = stat;
    };
    Piece fk[L::STEPS], fv[L::STEPS];
    if constexpr (GROUPS == 2) {
        TileLoad<T, DP, BN, WAVES, DMA> lk, lv;
        lk.init(a.ldk, a.D, wave);
        lv.init(a.ldv, a.D, wave);
        lk.issue(sk, (const T*)a.k + (sp.first + first) * a.ldk + at, sp.len - first);
        lv.issue(sv, (const T*)a.v + (sp.first + first) * a.ldv + at, sp.len - first);
        lk.store(sk);
        lv.store(sv);
    } else {
        load_row<T, DP>(fk, (const T*)a.k + row * a.ldk + at, there, a.D);
        load_row<T, DP>(fv, (const T*)a.v + row * a.ldv + at, there, a.D);
    }
    if (i0 < i1) issue(i0, sq0, sd0);
    const float c = a.scale * kLog2e;
    floatx16 dk[DP / 32] = {}, dv[DP / 32] = {};
    store(sq0, sd0, st0);
    auto step = [&](int i, const char* sq, const char* sd, const float* st, char* tq, char* td, float* ts) TT_INLINE {
        landed_barrier();
        if (i + 1 < i1) issue(i + 1, tq, td);
        const int q0 = (begin + i % per) * BM;
#pragma unroll
        for (int n = 0; n < BLOCKS / GROUPS; ++n) {
            const int b = GROUPS * n + group, first_q = q0 + 32 * b;
            if (first_q >= sp.len || (a.causal && first_q + 31 < k0)) continue;
            floatx16 s = {}, dp = {};
#pragma unroll
            for (int x = 0; x < L::STEPS; ++x) {
                if constexpr (GROUPS == 2) {
                    fk[x] = L::row_piece(sk, mine * kQueries, x);
                    fv[x] = L::row_piece(sv, mine * kQueries, x);
                }
                s = mma_rows<T>(L::row_piece(sq, 32 * b, x), fk[x], s);
                dp = mma_rows<T>(L::row_piece(sd, 32 * b, x), fv[x], dp);
            }
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                float lg[4], dg[4];
                const int q = 32 * b + block_row(4 * g);
                __builtin_memcpy(lg, st + q, 16);
                __builtin_memcpy(dg, st + BM + q, 16);
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
        if (i + 1 < i1) store(tq, td, ts);
    };
    for (int i = i0; i < i1; i += 2) {
        step(i, sq0, sd0, st0, sq1, sd1, st1);
        if (i + 1 < i1) step(i + 1, sq1, sd1, st1, sq0, sd0, st0);
    }
    if constexpr (GROUPS == 2) {
        // the first group takes the second's dk, the second the first's dv
        static_assert(BM * L::ROW >= kWaves * 64 * 64, "room for 32 columns of the sums");
        char* to = (group ? sq0 : sd0) + mine * 4096 + lane * 16;
        const char* from = (group ? sd0 : sq0) + mine * 4096 + lane * 16;
#pragma unroll
        for (int j = 0; j < DP / 32; ++j) {
            __syncthreads();
#pragma unroll
            for (int g = 0; g < 4; ++g)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    reinterpret_cast<float*>(to + g * 1024)[e] = group ? dk[j][4 * g + e] : dv[j][4 * g + e];
            __syncthreads();
#pragma unroll
            for (int g = 0; g < 4; ++g)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float f = reinterpret_cast<const float*>(from + g * 1024)[e];
                    if (group) dv[j][4 * g + e] += f;
                    else dk[j][4 * g + e] += f;
                }
        }
    }
    if (!there) return;
    const bool has_dk = GROUPS == 1 || group == 0, has_dv = GROUPS == 1 || group == 1;
    if (a.splits > 1) {
        float* p = a.part + ((int64_t)split * a.rows + row) * a.kv * a.D + at;
        if (has_dk) store_columns<float, DP>(p, dk, 1.f, a.D);
        if (has_dv) store_columns<float, DP>(p + (int64_t)a.splits * a.rows * a.kv * a.D, dv, 1.f, a.D);
    } else {
        if (has_dk) store_columns<T, DP>((T*)a.dk + row * a.lddk + at, dk, a.scale, a.D);
        if (has_dv) store_columns<T, DP>((T*)a.dv + row * a.lddv + at, dv, 1.f, a.D);
    }
}

// dk (blockIdx.y = 0) and dv from the splits' sums, in their order.
template <class T>
__global__ __launch_bounds__(256) void k_attend_join(const AttendArgs a) {
    const int N = a.kv * a.D, per = (N + 7) / 8;
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x, row = i / per;
    const int n = (int)(i - row * per) * 8, left = N - n;
    if (row >= a.rows || row < a.offsets[0] || row >= a.offsets[a.seqs]) return;   // rows of no sequence stay
    const bool second = blockIdx.y == 1;
    const float* p = a.part + ((int64_t)second * a.splits * a.rows + row) * N + n;
    float o[8] = {};
#pragma unroll 4
    for (int s = 0; s < a.splits; ++s) {
        const Raw8<float> f = load8n(p + (int64_t)s * a.rows * N, left, 0.f);
#pragma unroll
        for (int e = 0; e < 8; ++e) o[e] += f.at(e);
    }
    if (!second)
#pragma unroll
        for (int e = 0; e < 8; ++e) o[e] *= a.scale;
    store8n((T*)(second ? a.dv : a.dk) + row * (second ? a.lddv : a.lddk) + n, o, left);
}

// Splits of dk's and dv's sums: as many as bring the workgroups to kMinGroups.
constexpr int64_t kMinGroups = 512, kMaxSplits = 16;
inline int64_t splits_of(int64_t rows, int64_t seqs, int64_t kv) {
    const int64_t n = std::max<int64_t>(1, ((rows + kWaves * kQueries - 1) / (kWaves * kQueries) + seqs / 2) * kv);
    return std::max<int64_t>(1, std::min(kMaxSplits, kMinGroups / n));
}

// Whether rows start at whole 16-byte pieces, and their heads are made of them.
bool pieces(const void* p, int64_t ld, int D, size_t size) {
    return ((uintptr_t)p & 15) == 0 && ld * size % 16 == 0 && D * size % 16 == 0;
}

template <class T, int DP>
tt_status attend_launch(const AttendArgs& a, bool backward) {
    const bool keys = pieces(a.k, a.ldk, a.D, sizeof(T)) && pieces(a.v, a.ldv, a.D, sizeof(T));
    const int64_t tiles = a.rows / (kWaves * kQueries) + a.seqs;
    const dim3 grid((unsigned)(tiles * a.heads)), block(kWaves * 64);
    if (!backward) {
        TT_LAUNCH(nullptr, "k_attend", a.s, (keys ? k_attend<T, DP, true> : k_attend<T, DP, false>), grid, block, 0, a.s, a);
        TT_LAUNCH_CHECK();
        return TT_OK;
    }
    const bool queries = pieces(a.q, a.ldq, a.D, sizeof(T)) && pieces(a.dout, a.lddo, a.D, sizeof(T)) &&
                         (DP <= 64 || keys);
    auto dq = keys ? k_attend_dq<T, DP, true> : k_attend_dq<T, DP, false>;
    TT_LAUNCH(nullptr, "k_attend_dq", a.s, dq, grid, block, 0, a.s, a);
    TT_LAUNCH_CHECK();
    const dim3 keys_grid((unsigned)(tiles * a.splits * a.kv));
    if constexpr (sizeof(T) == 2 && DP > 64) {
        auto dkv = queries ? k_attend_dkv<T, DP, true, 2> : k_attend_dkv<T, DP, false, 2>;
        TT_LAUNCH(nullptr, "k_attend_dkv", a.s, dkv, keys_grid, dim3(2 * kWaves * 64), 0, a.s, a);
    } else {
        auto dkv = queries ? k_attend_dkv<T, DP, true, 1> : k_attend_dkv<T, DP, false, 1>;
        TT_LAUNCH(nullptr, "k_attend_dkv", a.s, dkv, keys_grid, block, 0, a.s, a);
    }
    TT_LAUNCH_CHECK();
    if (a.splits > 1) {
        const dim3 join(grid_for(a.rows * (((int64_t)a.kv * a.D + 7) / 8), 256), 2);
        TT_LAUNCH(nullptr, "k_attend_join", a.s, (k_attend_join<T>), join, dim3(256), 0, a.s, a);
        TT_LAUNCH_CHECK();
    }
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

inline size_t delta_bytes(int64_t rows, int64_t heads) {
    return ((size_t)rows * heads * sizeof(float) + 255) & ~size_t(255);
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
    // delta; the splits' sums, of which fewer rows have at most kMinGroups workgroups'
    const int64_t most = kMinGroups * kWaves * kQueries;
    const int64_t sums = std::min(rows * kv_heads * kMaxSplits, most) * 2 * dim;
    return delta_bytes(rows, heads) + std::max<size_t>(256, ((size_t)sums * sizeof(float) + 255) & ~size_t(255));
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
    a.part = (float*)((char*)workspace + delta_bytes(rows, heads));
    a.splits = (int)splits_of(rows, seqs, kv_heads);
    return attend_by_type(dtype, a, true);
}
