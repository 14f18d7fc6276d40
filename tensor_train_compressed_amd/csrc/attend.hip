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
// What bounds it, and what it measures: one prompt of 8192 rows, 32 and 8 heads of 128 bf16, causal,
// 555 us, 990 TFLOP/s of what is not masked. Without the loads of tiles 480, without the softmax
// 480, without both 405 (1360 TFLOP/s), all at 1.9 GHz of 2.4: matrix and vector instructions of
// a SIMD's two waves overlap in part, and power holds the clock. The matrix cores are busy 55% of the time, LDS 27%,
// with no bank conflict. Measured the same or slower: a block of keys ahead, its scores formed beside the weights
// of the one before, instruction by instruction (560 to 600); two blocks of queries a wave (its accumulators
// spill); priorities of waves (570).
//
// The backward forms scores twice, once by queries (dq) and once by keys (dk and dv): seven
// products instead of five, but each result is summed by one wave in a fixed order, without
// atomics. Of the same prompt dq takes 740 us (1110 TFLOP/s; matrix cores busy 65%, LDS 33%), dk and dv 1135
// (970; 50%, 44%).
//
// Workgroups: heads that share keys are launched together and, where 8 divides the key
// heads, on one XCD, whose L2 then holds their keys; of a sequence the tiles with the most
// work come first.
#include "attend.h"

namespace tt {
namespace {

template <class T, int DP, bool DMA, int WAVES>
__global__ __launch_bounds__(WAVES * 64, (waves_of<T, DP, DMA, FWD>())) void k_attend(const AttendArgs a) {
    typedef Tile<T, DP> L;
    constexpr int BN = tile_rows<T, DP, WAVES>(), BLOCKS = BN / 32, BM = WAVES * kQueries;
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
    TileLoad<T, DP, BN, WAVES, DMA> lk, lv;
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
            auto hide = [&]() TT_INLINE {
                if (next > whole) {
#pragma unroll
                    for (int b = 0; b < BLOCKS; ++b)
#pragma unroll
                        for (int r = 0; r < 16; ++r)
                            if (k0 + 32 * b + block_row(r) >= limit) s[b][r] = -INFINITY;
                }
            };
            auto rescale = [&](float f) TT_INLINE {
#pragma unroll
                for (int j = 0; j < DP / 32; ++j) o[j] *= f;
            };
            if constexpr (sizeof(T) == 2 && BLOCKS == 2) {
                // slot by slot: products of scores, the blocks in turn, then of outputs
                constexpr int N = 2 * L::STEPS, J = DP / 32, A = DP == 128 ? 3 : AHEAD;   // (four would spill)
                Piece f[A];
                auto fetch = [&](auto slot) TT_INLINE {
                    constexpr int u = slot, t = u - N;
                    if constexpr (u < N) f[u % A] = L::row_piece(sk, 32 * (u % 2), u / 2);
                    else if constexpr (t < 4 * J) f[u % A] = L::column_piece(sv, 16 * (t / J), t % J);
                };
                each<A>(fetch);
                each<N>([&](auto slot) TT_INLINE {
                    constexpr int u = slot;
                    __builtin_amdgcn_sched_barrier(0);
                    s[u % 2] = mma16<T>(f[u % A], fq[u / 2], s[u % 2]);
                    fetch(std::integral_constant<int, u + A>{});
                });
                __builtin_amdgcn_sched_barrier(0);
                hide();
                sm.step(s, c, rescale);
                Weights<T> w[2];
                w[0].set(s[0]);
                w[1].set(s[1]);
                each<4 * J>([&](auto slot) TT_INLINE {
                    constexpr int t = slot, j = t % J, h = t / J;
                    __builtin_amdgcn_sched_barrier(0);
                    o[j] = mma16<T>(f[(t + N) % A], w[h / 2].w[h % 2], o[j]);
                    fetch(std::integral_constant<int, t + N + A>{});
                });
                __builtin_amdgcn_sched_barrier(0);
            } else {
#pragma unroll
                for (int x = 0; x < L::STEPS; ++x)
#pragma unroll
                    for (int b = 0; b < BLOCKS; ++b) s[b] = mma_rows<T>(L::row_piece(sk, 32 * b, x), fq[x], s[b]);
                hide();
                sm.step(s, c, rescale);
#pragma unroll
                for (int b = 0; b < BLOCKS; ++b) {
                    Weights<T> w;
                    w.set(s[b]);
#pragma unroll
                    for (int j = 0; j < DP / 32; ++j) o[j] = mma_columns<T, DP>(sv, 32 * b, j, w, o[j]);
                }
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

template <class T, int DP>
tt_status attend_launch(const AttendArgs& a) {
    const bool whole = keys_in_pieces<T>(a), few = whole && short_sequences(a);
    const int waves = few ? 1 : kWaves;
    const dim3 grid((unsigned)(tiles_of(a, waves * kQueries) * a.heads));
    auto k = few ? k_attend<T, DP, true, 1> : whole ? k_attend<T, DP, true, kWaves> : k_attend<T, DP, false, kWaves>;
    TT_LAUNCH(nullptr, "k_attend", a.s, k, grid, dim3(waves * 64), 0, a.s, a);
    TT_LAUNCH_CHECK();
    return TT_OK;
}

constexpr int64_t kMaxLd = (int64_t(1) << 22) - 1;

tt_status attend_sizes(int32_t dtype, int64_t rows, int64_t heads, int64_t kv, int64_t dim) {
    if (!dtype_ok(dtype) || rows < 0 || heads < 1 || kv < 1 || dim < 1 || heads % kv != 0) return TT_ERR_INVALID_ARG;
    if (dim > 128 || rows > INT32_MAX || heads > (int64_t(1) << 22)) return TT_ERR_UNSUPPORTED;
    return TT_OK;
}

// Of one number a row and head: delta, base, ref.
inline size_t stat_bytes(int64_t rows, int64_t heads) {
    return ((size_t)rows * heads * sizeof(float) + 255) & ~size_t(255);
}

// The arguments that every call takes.
tt_status attend_args(AttendArgs& a, int32_t dtype, const void* q, int64_t ldq, const void* k, int64_t ldk,
                      const void* v, int64_t ldv, const int64_t* offsets, int64_t seqs, int64_t rows, int64_t heads,
                      int64_t kv, int64_t dim, int32_t causal, float scale, void* stream) {
    const tt_status st = attend_sizes(dtype, rows, heads, kv, dim);
    if (st != TT_OK) return st;
    if (seqs < 0 || !scale_ok(scale)) return TT_ERR_INVALID_ARG;
    if (ldq < heads * dim || ldk < kv * dim || ldv < kv * dim) return TT_ERR_INVALID_ARG;
    if (rows > 0 && seqs > 0 && (!q || !k || !v || !offsets)) return TT_ERR_INVALID_ARG;
    if (ldq > kMaxLd || ldk > kMaxLd || ldv > kMaxLd || seqs > INT32_MAX) return TT_ERR_UNSUPPORTED;
    // (a launch's threads, 512 a workgroup at most, must stay below 2^32)
    if ((rows / kQueries + seqs) * heads > int64_t(1) << 22) return TT_ERR_UNSUPPORTED;
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
    // delta, base and ref; the splits' sums, at most kGroups workgroups' at these and at fewer rows
    const int64_t most = kGroups * kWaves * kQueries;
    const int64_t sums = std::min(rows * kv_heads * kMaxSplits, most) * 2 * dim;
    return 3 * stat_bytes(rows, heads) + std::max<size_t>(256, ((size_t)sums * sizeof(float) + 255) & ~size_t(255));
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
    if (rows == 0 || seqs == 0) return TT_OK;
    return by_type(dtype, a, [&](auto* t, auto dim) { return attend_launch<std::remove_pointer_t<decltype(t)>, dim>(a); });
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
    a.stats = (float*)workspace;
    a.apart = (uint32_t)(stat_bytes(rows, heads) / sizeof(float));   // (below 2^28: rows * heads are below 2^27)
    a.part = (float*)((char*)workspace + 3 * stat_bytes(rows, heads));
    a.splits = (int)splits_of(rows, seqs, kv_heads);
    if (rows == 0 || seqs == 0) return TT_OK;
    const tt_status dq_st = attend_dq(dtype, a);
    return dq_st != TT_OK ? dq_st : attend_dkv(dtype, a);
}
