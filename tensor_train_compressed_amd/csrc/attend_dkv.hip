// The backward of attention over packed prompts, by keys: dk and dv (formulas and layout:
// attend.hip).
#include "attend.h"

namespace tt {
namespace {

// dk and dv: a wave keeps 32 keys and goes over the queries of every head that reads them.
//
// KEYS: waves of a tile of keys. GROUPS = 2: two waves a SIMD, where the registers for keys, values and both sums are too
// many for two (heads of more than 64): the second four waves have the first's keys and take
// the other half of each tile of queries, keys and values are read from LDS, and the halves' sums
// meet at the end. One prompt of 8192 rows, 32 and 8 heads of 128 bf16: 1135 us; one wave a SIMD with keys and
// values in registers 1500, and 1300 to 1400 with one block's weights formed beside the other's
// products. Without the loads of tiles 1000 to 1075.
//
// The (head, tile of queries) pairs of a tile of keys are split over a.splits workgroups where
// there are too few of these to fill the chip; sums then go to the workspace and are joined by
// k_attend_join.
template <class T, int DP, bool DMA, int GROUPS, int KEYS>
__global__ __launch_bounds__(GROUPS * KEYS * 64, (waves_of<T, DP, DMA, DKV>())) void k_attend_dkv(const AttendArgs a) {
    typedef Tile<T, DP> L;
    constexpr int BM = tile_rows<T, DP, KEYS>(), BLOCKS = BM / 32, BN = KEYS * kQueries, WAVES = GROUPS * KEYS;
    static_assert(BLOCKS % GROUPS == 0, "a group takes whole blocks");
    constexpr int STAT = 3 * BM + 4, ROLES = WAVES * 64 >= 3 * BM ? 3 : 2;
    __shared__ __align__(16) char sq0[BM * L::ROW], sd0[BM * L::ROW], sq1[BM * L::ROW], sd1[BM * L::ROW];
    __shared__ __align__(16) float st0[STAT], st1[STAT];   // a tile's delta, base and ref, and whether any ref is not 0
    __shared__ __align__(16) char sk[GROUPS == 2 ? BN * L::ROW : 16], sv[GROUPS == 2 ? BN * L::ROW : 16];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int group = wave / KEYS, mine = wave % KEYS;   // of keys
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
    const int all = per * heads, share = (all + a.splits - 1) / a.splits;
    const int i0 = min(all, split * share), i1 = min(all, i0 + share);
    TileLoad<T, DP, BM, WAVES, DMA> lq, ld;
    lq.init(a.ldq, a.D, wave);
    ld.init(a.lddo, a.D, wave);
    // delta, base or ref, by threadIdx.x / BM, of query threadIdx.x % BM of the tile; where there are too few threads for
    // three, ref apart
    float stat = 0.f, ref = 0.f;
    auto issue = [&](int i, char* tq, char* td) TT_INLINE {
        const int head = kv * heads + i / per, q0 = (begin + i % per) * BM, left = sp.len - q0;
        const int64_t r = sp.first + q0;
        lq.issue(tq, (const T*)a.q + r * a.ldq + (int64_t)head * a.D, left);
        ld.issue(td, (const T*)a.dout + r * a.lddo + (int64_t)head * a.D, left);
        // (tiles of 64 rows: a wave has one role)
        const int x = BM == 64 ? lane : threadIdx.x % BM, role = BM == 64 ? wave : threadIdx.x / BM;
        stat = role == 1 ? INFINITY : 0.f;
        if (ROLES == 2) ref = 0.f;
        if (role < ROLES && x < left) {
            const float* p = a.stats + (int64_t)head * a.rows + r;
            stat = (p + role * a.apart)[x] - (role == 1 ? weight_bits<T>() : 0.f);
            if (ROLES == 2) ref = p[2 * a.apart + x];
        }
    };
    auto store = [&](char* tq, char* td, float* ts) TT_INLINE {
        lq.store(tq);
        ld.store(td);
        if (BM == 64 ? wave < ROLES : threadIdx.x < ROLES * BM) ts[threadIdx.x] = stat;
        if (ROLES == 2 && threadIdx.x < BM) ts[2 * BM + threadIdx.x] = ref;
        static_assert(ROLES == 3 ? BM % 64 == 0 || BM == 32 : WAVES == 1, "one wave holds a tile's refs");
        const int holder = ROLES == 3 ? 2 * BM / 64 : 0;
        if (wave == holder) {
            const bool any = __ballot(ROLES == 3 ? stat != 0.f && (BM == 64 || threadIdx.x / BM == 2) : ref != 0.f) != 0;
            if (lane == 0) reinterpret_cast<int*>(ts)[3 * BM] = any;
        }
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
    // the first group's products go before the second's, whose weights are formed meanwhile
    if (GROUPS == 2 && group == 0) __builtin_amdgcn_s_setprio(1);
    const float c = a.scale * kLog2e;
    floatx16 dk[DP / 32] = {}, dv[DP / 32] = {};
    Range<T> range;   // of the keys
    range.init();
    store(sq0, sd0, st0);
    auto step = [&](int i, const char* sq, const char* sd, const float* st, char* tq, char* td, float* ts) TT_INLINE {
        landed_barrier();
        if (i + 1 < i1) issue(i + 1, tq, td);
        const int q0 = (begin + i % per) * BM;
        const bool far = __builtin_amdgcn_readfirstlane(reinterpret_cast<const int*>(st)[3 * BM]) != 0;
        auto weights = [&](int b, floatx16& s, floatx16& dp) TT_INLINE {
            if (far) {
#pragma unroll
                for (int g = 0; g < 4; ++g) {
                    float m[4];
                    __builtin_memcpy(m, st + 2 * BM + 32 * b + block_row(4 * g), 16);
#pragma unroll
                    for (int e = 0; e < 4; ++e) s[4 * g + e] -= m[e];
                }
            }
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                float lg[4], dg[4];
                const int q = 32 * b + block_row(4 * g);
                __builtin_memcpy(dg, st + q, 16);
                __builtin_memcpy(lg, st + BM + q, 16);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int r = 4 * g + e;
                    s[r] = exp2_hw(fmaf(s[r], c, -lg[e]));
                    dp[r] = s[r] * (dp[r] - dg[e]);
                }
            }
        };
        if constexpr (sizeof(T) == 2) {
#pragma unroll
            for (int n = 0; n < BLOCKS / GROUPS; ++n) {
                const int b = GROUPS * n + group, first_q = q0 + 32 * b;
                if (first_q >= sp.len || (a.causal && first_q + 31 < k0)) continue;
                // slot by slot: 2 STEPS products of scores, 4 DP / 32 of sums
                constexpr int N = 2 * L::STEPS, A = GROUPS == 2 ? 2 : AHEAD;
                floatx16 s = {}, dp = {};
                Weights<T> ws, wd;
                Piece f[A], g[A];
                auto fetch = [&](auto slot) TT_INLINE {
                    constexpr int u = slot, t = u - N;
                    if constexpr (u < N) {
                        f[u % A] = L::row_piece(u % 2 ? sd : sq, 32 * b, u / 2);
                        if constexpr (GROUPS == 2) g[u % A] = L::row_piece(u % 2 ? sv : sk, mine * kQueries, u / 2);
                    } else if constexpr (u < N + 4 * (DP / 32)) {
                        f[u % A] = L::column_piece(t % 2 ? sq : sd, 32 * b + 16 * (t / 2 / (DP / 32)), t / 2 % (DP / 32));
                    }
                };
                each<A>(fetch);
                each<N>([&](auto slot) TT_INLINE {
                    constexpr int u = slot;
                    __builtin_amdgcn_sched_barrier(0);
                    const Piece x = f[u % A];
                    Piece y;
                    if constexpr (GROUPS == 2) y = g[u % A];
                    else y = u % 2 ? fv[u / 2] : fk[u / 2];
                    if constexpr (u % 2) dp = mma16<T>(x, y, dp);
                    else s = mma16<T>(x, y, s);
                    fetch(std::integral_constant<int, u + A>{});
                });
                __builtin_amdgcn_sched_barrier(0);
                weights(b, s, dp);
                if (first_q + 32 > sp.len || (a.causal && first_q < k0 + 31)) {
#pragma unroll
                    for (int r = 0; r < 16; ++r) {
                        const int q = first_q + block_row(r);
                        if (q >= sp.len || (a.causal && q < ki)) s[r] = dp[r] = 0.f;
                    }
                }
                ws.set(s);
                if constexpr (Range<T>::kOn) {
                    const float f = exp2_hw(range.up);
#pragma unroll
                    for (int r = 0; r < 16; ++r) dp[r] *= f;
                }
                range.step(dp, [&](float f) TT_INLINE {
#pragma unroll
                    for (int j = 0; j < DP / 32; ++j) dk[j] *= f;
                });
                wd.set(dp);
                each<4 * (DP / 32)>([&](auto slot) TT_INLINE {
                    constexpr int t = slot, j = t / 2 % (DP / 32), h = t / 2 / (DP / 32);
                    __builtin_amdgcn_sched_barrier(0);
                    const Piece x = f[(t + N) % A];
                    if constexpr (t % 2) dk[j] = mma16<T>(x, wd.w[h], dk[j]);
                    else dv[j] = mma16<T>(x, ws.w[h], dv[j]);
                    fetch(std::integral_constant<int, t + N + A>{});
                });
                __builtin_amdgcn_sched_barrier(0);
            }
        } else {
#pragma unroll
            for (int n = 0; n < BLOCKS / GROUPS; ++n) {
                const int b = GROUPS * n + group, first_q = q0 + 32 * b;
                if (first_q >= sp.len || (a.causal && first_q + 31 < k0)) continue;
                floatx16 s = {}, dp = {};
#pragma unroll
                for (int x = 0; x < L::STEPS; ++x) {
                    s = mma_rows<T>(L::row_piece(sq, 32 * b, x), fk[x], s);
                    dp = mma_rows<T>(L::row_piece(sd, 32 * b, x), fv[x], dp);
                }
                weights(b, s, dp);
                if (first_q + 32 > sp.len || (a.causal && first_q < k0 + 31)) {
#pragma unroll
                    for (int r = 0; r < 16; ++r) {
                        const int q = first_q + block_row(r);
                        if (q >= sp.len || (a.causal && q < ki)) s[r] = dp[r] = 0.f;
                    }
                }
                Weights<T> ws, wd;
                ws.set(s);
                wd.set(dp);
#pragma unroll
                for (int j = 0; j < DP / 32; ++j) {
                    dv[j] = mma_columns<T, DP>(sd, 32 * b, j, ws, dv[j]);
                    dk[j] = mma_columns<T, DP>(sq, 32 * b, j, wd, dk[j]);
                }
            }
        }
        if (i + 1 < i1) store(tq, td, ts);
    };
    for (int i = i0; i < i1; i += 2) {
        step(i, sq0, sd0, st0, sq1, sd1, st1);
        if (i + 1 < i1) step(i + 1, sq1, sd1, st1, sq0, sd0, st0);
    }
    if constexpr (Range<T>::kOn) {
        const float wb = exp2f(-weight_bits<T>());
#pragma unroll
        for (int j = 0; j < DP / 32; ++j) {
            dk[j] = dk[j] * range.back() * wb;
            dv[j] *= wb;
        }
    }
    if constexpr (GROUPS == 2) {
        landed_barrier();   // (keys and values of a split without queries may be under way)
        // the first group takes the second's dk, the second the first's dv
        static_assert(BM * L::ROW >= KEYS * 64 * 64, "room for 32 columns of the sums");
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

template <class T, int DP>
tt_status dkv_launch(const AttendArgs& a) {
    const bool whole = queries_in_pieces<T>(a) && keys_in_pieces<T>(a), few = whole && short_sequences(a);
    constexpr int GROUPS = sizeof(T) == 2 && DP > 64 ? 2 : 1;
    const dim3 grid((unsigned)(tiles_of(a, (few ? 1 : kWaves) * kQueries) * a.splits * a.kv));
    auto k = few     ? k_attend_dkv<T, DP, true, 1, 1>
             : whole ? k_attend_dkv<T, DP, true, GROUPS, kWaves>
                     : k_attend_dkv<T, DP, false, GROUPS, kWaves>;
    TT_LAUNCH(nullptr, "k_attend_dkv", a.s, k, grid, dim3(few ? 64 : GROUPS * kWaves * 64), 0, a.s, a);
    TT_LAUNCH_CHECK();
    if (a.splits == 1) return TT_OK;
    const dim3 join(grid_for(a.rows * (((int64_t)a.kv * a.D + 7) / 8), 256), 2);
    TT_LAUNCH(nullptr, "k_attend_join", a.s, (k_attend_join<T>), join, dim3(256), 0, a.s, a);
    TT_LAUNCH_CHECK();
    return TT_OK;
}

}  // namespace

tt_status attend_dkv(int32_t dtype, const AttendArgs& a) {
    return by_type(dtype, a, [&](auto* t, auto dim) { return dkv_launch<std::remove_pointer_t<decltype(t)>, dim>(a); });
}

}  // namespace tt
