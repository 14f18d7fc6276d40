// The backward of attention over packed prompts, by queries: dq, and what the pass by keys
// takes of a row, delta and what its weights are relative to (formulas and layout: attend.hip).
#include "attend.h"

namespace tt {
namespace {

// delta is dout . out, with out as it was rounded to T, or the same as sum p (dout . v), which
// rounds nothing. The first is off by what the roundings of out add up to, common to all of a row's ds;
// rows of few keys, whose out and ds are largest, would make that the largest error of dq and
// dk (2-norm errors 0.0026 instead of 0.0017 for rounding the results alone). Tiles of up to this many keys
// are gone over once more for the second.
constexpr int kExact = 256;

// What a sweep over the keys forms: maximum and sum of a row's weights, delta, dq.
enum Sweep { STATS, DELTA, GRADIENT };

template <class T, int DP, bool DMA, int WAVES>
__global__ __launch_bounds__(WAVES * 64, (waves_of<T, DP, DMA, DQ>())) void k_attend_dq(const AttendArgs a) {
    typedef Tile<T, DP> L;
    constexpr int BN = tile_rows<T, DP, WAVES>(), BLOCKS = BN / 32, BM = WAVES * kQueries;
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
    TileLoad<T, DP, BN, WAVES, DMA> lk, lv;
    lk.init(a.ldk, a.D, wave);
    lv.init(a.ldv, a.D, wave);
    auto issue_first = [&]() TT_INLINE {
        lk.issue(sk0, pk, sp.len);
        lv.issue(sv0, pv, sp.len);
    };
    auto store_first = [&]() TT_INLINE {
        lk.store(sk0);
        lv.store(sv0);
    };
    issue_first();
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
    // weights are 2^(c (s - ref) - base); ref is 0 where lse is taken as it is
    float lse = 0.f, base = INFINITY, ref = 0.f;
    if (there) {
        lse = a.lse[(int64_t)job.head * a.rows + row];
        base = log2_sum(lse);
    }
    const float c = a.scale * kLog2e;
    floatx16 dq[DP / 32] = {};
    float sum = 0.f;   // of p (dout . v)
    bool far = false;  // any of the wave's rows has a ref
    Softmax<T> sm;
    Range<T> range;
    range.init();
    store_first();
    auto step = [&](auto sweep, int k0, const char* sk, const char* sv, char* tk, char* tv) TT_INLINE {
        constexpr Sweep SWEEP = sweep;
        landed_barrier();
        const int next = k0 + BN;
        if (next < last) {
            lk.issue(tk, pk + next * a.ldk, sp.len - next);
            if constexpr (SWEEP != STATS) lv.issue(tv, pv + next * a.ldv, sp.len - next);
        }
        if (k0 < mine) {
#pragma unroll
            for (int b = 0; b < BLOCKS; ++b) {
                if constexpr (SWEEP == STATS) {
                    floatx16 s[1] = {};
#pragma unroll
                    for (int x = 0; x < L::STEPS; ++x) s[0] = mma_rows<T>(L::row_piece(sk, 32 * b, x), fq[x], s[0]);
#pragma unroll
                    for (int r = 0; r < 16; ++r)
                        if (k0 + 32 * b + block_row(r) >= limit) s[0][r] = -INFINITY;
                    sm.step(s, c, [](float) {});
                    continue;
                }
                floatx16 s = {}, dp = {};
                auto weights = [&]() TT_INLINE {
                    if (far) {
#pragma unroll
                        for (int r = 0; r < 16; ++r) s[r] -= ref;
                    }
                    const float z = SWEEP == GRADIENT ? range.up - base : -base;
#pragma unroll
                    for (int r = 0; r < 16; ++r)
                        s[r] = exp2_hw(fmaf(s[r], c, z)) * (SWEEP == DELTA ? dp[r] : dp[r] - delta);
                    if (k0 + 32 * (b + 1) > whole) {
#pragma unroll
                        for (int r = 0; r < 16; ++r)
                            if (k0 + 32 * b + block_row(r) >= limit) s[r] = 0.f;
                    }
                    if constexpr (SWEEP == DELTA)
#pragma unroll
                        for (int r = 0; r < 16; ++r) sum += s[r];
                };
                Weights<T> w;
                if constexpr (sizeof(T) == 2) {
                    constexpr int N = 2 * L::STEPS, J = DP / 32;
                    Piece f[AHEAD];
                    auto fetch = [&](auto slot) TT_INLINE {
                        constexpr int u = slot, t = u - N;
                        if constexpr (u < N) f[u % AHEAD] = L::row_piece(u % 2 ? sv : sk, 32 * b, u / 2);
                        else if constexpr (SWEEP == GRADIENT && t < 2 * J)
                            f[u % AHEAD] = L::column_piece(sk, 32 * b + 16 * (t / J), t % J);
                    };
                    each<AHEAD>(fetch);
                    each<N>([&](auto slot) TT_INLINE {
                        constexpr int u = slot;
                        __builtin_amdgcn_sched_barrier(0);
                        if constexpr (u % 2) dp = mma16<T>(f[u % AHEAD], fd[u / 2], dp);
                        else s = mma16<T>(f[u % AHEAD], fq[u / 2], s);
                        fetch(std::integral_constant<int, u + AHEAD>{});
                    });
                    __builtin_amdgcn_sched_barrier(0);
                    weights();
                    if constexpr (SWEEP == DELTA) continue;
                    range.step(s, [&](float f) TT_INLINE {
#pragma unroll
                        for (int j = 0; j < J; ++j) dq[j] *= f;
                    });
                    w.set(s);
                    each<2 * J>([&](auto slot) TT_INLINE {
                        constexpr int t = slot, j = t % J;
                        __builtin_amdgcn_sched_barrier(0);
                        dq[j] = mma16<T>(f[(t + N) % AHEAD], w.w[t / J], dq[j]);
                        fetch(std::integral_constant<int, t + N + AHEAD>{});
                    });
                    __builtin_amdgcn_sched_barrier(0);
                } else {
#pragma unroll
                    for (int x = 0; x < L::STEPS; ++x) {
                        s = mma_rows<T>(L::row_piece(sk, 32 * b, x), fq[x], s);
                        dp = mma_rows<T>(L::row_piece(sv, 32 * b, x), fd[x], dp);
                    }
                    weights();
                    w.set(s);
#pragma unroll
                    for (int j = 0; j < DP / 32; ++j) dq[j] = mma_columns<T, DP>(sk, 32 * b, j, w, dq[j]);
                }
            }
        }
        if (next < last) {
            lk.store(tk);
            if constexpr (SWEEP != STATS) lv.store(tv);
        }
    };
    auto over = [&](auto sweep) TT_INLINE {
        for (int k0 = 0; k0 < last; k0 += 2 * BN) {
            step(sweep, k0, sk0, sv0, sk1, sv1);
            if (k0 + BN < last) step(sweep, k0 + BN, sk1, sv1, sk0, sv0);
        }
    };
    auto again = [&]() TT_INLINE {
        __syncthreads();
        issue_first();
        store_first();
    };
    const bool past = !(fabsf(lse) <= trusted_lse<T>());
    int any = __ballot(past) != 0;
    if constexpr (WAVES > 1) {   // (the waves', in a tile's place that nothing was sent for yet)
        int* flags = reinterpret_cast<int*>(sk1);
        if (lane == 0) flags[wave] = any;
        landed_barrier();
#pragma unroll
        for (int w = 0; w < WAVES; ++w) any |= flags[w];
        any = __builtin_amdgcn_readfirstlane(any);
    }
    if (any) {
        sm.init();
        over(std::integral_constant<Sweep, STATS>{});
        const float total = sm.total();
        if (past) {
            ref = sm.m == -INFINITY ? 0.f : sm.m;
            base = total == 0.f ? INFINITY : log2f(total) - Softmax<T>::kBias - Softmax<T>::rest(ref, sm.mc, c);
        }
        far = __ballot(ref != 0.f) != 0;
        again();
    }
    if constexpr (sizeof(T) == 2) {
        if (last <= kExact) {
            over(std::integral_constant<Sweep, DELTA>{});
            delta = halves_sum(sum);
            again();
        }
    }
    if (there && lane < 32) {
        float* p = a.stats + (int64_t)job.head * a.rows + row;
        p[0] = delta;
        p[a.apart] = base;
        p[2 * a.apart] = ref;
    }
    over(std::integral_constant<Sweep, GRADIENT>{});
    if constexpr (Range<T>::kOn) {
#pragma unroll
        for (int j = 0; j < DP / 32; ++j) dq[j] *= range.back();
    }
    if (there) store_columns<T, DP>((T*)a.dq + row * a.lddq + at, dq, a.scale, a.D);
}

template <class T, int DP>
tt_status dq_launch(const AttendArgs& a) {
    const bool whole = keys_in_pieces<T>(a), few = whole && short_sequences(a);
    const int waves = few ? 1 : kWaves;
    const dim3 grid((unsigned)(tiles_of(a, waves * kQueries) * a.heads));
    auto k = few ? k_attend_dq<T, DP, true, 1> : whole ? k_attend_dq<T, DP, true, kWaves> : k_attend_dq<T, DP, false, kWaves>;
    TT_LAUNCH(nullptr, "k_attend_dq", a.s, k, grid, dim3(waves * 64), 0, a.s, a);
    TT_LAUNCH_CHECK();
    return TT_OK;
}

}  // namespace

tt_status attend_dq(int32_t dtype, const AttendArgs& a) {
    return by_type(dtype, a, [&](auto* t, auto dim) { return dq_launch<std::remove_pointer_t<decltype(t)>, dim>(a); });
}

}  // namespace tt
