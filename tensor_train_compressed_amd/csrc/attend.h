// Shared by the kernels of attention over packed prompts (attend.hip, attend_dq.hip,
// attend_dkv.hip).
#pragma once

#include "tt_attend.h"

namespace tt {

struct AttendArgs {
    const void *q, *k, *v, *out, *dout;
    int64_t ldq, ldk, ldv, ldo, lddo;
    void *o, *dq, *dk, *dv;
    int64_t lddq, lddk, lddv;
    const int64_t* offsets;
    int64_t seqs, rows;
    int heads, kv, D, causal;
    float scale;
    float* lse;                  // [heads][rows]
    // the backward's, [3][apart], of each the first [heads][rows]: delta, base and ref; weights are
    // 2^(c (s - ref) - base)
    float* stats;
    uint32_t apart;
    float* part;          // dk's, then dv's sums [splits][rows][kv * D]
    int splits;
    hipStream_t s;
};

// f(0), .., f(N - 1) with constant arguments.
template <int N, class F, int I = 0>
__device__ __forceinline__ void each(F f) {
    if constexpr (I < N) {
        f(std::integral_constant<int, I>{});
        each<N, F, I + 1>(f);
    }
}

// Fragments under way from LDS ahead of the product that takes them (read right before it: forward
// of the long prompt below 577 us instead of 555).
constexpr int AHEAD = 4;

constexpr int kQueries = 32;   // a wave's

// Waves of a workgroup: four, or one where sequences are short on average (and rows in whole pieces), whose
// tiles the other three would have no part in. 16384 rows in sequences of equal length, us of the
// forward and of the backward, one wave and four:
//   rows a sequence      20                 64                96                128               192
//   4 heads of 32 fp32   17 45, 49 118      15 44, 20 59      25 68, 21 66      21 57, 29 85      25 68, 27 88
//   16 / 4 of 64 bf16    48 99, 128 211     45 96, 57 109     57 130, 53 112    46 106, 85 178    50 118, 57 129
//   32 / 8 of 128 bf16   206 437, 333 873   175 387, 181 440  179 452, 185 434  184 422, 174 494  193 460, 185 442
// The average also counts sequences without rows, and does not see one long sequence among many short ones; there
// four would take less (32 and 8 heads of 128 bf16): 7000 rows among 100 sequences of 10 803 2022, 546 1556; 8192 rows
// beside 255 empty sequences 944 2486, 590 1899.
constexpr int kWaves = 4;
constexpr int64_t kShort = 128;   // rows a sequence, on average, up to which

// Rows of a tile that goes through LDS.
template <class T, int DP, int WAVES>
constexpr int tile_rows() {
    return WAVES > 1 && Tile<T, DP>::ROW <= 256 ? 64 : 32;
}

// Waves a SIMD is to hold: two where their registers allow it without spilling (loads from where
// registers were spilled to wait for all that is under way to LDS, which took a kernel from 560 to
// 1230 us). dk and dv of 16-bit heads past 64 have two by their groups of waves; there rows that go through registers
// spill up to 43 of them (2948 unaligned rows, 8 heads of 127 bf16, dq, dk and dv: 533 us).
enum Pass { FWD, DQ, DKV };
template <class T, int DP, bool DMA, Pass PASS>
constexpr int waves_of() {
    if (sizeof(T) == 4) return DP == 32 || (DP == 64 && DMA && PASS != DKV) ? 2 : 1;
    if (PASS == DKV) return DP <= 64 ? 2 : 1;
    return DP <= 64 || DMA ? 2 : 1;
}

// A sum's f16 factors (the backward's ds), times a power of two 2^up that keeps the largest of a column that was
// seen between 2^9 and 2^15: none is past f16's range, and those down to 2^-23 of the largest keep their digits.
// The power falls where a factor outgrows it, and sums are multiplied by what it fell. Other types hold any factor.
// 2048 rows, heads of 64, dout of size 1e-4: dq's 2-norm error 1.6e-2 without it, 2.4e-3 with, as for rounding dq alone.
// Its cost, dq, dk and dv together: 8192 rows, 32 and 8 heads of 128, 1900 -> 2000 us; 16 and 2 heads of 64 in 8
// sequences 185 -> 200.
template <class T>
struct Range {
    static constexpr bool kOn = std::is_same<T, f16>::value;
    static constexpr float kMost = 32768.f;
    float up;
    __device__ __forceinline__ void init() { up = kOn ? 60.f : 0.f; }   // (f16's products, of at most 2^53, stay finite)
    // Takes factors that are multiplied by 2^up already.
    template <class F>
    __device__ __forceinline__ void step(floatx16& x, F rescale) {
        if constexpr (kOn) {
            float top = 0.f;
#pragma unroll
            for (int r = 0; r < 16; ++r) top = fmaxf(top, fabsf(x[r]));
            top = halves_max(top);
            if (__ballot(top > kMost)) {
                // top is below 2^e: to below 2^10 (infinite: it stays)
                const int e = top > kMost && top < INFINITY ? 10 - __builtin_amdgcn_frexp_expf(top) : 0;
                const float a = ldexpf(1.f, e);
                up += (float)e;
#pragma unroll
                for (int r = 0; r < 16; ++r) x[r] *= a;
                rescale(a);
            }
        }
    }
    // What sums are multiplied by at the end.
    __device__ __forceinline__ float back() const { return ldexpf(1.f, -(int)up); }
};
// Weights on their way to f16, which are 1 at most, in powers of two: those down to 2^-28 keep their digits.
template <class T>
constexpr float weight_bits() {
    return Range<T>::kOn ? 14.f : 0.f;
}

// The workgroup's tile and head: heads that share keys lie next to each other.
struct Job {
    int64_t tile;
    int kv, head;
};
__device__ __forceinline__ Job job_of(const AttendArgs& a) {
    const int i = blockIdx.x % a.heads, kv = i % a.kv;
    return {(int64_t)(blockIdx.x / a.heads), kv, kv * (a.heads / a.kv) + i / a.kv};
}

// What weights are relative to, in powers of two: 2^(c s - it). Rows that see nothing have
// none.
__device__ __forceinline__ float log2_sum(float lse) { return lse == -INFINITY ? INFINITY : lse * kLog2e; }
// Up to where the backward takes lse for that. Its four roundings (on the way to lse and back) are an
// exponent's error of 2^-22 |lse|, which no sum takes out of the weights again: up to here no more than what fp32's scores
// are off by themselves, with 16-bit types (6e-5) an eighth of f16's rounding of a weight. Rows past it have
// their maximum and sum formed again, kept apart, so that weights are never above 1; the workgroups of dq
// that hold such rows go over their keys once more for it. One prompt of 8192 rows, 32 and 8 heads of 128
// bf16, dq, dk and dv: 1910 us, with all rows past it 2170; 2048 rows, 8 heads of 64 fp32: 326 and 423.
template <class T>
constexpr float trusted_lse() {
    return sizeof(T) == 4 ? 32.f : 256.f;
}

// Whether rows start at whole 16-byte pieces, and their heads are made of them.
inline bool pieces(const void* p, int64_t ld, int D, size_t size) {
    return ((uintptr_t)p & 15) == 0 && ld * size % 16 == 0 && D * size % 16 == 0;
}
template <class T>
bool keys_in_pieces(const AttendArgs& a) {
    return pieces(a.k, a.ldk, a.D, sizeof(T)) && pieces(a.v, a.ldv, a.D, sizeof(T));
}
template <class T>
bool queries_in_pieces(const AttendArgs& a) {
    return pieces(a.q, a.ldq, a.D, sizeof(T)) && pieces(a.dout, a.lddo, a.D, sizeof(T));
}
inline bool short_sequences(const AttendArgs& a) { return a.rows <= kShort * a.seqs; }
// Tiles of `size` rows that the sequences have at most.
inline int64_t tiles_of(const AttendArgs& a, int64_t size) { return a.rows / size + a.seqs; }

// f of the kernels' element type and of the heads' padded size.
template <class T, class F>
tt_status by_dim(const AttendArgs& a, F f) {
    if (a.D <= 32) return f((T*)nullptr, std::integral_constant<int, 32>{});
    if (a.D <= 64) return f((T*)nullptr, std::integral_constant<int, 64>{});
    if (a.D <= 96) return f((T*)nullptr, std::integral_constant<int, 96>{});
    return f((T*)nullptr, std::integral_constant<int, 128>{});
}
template <class F>
tt_status by_type(int32_t dtype, const AttendArgs& a, F f) {
    if (dtype == TT_F32) return by_dim<float>(a, f);
    if (dtype == TT_BF16) return by_dim<bf16>(a, f);
    return by_dim<f16>(a, f);
}

// The backward's two passes (attend_dq.hip, attend_dkv.hip): dq, with delta for the other; dk
// and dv, whose sums may be split over workgroups.
tt_status attend_dq(int32_t dtype, const AttendArgs& a);
tt_status attend_dkv(int32_t dtype, const AttendArgs& a);
// Splits: where tiles of keys are fewer than would fill the chip twice, as many as bring them to
// kGroups workgroups. 140 tiles of 64 wide heads, 8 to a key head (8192 rows in 8 sequences):
// 510 us in one split, 185 in 3, 108 in 7 and 113 in 15, with 0, 6, 11 and 20 to join them; 512
// tiles of 128 wide heads: 1230 in one, 1257 in two and 26 to join.
constexpr int64_t kFull = 512, kGroups = 1024, kMaxSplits = 16;
inline int64_t splits_of(int64_t rows, int64_t seqs, int64_t kv) {
    const int64_t n = std::max<int64_t>(1, ((rows + kWaves * kQueries - 1) / (kWaves * kQueries) + seqs / 2) * kv);
    return n >= kFull ? 1 : std::max<int64_t>(1, std::min(kMaxSplits, kGroups / n));
}

}  // namespace tt
