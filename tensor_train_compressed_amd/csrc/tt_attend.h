// Shared by the attention kernels (attend*.hip, paged.hip): 32 x 32 products on the
// matrix cores from tiles in LDS, whose rows are keys, values or queries of one head.
//
// A 16-byte piece of a row is what a lane takes at once. Products come in two forms:
//
// by rows   D[m][n] += sum_d A[m][d] B[n][d]   scores: both operands by rows, a lane's
//           piece of the summed dim from LDS (A) and from its registers (B)
// by columns D[c][n] += sum_r A[r][c] P[r][n]  outputs: A's rows are summed over; P is
//           such a product's own result, rounded, in the registers where it was formed
//
// A 32 x 32 result lies with lane l holding column n = l % 32 and rows
// 8 (r / 4) + 4 (l / 32) + r % 4 in register r. By columns the sum over rows may take them in
// any order as long as both operands have the same: a lane's registers are then the
// fragment of P as they are, with no exchange between lanes, and A's is read by the
// transposing load of the same four rows.
#pragma once

#include "tt_dense.h"

namespace tt {

typedef float floatx16 __attribute__((ext_vector_type(16)));
typedef uint32_t Piece __attribute__((ext_vector_type(4)));
typedef bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef f16 f16x8 __attribute__((ext_vector_type(8)));

// Lambdas of a kernel's loop are part of it, whatever their size.
#define TT_INLINE __attribute__((always_inline))

// A scale whose product with log2 e is finite, too.
inline bool scale_ok(float scale) { return scale > 0.f && scale < 2e38f; }

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

// [m c], rounded before anything else is done with it: sums relative to it stay exact.
__device__ __forceinline__ float product(float m, float c) {
    float mc = m * c;
    asm("" : "+v"(mc));
    return mc;
}

__device__ __forceinline__ float exp2_hw(float x) { return __builtin_amdgcn_exp2f(x); }

// op of the two halves of a wave (a lane's and the lane's 32 further).
template <class Op>
__device__ __forceinline__ float halves(float v, Op op) {
    const unsigned u = __builtin_bit_cast(unsigned, v);
    const auto p = __builtin_amdgcn_permlane32_swap(u, u, false, false);
    const unsigned a = p[0], b = p[1];
    return op(__builtin_bit_cast(float, a), __builtin_bit_cast(float, b));
}
__device__ __forceinline__ float halves_sum(float v) {
    return halves(v, [](float a, float b) { return a + b; });
}
__device__ __forceinline__ float halves_max(float v) {
    return halves(v, [](float a, float b) { return fmaxf(a, b); });
}

template <class T>
__device__ __forceinline__ floatx16 mma16(Piece a, Piece b, floatx16 c) {
    if constexpr (std::is_same<T, bf16>::value)
        return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0,
                                                       0, 0);
    else
        return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0,
                                                      0, 0);
}

// A step by rows: the two halves of a wave hold two pieces of the summed dim.
template <class T>
__device__ __forceinline__ floatx16 mma_rows(Piece a, Piece b, floatx16 c) {
    if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int e = 0; e < 4; ++e)
            c = __builtin_amdgcn_mfma_f32_32x32x2f32(__builtin_bit_cast(float, (uint32_t)a[e]),
                                                     __builtin_bit_cast(float, (uint32_t)b[e]), c, 0, 0, 0);
        return c;
    } else {
        return mma16<T>(a, b, c);
    }
}

// The n (0 .. 16 / sizeof(T)) leading elements of a piece, zeros behind them, at any
// alignment.
template <class T>
__device__ __forceinline__ Piece load_piece(const T* __restrict__ p, int n) {
    constexpr int P = 16 / sizeof(T);
    Piece r = {0, 0, 0, 0};
    if (n >= P) {
        __builtin_memcpy(&r, p, 16);
        return r;
    }
    if (n <= 0) return r;
#pragma unroll
    for (int i = 0; i < P; ++i) {
        if (i >= n) continue;
        if constexpr (sizeof(T) == 4) r[i] = bits_of(p[i]);
        else r[i >> 1] |= bits_of(p[i]) << (i & 1) * 16;
    }
    return r;
}

// A tile in LDS: rows of DP elements in 16-byte pieces, a row's in the order
// piece ^ key(row). The keys put the same piece of 16 consecutive rows, and the
// four pieces that a transposing load takes of 8 consecutive ones, into all
// 64 banks.
template <class T, int DP>
struct Tile {
    static constexpr int P = 16 / sizeof(T);               // elements of a piece
    static constexpr int PIECES = DP / P;
    static constexpr int SLOTS = PIECES <= 4 ? 4 : PIECES <= 8 ? 8 : PIECES <= 16 ? 16 : 32;
    static constexpr int ROW = SLOTS * 16;                 // bytes
    static constexpr int STEPS = PIECES / 2;               // of a product by rows
    static __device__ __forceinline__ int key(int row) {
        if (SLOTS == 4) return (row >> 2) & 3;
        if (SLOTS == 8) return ((row >> 1) & 1) << 2 | ((row >> 2) & 3);
        return (row & 3) << 2 | ((row >> 2) & 3);
    }
    static __device__ __forceinline__ int at(int row, int piece) { return row * ROW + (piece ^ key(row)) * 16; }

    // Of a product by rows: this lane's piece of step c of row (base +) lane % 32.
    static __device__ __forceinline__ Piece row_piece(const char* lds, int base, int c) {
        const int lane = threadIdx.x & 63;
        return *reinterpret_cast<const Piece*>(lds + at(base + (lane & 31), 2 * c + (lane >> 5)));
    }

    // Of a product by columns, 16-bit types: columns 32 j + lane % 32 of the rows
    // row0 + 4 h + {0..3, 8..11}, h = lane / 32.
    static __device__ __forceinline__ Piece column_piece(const char* lds, int row0, int j) {
        typedef short s16x4 __attribute__((ext_vector_type(4)));
        const int lane = threadIdx.x & 63, li = lane & 15;
        const int row = row0 + 4 * (lane >> 5) + (li >> 2), piece = 4 * j + ((lane >> 4) & 1) * 2 + ((li >> 1) & 1);
        auto take = [&](int r) {
            const char* p = lds + at(r, piece) + (li & 1) * 8;
            return __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4*)p);
        };
        const s16x4 a = take(row), b = take(row + 8);
        return __builtin_bit_cast(Piece, __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7));
    }
    // fp32: column 32 j + lane % 32 of row `row`.
    static __device__ __forceinline__ float column_value(const char* lds, int row, int j) {
        const int c = 32 * j + (threadIdx.x & 31);
        return *reinterpret_cast<const float*>(lds + at(row, c >> 2) + (c & 3) * 4);
    }
};

// A 32 x 32 product's result as the second operand of one by columns. 16-bit types: rounded
// to T, once or in two parts, the second what the first rounds off. Outputs' 2-norm errors of bf16 (f16) are
// 0.0017 (2.1e-4) for their own rounding alone and in two parts, 0.0023 (2.8e-4) in one. Over a paged cache, bound by
// memory, two parts take 373 us for 369 (64 sequences of 8000 tokens) and 33.2 for 32.9 (one of 32768), and are taken;
// over packed prompts 750 for 550 (8192 rows, 32 and 8 heads of 128) and 70 for 58 (16 and 2 heads of 64 in 8
// sequences), and one is.
template <class T>
struct Weights {
    Piece w[2];
    __device__ __forceinline__ void set(const floatx16& s) {
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i) w[t][i] = word_of<T>(s[8 * t + 2 * i], s[8 * t + 2 * i + 1]);
    }
    // s less what was taken of it.
    __device__ __forceinline__ floatx16 rest(const floatx16& s) const {
        floatx16 r;
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            Raw8<T> x;
            __builtin_memcpy(&x, &w[t], 16);
#pragma unroll
            for (int e = 0; e < 8; ++e) r[8 * t + e] = s[8 * t + e] - x.at(e);
        }
        return r;
    }
};
template <>
struct Weights<float> {
    floatx16 w;
    __device__ __forceinline__ void set(const floatx16& s) { w = s; }
};

// c += sum over the 32 rows from row0 of (columns 32 j ..) x p.
template <class T, int DP>
__device__ __forceinline__ floatx16 mma_columns(const char* lds, int row0, int j, const Weights<T>& p, floatx16 c) {
    typedef Tile<T, DP> L;
    if constexpr (sizeof(T) == 4) {
        const int h = (threadIdx.x >> 5) & 1;
#pragma unroll
        for (int r = 0; r < 16; ++r)
            c = __builtin_amdgcn_mfma_f32_32x32x2f32(L::column_value(lds, row0 + 8 * (r / 4) + 4 * h + r % 4, j), p.w[r],
                                                     c, 0, 0, 0);
    } else {
#pragma unroll
        for (int t = 0; t < 2; ++t) c = mma16<T>(L::column_piece(lds, row0 + 16 * t, j), p.w[t], c);
    }
    return c;
}

// This lane's pieces of a row as the second operand of products by rows.
template <class T, int DP>
using RowPieces = Piece[Tile<T, DP>::STEPS];
template <class T, int DP>
__device__ __forceinline__ void load_row(RowPieces<T, DP>& f, const T* __restrict__ row, bool there, int D) {
    constexpr int P = Tile<T, DP>::P;
    const int h = (threadIdx.x >> 5) & 1;
#pragma unroll
    for (int c = 0; c < Tile<T, DP>::STEPS; ++c) {
        const int e = (2 * c + h) * P;
        f[c] = load_piece(row + e, there ? min(P, D - e) : 0);
    }
}

// A tile's rows on their way to LDS; rows from `left` on, and pieces past D, become zeros.
//
// DMA: straight to LDS, 16 bytes a lane, for rows that start at whole pieces and D of whole
// pieces. What lies past the rows or past D has an offset outside the buffer's
// descriptor, for which the load delivers zeros. Otherwise through registers, read when
// the loads are issued and stored once the tile is wanted.
template <class T, int DP, int ROWS, int WAVES, bool DMA>
struct TileLoad {
    typedef Tile<T, DP> L;
    static constexpr int N = ROWS * L::SLOTS / (WAVES * 64);   // pieces of a lane
    static_assert(ROWS * L::SLOTS % (WAVES * 64) == 0, "whole pieces a lane");
    Piece r[DMA ? 1 : N];
    uint32_t off[DMA ? N : 1];
    int64_t ld;       // elements from row to row
    int D, wave;
    // slot i of this lane
    __device__ __forceinline__ int slot(int i) const { return (wave * N + i) * 64 + (threadIdx.x & 63); }
    __device__ __forceinline__ int row(int i) const { return slot(i) / L::SLOTS; }
    __device__ __forceinline__ int piece(int i) const { return (slot(i) % L::SLOTS) ^ L::key(row(i)); }
    __device__ __forceinline__ void init(int64_t ld_, int D_, int wave_) {
        ld = ld_;
        D = D_;
        wave = wave_;
        if constexpr (DMA) {
#pragma unroll
            for (int i = 0; i < N; ++i)
                off[i] = piece(i) * L::P < D ? (uint32_t)((row(i) * ld + piece(i) * L::P) * sizeof(T)) : 0x80000000u;
        }
    }
    __device__ __forceinline__ void issue(char* lds, const T* __restrict__ p, int left) {
        if constexpr (DMA) {
#ifdef __HIP_DEVICE_COMPILE__   // the descriptor's type is the device compiler's
            const int64_t bytes = left * ld * (int64_t)sizeof(T);
            const int records = left <= 0 ? 0 : bytes < 0x7FFFFFFF ? (int)bytes : 0x7FFFFFFF;
            const auto rsrc = __builtin_amdgcn_make_buffer_rsrc((void*)p, 0, records, 0x00020000);
#pragma unroll
            for (int i = 0; i < N; ++i)
                __builtin_amdgcn_raw_ptr_buffer_load_lds(
                    rsrc, (__attribute__((address_space(3))) void*)(lds + (wave * N + i) * 1024), 16, off[i], 0, 0, 0);
#endif
        } else {
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const int e = piece(i) * L::P;
                r[i] = load_piece(p + row(i) * ld + e, row(i) < left ? max(0, min(L::P, D - e)) : 0);
            }
        }
    }
    __device__ __forceinline__ void store(char* lds) const {
        if constexpr (!DMA) {
#pragma unroll
            for (int i = 0; i < N; ++i) *reinterpret_cast<Piece*>(lds + slot(i) * 16) = r[i];
        }
    }
};

// Waits until this wave's loads to LDS have arrived and its LDS accesses are done, then
// for the workgroup's other waves.
__device__ __forceinline__ void landed_barrier() {
    __atomic_signal_fence(__ATOMIC_SEQ_CST);
    __builtin_amdgcn_s_waitcnt(0x0070);   // vmcnt(0) lgkmcnt(0)
    __builtin_amdgcn_s_barrier();
    __atomic_signal_fence(__ATOMIC_SEQ_CST);
}

// Where the n-th register of a lane's half lies in a block of 32 rows.
__device__ __forceinline__ int block_row(int r) { return 8 * (r / 4) + 4 * ((threadIdx.x >> 5) & 1) + r % 4; }

// Stores a product by columns (its columns c are a row's elements): row pointer of lane
// % 32's row, `scale` its own.
template <class T, int DP>
__device__ __forceinline__ void store_columns(T* __restrict__ row, const floatx16 (&o)[DP / 32], float scale, int D) {
#pragma unroll
    for (int j = 0; j < DP / 32; ++j)
#pragma unroll
        for (int g = 0; g < 4; ++g) {
            const int d = 32 * j + block_row(4 * g);
            const float f[4] = {o[j][4 * g] * scale, o[j][4 * g + 1] * scale, o[j][4 * g + 2] * scale,
                                o[j][4 * g + 3] * scale};
            store4n(row + d, f, D - d);
        }
}

// The running softmax of a wave's 32 columns (queries): the reference m that weights are
// relative to, this half's part of their sum. Weights are 2^(c s - c m + kBias): with f16 the
// bias keeps weights down to 2^-22 of the largest among f16's full-precision numbers. The reference follows the
// maximum only when that has grown by 2^kSlack, so that most tiles rescale nothing.
template <class T>
struct Softmax {
    static constexpr float kBias = std::is_same<T, f16>::value ? 8.f : 0.f;
    static constexpr float kSlack = std::is_same<T, f16>::value ? 6.f : 8.f;
    // From here on differences come before products: the rounding of c m, which all
    // weights share, would be large beside the range of 2^x. Weights are then relative to c m itself,
    // up to here to c m rounded (mc); where both meet (a reference that moves past the border, a row
    // beside one past it, parts that are joined), `rest` is what one has and the other has not.
    static constexpr float kFar = 1048576.f;
    static __device__ __forceinline__ float rest(float m, float mc, float c) {
        return fabsf(mc) > kFar ? 0.f : fmaf(m, c, -mc);
    }
    float m, mc, l;   // mc: c m rounded (0 while nothing was seen)
    __device__ __forceinline__ void init() {
        m = -INFINITY;
        mc = 0.f;
        l = 0.f;
    }
    // Takes the scores s (masked ones -inf) to weights; rescale(a) where outputs must be
    // multiplied by a.
    template <int N, class F>
    __device__ __forceinline__ void step(floatx16 (&s)[N], float c, F rescale) {
        float top = s[0][0];
#pragma unroll
        for (int b = 0; b < N; ++b)
#pragma unroll
            for (int r = 0; r < 16; ++r) top = fmaxf(top, s[b][r]);
        top = halves_max(top);
        const bool grown = m == -INFINITY ? top > -INFINITY : (top - m) * c > kSlack;
        if (__ballot(grown)) {
            const float to = fmaxf(m, top), toc = to == -INFINITY ? 0.f : product(to, c);
            // nothing seen before: what was summed is 0
            const float a = moved(m, to, c);
            m = to;
            mc = toc;
            l *= a;
            rescale(a);
        }
        float sum = 0.f;
        if (__ballot(fabsf(mc) > kFar)) {
            const float z = m == -INFINITY ? 0.f : m, add = kBias + rest(z, mc, c);
#pragma unroll
            for (int b = 0; b < N; ++b)
#pragma unroll
                for (int r = 0; r < 16; ++r) {
                    s[b][r] = exp2_hw(fmaf(s[b][r] - z, c, add));
                    sum += s[b][r];
                }
        } else {
            const float z = kBias - mc;
#pragma unroll
            for (int b = 0; b < N; ++b)
#pragma unroll
                for (int r = 0; r < 16; ++r) {
                    s[b][r] = exp2_hw(fmaf(s[b][r], c, z));
                    sum += s[b][r];
                }
        }
        l += sum;
    }
    // What sums relative to maximum m are multiplied by to be relative to `to`.
    static __device__ __forceinline__ float moved(float m, float to, float c) {
        if (m == -INFINITY) return 0.f;
        const float mc = product(m, c), toc = product(to, c);
        if (fabsf(mc) <= kFar && fabsf(toc) <= kFar) return exp2_hw(mc - toc);
        return exp2_hw((m - to) * c - rest(m, mc, c) + rest(to, toc, c));
    }
    // Both halves' sum; the log of the sum of e^score.
    __device__ __forceinline__ float total() const { return halves_sum(l); }
    __device__ __forceinline__ float log_sum(float total) const {
        return total == 0.f ? -INFINITY : kLn2 * (mc - kBias + log2f(total));
    }
};

// A sequence's tile of `size` rows.
struct Span {
    int64_t first;   // row of the sequence's first
    int len, tile, tiles;
};
// Of tile t (as counted over all sequences: sequence s has those from offsets[s] / size + s
// on, which are at least as many as it needs); false where t is none. A wave looks
// through 64 sequences at a time. Offsets are kept within [0, rows].
__device__ __forceinline__ bool find_tile(const int64_t* __restrict__ offsets, int64_t seqs, int64_t rows, int size,
                                          int64_t t, Span& sp) {
    const int lane = threadIdx.x & 63;
    auto at = [&](int64_t s) {
        const int64_t o = offsets[s];
        return o < 0 ? 0 : o > rows ? rows : o;
    };
    int64_t lo = 0, hi = seqs;
    while (hi - lo > 1) {
        const int64_t step = (hi - lo + 63) / 64, s = lo + lane * step;
        const int n = __popcll(__ballot(s < hi && at(s) / size + s <= t));
        if (n == 0) return false;
        lo += (n - 1) * step;
        hi = lo + step < hi ? lo + step : hi;
    }
    const int64_t first = at(lo), end = at(lo + 1), tile = t - (first / size + lo);
    sp.first = first;
    sp.len = end > first ? (int)(end - first) : 0;
    sp.tiles = (sp.len + size - 1) / size;
    sp.tile = (int)tile;
    return tile >= 0 && tile < sp.tiles;
}

}  // namespace tt
