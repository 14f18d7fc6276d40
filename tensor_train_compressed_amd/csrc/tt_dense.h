// Helpers shared by the dense operators (norm.hip, gate.hip, distill.hip):
// element types, loads and stores of eight elements at any alignment, group
// sums. Written for gfx950 (wave64).
#pragma once

#include "tt_internal.h"

#include <hip/hip_bf16.h>
#include <hip/hip_fp16.h>

#include <cstddef>
#include <type_traits>

// Not part of the library's interface; for its tests. How often a workgroup of
// tt_emb_distill_train polls for the other parts of its row before it forms them
// itself (negative: the default), for every later call of the process. Returns what
// it was. Every count gives the same bits.
extern "C" int32_t tt_distill_set_polls(int32_t n);

namespace tt {

typedef __bf16 bf16;
typedef _Float16 f16;

inline bool dtype_ok(int32_t d) { return d == TT_F32 || d == TT_BF16 || d == TT_F16; }

template <class T>
__device__ __forceinline__ uint32_t bits_of(T v) {
    if constexpr (sizeof(T) == 4) return __builtin_bit_cast(uint32_t, v);
    else return __builtin_bit_cast(uint16_t, v);
}

// Two values rounded to the nearest T, in one word (bf16: one instruction; rounded
// one by one they would take two and a third to join them).
template <class T>
__device__ __forceinline__ uint32_t word_of(float a, float b) {
    typedef float floatx2 __attribute__((ext_vector_type(2)));
    typedef T Tx2 __attribute__((ext_vector_type(2)));
    return __builtin_bit_cast(uint32_t, __builtin_convertvector((floatx2{a, b}), Tx2));
}

// Eight consecutive elements as they sit in memory, kept as 32-bit words (an
// array of 16-bit elements would take a register each). Rows of any width and
// stride are served by one code path: the copies below take the element's own
// alignment, and gfx950 executes 16-byte global accesses at any address.
template <class T>
struct alignas(16) Raw8 {
    uint32_t w[2 * sizeof(T)];

    __device__ __forceinline__ float at(int e) const {
        if constexpr (sizeof(T) == 4) {
            return __builtin_bit_cast(float, w[e]);
        } else {
            const uint32_t x = w[e >> 1];
            if constexpr (std::is_same<T, bf16>::value)
                return __builtin_bit_cast(float, (e & 1) ? x & 0xFFFF0000u : x << 16);
            else
                return (float)__builtin_bit_cast(T, (uint16_t)((e & 1) ? x >> 16 : x & 0xFFFFu));
        }
    }
    // Rounded to the nearest T.
    __device__ __forceinline__ void set(const float (&f)[8]) {
#pragma unroll
        for (int i = 0; i < (int)(2 * sizeof(T)); ++i) {
            if constexpr (sizeof(T) == 4) w[i] = bits_of(f[i]);
            else w[i] = word_of<T>(f[2 * i], f[2 * i + 1]);
        }
    }
};

template <class T>
__device__ __forceinline__ Raw8<T> load8(const T* __restrict__ p) {
    Raw8<T> r;
    __builtin_memcpy(&r, p, sizeof(r));
    return r;
}

// The first n (0..8) of them, `fill` in the place of the others.
template <class T>
__device__ __forceinline__ Raw8<T> load8n(const T* __restrict__ p, int n, T fill) {
    if (n >= 8) return load8(p);
    Raw8<T> r;
#pragma unroll
    for (int i = 0; i < (int)(2 * sizeof(T)); ++i) {
        if constexpr (sizeof(T) == 4) {
            r.w[i] = bits_of(i < n ? p[i] : fill);
        } else {
            r.w[i] = bits_of(2 * i < n ? p[2 * i] : fill) | bits_of(2 * i + 1 < n ? p[2 * i + 1] : fill) << 16;
        }
    }
    return r;
}

// Keeps the raw words as what later passes unpack again: the compiler would
// otherwise hold the floats, twice the registers, from one pass to the next.
template <class T, int N>
__device__ __forceinline__ void keep_raw(Raw8<T> (&r)[N]) {
#pragma unroll
    for (int v = 0; v < N; ++v)
#pragma unroll
        for (int i = 0; i < (int)(2 * sizeof(T)); ++i) asm volatile("" : "+v"(r[v].w[i]));
}

template <class T>
__device__ __forceinline__ void store8n(T* __restrict__ p, const float (&f)[8], int n) {
    if (n >= 8) {
        Raw8<T> r;
        r.set(f);
        __builtin_memcpy(p, &r, sizeof(r));
        return;
    }
#pragma unroll
    for (int e = 0; e < 8; ++e)
        if (e < n) p[e] = (T)f[e];
}

template <class T>
__device__ __forceinline__ void store4n(T* __restrict__ p, const float (&f)[4], int n) {
    if (n >= 4) {
        struct alignas(8) {
            T v[4];
        } r = {(T)f[0], (T)f[1], (T)f[2], (T)f[3]};
        __builtin_memcpy(p, &r, sizeof(r));
        return;
    }
#pragma unroll
    for (int e = 0; e < 4; ++e)
        if (e < n) p[e] = (T)f[e];
}

// Eight, past the caches.
template <class T>
__device__ __forceinline__ void store8n_apart(T* __restrict__ p, const float (&f)[8], int n) {
    if (n < 8) return store8n(p, f, n);
    typedef uint32_t u32x4 __attribute__((ext_vector_type(4), aligned(2)));
    Raw8<T> r;
    r.set(f);
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) / 2; ++i) {
        const u32x4 q = {r.w[4 * i], r.w[4 * i + 1], r.w[4 * i + 2], r.w[4 * i + 3]};
        __builtin_nontemporal_store(q, reinterpret_cast<u32x4*>(p) + i);
    }
}

// v of another lane, by moves in the vector unit: lane ^ 1, lane ^ 2, the lane
// mirrored within 8 and within 16 (after the steps before, mirrored lanes hold
// what lane ^ 4 and lane ^ 8 hold).
template <int CTRL>
__device__ __forceinline__ float dpp(float v) {
    return __builtin_bit_cast(
        float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), CTRL, 0xF, 0xF, false));
}

// op over the 2^k consecutive lanes a lane belongs to (WIDTH <= 64).
template <int WIDTH, class Op>
__device__ __forceinline__ float lanes_reduce(float v, Op op) {
    if (WIDTH > 1) v = op(v, dpp<0xB1>(v));
    if (WIDTH > 2) v = op(v, dpp<0x4E>(v));
    if (WIDTH > 4) v = op(v, dpp<0x141>(v));
    if (WIDTH > 8) v = op(v, dpp<0x140>(v));
    if (WIDTH > 16) {
        const unsigned u = __builtin_bit_cast(unsigned, v);
        const auto p = __builtin_amdgcn_permlane16_swap(u, u, false, false);
        const unsigned a = p[0], b = p[1];
        v = op(__builtin_bit_cast(float, a), __builtin_bit_cast(float, b));
    }
    if (WIDTH > 32) {
        const unsigned u = __builtin_bit_cast(unsigned, v);
        const auto p = __builtin_amdgcn_permlane32_swap(u, u, false, false);
        const unsigned a = p[0], b = p[1];
        v = op(__builtin_bit_cast(float, a), __builtin_bit_cast(float, b));
    }
    return v;
}
template <int WIDTH>
__device__ __forceinline__ float lanes_sum(float v) {
    return lanes_reduce<WIDTH>(v, [](float a, float b) { return a + b; });
}
template <int WIDTH>
__device__ __forceinline__ float lanes_max(float v) {
    return lanes_reduce<WIDTH>(v, [](float a, float b) { return fmaxf(a, b); });
}

}  // namespace tt
