// Helpers shared by the dense operators (norm.hip, gate.hip, distill.hip):
// element types, loads and stores of eight elements at any alignment, group
// sums. Written for gfx950 (wave64).
#pragma once

#include "tt_internal.h"

#include <hip/hip_bf16.h>
#include <hip/hip_fp16.h>

#include <cstddef>

namespace tt {

typedef __bf16 bf16;
typedef _Float16 f16;

inline bool dtype_ok(int32_t d) { return d == TT_F32 || d == TT_BF16 || d == TT_F16; }
inline int dtype_bytes(int32_t d) { return d == TT_F32 ? 4 : 2; }

// Eight consecutive elements as they sit in memory. Rows of any width and
// stride are served by one code path: the copies below take the element's own
// alignment, and gfx950 executes 16-byte global accesses at any address.
template <class T>
struct alignas(16) Raw8 {
    T v[8];
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
    for (int e = 0; e < 8; ++e) r.v[e] = fill;
#pragma unroll
    for (int e = 0; e < 8; ++e)
        if (e < n) r.v[e] = p[e];
    return r;
}

template <class T>
__device__ __forceinline__ void store8n(T* __restrict__ p, const Raw8<T>& r, int n) {
    if (n >= 8) {
        __builtin_memcpy(p, &r, sizeof(r));
        return;
    }
#pragma unroll
    for (int e = 0; e < 8; ++e)
        if (e < n) p[e] = r.v[e];
}

// Sum over the 2^k consecutive lanes a lane belongs to (width <= 64).
template <int WIDTH>
__device__ __forceinline__ float lanes_sum(float v) {
#pragma unroll
    for (int d = 1; d < WIDTH; d <<= 1) v += __shfl_xor(v, d, 64);
    return v;
}

template <int WIDTH>
__device__ __forceinline__ float lanes_max(float v) {
#pragma unroll
    for (int d = 1; d < WIDTH; d <<= 1) v = fmaxf(v, __shfl_xor(v, d, 64));
    return v;
}

}  // namespace tt
