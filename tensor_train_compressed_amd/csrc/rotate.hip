// Norms of queries and keys for each head with the rotation by position, forward
// and backward, and the form that serves: keys and values go into the paged cache.
//
//   r = 1/sqrt(mean(x^2) + eps),  n = x r,  u = n w          (x: a head's dim elements)
//   angle_p = position freq_p;  of the pair (a, b):
//   y_a = u_a cos - u_b sin,  y_b = u_a sin + u_b cos;       y = u past the pairs
//   g = the rotation back of dy,  dw = sum over rows and heads of g n
//   t = g w,  dx = r (t - n mean(t n))
//
// Everything is held in fp32 and rounded once, at the store; angles are formed as
// turns in fp64 (position freq / 2 pi less its whole turns), so that positions far
// along keep the digits of their angle, and go to sine and cosine in fp32.
//
// Bound by memory (forward: 8192 rows of 32 and 8 heads of 128 bf16 in 31 us, 5.4 TB/s): a head is
// read once and stays in registers. A head is cut into
// chunks of 8 pairs, one a lane, so that both of a pair are the lane's own whatever
// the pairing and the rotated part; what is not rotated goes in chunks of 16. A wave
// takes one row and goes over its heads 64 / lanes-a-head at a time, with the
// row's sines and cosines formed once, a lane a pair, and passed through LDS.
#include "tt_dense.h"

namespace tt {
namespace {

constexpr int kMaxDim = 256;
constexpr int kThreads = 256, kWaves = kThreads / 64;

struct RotateArgs {
    const void *q, *k, *v;            // v: append only
    int64_t ldq, ldk, ldv;
    const void *wq, *wk;
    const int64_t* positions;
    const double* freq;
    const void *dyq, *dyk;            // backward
    int64_t lddyq, lddyk;
    void *oq, *ok, *ov;               // y; dx in the backward
    int64_t ldoq, ldok;
    const int64_t* slots;             // append: a row's place in the cache, ok and ov
    int64_t nslots;
    float* part;                      // backward: [q_groups + k_groups][dim]
    int q_groups, k_groups;
    void *dwq, *dwk;
    int64_t rows;
    int heads, kv, dim, half;         // half: pairs
    bool neighbours;
    float eps;
    int slabs, per;                   // a row's heads go in `slabs` waves of `per` rounds each
    hipStream_t s;
};

// Chunks of a head: pairs by eights, then the rest by sixteens.
__host__ __device__ inline int chunks_of(int dim, int half) { return (half + 7) / 8 + (dim - 2 * half + 15) / 16; }

// A lane's chunk: two pieces of up to 8 elements at o0 and o1 of the head.
struct Chunk {
    int o0, n0, o1, n1, p, np;        // p, np: its pairs (np = 0: not rotated)
};
__device__ __forceinline__ Chunk chunk_of(const RotateArgs& a, int c) {
    Chunk k{};
    const int turned = (a.half + 7) / 8;
    if (c < turned) {
        k.p = c * 8;
        k.np = min(8, a.half - k.p);
        k.o0 = a.neighbours ? 2 * k.p : k.p;
        k.o1 = a.neighbours ? 2 * k.p + 8 : k.p + a.half;
        k.n0 = a.neighbours ? min(8, 2 * k.np) : k.np;
        k.n1 = a.neighbours ? max(0, 2 * k.np - 8) : k.np;
    } else {
        k.o0 = 2 * a.half + (c - turned) * 16;
        k.o1 = k.o0 + 8;
        k.n0 = min(8, max(0, a.dim - k.o0));
        k.n1 = min(8, max(0, a.dim - k.o1));
    }
    return k;
}

// Sine and cosine of a row's angles, one pair a lane, into this wave's LDS; then
// this lane's chunk of them (cos 1, sin 0 where nothing is rotated).
__device__ __forceinline__ void turns_of(const RotateArgs& a, int64_t row, const Chunk& k, float2* sm, float (&c)[8],
                                         float (&s)[8]) {
    const int lane = threadIdx.x & 63;
    const double pos = (double)a.positions[row];
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    for (int p = lane; p < a.half; p += 64) {
        double t = pos * a.freq[p] * 0.15915494309189533577;   // turns
        t -= rint(t);
        float sn, cs;
        sincospif((float)(2.0 * t), &sn, &cs);
        sm[p] = make_float2(cs, sn);
    }
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float2 v = i < k.np ? sm[k.p + i] : make_float2(1.f, 0.f);
        c[i] = v.x;
        s[i] = v.y;
    }
}

// The rotation of a chunk x[0..7], x[8..15] by its angles (sign -1: back). Elements that
// are not rotated stay as they are, whatever lies beside them.
__device__ __forceinline__ void turn(float (&x)[16], const Chunk& k, const float (&c)[8], const float (&s)[8],
                                     bool neighbours, float sign) {
    if (k.np == 0) return;
    if (neighbours) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float a = x[2 * i], b = x[2 * i + 1], sn = sign * s[i];
            x[2 * i] = a * c[i] - b * sn;
            x[2 * i + 1] = a * sn + b * c[i];
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float a = x[i], b = x[8 + i], sn = sign * s[i];
            x[i] = a * c[i] - b * sn;
            x[8 + i] = a * sn + b * c[i];
        }
    }
}

template <class T>
__device__ __forceinline__ void load_chunk(const T* __restrict__ p, const Chunk& k, float (&x)[16]) {
    const Raw8<T> a = load8n(p + k.o0, k.n0, (T)0.f), b = load8n(p + k.o1, k.n1, (T)0.f);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        x[e] = a.at(e);
        x[8 + e] = b.at(e);
    }
}
template <class T>
__device__ __forceinline__ void store_chunk(T* __restrict__ p, const Chunk& k, const float (&x)[16]) {
    float a[8], b[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        a[e] = x[e];
        b[e] = x[8 + e];
    }
    store8n(p + k.o0, a, k.n0);
    store8n(p + k.o1, b, k.n1);
}

template <int LANES>
__device__ __forceinline__ float rstd_of(const float (&x)[16], float inv_dim, float eps) {
    float sum = 0.f;
#pragma unroll
    for (int e = 0; e < 16; ++e) sum = fmaf(x[e], x[e], sum);
    return 1.f / sqrtf(lanes_sum<LANES>(sum) * inv_dim + eps);
}

// Forward, and the form that appends to the cache (keys and values of a row whose
// slot lies outside it go nowhere). A wave takes a slab of a row's heads.
template <class T, class W, int LANES>
__global__ __launch_bounds__(kThreads) void k_rotate(const RotateArgs a) {
    constexpr int HEADS = 64 / LANES;     // a round
    __shared__ float2 sm[kWaves][kMaxDim / 2];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t job = (int64_t)blockIdx.x * kWaves + wave, row = job / a.slabs;
    if (row >= a.rows) return;
    const int slab = (int)(job % a.slabs);
    const Chunk k = chunk_of(a, lane % LANES);
    float c[8], s[8], wq[16], wk[16];
    turns_of(a, row, k, sm[wave], c, s);
    load_chunk((const W*)a.wq, k, wq);
    load_chunk((const W*)a.wk, k, wk);
    const float inv_dim = 1.f / (float)a.dim;
    const int64_t slot = a.slots ? a.slots[row] : row;
    const bool kept = !a.slots || (slot >= 0 && slot < a.nslots);
    const int all = a.heads + a.kv * (a.slots ? 2 : 1);
    for (int r = 0; r < a.per; ++r) {
        const int h = (slab * a.per + r) * HEADS + lane / LANES;
        const bool is_q = h < a.heads, is_v = h >= a.heads + a.kv;
        const int hk = h - a.heads - (is_v ? a.kv : 0);
        if (h >= all) continue;           // (a head's lanes go together)
        const T* src = is_q ? (const T*)a.q + row * a.ldq + (int64_t)h * a.dim
                            : (is_v ? (const T*)a.v + row * a.ldv : (const T*)a.k + row * a.ldk) + (int64_t)hk * a.dim;
        T* dst = is_q ? (T*)a.oq + row * a.ldoq + (int64_t)h * a.dim
                      : (T*)(is_v ? a.ov : a.ok) + slot * a.ldok + (int64_t)hk * a.dim;
        if (is_v) {
            const Raw8<T> x0 = load8n(src + k.o0, k.n0, (T)0.f), x1 = load8n(src + k.o1, k.n1, (T)0.f);
            if (!kept) continue;
            auto copy = [](T* p, const Raw8<T>& x, int n) {
                if (n >= 8) {
                    __builtin_memcpy(p, &x, sizeof(x));
                    return;
                }
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    if (e >= n) continue;
                    if constexpr (sizeof(T) == 4) p[e] = __builtin_bit_cast(T, x.w[e]);
                    else p[e] = __builtin_bit_cast(T, (uint16_t)(x.w[e >> 1] >> (e & 1) * 16));
                }
            };
            copy(dst + k.o0, x0, k.n0);
            copy(dst + k.o1, x1, k.n1);
            continue;
        }
        float x[16];
        load_chunk(src, k, x);
        const float rstd = rstd_of<LANES>(x, inv_dim, a.eps);
#pragma unroll
        for (int e = 0; e < 16; ++e) x[e] = x[e] * rstd * (is_q ? wq[e] : wk[e]);
        turn(x, k, c, s, a.neighbours, 1.f);
        if (is_q || kept) store_chunk(dst, k, x);
    }
}

// Backward: the first q_groups workgroups take queries, the others keys, so that a wave holds one
// weight and one sum. A wave takes whole rows, and sums dw of its heads in registers. 8192 rows
// of 32 and 8 heads of 128 bf16: 57 us, 4.4 TB/s; the same with the next round's pieces fetched
// ahead (219 registers) or both weights in a wave (170), 66 with registers for a fourth wave a SIMD.
template <class T, class W, int LANES>
__global__ __launch_bounds__(kThreads) void k_rotate_back(const RotateArgs a) {
    constexpr int HEADS = 64 / LANES;
    __shared__ float2 sm[kWaves][kMaxDim / 2];
    __shared__ float sum[kWaves][LANES * 16];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const bool is_q = (int)blockIdx.x < a.q_groups;
    const int group = is_q ? blockIdx.x : blockIdx.x - a.q_groups, groups = is_q ? a.q_groups : a.k_groups;
    const int heads = is_q ? a.heads : a.kv;
    const T *x0 = (const T*)(is_q ? a.q : a.k), *dy0 = (const T*)(is_q ? a.dyq : a.dyk);
    T* dx0 = (T*)(is_q ? a.oq : a.ok);
    const int64_t ldx = is_q ? a.ldq : a.ldk, lddy = is_q ? a.lddyq : a.lddyk, lddx = is_q ? a.ldoq : a.ldok;
    const Chunk k = chunk_of(a, lane % LANES);
    float w[16], dw[16] = {};
    load_chunk((const W*)(is_q ? a.wq : a.wk), k, w);
    const float inv_dim = 1.f / (float)a.dim;
    for (int64_t row = (int64_t)group * kWaves + wave; row < a.rows; row += (int64_t)groups * kWaves) {
        float c[8], s[8];
        turns_of(a, row, k, sm[wave], c, s);
        for (int h = lane / LANES; h < heads; h += HEADS) {
            const int64_t at = (int64_t)h * a.dim;
            float x[16], g[16];
            load_chunk(x0 + row * ldx + at, k, x);
            load_chunk(dy0 + row * lddy + at, k, g);
            const float rstd = rstd_of<LANES>(x, inv_dim, a.eps);
            turn(g, k, c, s, a.neighbours, -1.f);
            float tn = 0.f;
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                x[e] *= rstd;             // n
                dw[e] = fmaf(g[e], x[e], dw[e]);
                g[e] *= w[e];
                tn = fmaf(g[e], x[e], tn);
            }
            tn = lanes_sum<LANES>(tn) * inv_dim;
#pragma unroll
            for (int e = 0; e < 16; ++e) x[e] = rstd * (g[e] - x[e] * tn);
            store_chunk(dx0 + row * lddx + at, k, x);
        }
    }
    // the heads of a round lie LANES lanes apart
#pragma unroll
    for (int e = 0; e < 16; ++e) {
#pragma unroll
        for (int m = LANES; m < 64; m *= 2) dw[e] += __shfl_xor(dw[e], m);
        if (lane < LANES) sum[wave][lane * 16 + e] = dw[e];
    }
    __syncthreads();
    for (int j = threadIdx.x; j < LANES * 16; j += kThreads) {
        const int e = j % 16;
        const Chunk m = chunk_of(a, j / 16);
        const int at = e < 8 ? m.o0 + e : m.o1 + e - 8;
        if (e < 8 ? e >= m.n0 : e - 8 >= m.n1) continue;
        float t = 0.f;
#pragma unroll
        for (int v = 0; v < kWaves; ++v) t += sum[v][j];
        a.part[(int64_t)blockIdx.x * a.dim + at] = t;
    }
}

// dw from the groups' sums, in their order: a workgroup takes 16 elements of one weight
// (blockIdx.y), 64 groups at a time.
constexpr int kJoinRows = 64;
template <class W>
__global__ __launch_bounds__(16 * kJoinRows) void k_rotate_join(const float* __restrict__ part, int q_groups,
                                                                int k_groups, int dim, W* __restrict__ dwq,
                                                                W* __restrict__ dwk) {
    __shared__ float sm[kJoinRows][17];
    const int x = threadIdx.x % 16, y = threadIdx.x / 16, i = blockIdx.x * 16 + x;
    const int groups = blockIdx.y ? k_groups : q_groups;
    const float* p = part + (blockIdx.y ? (int64_t)q_groups * dim : 0) + i;
    float t = 0.f;
    if (i < dim) {
#pragma unroll 4
        for (int g = y; g < groups; g += kJoinRows) t += p[(int64_t)g * dim];
    }
    sm[y][x] = t;
    __syncthreads();
    if (y > 0 || i >= dim) return;
    t = 0.f;
#pragma unroll
    for (int j = 0; j < kJoinRows; ++j) t += sm[j][x];
    (blockIdx.y ? dwk : dwq)[i] = (W)t;
}

// Workgroups of the backward, shared by queries and keys as their heads are: the three a CU that
// registers allow (768: 57 us; 512: 66; 1024: 63).
constexpr int64_t kMaxGroups = 768;
struct BackGroups {
    int64_t q, k;
};
inline BackGroups back_groups(int64_t rows, int64_t heads, int64_t kv) {
    const int64_t most = (rows + kWaves - 1) / kWaves;
    const int64_t q = std::max<int64_t>(1, kMaxGroups * heads / (heads + kv));
    return {std::min(most, q), std::min(most, std::max<int64_t>(1, kMaxGroups - q))};
}

template <class T, class W, int LANES>
tt_status rotate_launch(RotateArgs a, bool backward) {
    const int rounds = (a.heads + a.kv * (a.slots ? 2 : 1) + 64 / LANES - 1) / (64 / LANES);
    const dim3 block(kThreads);
    if (backward) {
        const BackGroups g = back_groups(a.rows, a.heads, a.kv);
        a.q_groups = (int)g.q;
        a.k_groups = (int)g.k;
        if (a.rows > 0) {
            TT_LAUNCH(nullptr, "k_rotate_back", a.s, (k_rotate_back<T, W, LANES>), dim3(a.q_groups + a.k_groups), block, 0,
                      a.s, a);
            TT_LAUNCH_CHECK();
        }
        TT_LAUNCH(nullptr, "k_rotate_join", a.s, (k_rotate_join<W>), dim3((a.dim + 15) / 16, 2), dim3(16 * kJoinRows), 0,
                  a.s, a.part, a.q_groups, a.k_groups, a.dim, (W*)a.dwq, (W*)a.dwk);
        TT_LAUNCH_CHECK();
        return TT_OK;
    }
    if (a.rows == 0) return TT_OK;
    // few rows: their heads over more waves
    a.slabs = (int)std::min<int64_t>(rounds, std::max<int64_t>(1, 4096 / a.rows));
    a.per = (rounds + a.slabs - 1) / a.slabs;
    a.slabs = (rounds + a.per - 1) / a.per;
    const int64_t groups = (a.rows * a.slabs + kWaves - 1) / kWaves;
    TT_LAUNCH(nullptr, "k_rotate", a.s, (k_rotate<T, W, LANES>), dim3((unsigned)groups), block, 0, a.s, a);
    TT_LAUNCH_CHECK();
    return TT_OK;
}

template <class T, class W>
tt_status rotate_by_lanes(const RotateArgs& a, bool backward) {
    const int n = chunks_of(a.dim, a.half);
    if (n <= 2) return rotate_launch<T, W, 2>(a, backward);
    if (n <= 4) return rotate_launch<T, W, 4>(a, backward);
    if (n <= 8) return rotate_launch<T, W, 8>(a, backward);
    if (n <= 16) return rotate_launch<T, W, 16>(a, backward);
    return rotate_launch<T, W, 32>(a, backward);
}

tt_status rotate_by_type(int32_t dtype, int32_t wdtype, const RotateArgs& a, bool backward) {
    if (dtype == TT_F32) return rotate_by_lanes<float, float>(a, backward);
    if (dtype == TT_BF16)
        return wdtype == TT_F32 ? rotate_by_lanes<bf16, float>(a, backward) : rotate_by_lanes<bf16, bf16>(a, backward);
    return wdtype == TT_F32 ? rotate_by_lanes<f16, float>(a, backward) : rotate_by_lanes<f16, f16>(a, backward);
}

tt_status rotate_sizes(int32_t dtype, int64_t rows, int64_t heads, int64_t kv, int64_t dim) {
    if (!dtype_ok(dtype) || rows < 0 || heads < 1 || kv < 1 || dim < 1) return TT_ERR_INVALID_ARG;
    // (a row's waves are 2^15 at most, rows that are many have one each)
    if (rows > (int64_t(1) << 24) || heads > 4096 || kv > 4096 || dim > kMaxDim) return TT_ERR_UNSUPPORTED;
    return TT_OK;
}

// The arguments that every call takes.
tt_status rotate_args(RotateArgs& a, int32_t dtype, int32_t wdtype, const void* q, int64_t ldq, const void* k,
                      int64_t ldk, const void* wq, const void* wk, const int64_t* positions, const double* freq,
                      int64_t rot, int32_t pairs, int64_t rows, int64_t heads, int64_t kv, int64_t dim, float eps,
                      void* stream) {
    const tt_status st = rotate_sizes(dtype, rows, heads, kv, dim);
    if (st != TT_OK) return st;
    if (!dtype_ok(wdtype) || rot < 0 || rot > dim || rot % 2 != 0 || !(eps >= 0.f) || eps == INFINITY)
        return TT_ERR_INVALID_ARG;
    if (pairs != TT_PAIRS_HALVES && pairs != TT_PAIRS_NEIGHBOURS) return TT_ERR_INVALID_ARG;
    if (wdtype != dtype && wdtype != TT_F32) return TT_ERR_UNSUPPORTED;
    if (ldq < heads * dim || ldk < kv * dim || !wq || !wk || (rot > 0 && !freq)) return TT_ERR_INVALID_ARG;
    if (rows > 0 && (!q || !k || !positions)) return TT_ERR_INVALID_ARG;
    a = RotateArgs{};
    a.q = q; a.k = k; a.ldq = ldq; a.ldk = ldk;
    a.wq = wq; a.wk = wk; a.positions = positions; a.freq = freq;
    a.rows = rows; a.heads = (int)heads; a.kv = (int)kv; a.dim = (int)dim; a.half = (int)rot / 2;
    a.neighbours = pairs == TT_PAIRS_NEIGHBOURS;
    a.eps = eps;
    a.s = (hipStream_t)stream;
    return TT_OK;
}

}  // namespace
}  // namespace tt

using namespace tt;

extern "C" size_t tt_emb_rotate_workspace_bytes(int32_t dtype, int64_t rows, int64_t heads, int64_t kv_heads,
                                                int64_t dim) {
    if (rotate_sizes(dtype, rows, heads, kv_heads, dim) != TT_OK) return 0;
    const BackGroups g = back_groups(rows, heads, kv_heads);
    return std::max<size_t>(256, ((size_t)(g.q + g.k) * dim * sizeof(float) + 255) & ~size_t(255));
}

extern "C" tt_status tt_emb_rotate_forward(int32_t dtype, int32_t wdtype, const void* q, int64_t ldq, const void* k,
                                           int64_t ldk, const void* q_weight, const void* k_weight,
                                           const int64_t* positions, const double* freq, int64_t rot, int32_t pairs,
                                           void* q_out, int64_t ldqo, void* k_out, int64_t ldko, int64_t rows,
                                           int64_t heads, int64_t kv_heads, int64_t dim, float eps, void* stream) {
    RotateArgs a;
    const tt_status st = rotate_args(a, dtype, wdtype, q, ldq, k, ldk, q_weight, k_weight, positions, freq, rot, pairs,
                                     rows, heads, kv_heads, dim, eps, stream);
    if (st != TT_OK) return st;
    if (ldqo < heads * dim || ldko < kv_heads * dim || (rows > 0 && (!q_out || !k_out))) return TT_ERR_INVALID_ARG;
    a.oq = q_out; a.ldoq = ldqo;
    a.ok = k_out; a.ldok = ldko;
    return rotate_by_type(dtype, wdtype, a, false);
}

extern "C" tt_status tt_emb_rotate_append(int32_t dtype, int32_t wdtype, const void* q, int64_t ldq, const void* k,
                                          int64_t ldk, const void* v, int64_t ldv, const void* q_weight,
                                          const void* k_weight, const int64_t* positions, const double* freq,
                                          int64_t rot, int32_t pairs, const int64_t* slots, void* q_out, int64_t ldqo,
                                          void* k_pages, void* v_pages, int64_t num_slots, int64_t rows, int64_t heads,
                                          int64_t kv_heads, int64_t dim, float eps, void* stream) {
    RotateArgs a;
    const tt_status st = rotate_args(a, dtype, wdtype, q, ldq, k, ldk, q_weight, k_weight, positions, freq, rot, pairs,
                                     rows, heads, kv_heads, dim, eps, stream);
    if (st != TT_OK) return st;
    if (ldqo < heads * dim || ldv < kv_heads * dim || num_slots < 0) return TT_ERR_INVALID_ARG;
    if (rows > 0 && (!v || !q_out || !slots || (num_slots > 0 && (!k_pages || !v_pages)))) return TT_ERR_INVALID_ARG;
    a.v = v; a.ldv = ldv;
    a.oq = q_out; a.ldoq = ldqo;
    a.ok = k_pages; a.ov = v_pages; a.ldok = kv_heads * dim;
    a.slots = slots; a.nslots = num_slots;
    return rotate_by_type(dtype, wdtype, a, false);
}

extern "C" tt_status tt_emb_rotate_backward(int32_t dtype, int32_t wdtype, const void* q, int64_t ldq, const void* k,
                                            int64_t ldk, const void* q_weight, const void* k_weight,
                                            const int64_t* positions, const double* freq, int64_t rot, int32_t pairs,
                                            const void* dq_out, int64_t lddqo, const void* dk_out, int64_t lddko,
                                            void* dq, int64_t lddq, void* dk, int64_t lddk, void* dq_weight,
                                            void* dk_weight, int64_t rows, int64_t heads, int64_t kv_heads, int64_t dim,
                                            float eps, void* workspace, size_t workspace_bytes, void* stream) {
    RotateArgs a;
    const tt_status st = rotate_args(a, dtype, wdtype, q, ldq, k, ldk, q_weight, k_weight, positions, freq, rot, pairs,
                                     rows, heads, kv_heads, dim, eps, stream);
    if (st != TT_OK) return st;
    if (lddqo < heads * dim || lddq < heads * dim || lddko < kv_heads * dim || lddk < kv_heads * dim)
        return TT_ERR_INVALID_ARG;
    if (!dq_weight || !dk_weight || (rows > 0 && (!dq_out || !dk_out || !dq || !dk))) return TT_ERR_INVALID_ARG;
    if (!workspace || ((uintptr_t)workspace & 255) != 0) return TT_ERR_INVALID_ARG;
    if (workspace_bytes < tt_emb_rotate_workspace_bytes(dtype, rows, heads, kv_heads, dim)) return TT_ERR_WORKSPACE;
    a.dyq = dq_out; a.lddyq = lddqo;
    a.dyk = dk_out; a.lddyk = lddko;
    a.oq = dq; a.ldoq = lddq;
    a.ok = dk; a.ldok = lddk;
    a.dwq = dq_weight; a.dwk = dk_weight;
    a.part = (float*)workspace;
    return rotate_by_type(dtype, wdtype, a, true);
}
