// The gated feed-forward block, forward and backward:
//
//   g = x Wg^T,  u = x Wu^T,  out = act(g) u            (x [M][K], Wg, Wu [H][K])
//   dg = dout u act'(g),  du = dout act(g)
//   dx = dg Wg + du Wu,  dWg = dg^T x,  dWu = du^T x
//
// Every product is one matrix-core kernel over operands whose summed index is
// contiguous: D[m][n] = sum_k A[m][k] B[n][k]. The forward has that form as it
// stands and forms both projections in one launch, act(g) u in its epilogue.
// The backward lays out what it needs in the workspace: one pass over g, u and
// dout writes [dg | du] and its transpose, and x and the weights are
// transposed.
//
// Types. bf16 and f16 operands go to the matrix cores as they are; dg and du
// are rounded to them (half a step of 2^-8 or 2^-11, the size of the error that
// the rounding of dx, dWg and dWu themselves has). fp32 operands are cut into
// three bf16 planes, x = x0 + x1 + x2 exactly (8 digits each), and a product
// is the sum of the six plane products down to 2^-16; the three left out are
// below 2^-24 of |a||b|, the rounding of an fp32 product. Six bf16 products
// take 6/16 of the matrix cores' time for an fp32 one. Sums are fp32 throughout.
#include "tt_dense.h"

namespace tt {
namespace {

typedef float floatx4 __attribute__((ext_vector_type(4)));
typedef bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef f16 f16x8 __attribute__((ext_vector_type(8)));

template <class E>
struct Frag;
template <>
struct Frag<bf16> {
    typedef bf16x8 V;
    static __device__ __forceinline__ floatx4 mma(V a, V b, floatx4 c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
    }
};
template <>
struct Frag<f16> {
    typedef f16x8 V;
    static __device__ __forceinline__ floatx4 mma(V a, V b, floatx4 c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
    }
};

// What a tensor of type T is on the matrix cores: E elements, P planes.
template <class T>
struct Mat {
    typedef T E;
    static constexpr int P = 1;
};
template <>
struct Mat<float> {
    typedef bf16 E;
    static constexpr int P = 3;
};

constexpr int kActs = 3;
template <int ACT>
__device__ __forceinline__ float act_of(float g) {
    if (ACT == TT_ACT_SILU) return g / (1.f + expf(-g));
    if (ACT == TT_ACT_GELU) return 0.5f * g * erfcf(-0.70710678118654752f * g);
    return g > 0.f ? g : g == g ? 0.f : g;   // NaN stays NaN
}
// The activation and its derivative.
template <int ACT>
__device__ __forceinline__ void act_grad(float g, float& a, float& da) {
    if (ACT == TT_ACT_SILU) {
        const float s = 1.f / (1.f + expf(-g));
        a = g * s;
        da = s * (1.f + g * (1.f - s));
    } else if (ACT == TT_ACT_GELU) {
        const float cdf = 0.5f * erfcf(-0.70710678118654752f * g);
        a = g * cdf;
        da = cdf + g * (0.39894228040143268f * expf(-0.5f * g * g));
    } else {
        a = g > 0.f ? g : g == g ? 0.f : g;
        da = g > 0.f ? 1.f : 0.f;
    }
}

// ---------------------------------------------------------------------------
// Laying out operands.

// The planes of eight values, written `plane` elements apart.
template <int P, class E>
__device__ __forceinline__ void put_planes(E* __restrict__ dst, int64_t plane, const float (&f)[8]) {
    if constexpr (P == 1) {
        Raw8<E> o;
        o.set(f);
        *reinterpret_cast<Raw8<E>*>(dst) = o;
    } else {
        float o[3][8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float x = f[e];
            bf16 x0 = (bf16)x;
            const bool fin = fabsf(x) <= 3.402823466e38f;
            if (fin && !(fabsf((float)x0) <= 3.402823466e38f))   // rounded up to infinity: cut instead
                x0 = (bf16)__uint_as_float(__float_as_uint(x) & 0xFFFF0000u);
            const float r = fin ? x - (float)x0 : 0.f;
            const bf16 x1 = (bf16)r;
            o[0][e] = (float)x0;
            o[1][e] = (float)x1;
            o[2][e] = r - (float)x1;
        }
#pragma unroll
        for (int p = 0; p < 3; ++p) {
            Raw8<bf16> q;
            q.set(o[p]);
            *reinterpret_cast<Raw8<bf16>*>(dst + p * plane) = q;
        }
    }
}

// dst[p][r][c] for c < ldd: src's rows, zeros past `cols` (ldd a multiple of 64).
template <class T>
__global__ __launch_bounds__(256) void k_gate_pack(const T* __restrict__ src, int64_t ld, int64_t rows, int cols,
                                                   typename Mat<T>::E* __restrict__ dst, int64_t ldd,
                                                   int64_t plane) {
    const int64_t per = ldd / 8, i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    const int64_t r = i / per;
    const int c = (int)(i % per) * 8;
    if (r >= rows) return;
    const Raw8<T> v = load8n(src + r * ld + c, cols - c, (T)0.f);
    float f[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] = v.at(e);
    put_planes<Mat<T>::P>(dst + r * ldd + c, plane, f);
}

// A 64 x 64 tile in LDS, written by rows and read by columns.
struct Tile64 {
    float v[64][65];
};

// dst[p][c][r] for r < rowsp (a multiple of 64): src's columns, zeros past `rows`.
template <class T>
__global__ __launch_bounds__(256) void k_gate_turn(const T* __restrict__ src, int64_t ld, int64_t rows, int cols,
                                                   typename Mat<T>::E* __restrict__ dst, int64_t ldd,
                                                   int64_t plane) {
    __shared__ Tile64 t;
    const int64_t r0 = (int64_t)blockIdx.x * 64;
    const int c0 = blockIdx.y * 64;
    const int a = threadIdx.x >> 3, b = (threadIdx.x & 7) * 8;
#pragma unroll
    for (int i = 0; i < 64; i += 32) {
        const int64_t r = r0 + a + i;
        const Raw8<T> v = load8n(src + r * ld + c0 + b, r < rows ? cols - c0 - b : 0, (T)0.f);
#pragma unroll
        for (int e = 0; e < 8; ++e) t.v[a + i][b + e] = v.at(e);
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 64; i += 32) {
        if (c0 + a + i >= cols) continue;
        float f[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] = t.v[b + e][a + i];
        put_planes<Mat<T>::P>(dst + (int64_t)(c0 + a + i) * ldd + r0 + b, plane, f);
    }
}

// dg and du of a 64 x 64 tile: into gu [M][2 Hp] (dg, then du) and turned into
// gut [2 Hp][Mp]. Zeros in [H, Hp) and in gut past M.
template <class T, int ACT>
__global__ __launch_bounds__(256) void k_gate_grad(const float* __restrict__ gate, const float* __restrict__ up,
                                                   const T* __restrict__ dout, int64_t ldo, int64_t M, int H, int Hp,
                                                   int64_t Mp, typename Mat<T>::E* __restrict__ gu, int64_t gu_plane,
                                                   typename Mat<T>::E* __restrict__ gut, int64_t gut_plane) {
    constexpr int P = Mat<T>::P;
    __shared__ Tile64 tg, tu;
    const int64_t m0 = (int64_t)blockIdx.x * 64;
    const int h0 = blockIdx.y * 64;
    const int a = threadIdx.x >> 3, b = (threadIdx.x & 7) * 8;
#pragma unroll
    for (int i = 0; i < 64; i += 32) {
        const int64_t m = m0 + a + i;
        const int n = m < M ? H - h0 - b : 0;
        const Raw8<float> g = load8n(gate + m * H + h0 + b, n, 0.f);
        const Raw8<float> u = load8n(up + m * H + h0 + b, n, 0.f);
        const Raw8<T> d = load8n(dout + m * ldo + h0 + b, n, (T)0.f);
        float dg[8], du[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            float av, da;
            act_grad<ACT>(g.at(e), av, da);
            const float o = d.at(e);
            dg[e] = e < n ? o * u.at(e) * da : 0.f;
            du[e] = e < n ? o * av : 0.f;
            tg.v[a + i][b + e] = dg[e];
            tu.v[a + i][b + e] = du[e];
        }
        if (m < M) {
            put_planes<P>(gu + m * 2 * Hp + h0 + b, gu_plane, dg);
            put_planes<P>(gu + m * 2 * Hp + Hp + h0 + b, gu_plane, du);
        }
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 64; i += 32) {
        float fg[8], fu[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            fg[e] = tg.v[b + e][a + i];
            fu[e] = tu.v[b + e][a + i];
        }
        put_planes<P>(gut + (int64_t)(h0 + a + i) * Mp + m0 + b, gut_plane, fg);
        put_planes<P>(gut + (int64_t)(Hp + h0 + a + i) * Mp + m0 + b, gut_plane, fu);
    }
}

// ---------------------------------------------------------------------------
// The product. A workgroup of four waves forms a 128 x 128 tile of D, 64 of
// the summed index at a time: both operands' tiles go from memory straight to
// LDS, the next ones while the matrix cores work on these. A tile's row is 128
// bytes, eight 16-byte pieces that are stored in the order piece ^ key(row),
// so that the 16 rows a wave reads at once lie in different banks.

constexpr int kBK = 64;

struct Operand {
    const void* p;     // rows of `ld` elements, the summed index contiguous
    int64_t ld, plane; // elements from row to row, from plane to plane
    int64_t rows;      // rows past the last one are read as the last one (their results are dropped)
};

struct Product {
    Operand a, b, b2;   // b2: the second projection's weight (forward)
    int64_t M;
    int N, kp;          // kp: summed length, a multiple of kBK (both operands hold zeros past the real one)
    void *out, *out2;   // out2: of the second half of a's rows (weight gradients), blockIdx.z = 1
    int64_t ldo;
    float *gate, *up;   // forward, or null: g and u, [M][N]
};

enum { EPI_FWD, EPI_OUT };

// The planes of the six products of fp32 operands, the smallest products first.
__device__ __forceinline__ int plane_a(int s) { return (0x001102 >> (4 * s)) & 3; }   // 2 0 1 1 0 0
__device__ __forceinline__ int plane_b(int s) { return (0x010120 >> (4 * s)) & 3; }   // 0 2 1 0 1 0

template <int ROWS, int GROUP>
__device__ __forceinline__ int lds_key(int row) {
    return (row & 3) | (((row / GROUP) & 1) << 2);
}

// Loads a wave's part of a ROWS x kBK tile: offsets of its 16-byte pieces
// (bytes from the tile's first row), one instruction for 8 rows.
template <int ROWS, int GROUP, int WAVES>
struct TileLoad {
    static constexpr int N = ROWS / 8 / WAVES;
    uint32_t off[N];
    const char* base;
    __device__ __forceinline__ void init(const Operand& o, int64_t row0) {
        base = (const char*)o.p + row0 * o.ld * 2;
        const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int r = (wave * N + i) * 8 + (lane >> 3), c = (lane & 7) ^ lds_key<ROWS, GROUP>(r);
            const int64_t last = o.rows - 1 - row0;
            off[i] = (uint32_t)((r < last ? r : last) * o.ld * 2 + c * 16);
        }
    }
    // k: bytes along the row (and to the plane)
    __device__ __forceinline__ void load(char* lds, int64_t k) const {
        const int wave = threadIdx.x >> 6;
#pragma unroll
        for (int i = 0; i < N; ++i)
            __builtin_amdgcn_global_load_lds((__attribute__((address_space(1))) void*)(base + k + off[i]),
                                             (__attribute__((address_space(3))) void*)(lds + (wave * N + i) * 1024),
                                             16, 0, 0);
    }
};

__device__ __forceinline__ void loads_done_barrier() {
    __builtin_amdgcn_s_waitcnt(0x0f70);   // vmcnt(0): this wave's loads to LDS have landed
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup");
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup");
}

template <class T, int EPI, int ACT>
__global__ __launch_bounds__(256, 2) void k_gate_mm(const Product q) {
    typedef typename Mat<T>::E E;
    typedef typename Frag<E>::V V;
    constexpr int P = Mat<T>::P, SEGS = P == 1 ? 1 : 6;
    constexpr int TM = 128, TN = 128, FM = 4, FN = 4, WAVES = 4;
    constexpr int FH = EPI == EPI_FWD ? FN / 2 : FN;   // fragments of consecutive columns
    constexpr int GROUP = 4 * FH;                      // consecutive columns a lane ends up with
    constexpr int NB = EPI == EPI_FWD ? TN / 2 : TN;   // columns of D a workgroup forms
    __shared__ __align__(16) char sa0[TM * 128], sb0[TN * 128], sa1[TM * 128], sb1[TN * 128];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, wm = wave >> 1, wn = wave & 1;
    const int n0 = blockIdx.x * NB;
    const int64_t m0 = (int64_t)blockIdx.y * TM;
    Operand oa = q.a;
    if (EPI == EPI_OUT) oa.p = (const char*)oa.p + blockIdx.z * oa.rows * oa.ld * 2;

    TileLoad<TM, 4, WAVES> la;
    TileLoad<NB, GROUP, WAVES> lb, lb2;
    la.init(oa, m0);
    lb.init(q.b, n0);
    if (EPI == EPI_FWD) lb2.init(q.b2, n0);
    const int nk = q.kp / kBK, steps = nk * SEGS;
    auto load = [&](char* sa, char* sb, int step) {
        const int s = SEGS == 1 ? 0 : step / nk;
        const int64_t k = (int64_t)(step - s * nk) * (kBK * 2);
        la.load(sa, k + (SEGS == 1 ? 0 : plane_a(s) * oa.plane * 2));
        lb.load(sb, k + (SEGS == 1 ? 0 : plane_b(s) * q.b.plane * 2));
        if (EPI == EPI_FWD) lb2.load(sb + NB * 128, k + (SEGS == 1 ? 0 : plane_b(s) * q.b2.plane * 2));
    };

    floatx4 acc[FM][FN];
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j) acc[i][j] = floatx4{0.f, 0.f, 0.f, 0.f};

    const int li = lane & 15, lk = lane >> 4;
    auto compute = [&](const char* sa, const char* sb) {
#pragma unroll
        for (int h = 0; h < kBK / 32; ++h) {
            V fa[FM], fb[FN];
#pragma unroll
            for (int i = 0; i < FM; ++i) {
                const int r = wm * FM * 16 + i * 16 + li;
                fa[i] = *reinterpret_cast<const V*>(sa + r * 128 + ((h * 4 + lk) ^ lds_key<TM, 4>(r)) * 16);
            }
#pragma unroll
            for (int j = 0; j < FN; ++j) {
                const int w = wn * FH * 16 + (li >> 2) * GROUP + (j % FH) * 4 + (li & 3);
                const int r = (j / FH) * NB + w;
                fb[j] = *reinterpret_cast<const V*>(sb + r * 128 + ((h * 4 + lk) ^ lds_key<NB, GROUP>(w)) * 16);
            }
#pragma unroll
            for (int i = 0; i < FM; ++i)
#pragma unroll
                for (int j = 0; j < FN; ++j) acc[i][j] = Frag<E>::mma(fb[j], fa[i], acc[i][j]);
        }
    };

    if (steps > 0) load(sa0, sb0, 0);
    for (int s = 0; s < steps; s += 2) {
        loads_done_barrier();
        if (s + 1 < steps) load(sa1, sb1, s + 1);
        compute(sa0, sb0);
        if (s + 1 >= steps) break;
        loads_done_barrier();
        if (s + 2 < steps) load(sa0, sb0, s + 2);
        compute(sa1, sb1);
    }

    // acc[i][j][r] is D[m][n] with m = .. + i*16 + lane%16 and n consecutive over (j, r)
    const int nb = n0 + wn * FH * 16 + lk * GROUP;
#pragma unroll
    for (int i = 0; i < FM; ++i) {
        const int64_t m = m0 + wm * FM * 16 + i * 16 + li;
        if (m >= q.M) continue;
        T* po = (T*)(blockIdx.z ? q.out2 : q.out) + m * q.ldo + nb;
#pragma unroll
        for (int v = 0; v < GROUP; v += 8) {
            const int n = q.N - nb - v;
            if (n <= 0) continue;
            float o[8], g[8], u[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int j = (v + e) / 4, r = e & 3;
                if constexpr (EPI == EPI_FWD) {
                    g[e] = acc[i][j][r];
                    u[e] = acc[i][j + FH][r];
                    o[e] = act_of<ACT>(g[e]) * u[e];
                } else {
                    o[e] = acc[i][j][r];
                }
            }
            store8n(po + v, o, n);
            if constexpr (EPI == EPI_FWD)
                if (q.gate) {
                    store8n(q.gate + m * q.N + nb + v, g, n);
                    store8n(q.up + m * q.N + nb + v, u, n);
                }
        }
    }
}

// ---------------------------------------------------------------------------
// Host side.

inline int64_t up64(int64_t n) { return (n + 63) & ~int64_t(63); }

// Where the operands lie in the workspace (offsets in bytes, 0 where a
// direction does not need them).
struct GateSpace {
    int64_t Kp, Hp, Mp;
    size_t x, w, w2, forward;                 // packed operands of the forward
    size_t gu, gut, wt, xt, backward;         // of the backward
    GateSpace(int32_t dtype, int64_t M, int64_t K, int64_t H) {
        const size_t e = dtype == TT_F32 ? 6 : 2;   // bytes of an element, all planes
        Kp = up64(K);
        Hp = up64(H);
        Mp = up64(M);
        size_t at = 0;
        auto take = [&](int64_t n) {
            const size_t o = at;
            at += ((size_t)n * e + 255) & ~size_t(255);
            return o;
        };
        x = take(M * Kp);
        w = take(H * Kp);
        w2 = take(H * Kp);
        forward = at;
        at = 0;
        gu = take(M * 2 * Hp);
        gut = take(2 * Hp * Mp);
        wt = take(K * 2 * Hp);
        xt = take(K * Mp);
        backward = at;
    }
};

struct GateArgs {
    const void *x, *wg, *wu, *dout;
    void *out, *dx, *dwg, *dwu;
    int64_t ldx, ldout, lddout, lddx, M, K, H;
    float *gate, *up;
    int act;
    char* ws;
    hipStream_t s;
};

// Operand rows as they are, or packed into `dst`, when their alignment or
// width does not suit the product's loads.
template <class T>
tt_status as_operand(Operand& o, const void* src, int64_t ld, int64_t rows, int64_t cols, char* dst, hipStream_t s) {
    const int64_t cp = up64(cols);
    if (Mat<T>::P == 1 && cols % kBK == 0 && ld % 8 == 0 && ((uintptr_t)src & 15) == 0) {
        o = Operand{src, ld, 0, rows};
        return TT_OK;
    }
    o = Operand{dst, cp, rows * cp, rows};
    TT_LAUNCH(nullptr, "k_gate_pack", s, (k_gate_pack<T>), dim3(grid_for(rows * (cp / 8), 256)), dim3(256), 0, s,
              (const T*)src, ld, rows, (int)cols, (typename Mat<T>::E*)dst, cp, rows * cp);
    TT_LAUNCH_CHECK();
    return TT_OK;
}

template <class T>
tt_status turn(const void* src, int64_t ld, int64_t rows, int64_t cols, char* dst, int64_t ldd, int64_t plane,
               hipStream_t s) {
    if (rows == 0) return TT_OK;
    TT_LAUNCH(nullptr, "k_gate_turn", s, (k_gate_turn<T>), dim3(grid_for(rows, 64), grid_for(cols, 64)), dim3(256),
              0, s, (const T*)src, ld, rows, (int)cols, (typename Mat<T>::E*)dst, ldd, plane);
    TT_LAUNCH_CHECK();
    return TT_OK;
}

template <class T, int EPI, int ACT>
tt_status product(const Product& q, int z, hipStream_t s) {
    const int nb = EPI == EPI_FWD ? 64 : 128;
    TT_LAUNCH(nullptr, "k_gate_mm", s, (k_gate_mm<T, EPI, ACT>),
              dim3(grid_for(q.N, nb), grid_for(q.M, 128), z), dim3(256), 0, s, q);
    TT_LAUNCH_CHECK();
    return TT_OK;
}

template <class T, int ACT>
tt_status gate_forward(const GateArgs& a, const GateSpace& sp) {
    Product q{};
    tt_status st = as_operand<T>(q.a, a.x, a.ldx, a.M, a.K, a.ws + sp.x, a.s);
    if (st == TT_OK) st = as_operand<T>(q.b, a.wg, a.K, a.H, a.K, a.ws + sp.w, a.s);
    if (st == TT_OK) st = as_operand<T>(q.b2, a.wu, a.K, a.H, a.K, a.ws + sp.w2, a.s);
    if (st != TT_OK) return st;
    q.M = a.M;
    q.N = (int)a.H;
    q.kp = (int)sp.Kp;
    q.out = a.out;
    q.ldo = a.ldout;
    q.gate = a.gate;
    q.up = a.up;
    return product<T, EPI_FWD, ACT>(q, 1, a.s);
}

template <class T, int ACT>
tt_status gate_backward(const GateArgs& a, const GateSpace& sp) {
    typedef typename Mat<T>::E E;
    const int64_t gu_plane = a.M * 2 * sp.Hp, gut_plane = 2 * sp.Hp * sp.Mp, wt_plane = a.K * 2 * sp.Hp,
                  xt_plane = a.K * sp.Mp;
    E *gu = (E*)(a.ws + sp.gu), *gut = (E*)(a.ws + sp.gut);
    char *wt = a.ws + sp.wt, *xt = a.ws + sp.xt;
    tt_status st = turn<T>(a.x, a.ldx, a.M, a.K, xt, sp.Mp, xt_plane, a.s);
    if (a.M > 0) {
        TT_LAUNCH(nullptr, "k_gate_grad", a.s, (k_gate_grad<T, ACT>), dim3(grid_for(a.M, 64), grid_for(a.H, 64)),
                  dim3(256), 0, a.s, a.gate, a.up, (const T*)a.dout, a.lddout, a.M, (int)a.H, (int)sp.Hp, sp.Mp, gu,
                  gu_plane, gut, gut_plane);
        TT_LAUNCH_CHECK();
        // the turned weights side by side: [K][Hp of Wg | Hp of Wu]
        if (st == TT_OK) st = turn<T>(a.wg, a.K, a.H, a.K, wt, 2 * sp.Hp, wt_plane, a.s);
        if (st == TT_OK) st = turn<T>(a.wu, a.K, a.H, a.K, wt + sp.Hp * 2, 2 * sp.Hp, wt_plane, a.s);
        Product q{};
        q.a = Operand{gu, 2 * sp.Hp, gu_plane, a.M};
        q.b = Operand{wt, 2 * sp.Hp, wt_plane, a.K};
        q.M = a.M;
        q.N = (int)a.K;
        q.kp = (int)(2 * sp.Hp);
        q.out = a.dx;
        q.ldo = a.lddx;
        if (st == TT_OK) st = product<T, EPI_OUT, 0>(q, 1, a.s);
    }
    if (st != TT_OK) return st;
    Product q{};
    q.a = Operand{gut, sp.Mp, gut_plane, sp.Hp};
    q.b = Operand{xt, sp.Mp, xt_plane, a.K};
    q.M = a.H;
    q.N = (int)a.K;
    q.kp = (int)sp.Mp;
    q.out = a.dwg;
    q.out2 = a.dwu;
    q.ldo = a.K;
    return product<T, EPI_OUT, 0>(q, 2, a.s);
}

template <class T, int ACT>
tt_status gate_run(const GateArgs& a, const GateSpace& sp, bool backward) {
    return backward ? gate_backward<T, ACT>(a, sp) : gate_forward<T, ACT>(a, sp);
}

template <class T>
tt_status gate_by_act(const GateArgs& a, const GateSpace& sp, bool backward) {
    if (a.act == TT_ACT_SILU) return gate_run<T, TT_ACT_SILU>(a, sp, backward);
    if (a.act == TT_ACT_GELU) return gate_run<T, TT_ACT_GELU>(a, sp, backward);
    return gate_run<T, TT_ACT_RELU>(a, sp, backward);
}

tt_status gate_by_type(int32_t dtype, const GateArgs& a, bool backward) {
    const GateSpace sp(dtype, a.M, a.K, a.H);
    if (dtype == TT_F32) return gate_by_act<float>(a, sp, backward);
    if (dtype == TT_BF16) return gate_by_act<bf16>(a, sp, backward);
    return gate_by_act<f16>(a, sp, backward);
}

constexpr int64_t kGateMaxWidth = 1 << 20;
constexpr int64_t kGateMaxRows = int64_t(1) << 22;   // 64-row tiles within a grid's second dimension

tt_status gate_check(int32_t dtype, int64_t M, int64_t K, int64_t H) {
    if (!dtype_ok(dtype) || M < 0 || K < 1 || H < 1) return TT_ERR_INVALID_ARG;
    if (M >= kGateMaxRows || K >= kGateMaxWidth || H >= kGateMaxWidth) return TT_ERR_UNSUPPORTED;
    return TT_OK;
}

// A row stride that the product's 32-bit offsets within a tile can take.
bool stride_ok(int64_t ld) { return ld < (int64_t(1) << 22); }

}  // namespace
}  // namespace tt

using namespace tt;

extern "C" size_t tt_emb_gate_workspace_bytes(int32_t dtype, int64_t rows, int64_t dim, int64_t hidden) {
    if (gate_check(dtype, rows, dim, hidden) != TT_OK) return 0;
    const GateSpace sp(dtype, rows, dim, hidden);
    return std::max<size_t>(256, std::max(sp.forward, sp.backward));
}

extern "C" tt_status tt_emb_gate_forward(int32_t dtype, const void* x, int64_t ldx, const void* w_gate,
                                         const void* w_up, void* out, int64_t ldout, float* gate, float* up,
                                         int64_t rows, int64_t dim, int64_t hidden, int32_t act, void* workspace,
                                         size_t workspace_bytes, void* stream) {
    const tt_status st = gate_check(dtype, rows, dim, hidden);
    if (st != TT_OK) return st;
    if (act < 0 || act >= kActs || !w_gate || !w_up || ldx < dim || ldout < hidden || !gate != !up)
        return TT_ERR_INVALID_ARG;
    if ((rows > 0 && (!x || !out)) || !workspace || ((uintptr_t)workspace & 255) != 0) return TT_ERR_INVALID_ARG;
    if (!stride_ok(ldx)) return TT_ERR_UNSUPPORTED;
    if (workspace_bytes < tt_emb_gate_workspace_bytes(dtype, rows, dim, hidden)) return TT_ERR_WORKSPACE;
    if (rows == 0) return TT_OK;
    GateArgs a{};
    a.x = x; a.wg = w_gate; a.wu = w_up; a.out = out;
    a.ldx = ldx; a.ldout = ldout; a.M = rows; a.K = dim; a.H = hidden;
    a.gate = gate; a.up = up; a.act = act; a.ws = (char*)workspace; a.s = (hipStream_t)stream;
    return gate_by_type(dtype, a, false);
}

extern "C" tt_status tt_emb_gate_backward(int32_t dtype, const void* x, int64_t ldx, const void* w_gate,
                                          const void* w_up, const float* gate, const float* up, const void* dout,
                                          int64_t lddout, void* dx, int64_t lddx, void* dw_gate, void* dw_up,
                                          int64_t rows, int64_t dim, int64_t hidden, int32_t act, void* workspace,
                                          size_t workspace_bytes, void* stream) {
    const tt_status st = gate_check(dtype, rows, dim, hidden);
    if (st != TT_OK) return st;
    if (act < 0 || act >= kActs || !w_gate || !w_up || !dw_gate || !dw_up || ldx < dim || lddout < hidden ||
        lddx < dim)
        return TT_ERR_INVALID_ARG;
    if (rows > 0 && (!x || !gate || !up || !dout || !dx)) return TT_ERR_INVALID_ARG;
    if (!workspace || ((uintptr_t)workspace & 255) != 0) return TT_ERR_INVALID_ARG;
    if (!stride_ok(ldx)) return TT_ERR_UNSUPPORTED;
    if (workspace_bytes < tt_emb_gate_workspace_bytes(dtype, rows, dim, hidden)) return TT_ERR_WORKSPACE;
    GateArgs a{};
    a.x = x; a.wg = w_gate; a.wu = w_up; a.dout = dout; a.dx = dx; a.dwg = dw_gate; a.dwu = dw_up;
    a.ldx = ldx; a.lddout = lddout; a.lddx = lddx; a.M = rows; a.K = dim; a.H = hidden;
    a.gate = const_cast<float*>(gate); a.up = const_cast<float*>(up);
    a.act = act; a.ws = (char*)workspace; a.s = (hipStream_t)stream;
    return gate_by_type(dtype, a, true);
}
