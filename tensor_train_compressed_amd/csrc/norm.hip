// Layer norm over the last dimension, forward and backward, with the
// reduction of the weight's and the bias's gradients.
//
//   mean = sum_j x_j / n,  var = sum_j (x_j - mean)^2 / n,  rstd = 1/sqrt(var + eps)
//   xhat = (x - mean) rstd,  y = xhat w + b
//   a = dy w,  dx = rstd (a - sum(a)/n - xhat sum(a xhat)/n)
//   dw_j = sum_rows dy_j xhat_j,  db_j = sum_rows dy_j
//
// Everything is held in fp32; inputs and outputs are rounded once, at the
// store. Both passes are bound by memory: a row is read once and stays in the
// registers of the threads that share it. The variance is formed from the
// centred values there, not from a sum of squares, which would lose the digits
// of rows with a large offset; the centred values' own mean, what the first sum
// was off by, is taken off them too. The threads of a workgroup keep their columns
// for all the rows they take, so that w and b are read once a thread, and dw
// and db are summed in registers over those rows.
#include "tt_dense.h"

namespace tt {
namespace {

// How many threads share a row, and how many elements each of them holds:
// rows up to 256 wide take 16 or 32 lanes (four or two rows a wave), wider ones a
// wave or a workgroup (65536 x 256 bf16 backward 21 us on 32 lanes, 44 on 64 of
// which half have no element). 8 or 16 elements a thread keep the backward, which holds x
// and dy of its columns in their own type and w, dw and db, under 128 registers.
struct NormShape {
    int threads, elems;
};
inline NormShape norm_shape(int64_t dim) {
    if (dim <= 128) return {16, 8};
    if (dim <= 256) return {32, 8};
    if (dim <= 512) return {64, 8};
    if (dim <= 1024) return {64, 16};
    if (dim <= 2048) return {256, 8};
    if (dim <= 4096) return {256, 16};
    if (dim <= 8192) return {512, 16};
    return {1024, 16};
}
constexpr int64_t kNormMaxDim = 16384;

template <int TPR>
constexpr int norm_block() {
    return TPR < 256 ? 256 : TPR;
}

// Sums of two values over the TPR threads of a row. Rows of more than a wave
// go through LDS; `slot` alternates between calls, so that one barrier a call
// is enough (a slot is written again two calls later, after a barrier that
// every reader of it has passed).
template <int TPR>
__device__ __forceinline__ void row_sum2(float& a, float& b, float (*sm)[2][16], int& slot) {
    constexpr int W = TPR < 64 ? TPR : 64;
    a = lanes_sum<W>(a);
    b = lanes_sum<W>(b);
    if constexpr (TPR > 64) {
        const int wave = threadIdx.x >> 6;
        if ((threadIdx.x & 63) == 0) {
            sm[slot][0][wave] = a;
            sm[slot][1][wave] = b;
        }
        __syncthreads();
        a = b = 0.f;
#pragma unroll
        for (int w = 0; w < TPR / 64; ++w) {
            a += sm[slot][0][w];
            b += sm[slot][1][w];
        }
        slot ^= 1;
    }
}

template <class T, class WT, int TPR, int E>
__global__ __launch_bounds__(norm_block<TPR>()) void k_norm_fwd(
    const T* __restrict__ x, int64_t ldx, const WT* __restrict__ weight, const WT* __restrict__ bias,
    T* __restrict__ y, int64_t ldy, float* __restrict__ mean_out, float* __restrict__ rstd_out, int64_t rows,
    int dim, float eps) {
    constexpr int GPB = norm_block<TPR>() / TPR, NV = E / 8;
    __shared__ float sm[2][2][16];
    int slot = 0;
    const int t = threadIdx.x % TPR;
    const float inv_n = 1.f / (float)dim;
    float w[E], b[E];
#pragma unroll
    for (int v = 0; v < NV; ++v) {
        const int c = (v * TPR + t) * 8, n = dim - c;
        const Raw8<WT> rw = load8n(weight + c, n, (WT)0.f);
        const Raw8<WT> rb = bias ? load8n(bias + c, n, (WT)0.f) : Raw8<WT>{};
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            w[v * 8 + e] = rw.at(e);
            b[v * 8 + e] = bias ? rb.at(e) : 0.f;
        }
    }
    Raw8<T> rx[NV];
    auto fetch = [&](int64_t r) {
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int c = (v * TPR + t) * 8;
            rx[v] = load8n(x + r * ldx + c, dim - c, (T)0.f);
        }
    };
    // rows of one wave or less need no barrier, so its groups may end apart
    const int64_t step = (int64_t)gridDim.x * GPB;
    int64_t r = (int64_t)blockIdx.x * GPB + threadIdx.x / TPR;
    if (r < rows) fetch(r);
    for (; r < rows; r += step) {
        float f[E];
        float s = 0.f, q = 0.f;
#pragma unroll
        for (int v = 0; v < NV; ++v)
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                f[v * 8 + e] = rx[v].at(e);
                s += f[v * 8 + e];
            }
        if (r + step < rows) fetch(r + step);   // under way while this row is reduced
        row_sum2<TPR>(s, q, sm, slot);
        float mean = s * inv_n, var = 0.f;
        mean = fmaf(fmaf(-mean, (float)dim, s), inv_n, mean);   // s / n: a row of one value has that mean
        s = 0.f;
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int n = dim - (v * TPR + t) * 8;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float d = f[v * 8 + e] - mean;
                f[v * 8 + e] = d;
                if (e < n) {
                    s += d;
                    var += d * d;
                }
            }
        }
        row_sum2<TPR>(s, var, sm, slot);
        const float off = s * inv_n;
        mean += off;
        var -= s * off;
        const float rstd = 1.f / sqrtf((var < 0.f ? 0.f : var) * inv_n + eps);
        T* py = y + r * ldy;
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int c = (v * TPR + t) * 8;
            float o[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) o[e] = (f[v * 8 + e] - off) * rstd * w[v * 8 + e] + b[v * 8 + e];
            store8n(py + c, o, dim - c);
        }
        if (t == 0 && mean_out) {
            mean_out[r] = mean;
            rstd_out[r] = rstd;
        }
    }
}

// The workgroup's sums of dw and db go to part[blockIdx.x][0 or 1][dim], those of an
// only workgroup straight to dweight and dbias.
// 16384 x 4096 bf16: 83 us, 4.8 TB/s, what a large copy reaches; with the next two
// rows under way instead of one the same, and 32768 x 128 fp32 10.6 us for 8.9.
template <class T, class WT, int TPR, int E>
__global__ __launch_bounds__(norm_block<TPR>()) void k_norm_bwd(
    const T* __restrict__ x, int64_t ldx, const WT* __restrict__ weight, const float* __restrict__ mean_in,
    const float* __restrict__ rstd_in, const T* __restrict__ dy, int64_t lddy, T* __restrict__ dx, int64_t lddx,
    float* __restrict__ part, WT* __restrict__ dweight, WT* __restrict__ dbias, int64_t rows, int dim) {
    constexpr int GPB = norm_block<TPR>() / TPR, NV = E / 8;
    __shared__ float sm[2][2][16];
    int slot = 0;
    const int t = threadIdx.x % TPR;
    const float inv_n = 1.f / (float)dim;
    float w[E], dw[E], db[E];
#pragma unroll
    for (int v = 0; v < NV; ++v) {
        const int c = (v * TPR + t) * 8;
        const Raw8<WT> rw = load8n(weight + c, dim - c, (WT)0.f);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            w[v * 8 + e] = rw.at(e);
            dw[v * 8 + e] = db[v * 8 + e] = 0.f;
        }
    }
    // a row's x and dy stay as they were read, and are unpacked before and after the
    // sums; the next row's are under way meanwhile where registers allow it (4096 x
    // 16384 fp32 264 us with them spilt, 190 without the next row; bf16 142 and 112)
    constexpr bool AHEAD = TPR < 1024;
    Raw8<T> nx[NV], ng[NV];
    float mean_n, rstd_n;
    auto fetch = [&](int64_t r) {
        mean_n = mean_in[r];
        rstd_n = rstd_in[r];
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int c = (v * TPR + t) * 8, n = dim - c;
            // past the row's end x is its last value: its xhat is as large as the others', where
            // that of 0 may be infinite (a row of one value, far from 0: rstd is 1/sqrt(eps))
            nx[v] = load8n(x + r * ldx + c, n, n < 8 ? x[r * ldx + dim - 1] : (T)0.f);
            ng[v] = load8n(dy + r * lddy + c, n, (T)0.f);
        }
    };
    const int64_t step = (int64_t)gridDim.x * GPB;
    int64_t r = (int64_t)blockIdx.x * GPB + threadIdx.x / TPR;
    if (AHEAD && r < rows) fetch(r);
    for (; r < rows; r += step) {
        if (!AHEAD) fetch(r);
        const float mean = mean_n, rstd = rstd_n;
        Raw8<T> rx[NV], rg[NV];
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            rx[v] = nx[v];
            rg[v] = ng[v];
        }
        if (AHEAD && r + step < rows) fetch(r + step);
        float s = 0.f, q = 0.f;
#pragma unroll
        for (int v = 0; v < NV; ++v)
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int k = v * 8 + e;
                const float g = rg[v].at(e), h = (rx[v].at(e) - mean) * rstd;   // dy (0 past the row's end), xhat
                const float a = g * w[k];
                s += a;
                q += a * h;
                dw[k] += g * h;
                db[k] += g;
            }
        row_sum2<TPR>(s, q, sm, slot);
        s *= inv_n;
        q *= inv_n;
        keep_raw(rx);
        keep_raw(rg);
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int c = (v * TPR + t) * 8;
            float o[8];
#pragma unroll
            for (int e = 0; e < 8; ++e)
                o[e] = rstd * (rg[v].at(e) * w[v * 8 + e] - s - (rx[v].at(e) - mean) * rstd * q);
            store8n(dx + r * lddx + c, o, dim - c);
        }
    }
    float* pw = part + (int64_t)blockIdx.x * 2 * dim;
    auto put = [&](int k, int c, float a) {
        if (gridDim.x > 1) pw[k * dim + c] = a;
        else if (k == 0) dweight[c] = (WT)a;
        else if (dbias) dbias[c] = (WT)a;
    };
    if constexpr (GPB == 1) {
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int c = (v * TPR + t) * 8;
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (c + e < dim) {
                    put(0, c + e, dw[v * 8 + e]);
                    put(1, c + e, db[v * 8 + e]);
                }
        }
    } else {
        // the workgroup's groups hold the same columns: sum them in order
        constexpr int COLS = TPR * E;
        __shared__ float sw[GPB][2][COLS];
        const int g = threadIdx.x / TPR;
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int c = (v * TPR + t) * 8;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                sw[g][0][c + e] = dw[v * 8 + e];
                sw[g][1][c + e] = db[v * 8 + e];
            }
        }
        __syncthreads();
        for (int i = threadIdx.x; i < 2 * COLS; i += norm_block<TPR>()) {
            const int k = i / COLS, c = i % COLS;
            if (c >= dim) continue;
            float a = 0.f;
#pragma unroll
            for (int j = 0; j < GPB; ++j) a += sw[j][k][c];
            put(k, c, a);
        }
    }
}

// Sums the workgroups' parts over `parts` in a fixed order: 16 columns a
// workgroup, its 64 rows of threads each taking every 64th part.
template <class WT>
__global__ __launch_bounds__(1024) void k_norm_wgrad(const float* __restrict__ part, int parts, int dim,
                                                     WT* __restrict__ dweight, WT* __restrict__ dbias) {
    __shared__ float sm[64][17];
    const int lc = threadIdx.x & 15, s = threadIdx.x >> 4;
    const int c = blockIdx.x * 16 + lc, k = blockIdx.y;
    float a = 0.f;
    if (c < dim)
#pragma unroll 8
        for (int p = s; p < parts; p += 64) a += part[((int64_t)p * 2 + k) * dim + c];
    sm[s][lc] = a;
    __syncthreads();
    for (int d = 32; d > 0; d >>= 1) {
        if (s < d) sm[s][lc] += sm[s + d][lc];
        __syncthreads();
    }
    if (s == 0 && c < dim) (k ? dbias : dweight)[c] = (WT)sm[0][lc];
}

// Workgroups of the backward (and parts of dw, db): two of 256 threads a CU,
// fewer of the larger ones, so that the parts stay small beside the rows. A single
// one for a few rows a group, which needs no second launch: 64 x 128 fp32 11.3 ->
// 8.8 us, 4 x 4096 11.4 -> 10.3 (but 32 x 1000 10.9 -> 13.5, 4 x 16384 25.0 -> 27.9).
inline int64_t norm_bwd_blocks(int64_t rows, int64_t dim) {
    const NormShape sh = norm_shape(dim);
    const int64_t gpb = sh.threads < 256 ? 256 / sh.threads : 1;
    const int64_t most = sh.threads <= 512 ? 512 : 256;
    const int64_t n = (rows + gpb - 1) / gpb;
    const int64_t one = sh.threads <= 32 ? 8 : sh.threads <= 256 ? 4 : 1;
    return n <= one ? std::min<int64_t>(n, 1) : std::min(most, n);
}

inline int64_t norm_fwd_blocks(int64_t rows, int64_t dim) {
    const NormShape sh = norm_shape(dim);
    const int64_t gpb = sh.threads < 256 ? 256 / sh.threads : 1;
    const int64_t most = sh.threads <= 256 ? 2048 : sh.threads == 512 ? 1024 : 512;
    return std::min(most, (rows + gpb - 1) / gpb);
}

struct NormArgs {
    const void *x, *weight, *bias, *dy;
    void *y, *dx, *dweight, *dbias;
    int64_t ldx, ldy, lddy, lddx, rows, dim;
    float *mean, *rstd, *part;
    float eps;
    hipStream_t s;
};

template <class T, class WT, int TPR, int E>
tt_status norm_launch(const NormArgs& a, bool backward) {
    constexpr int BLOCK = norm_block<TPR>();
    if (!backward) {
        const unsigned grid = (unsigned)norm_fwd_blocks(a.rows, a.dim);
        TT_LAUNCH(nullptr, "k_norm_fwd", a.s, (k_norm_fwd<T, WT, TPR, E>), dim3(grid), dim3(BLOCK), 0, a.s,
                  (const T*)a.x, a.ldx, (const WT*)a.weight, (const WT*)a.bias, (T*)a.y, a.ldy, a.mean, a.rstd,
                  a.rows, (int)a.dim, a.eps);
        TT_LAUNCH_CHECK();
        return TT_OK;
    }
    const unsigned grid = (unsigned)norm_bwd_blocks(a.rows, a.dim);   // 0 rows: no parts, zero gradients
    if (grid) {
        TT_LAUNCH(nullptr, "k_norm_bwd", a.s, (k_norm_bwd<T, WT, TPR, E>), dim3(grid), dim3(BLOCK), 0, a.s,
                  (const T*)a.x, a.ldx, (const WT*)a.weight, a.mean, a.rstd, (const T*)a.dy, a.lddy, (T*)a.dx,
                  a.lddx, a.part, (WT*)a.dweight, (WT*)a.dbias, a.rows, (int)a.dim);
        TT_LAUNCH_CHECK();
        if (grid == 1) return TT_OK;
    }
    TT_LAUNCH(nullptr, "k_norm_wgrad", a.s, (k_norm_wgrad<WT>), dim3(grid_for(a.dim, 16), a.dbias ? 2 : 1),
              dim3(1024), 0, a.s, a.part, (int)grid, (int)a.dim, (WT*)a.dweight, (WT*)a.dbias);
    TT_LAUNCH_CHECK();
    return TT_OK;
}

template <class T, class WT>
tt_status norm_by_shape(const NormArgs& a, bool backward) {
    const NormShape sh = norm_shape(a.dim);
    switch (sh.threads) {
        case 16: return norm_launch<T, WT, 16, 8>(a, backward);
        case 32: return norm_launch<T, WT, 32, 8>(a, backward);
        case 64: return sh.elems == 8 ? norm_launch<T, WT, 64, 8>(a, backward) : norm_launch<T, WT, 64, 16>(a, backward);
        case 256:
            return sh.elems == 8 ? norm_launch<T, WT, 256, 8>(a, backward) : norm_launch<T, WT, 256, 16>(a, backward);
        case 512: return norm_launch<T, WT, 512, 16>(a, backward);
        default: return norm_launch<T, WT, 1024, 16>(a, backward);
    }
}

tt_status norm_by_type(int32_t dtype, int32_t wdtype, const NormArgs& a, bool backward) {
    if (dtype == TT_F32) return norm_by_shape<float, float>(a, backward);
    if (dtype == TT_BF16)
        return wdtype == TT_F32 ? norm_by_shape<bf16, float>(a, backward) : norm_by_shape<bf16, bf16>(a, backward);
    return wdtype == TT_F32 ? norm_by_shape<f16, float>(a, backward) : norm_by_shape<f16, f16>(a, backward);
}

// What both directions ask of their arguments.
tt_status norm_check(int32_t dtype, int32_t wdtype, int64_t rows, int64_t dim) {
    if (!dtype_ok(dtype) || !dtype_ok(wdtype) || rows < 0 || dim < 1) return TT_ERR_INVALID_ARG;
    if (wdtype != dtype && wdtype != TT_F32) return TT_ERR_UNSUPPORTED;
    if (dim > kNormMaxDim || rows > INT32_MAX) return TT_ERR_UNSUPPORTED;
    return TT_OK;
}

}  // namespace
}  // namespace tt

using namespace tt;

extern "C" size_t tt_emb_norm_workspace_bytes(int32_t dtype, int64_t rows, int64_t dim) {
    if (norm_check(dtype, dtype, rows, dim) != TT_OK) return 0;
    const size_t b = (size_t)norm_bwd_blocks(rows, dim) * 2 * (size_t)dim * sizeof(float);
    return std::max<size_t>(256, (b + 255) & ~size_t(255));
}

extern "C" tt_status tt_emb_norm_forward(int32_t dtype, int32_t wdtype, const void* x, int64_t ldx,
                                         const void* weight, const void* bias, void* y, int64_t ldy, float* mean,
                                         float* rstd, int64_t rows, int64_t dim, float eps, void* stream) {
    const tt_status st = norm_check(dtype, wdtype, rows, dim);
    if (st != TT_OK) return st;
    if (!weight || (rows > 0 && (!x || !y)) || !mean != !rstd || ldx < dim || ldy < dim) return TT_ERR_INVALID_ARG;
    if (!(eps >= 0.f)) return TT_ERR_INVALID_ARG;
    if (rows == 0) return TT_OK;
    NormArgs a{};
    a.x = x; a.weight = weight; a.bias = bias; a.y = y;
    a.ldx = ldx; a.ldy = ldy; a.rows = rows; a.dim = dim;
    a.mean = mean; a.rstd = rstd; a.eps = eps; a.s = (hipStream_t)stream;
    return norm_by_type(dtype, wdtype, a, false);
}

extern "C" tt_status tt_emb_norm_backward(int32_t dtype, int32_t wdtype, const void* x, int64_t ldx,
                                          const void* weight, const float* mean, const float* rstd, const void* dy,
                                          int64_t lddy, void* dx, int64_t lddx, void* dweight, void* dbias,
                                          int64_t rows, int64_t dim, void* workspace, size_t workspace_bytes,
                                          void* stream) {
    const tt_status st = norm_check(dtype, wdtype, rows, dim);
    if (st != TT_OK) return st;
    if (!weight || !dweight || !workspace || ldx < dim || lddy < dim || lddx < dim) return TT_ERR_INVALID_ARG;
    if (rows > 0 && (!x || !mean || !rstd || !dy || !dx)) return TT_ERR_INVALID_ARG;
    if (((uintptr_t)workspace & 255) != 0) return TT_ERR_INVALID_ARG;
    if (workspace_bytes < tt_emb_norm_workspace_bytes(dtype, rows, dim)) return TT_ERR_WORKSPACE;
    NormArgs a{};
    a.x = x; a.weight = weight; a.dy = dy; a.dx = dx; a.dweight = dweight; a.dbias = dbias;
    a.ldx = ldx; a.lddy = lddy; a.lddx = lddx; a.rows = rows; a.dim = dim;
    a.mean = const_cast<float*>(mean); a.rstd = const_cast<float*>(rstd); a.part = (float*)workspace;
    a.s = (hipStream_t)stream;
    return norm_by_type(dtype, wdtype, a, true);
}
