// Distillation from a teacher's top logits: per row, the divergence of the
// student's distribution over all V classes from the teacher's over the
// classes of its list, both at temperature t, and its gradient.
//
//   q = softmax(z / t),  p = softmax(list / t)
//   loss = t^2 sum_k p_k (log p_k - log q_{id_k})
//   dz_j = w t (q_j - sum_{k: id_k = j} p_k)          (w: the row's weight)
//
// An entry is absent when its id is outside [0, V) or its logit is -inf; a row
// whose list has no entry has loss 0 and gradient 0. Everything is held in
// fp32; exponents are formed as (z - max) * (log2 e / t), the difference first,
// so that the terms that matter (z near max) carry no error of a large product.
//
// Bound by memory: the logits are read and the gradient is written. A row is
// cut into chunks of 16,384 classes, one workgroup each, that stay in its
// registers (64 or 32 a thread); each chunk's maximum and sum of exponentials
// meet in the workspace.
#include "tt_dense.h"

namespace tt {
namespace {

constexpr int kThreads = 256;
constexpr int kVecs = 8;                                  // vectors of 8 classes a thread
constexpr int kChunk = kThreads * kVecs * 8;              // classes a workgroup holds
constexpr int kMaxTop = 1024;
constexpr int64_t kMaxClasses = int64_t(1) << 30;
constexpr float kMinT = 1e-18f, kMaxT = 1e18f;            // t^2 and 1/t within fp32's range

struct MaxSum {
    float m, s;   // the largest z, and sum exp((z - m)/t); m = -inf goes with s = 0
};

// Joins the (maximum, sum) of two parts of a row.
__device__ __forceinline__ MaxSum join(MaxSum a, MaxSum b, float c) {
    const float m = fmaxf(a.m, b.m);
    // a part of -inf only has s = 0 and joins without a NaN; one of +inf or NaN keeps it
    const float ea = a.m == m ? 1.f : exp2f((a.m - m) * c), eb = b.m == m ? 1.f : exp2f((b.m - m) * c);
    return {m, a.s * ea + b.s * eb};
}

__device__ __forceinline__ float block_max(float v, float* sm) {
    v = lanes_max<64>(v);
    __syncthreads();
    if ((threadIdx.x & 63) == 0) sm[threadIdx.x >> 6] = v;
    __syncthreads();
    return fmaxf(fmaxf(sm[0], sm[1]), fmaxf(sm[2], sm[3]));
}
__device__ __forceinline__ float block_sum(float v, float* sm) {
    v = lanes_sum<64>(v);
    __syncthreads();
    if ((threadIdx.x & 63) == 0) sm[threadIdx.x >> 6] = v;
    __syncthreads();
    return (sm[0] + sm[1]) + (sm[2] + sm[3]);
}

// The chunk's (maximum, sum) from its elements in registers.
template <class T>
__device__ __forceinline__ MaxSum chunk_stats(const Raw8<T> (&r)[kVecs], int n, float c, float* sm) {
    float m = -INFINITY;
#pragma unroll
    for (int v = 0; v < kVecs; ++v)
#pragma unroll
        for (int e = 0; e < 8; ++e) m = fmaxf(m, (float)r[v].v[e]);   // -inf past the row's end
    m = block_max(m, sm);
    const float shift = m == -INFINITY ? 0.f : m;
    float s = 0.f;
#pragma unroll
    for (int v = 0; v < kVecs; ++v)
#pragma unroll
        for (int e = 0; e < 8; ++e) s += exp2f(((float)r[v].v[e] - shift) * c);
    return {m, block_sum(s, sm)};
}

template <class T>
__device__ __forceinline__ void chunk_load(Raw8<T> (&r)[kVecs], const T* __restrict__ z, int n) {
#pragma unroll
    for (int v = 0; v < kVecs; ++v) {
        const int c = (v * kThreads + threadIdx.x) * 8;
        r[v] = load8n(z + c, n - c, (T)(-INFINITY));
    }
}

template <class T>
__global__ __launch_bounds__(kThreads) void k_distill_stats(const T* __restrict__ z, int64_t ldz, int64_t V,
                                                            int chunks, float c, MaxSum* __restrict__ part) {
    __shared__ float sm[4];
    const int64_t row = blockIdx.x / chunks, k = blockIdx.x % chunks;
    const int n = (int)min((int64_t)kChunk, V - k * kChunk);
    Raw8<T> r[kVecs];
    chunk_load(r, z + row * ldz + k * kChunk, n);
    const MaxSum a = chunk_stats(r, n, c, sm);
    if (threadIdx.x == 0) part[blockIdx.x] = a;
}

// The teacher's list of a row in LDS: ids (-1: absent) and probabilities.
struct List {
    int32_t id[kMaxTop];
    float x[kMaxTop];    // (logit - the largest) * c, in powers of two
    float p[kMaxTop];    // 2^x / sum
};

// Fills it; returns log2 of the sum of 2^x (0 for an empty list).
__device__ __forceinline__ float list_load(List& l, const int64_t* __restrict__ ids, const float* __restrict__ lg,
                                           int top, int64_t V, float c, float* sm) {
    float m = -INFINITY;
    for (int k = threadIdx.x; k < top; k += kThreads) {
        const int64_t id = ids[k];
        const float x = lg[k];
        const bool there = id >= 0 && id < V && !(x == -INFINITY);
        l.id[k] = there ? (int32_t)id : -1;
        l.x[k] = x;
        if (there) m = fmaxf(m, x);
    }
    m = block_max(m, sm);
    float s = 0.f;
    for (int k = threadIdx.x; k < top; k += kThreads) {
        const bool there = l.id[k] >= 0;
        l.x[k] = (l.x[k] - m) * c;
        l.p[k] = there ? exp2f(l.x[k]) : 0.f;
        s += l.p[k];
    }
    s = block_sum(s, sm);
    const bool some = __syncthreads_or(m != -INFINITY || s != 0.f);
    const float inv = some ? 1.f / s : 0.f;
    for (int k = threadIdx.x; k < top; k += kThreads) l.p[k] *= inv;
    __syncthreads();
    return some ? log2f(s) : 0.f;
}

// One workgroup a row: joins the chunks' statistics, forms the row's loss.
template <class T>
__global__ __launch_bounds__(kThreads) void k_distill_loss(const T* __restrict__ z, int64_t ldz, int64_t V,
                                                           int chunks, float t, float c,
                                                           const int64_t* __restrict__ ids,
                                                           const float* __restrict__ top_logits, int top,
                                                           const MaxSum* __restrict__ part, float* __restrict__ loss,
                                                           MaxSum* __restrict__ stats) {
    __shared__ float sm[4];
    __shared__ List l;
    const int64_t row = blockIdx.x;
    MaxSum a{-INFINITY, 0.f};
    for (int k = threadIdx.x; k < chunks; k += kThreads) a = join(a, part[row * chunks + k], c);
    const float m = block_max(a.m, sm);
    const float s = block_sum(a.m == m ? a.s : a.s * exp2f((a.m - m) * c), sm);
    const float lsum = list_load(l, ids + row * top, top_logits + row * top, top, V, c, sm);
    const float log2s = log2f(s);
    float d = 0.f;
    for (int k = threadIdx.x; k < top; k += kThreads) {
        const float p = l.p[k];
        if (l.id[k] < 0 || p == 0.f) continue;   // p log p -> 0
        d += p * ((l.x[k] - lsum) - (((float)z[row * ldz + l.id[k]] - m) * c - log2s));
    }
    d = block_sum(d, sm);
    if (threadIdx.x == 0) {
        loss[row] = t * t * 0.6931471805599453f * d;
        if (stats) stats[row] = {m, s};
    }
}

// One workgroup a chunk: w t q at every class, then the list's classes again
// with their p taken off.
template <class T>
__global__ __launch_bounds__(kThreads) void k_distill_grad(const T* __restrict__ z, int64_t ldz, int64_t V,
                                                           int chunks, float t, float c,
                                                           const int64_t* __restrict__ ids,
                                                           const float* __restrict__ top_logits, int top,
                                                           const MaxSum* __restrict__ stats,
                                                           const float* __restrict__ row_weight, T* __restrict__ dz,
                                                           int64_t lddz) {
    __shared__ float sm[4];
    __shared__ List l;
    const int64_t row = blockIdx.x / chunks, k = blockIdx.x % chunks;
    const int64_t c0 = k * kChunk;
    const int n = (int)min((int64_t)kChunk, V - c0);
    const T* zr = z + row * ldz + c0;
    T* dr = dz + row * lddz + c0;
    Raw8<T> r[kVecs];
    chunk_load(r, zr, n);
    list_load(l, ids + row * top, top_logits + row * top, top, V, c, sm);
    bool mine = false;
    for (int j = threadIdx.x; j < top; j += kThreads) mine |= l.id[j] >= 0;
    const bool some = __syncthreads_or(mine);
    const MaxSum a = stats[row];
    const float wt = t * row_weight[row], inv = 1.f / a.s;
#pragma unroll
    for (int v = 0; v < kVecs; ++v) {
        const int o = (v * kThreads + threadIdx.x) * 8;
        Raw8<T> g;
#pragma unroll
        for (int e = 0; e < 8; ++e)
            g.v[e] = (T)(some ? wt * (exp2f(((float)r[v].v[e] - a.m) * c) * inv) : 0.f);
        store8n(dr + o, g, n - o);
    }
    __syncthreads();   // the list's classes are written after the whole chunk
    for (int j = threadIdx.x; j < top; j += kThreads) {
        const int64_t id = (int64_t)l.id[j] - c0;
        if (l.id[j] < 0 || id < 0 || id >= n) continue;
        // a class that is listed more than once: every entry of it writes the same sum
        float p = 0.f;
        for (int i = 0; i < top; ++i) p += l.id[i] == l.id[j] ? l.p[i] : 0.f;
        dr[id] = (T)(wt * (exp2f(((float)zr[id] - a.m) * c) * inv - p));
    }
}

int64_t chunks_of(int64_t V) { return (V + kChunk - 1) / kChunk; }

struct DistillArgs {
    const void* z;
    int64_t ldz, rows, V;
    const int64_t* ids;
    const float* top_logits;
    int top;
    float t;
    const float* row_weight;
    float* loss;
    void* dz;
    int64_t lddz;
    MaxSum *part, *stats;   // stats: the caller's (forward's output, backward's input), or null
    hipStream_t s;
};

template <class T>
tt_status distill_launch(const DistillArgs& a, bool forward, bool backward) {
    const int chunks = (int)chunks_of(a.V);
    const float c = 1.4426950408889634f / a.t;
    const T* z = (const T*)a.z;
    const unsigned grid = (unsigned)(a.rows * chunks);
    if (forward) {
        TT_LAUNCH(nullptr, "k_distill_stats", a.s, (k_distill_stats<T>), dim3(grid), dim3(kThreads), 0, a.s, z, a.ldz,
                  a.V, chunks, c, a.part);
        TT_LAUNCH_CHECK();
        TT_LAUNCH(nullptr, "k_distill_loss", a.s, (k_distill_loss<T>), dim3((unsigned)a.rows), dim3(kThreads), 0, a.s,
                  z, a.ldz, a.V, chunks, a.t, c, a.ids, a.top_logits, a.top, a.part, a.loss, a.stats);
        TT_LAUNCH_CHECK();
    }
    if (backward) {
        TT_LAUNCH(nullptr, "k_distill_grad", a.s, (k_distill_grad<T>), dim3(grid), dim3(kThreads), 0, a.s, z, a.ldz,
                  a.V, chunks, a.t, c, a.ids, a.top_logits, a.top, a.stats, a.row_weight, (T*)a.dz, a.lddz);
        TT_LAUNCH_CHECK();
    }
    return TT_OK;
}

tt_status distill_by_type(int32_t dtype, const DistillArgs& a, bool forward, bool backward) {
    if (a.rows == 0) return TT_OK;
    if (dtype == TT_F32) return distill_launch<float>(a, forward, backward);
    if (dtype == TT_BF16) return distill_launch<bf16>(a, forward, backward);
    return distill_launch<f16>(a, forward, backward);
}

tt_status distill_check(int32_t dtype, int64_t rows, int64_t V) {
    if (!dtype_ok(dtype) || rows < 0 || V < 1) return TT_ERR_INVALID_ARG;
    if (V > kMaxClasses || rows > INT32_MAX || rows * chunks_of(V) > INT32_MAX) return TT_ERR_UNSUPPORTED;
    return TT_OK;
}

// The arguments that every call takes.
tt_status distill_args(DistillArgs& a, int32_t dtype, const void* z, int64_t ldz, const int64_t* ids,
                       const float* top_logits, int64_t top, float t, int64_t rows, int64_t V, void* stream) {
    const tt_status st = distill_check(dtype, rows, V);
    if (st != TT_OK) return st;
    if (ldz < V || top < 0 || !(t >= kMinT && t <= kMaxT)) return TT_ERR_INVALID_ARG;
    if (rows > 0 && (!z || (top > 0 && (!ids || !top_logits)))) return TT_ERR_INVALID_ARG;
    if (top > kMaxTop) return TT_ERR_UNSUPPORTED;
    a = DistillArgs{};
    a.z = z; a.ldz = ldz; a.rows = rows; a.V = V;
    a.ids = ids; a.top_logits = top_logits; a.top = (int)top; a.t = t;
    a.s = (hipStream_t)stream;
    return TT_OK;
}

// The workspace: the chunks' statistics, then the rows'.
tt_status distill_workspace(DistillArgs& a, int32_t dtype, void* ws, size_t bytes) {
    if (!ws || ((uintptr_t)ws & 255) != 0) return TT_ERR_INVALID_ARG;
    if (bytes < tt_emb_distill_workspace_bytes(dtype, a.rows, a.V)) return TT_ERR_WORKSPACE;
    a.part = (MaxSum*)ws;
    a.stats = a.part + a.rows * chunks_of(a.V);
    return TT_OK;
}

}  // namespace
}  // namespace tt

using namespace tt;

extern "C" size_t tt_emb_distill_workspace_bytes(int32_t dtype, int64_t rows, int64_t classes) {
    if (distill_check(dtype, rows, classes) != TT_OK) return 0;
    const size_t b = (size_t)rows * (size_t)(chunks_of(classes) + 1) * sizeof(MaxSum);
    return std::max<size_t>(256, (b + 255) & ~size_t(255));
}

extern "C" tt_status tt_emb_distill_forward(int32_t dtype, const void* logits, int64_t ld, const int64_t* ids,
                                            const float* top_logits, int64_t top, float* loss, float* stats,
                                            int64_t rows, int64_t classes, float temperature, void* workspace,
                                            size_t workspace_bytes, void* stream) {
    DistillArgs a;
    tt_status st = distill_args(a, dtype, logits, ld, ids, top_logits, top, temperature, rows, classes, stream);
    if (st != TT_OK) return st;
    if (rows > 0 && !loss) return TT_ERR_INVALID_ARG;
    if ((st = distill_workspace(a, dtype, workspace, workspace_bytes)) != TT_OK) return st;
    a.loss = loss;
    a.stats = (MaxSum*)stats;
    return distill_by_type(dtype, a, true, false);
}

extern "C" tt_status tt_emb_distill_backward(int32_t dtype, const void* logits, int64_t ld, const int64_t* ids,
                                             const float* top_logits, int64_t top, const float* stats,
                                             const float* row_weight, void* dlogits, int64_t ldd, int64_t rows,
                                             int64_t classes, float temperature, void* stream) {
    DistillArgs a;
    const tt_status st = distill_args(a, dtype, logits, ld, ids, top_logits, top, temperature, rows, classes, stream);
    if (st != TT_OK) return st;
    if (ldd < classes || (rows > 0 && (!stats || !row_weight || !dlogits))) return TT_ERR_INVALID_ARG;
    a.stats = (MaxSum*)const_cast<float*>(stats);
    a.row_weight = row_weight;
    a.dz = dlogits;
    a.lddz = ldd;
    return distill_by_type(dtype, a, false, true);
}

extern "C" tt_status tt_emb_distill_train(int32_t dtype, const void* logits, int64_t ld, const int64_t* ids,
                                          const float* top_logits, int64_t top, const float* row_weight, float* loss,
                                          void* dlogits, int64_t ldd, int64_t rows, int64_t classes,
                                          float temperature, void* workspace, size_t workspace_bytes, void* stream) {
    DistillArgs a;
    tt_status st = distill_args(a, dtype, logits, ld, ids, top_logits, top, temperature, rows, classes, stream);
    if (st != TT_OK) return st;
    if (ldd < classes || (rows > 0 && (!row_weight || !loss || !dlogits))) return TT_ERR_INVALID_ARG;
    if ((st = distill_workspace(a, dtype, workspace, workspace_bytes)) != TT_OK) return st;
    a.loss = loss;
    a.row_weight = row_weight;
    a.dz = dlogits;
    a.lddz = ldd;
    return distill_by_type(dtype, a, true, true);
}
