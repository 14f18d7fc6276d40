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
// fp32. Exponents are formed as c z - [c max], c = log2 e / t, in one fused operation
// from the exact product and the rounded [c max]: what that rounding adds, half a step
// of the product, is common to every term of a part and leaves with its sum, so that
// the terms that matter (z near max) carry no error of a large product. That holds
// while the half step is small beside the range of 2^x: past |c max| = 2^24, where it
// is 1 and grows with the product, the difference z - max comes first.
//
// Bound by memory: the logits are read and the gradient is written, each once
// where both are formed in one call. A row is cut into chunks of up to 16,384 classes,
// one workgroup each, that stay in its registers; the chunks' maxima and sums
// of exponentials meet in the workspace, where each workgroup of the row waits
// for the others' before it writes its part of the gradient. The workgroups of
// a CU are at different steps, which keeps memory busy while some form
// exponentials (two a class; the vector time is near the memory's). 4096 x 131072 bf16:
// 375 us, 5.7 TB/s; 96 x 10^6 fp32: 176 us, 4.4 TB/s.
#include "tt_dense.h"

#include <atomic>

namespace tt {
namespace {

constexpr int kThreads = 256;
constexpr int kPiece = kThreads * 8;                      // classes of one load by every thread
// Loads of 8 classes a thread holds at most: 32 registers of raw 16-bit logits,
// 64 of fp32 ones. Measured both ways: 4096 x 131072 bf16 370 us against 400
// with 64 registers (four workgroups a CU instead of eight); 96 x 10^6 fp32
// 180 us against 230 with 32 (123 workgroups a row to wait for instead of 62).
constexpr int kVecs = 8;
constexpr int kChunk = kPiece * kVecs;                    // classes a workgroup holds at most

// Chunks a row is cut into, and their classes (a multiple of kPiece). As few
// as registers allow when there are rows enough; a batch of few rows is cut
// further, down to chunks of two loads, to reach 1024 workgroups.
struct Cut {
    int chunks, classes;
};
inline Cut cut_of(int64_t rows, int64_t V) {
    const int64_t pieces = (V + kPiece - 1) / kPiece;
    int64_t n = (V + kChunk - 1) / kChunk;
    n = std::max(n, std::min((pieces + 1) / 2, (1024 + rows - 1) / std::max<int64_t>(rows, 1)));
    const int64_t per = (pieces + n - 1) / n;
    return {(int)((pieces + per - 1) / per), (int)(per * kPiece)};
}

constexpr int kMaxTop = 1024;
constexpr int64_t kMaxClasses = int64_t(1) << 30;
constexpr float kMinT = 1e-18f, kMaxT = 1e18f;            // t^2 and 1/t within fp32's range

struct alignas(8) MaxSum {
    float m, s;   // the largest z, and the sum of 2^exponent(z) at it; m = -inf goes with s = 0
};

// 2^x by the hardware instruction; results below 2^-126 are 0.
__device__ __forceinline__ float pow2(float x) { return __builtin_amdgcn_exp2f(x); }

// [c m], rounded before anything else is done with it.
__device__ __forceinline__ float times(float m, float c) {
    float mc = m * c;
    asm("" : "+v"(mc));
    return mc;
}
// Where the difference from the maximum comes first: products whose rounding would
// move every term by more than 2^(1/2), or overflow (rows or chunks masked with a large
// finite value; low temperatures).
__device__ __forceinline__ bool is_far(float mc) { return !(fabsf(mc) <= 16777216.f); }

// f(exponent), exponent(z) that of z at the maximum m; the same for the workgroup.
template <class F>
__device__ __forceinline__ void at_maximum(float m, float c, F f) {
    const float mc = times(m, c);
    if (is_far(mc)) f([=](float z) { return (z - m) * c; });
    else f([=](float z) { return fmaf(z, c, -mc); });
}
// exponent(m): what every exponent of a part with this maximum is too large by.
__device__ __forceinline__ float excess(float m, float c) {
    const float mc = times(m, c);
    return is_far(mc) ? 0.f : fmaf(m, c, -mc);
}

// A part's sum at the maximum m of the whole (a part of -inf only has s = 0
// and joins without a NaN).
__device__ __forceinline__ float at_max(MaxSum a, float m, float c) {
    return a.m == m ? a.s : a.s * pow2((a.m - m) * c + (excess(m, c) - excess(a.m, c)));
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

// A chunk's logits in registers; -inf past its end. Loads that lie past it as a
// whole are left out (n is the same for the workgroup).
template <class T>
__device__ __forceinline__ void chunk_load(Raw8<T> (&r)[kVecs], const T* __restrict__ z, int n) {
#pragma unroll
    for (int v = 0; v < kVecs; ++v) {
        const int c = v * kPiece + threadIdx.x * 8;
        if (v * kPiece < n) r[v] = load8n(z + c, n - c, (T)(-INFINITY));
    }
}

template <class T>
__device__ __forceinline__ MaxSum chunk_stats(Raw8<T> (&r)[kVecs], int n, float c, float* sm) {
    float m = -INFINITY;
#pragma unroll
    for (int v = 0; v < kVecs; ++v) {
        if (v * kPiece < n)
#pragma unroll
            for (int e = 0; e < 8; ++e) m = fmaxf(m, r[v].at(e));
    }
    keep_raw(r);
    m = block_max(m, sm);
    float s = 0.f;
    at_maximum(m == -INFINITY ? 0.f : m, c, [&](auto exponent) {
#pragma unroll
        for (int v = 0; v < kVecs; ++v) {
            if (v * kPiece < n)
#pragma unroll
                for (int e = 0; e < 8; ++e) s += pow2(exponent(r[v].at(e)));
        }
    });
    return {m, block_sum(s, sm)};
}

// The row's (maximum, sum) from its chunks', the same bits in every workgroup.
__device__ __forceinline__ MaxSum row_stats(const MaxSum* part, int chunks, float c, float* sm) {
    float m = -INFINITY, s = 0.f;
    for (int k = threadIdx.x; k < chunks; k += kThreads) m = fmaxf(m, part[k].m);
    m = block_max(m, sm);
    for (int k = threadIdx.x; k < chunks; k += kThreads) s += at_max(part[k], m, c);
    return {m, block_sum(s, sm)};
}

template <class T>
__global__ __launch_bounds__(kThreads) void k_distill_stats(const T* __restrict__ z, int64_t ldz, int64_t V,
                                                            Cut cut, float c, MaxSum* __restrict__ part) {
    __shared__ float sm[4];
    const int64_t row = blockIdx.x / cut.chunks, c0 = (int64_t)(blockIdx.x % cut.chunks) * cut.classes;
    const int n = (int)min((int64_t)cut.classes, V - c0);
    Raw8<T> r[kVecs];
    chunk_load(r, z + row * ldz + c0, n);
    const MaxSum a = chunk_stats(r, n, c, sm);
    if (threadIdx.x == 0) part[blockIdx.x] = a;
}

// The teacher's list of a row in LDS: ids (-1: absent) and probabilities.
struct List {
    alignas(16) int32_t id[kMaxTop];   // -1 up to a multiple of 4 past the list's end
    alignas(16) float p[kMaxTop];      // 2^x / sum
    float all[kMaxTop];                // of the entry's class, where it lies in this workgroup's chunk
    float x[kMaxTop];                  // (logit - the largest) * c, in powers of two
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
    if ((int)threadIdx.x < (-top & 3)) {
        l.id[top + threadIdx.x] = -1;
        l.p[top + threadIdx.x] = 0.f;
    }
    m = block_max(m, sm);
    float s = 0.f;
    for (int k = threadIdx.x; k < top; k += kThreads) {
        const bool there = l.id[k] >= 0;
        l.x[k] = (l.x[k] - m) * c;
        l.p[k] = there ? pow2(l.x[k]) : 0.f;
        s += l.p[k];
    }
    s = block_sum(s, sm);
    const bool some = __syncthreads_or(m != -INFINITY || s != 0.f);
    const float inv = some ? 1.f / s : 0.f;
    for (int k = threadIdx.x; k < top; k += kThreads) l.p[k] *= inv;
    __syncthreads();
    return some ? log2f(s) : 0.f;
}

// The row's loss from its list and statistics (thread 0 has it).
template <class T>
__device__ __forceinline__ float row_loss(const List& l, int top, float lsum, const T* __restrict__ zrow, MaxSum a,
                                          float t, float c, float* sm) {
    const float log2s = log2f(a.s);
    float d = 0.f;
    at_maximum(a.m, c, [&](auto exponent) {
        for (int k = threadIdx.x; k < top; k += kThreads) {
            const float p = l.p[k];
            if (l.id[k] < 0 || p == 0.f) continue;   // p log p -> 0
            d += p * ((l.x[k] - lsum) - (exponent((float)zrow[l.id[k]]) - log2s));
        }
    });
    return t * t * 0.6931471805599453f * block_sum(d, sm);
}

// The sums of p over each class that the list names in this chunk (a class may be
// listed more than once).
__device__ __forceinline__ void list_sums(List& l, int top, int64_t c0, int n) {
    for (int j = threadIdx.x; j < top; j += kThreads) {
        const int me = l.id[j];
        if (me < 0 || me < c0 || me >= c0 + n) continue;
        float p = 0.f;
#pragma unroll 1
        for (int i = 0; i < top; i += 4) {
            const int4 k = *reinterpret_cast<const int4*>(l.id + i);
            const float4 q = *reinterpret_cast<const float4*>(l.p + i);
            p += (k.x == me ? q.x : 0.f) + (k.y == me ? q.y : 0.f) + (k.z == me ? q.z : 0.f) + (k.w == me ? q.w : 0.f);
        }
        l.all[j] = p;
    }
}

// w t q at every class of a chunk, then the list's classes again with their p
// (l.all, formed while the row's other workgroups finish: 96 x 10^6 fp32 183 -> 176 us,
// 194 -> 169 with lists that spread over all classes) taken off, once the chunk is
// written. Measured at 4096 x 131072 bf16: 375 us; 442 with p taken off before the one
// store (registers hold it), 414 with each thread writing its own listed classes again.
template <class T>
__device__ __forceinline__ void chunk_grad(Raw8<T> (&r)[kVecs], const T* __restrict__ zc, int64_t c0, int n,
                                           const List& l, int top, MaxSum a, float wt, float c, bool apart,
                                           T* __restrict__ dc) {
    bool any = false;
    for (int j = threadIdx.x; j < top; j += kThreads) any |= l.id[j] >= 0;
    const bool some = __syncthreads_or(any);
    keep_raw(r);
    const float scale = wt * (1.f / a.s);
    auto write = [&](int v, const float (&g)[8]) {
        const int o = v * kPiece + threadIdx.x * 8;
        if (apart) store8n_apart(dc + o, g, n - o);
        else store8n(dc + o, g, n - o);
    };
    if (!some) {   // 0 whatever the logits are
        const float g[8] = {};
        for (int v = 0; v * kPiece < n; ++v) write(v, g);
        return;
    }
    at_maximum(a.m, c, [&](auto exponent) {
#pragma unroll
        for (int v = 0; v < kVecs; ++v) {
            if (v * kPiece >= n) continue;
            float g[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) g[e] = scale * pow2(exponent(r[v].at(e)));
            write(v, g);
        }
        __syncthreads();   // the list's classes are written after the whole chunk
        for (int j = threadIdx.x; j < top; j += kThreads) {
            const int64_t id = (int64_t)l.id[j] - c0;
            if (l.id[j] < 0 || id < 0 || id >= n) continue;
            const float p = l.all[j];   // every entry of a class writes the same
            dc[id] = (T)(scale * pow2(exponent((float)zc[id])) - wt * p);
        }
    });
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
    const MaxSum a = row_stats(part + row * chunks, chunks, c, sm);
    const float lsum = list_load(l, ids + row * top, top_logits + row * top, top, V, c, sm);
    const float d = row_loss(l, top, lsum, z + row * ldz, a, t, c, sm);
    if (threadIdx.x == 0) {
        loss[row] = d;
        if (stats) stats[row] = a;
    }
}

template <class T>
__global__ __launch_bounds__(kThreads) void k_distill_grad(const T* __restrict__ z, int64_t ldz, int64_t V, Cut cut,
                                                           float t, float c, const int64_t* __restrict__ ids,
                                                           const float* __restrict__ top_logits, int top,
                                                           const MaxSum* __restrict__ stats,
                                                           const float* __restrict__ row_weight, bool apart,
                                                           T* __restrict__ dz, int64_t lddz) {
    __shared__ float sm[4];
    __shared__ List l;
    const int64_t row = blockIdx.x / cut.chunks, c0 = (int64_t)(blockIdx.x % cut.chunks) * cut.classes;
    const int n = (int)min((int64_t)cut.classes, V - c0);
    Raw8<T> r[kVecs];
    chunk_load(r, z + row * ldz + c0, n);
    list_load(l, ids + row * top, top_logits + row * top, top, V, c, sm);
    list_sums(l, top, c0, n);
    chunk_grad(r, z + row * ldz + c0, c0, n, l, top, stats[row], t * row_weight[row], c, apart,
               dz + row * lddz + c0);
}

// Marks a chunk's place in the workspace as not yet written: no (maximum, sum)
// has these bits, a maximum is never NaN.
constexpr uint64_t kNoPart = ~uint64_t(0);

// Forward, or forward and backward, of a chunk that the workgroup keeps in
// registers. The row's workgroups post their (maximum, sum) in `part` and wait
// for the others'. They run at about the same time (consecutive workgroups);
// should one of them not have started yet, which the wait does not rely on,
// the waiting one forms the missing parts itself after `spins` polls, from
// the logits and in the same order, hence with the same bits.
template <class T, bool GRAD>
__global__ __launch_bounds__(kThreads, sizeof(T) == 2 ? 8 : 4) void k_distill_row(
    const T* __restrict__ z, int64_t ldz, int64_t V, Cut cut, float t, float c, const int64_t* __restrict__ ids,
    const float* __restrict__ top_logits, int top, uint64_t* __restrict__ part, int spins,
    const float* __restrict__ row_weight, float* __restrict__ loss, MaxSum* __restrict__ stats, bool apart,
    T* __restrict__ dz, int64_t lddz) {
    __shared__ float sm[4];
    __shared__ List l;
    __shared__ MaxSum row_part[kThreads];
    const int64_t row = blockIdx.x / cut.chunks;
    const int mine = blockIdx.x % cut.chunks;
    const int64_t c0 = (int64_t)mine * cut.classes;
    const T* zr = z + row * ldz;
    const int n = (int)min((int64_t)cut.classes, V - c0);
    Raw8<T> r[kVecs];
    chunk_load(r, zr + c0, n);
    const float lsum = list_load(l, ids + row * top, top_logits + row * top, top, V, c, sm);
    MaxSum a = chunk_stats(r, n, c, sm);
    if (cut.chunks > 1 && threadIdx.x == 0)
        __hip_atomic_store(part + row * cut.chunks + mine, __builtin_bit_cast(uint64_t, a), __ATOMIC_RELAXED,
                           __HIP_MEMORY_SCOPE_AGENT);
    if (GRAD) list_sums(l, top, c0, n);
    if (cut.chunks > 1) {
        uint64_t* rp = part + row * cut.chunks;
        uint64_t p = kNoPart;
        const bool polls = (int)threadIdx.x < cut.chunks;
        for (int i = 0; i < spins && polls && p == kNoPart; ++i) {
            p = __hip_atomic_load(rp + threadIdx.x, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            if (p == kNoPart) __builtin_amdgcn_s_sleep(2);
        }
        row_part[threadIdx.x] = __builtin_bit_cast(MaxSum, p);
        if (__syncthreads_or(polls && p == kNoPart)) {
            for (int k = 0; k < cut.chunks; ++k) {
                if (__builtin_bit_cast(uint64_t, row_part[k]) != kNoPart) continue;
                const int64_t k0 = (int64_t)k * cut.classes;
                const int kn = (int)min((int64_t)cut.classes, V - k0);
                chunk_load(r, zr + k0, kn);
                const MaxSum b = chunk_stats(r, kn, c, sm);
                __syncthreads();
                if (threadIdx.x == 0) row_part[k] = b;
                __syncthreads();
            }
            chunk_load(r, zr + c0, n);
        }
        a = row_stats(row_part, cut.chunks, c, sm);
    }
    if (mine == 0) {
        const float d = row_loss(l, top, lsum, zr, a, t, c, sm);
        if (threadIdx.x == 0) {
            loss[row] = d;
            if (stats) stats[row] = a;
        }
    }
    if (GRAD) chunk_grad(r, zr + c0, c0, n, l, top, a, t * row_weight[row], c, apart,
                         dz + row * lddz + c0);
}

// Gradients of this many bytes and more are stored past the caches, which keeps
// the logits there: 96 x 10^6 fp32 180 us instead of 207, and the forward that
// follows another batch's backward of 1021 x 50021 f16 23 us instead of 29.
// Smaller ones stay in the caches for whoever reads them next.
constexpr int64_t kApart = int64_t(64) << 20;

// Polls before a workgroup forms the missing parts itself: about 10 ms.
constexpr int kPolls = 1 << 15;
std::atomic<int> polls{kPolls};

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
tt_status distill_launch(const DistillArgs& a, const Cut& cut, bool forward, bool backward) {
    const float c = 1.4426950408889634f / a.t;
    const T* z = (const T*)a.z;
    const dim3 grid((unsigned)(a.rows * cut.chunks)), block(kThreads);
    const bool apart = a.rows * a.V * (int64_t)sizeof(T) >= kApart;
    if (forward && (cut.chunks == 1 || (backward && cut.chunks <= kThreads))) {
        // one kernel, the rows' chunks meeting in the workspace
        if (cut.chunks > 1) {
            const tt_status st = fill32(nullptr, a.part, ~0u, 2 * a.rows * cut.chunks, a.s);
            if (st != TT_OK) return st;
        }
        auto k = backward ? k_distill_row<T, true> : k_distill_row<T, false>;
        TT_LAUNCH(nullptr, "k_distill_row", a.s, k, grid, block, 0, a.s, z, a.ldz, a.V, cut, a.t, c, a.ids,
                  a.top_logits, a.top, (uint64_t*)a.part, polls.load(std::memory_order_relaxed), a.row_weight, a.loss, backward ? nullptr : a.stats,
                  apart, (T*)a.dz, a.lddz);
        TT_LAUNCH_CHECK();
        return TT_OK;
    }
    if (forward) {
        TT_LAUNCH(nullptr, "k_distill_stats", a.s, (k_distill_stats<T>), grid, block, 0, a.s, z, a.ldz, a.V, cut, c,
                  a.part);
        TT_LAUNCH_CHECK();
        TT_LAUNCH(nullptr, "k_distill_loss", a.s, (k_distill_loss<T>), dim3((unsigned)a.rows), block, 0, a.s, z,
                  a.ldz, a.V, cut.chunks, a.t, c, a.ids, a.top_logits, a.top, a.part, a.loss, a.stats);
        TT_LAUNCH_CHECK();
    }
    if (backward) {
        TT_LAUNCH(nullptr, "k_distill_grad", a.s, (k_distill_grad<T>), grid, block, 0, a.s, z, a.ldz, a.V, cut, a.t,
                  c, a.ids, a.top_logits, a.top, a.stats, a.row_weight, apart, (T*)a.dz, a.lddz);
        TT_LAUNCH_CHECK();
    }
    return TT_OK;
}

// Workgroups of a launch: its threads must stay below 2^32.
constexpr int64_t kMaxGroups = int64_t(1) << 23;

// More rows than one launch takes go in several.
template <class T>
tt_status distill_rows(const DistillArgs& a, bool forward, bool backward) {
    const Cut cut = cut_of(a.rows, a.V);
    const int64_t step = std::max<int64_t>(1, kMaxGroups / cut.chunks);
    for (int64_t r = 0; r < a.rows; r += step) {
        DistillArgs b = a;
        b.rows = std::min(step, a.rows - r);
        b.z = (const T*)a.z + r * a.ldz;
        b.ids = a.ids ? a.ids + r * a.top : nullptr;
        b.top_logits = a.top_logits ? a.top_logits + r * a.top : nullptr;
        b.part = a.part ? a.part + r * cut.chunks : nullptr;
        b.loss = a.loss ? a.loss + r : nullptr;
        b.stats = a.stats ? a.stats + r : nullptr;
        b.row_weight = a.row_weight ? a.row_weight + r : nullptr;
        b.dz = a.dz ? (T*)a.dz + r * a.lddz : nullptr;
        const tt_status st = distill_launch<T>(b, cut, forward, backward);
        if (st != TT_OK) return st;
    }
    return TT_OK;
}

tt_status distill_by_type(int32_t dtype, const DistillArgs& a, bool forward, bool backward) {
    if (dtype == TT_F32) return distill_rows<float>(a, forward, backward);
    if (dtype == TT_BF16) return distill_rows<bf16>(a, forward, backward);
    return distill_rows<f16>(a, forward, backward);
}

tt_status distill_check(int32_t dtype, int64_t rows, int64_t V) {
    if (!dtype_ok(dtype) || rows < 0 || V < 1) return TT_ERR_INVALID_ARG;
    if (V > kMaxClasses || rows > INT32_MAX || rows * cut_of(rows, V).chunks > INT32_MAX) return TT_ERR_UNSUPPORTED;
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

inline size_t workspace_of(int64_t parts) {
    return std::max<size_t>(256, ((size_t)parts * sizeof(MaxSum) + 255) & ~size_t(255));
}

// The workspace: the chunks' statistics, then the rows'.
tt_status distill_workspace(DistillArgs& a, void* ws, size_t bytes) {
    if (!ws || ((uintptr_t)ws & 255) != 0) return TT_ERR_INVALID_ARG;
    const int64_t parts = a.rows * cut_of(a.rows, a.V).chunks;
    if (bytes < workspace_of(parts + a.rows)) return TT_ERR_WORKSPACE;
    a.part = (MaxSum*)ws;
    a.stats = a.part + parts;
    return TT_OK;
}

}  // namespace
}  // namespace tt

using namespace tt;

extern "C" int32_t tt_distill_set_polls(int32_t n) { return polls.exchange(n < 0 ? kPolls : n); }

extern "C" size_t tt_emb_distill_workspace_bytes(int32_t dtype, int64_t rows, int64_t classes) {
    if (distill_check(dtype, rows, classes) != TT_OK) return 0;
    // what fewer rows, cut into more chunks each, need is no more than this either: theirs
    // are as few as a row takes, or at most the 1024 they are cut to reach and one a row
    const int64_t pieces = (classes + kPiece - 1) / kPiece, least = (classes + kChunk - 1) / kChunk;
    return workspace_of(std::max(rows * least, std::min(rows * ((pieces + 1) / 2), rows + 1024)) + rows);
}

extern "C" tt_status tt_emb_distill_forward(int32_t dtype, const void* logits, int64_t ld, const int64_t* ids,
                                            const float* top_logits, int64_t top, float* loss, float* stats,
                                            int64_t rows, int64_t classes, float temperature, void* workspace,
                                            size_t workspace_bytes, void* stream) {
    DistillArgs a;
    tt_status st = distill_args(a, dtype, logits, ld, ids, top_logits, top, temperature, rows, classes, stream);
    if (st != TT_OK) return st;
    if (rows > 0 && !loss) return TT_ERR_INVALID_ARG;
    if ((st = distill_workspace(a, workspace, workspace_bytes)) != TT_OK) return st;
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
    if ((st = distill_workspace(a, workspace, workspace_bytes)) != TT_OK) return st;
    a.loss = loss;
    a.row_weight = row_weight;
    a.dz = dlogits;
    a.lddz = ldd;
    return distill_by_type(dtype, a, true, true);
}
