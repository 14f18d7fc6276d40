// Attention of one new token a sequence over its keys and values in a paged cache.
//
//   s_j = scale q . k_j,  out = sum_j e^(s_j - m) v_j / sum_j e^(s_j - m)
//
// Bound by memory: the cache is read once, by the workgroup that answers every head of a
// key head (a wave's 32 columns are these heads; past 32 heads a key head, once for each 32 of
// them). A sequence's tokens are split over
// workgroups and, there, over waves, each with a softmax of its own; waves are joined in
// LDS and workgroups, where a sequence has several, by a second launch, in a fixed order.
// 64 sequences of 8000 tokens, 8 key heads of 128 bf16: 1.8 GB in 373 us, 4.8 TB/s; one of 32768:
// 134 MB in 25 us and 4.6 to join.
#include "tt_attend.h"

namespace tt {
namespace {

constexpr int kWaves = 4, kTokens = 32;           // tokens of a wave's tile
constexpr int kHeads = 32;                        // heads of a workgroup at most
// tokens a workgroup takes, where there are that many (32768 tokens, 8 key heads: 256 32 us and 9
// to join, 512 30 and 6, 1024 41 and 5)
constexpr int kMinChunk = 512;

struct PagedArgs {
    const void *q, *k, *v;
    int64_t ldq, pages, ldt, ldo;
    const int32_t* table;
    const int64_t* lengths;
    void* out;
    int page, most, seqs, heads, kv, group, blocks, splits, D;   // most: tokens of a sequence; blocks: of kHeads heads
    float scale;
    float* part;        // [seqs][heads][splits][DP], weighted sums
    float2* ml;         // [seqs][heads][splits], maximum and sum of weights
    hipStream_t s;
};

__device__ __forceinline__ int length_of(const PagedArgs& a, int seq) {
    const int64_t n = a.lengths[seq];
    return n < 0 ? 0 : n > a.most ? a.most : (int)n;
}
// Tokens of a workgroup.
__device__ __forceinline__ int chunk_of(const PagedArgs& a, int len) {
    const int n = (int)(((int64_t)len + a.splits - 1) / a.splits);
    return max(kMinChunk, (n + kWaves * kTokens - 1) / (kWaves * kTokens) * (kWaves * kTokens));
}

// DMA: keys and values go from memory straight to LDS, which needs whole, aligned 16-byte pieces;
// a wave sends for the next tile's keys when this one's scores are formed, and for its values after
// the outputs. Lanes without a piece (past D, or of tokens not seen) send for nothing: their
// places are zeros from the start, or written so. Otherwise through registers.
//
// Two workgroups a CU: 8 waves with up to 16 KB under way each. A token over 32768 bf16 (8 key
// heads of 128) took 40 us with one and registers that hold a tile under way.
template <class T, int DP, bool DMA>
__global__ __launch_bounds__(kWaves * 64, (DMA && sizeof(T) == 2) || DP == 32 ? 2 : 1) void k_attend_paged(const PagedArgs a) {
    typedef Tile<T, DP> L;
    constexpr int N = kTokens * L::SLOTS / 64, BYTES = kTokens * L::ROW;
    constexpr int HALF = BYTES / (DP * 4);   // heads whose sums the place of a tile of keys takes
    static_assert(2 * HALF >= kHeads, "room for a wave's sums");
    __shared__ __align__(16) char tk[kWaves][BYTES], tv[kWaves][BYTES];
    __shared__ float sm_m[kWaves][kHeads], sm_l[kWaves][kHeads];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    int b = blockIdx.x;
    const int kv = b % a.kv;
    b /= a.kv;
    const int block = b % a.blocks;
    b /= a.blocks;
    const int split = b % a.splits, seq = b / a.splits;
    const int len = length_of(a, seq), chunk = chunk_of(a, len), used = max(1, (len + chunk - 1) / chunk);
    if (split >= used) return;
    const int begin = split * chunk, end = min(len, begin + chunk);
    const int heads = min(kHeads, a.group - block * kHeads), head0 = kv * a.group + block * kHeads;
    const float c = a.scale * kLog2e;

    Piece fq[L::STEPS];
    load_row<T, DP>(fq, (const T*)a.q + seq * a.ldq + (int64_t)(head0 + (lane & 31)) * a.D, (lane & 31) < heads, a.D);
    const int32_t* table = a.table + seq * a.ldt;
    // the cache's row of token t0 + lane % 32, or -1
    auto row_of = [&](int t0) -> int64_t {
        const int t = t0 + (lane & 31);
        if (t >= end) return -1;
        const int64_t p = table[t / a.page];
        return p >= 0 && p < a.pages ? p * a.page + t % a.page : -1;
    };
    char *sk = tk[wave], *sv = tv[wave];
    auto slot_row = [&](int i) { return (i * 64 + lane) / L::SLOTS; };
    auto slot_element = [&](int i) { return (((i * 64 + lane) % L::SLOTS) ^ L::key(slot_row(i))) * L::P; };
    Piece rk[DMA ? 1 : N], rv[DMA ? 1 : N];
    int64_t row = -1;            // of the tile that is sent for
    uint32_t seen = 0;
    auto find = [&](int t0) TT_INLINE {
        row = row_of(t0);
        seen = (uint32_t)__ballot(row >= 0);
    };
    // Sends for the tile's keys or values.
    auto send = [&](const void* from, char* lds, Piece (&r)[DMA ? 1 : N]) TT_INLINE {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int x = slot_row(i), e = slot_element(i);
            const T* p = (const T*)from + (__shfl(row, x) * a.kv + kv) * a.D + e;
            const bool there = seen >> x & 1;
            if constexpr (DMA) {
#ifdef __HIP_DEVICE_COMPILE__
                if (there && e < a.D)
                    __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)p,
                                                     (__attribute__((address_space(3))) void*)(lds + i * 1024), 16, 0, 0);
                else
                    *reinterpret_cast<Piece*>(lds + (i * 64 + lane) * 16) = Piece{0, 0, 0, 0};
#endif
            } else {
                r[i] = load_piece(p, there ? max(0, min(L::P, a.D - e)) : 0);
            }
        }
    };
    // Until all that this wave has sent for is in LDS.
    auto arrive = [&]() TT_INLINE {
        if constexpr (DMA) {
            __atomic_signal_fence(__ATOMIC_SEQ_CST);
            __builtin_amdgcn_s_waitcnt(0x0070);   // vmcnt(0) lgkmcnt(0)
            __atomic_signal_fence(__ATOMIC_SEQ_CST);
        } else {
            __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
            __builtin_amdgcn_wave_barrier();
#pragma unroll
            for (int i = 0; i < N; ++i) {
                *reinterpret_cast<Piece*>(sk + (i * 64 + lane) * 16) = rk[i];
                *reinterpret_cast<Piece*>(sv + (i * 64 + lane) * 16) = rv[i];
            }
        }
        __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
        __builtin_amdgcn_wave_barrier();
        __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
    };
    // Until this wave's reads of a tile are done, which the next one's pieces are to overwrite.
    auto taken = [&]() TT_INLINE {
        __atomic_signal_fence(__ATOMIC_SEQ_CST);
        __builtin_amdgcn_s_waitcnt(0xC07F);       // lgkmcnt(0)
        __atomic_signal_fence(__ATOMIC_SEQ_CST);
    };
    floatx16 o[DP / 32] = {};
    Softmax<T> sm;
    sm.init();
    int t0 = begin + wave * kTokens;
    if (t0 < end) {
        find(t0);
        send(a.k, sk, rk);
        send(a.v, sv, rv);
    }
    for (; t0 < end; t0 += kWaves * kTokens) {
        arrive();
        const uint32_t here = seen;
        const int next = t0 + kWaves * kTokens;
        if (next < end) find(next);
        if (!DMA && next < end) {
            send(a.k, sk, rk);
            send(a.v, sv, rv);
        }
        floatx16 s[1] = {};
#pragma unroll
        for (int x = 0; x < L::STEPS; ++x) s[0] = mma_rows<T>(L::row_piece(sk, 0, x), fq[x], s[0]);
        if (DMA && next < end) {
            taken();
            send(a.k, sk, rk);
        }
        if (here != ~0u) {
#pragma unroll
            for (int r = 0; r < 16; ++r)
                if (!(here >> block_row(r) & 1)) s[0][r] = -INFINITY;
        }
        sm.step(s, c, [&](float f) {
#pragma unroll
            for (int j = 0; j < DP / 32; ++j) o[j] *= f;
        });
        Weights<T> w;
        w.set(s[0]);
        if constexpr (sizeof(T) == 2) {
            // the second part (see Weights)
            Weights<T> low;
            s[0] = w.rest(s[0]);
            low.set(s[0]);
#pragma unroll
            for (int j = 0; j < DP / 32; ++j)
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    const Piece x = L::column_piece(sv, 16 * t, j);
                    o[j] = mma16<T>(x, w.w[t], o[j]);
                    o[j] = mma16<T>(x, low.w[t], o[j]);
                }
        } else {
#pragma unroll
            for (int j = 0; j < DP / 32; ++j) o[j] = mma_columns<T, DP>(sv, 0, j, w, o[j]);
        }
        if (DMA && next < end) {
            taken();
            send(a.v, sv, rv);
        }
    }

    // the waves' sums, joined at the largest maximum; a head's row of sums lies in LDS in
    // 16-byte pieces in the order piece ^ head
    const float total = sm.total();
    if (lane < kHeads) {
        sm_m[wave][lane] = sm.m;
        sm_l[wave][lane] = total;
    }
    __syncthreads();
    const int h = lane & 31;
    constexpr int KEY = (DP % 64 == 0 ? 16 : 8) - 1;   // (orders within 16 or 8 pieces, of which a row has whole lots)
    {
        float top = sm_m[0][h];
#pragma unroll
        for (int w = 1; w < kWaves; ++w) top = fmaxf(top, sm_m[w][h]);
        const float f = Softmax<T>::moved(sm.m, top, c);
        if (h < heads) {
            char* p = h < HALF ? sk + h * DP * 4 : sv + (h - HALF) * DP * 4;
#pragma unroll
            for (int j = 0; j < DP / 32; ++j)
#pragma unroll
                for (int g = 0; g < 4; ++g) {
                    const float4 v = make_float4(o[j][4 * g] * f, o[j][4 * g + 1] * f, o[j][4 * g + 2] * f,
                                                 o[j][4 * g + 3] * f);
                    *reinterpret_cast<float4*>(p + (((32 * j + block_row(4 * g)) / 4) ^ (h & KEY)) * 16) = v;
                }
        }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < heads * (DP / 4); i += kWaves * 64) {
        const int n = i / (DP / 4), d = i % (DP / 4) * 4;
        float top = sm_m[0][n], l = 0.f, v[4] = {};
#pragma unroll
        for (int w = 1; w < kWaves; ++w) top = fmaxf(top, sm_m[w][n]);
#pragma unroll
        for (int w = 0; w < kWaves; ++w) {
            l += sm_l[w][n] * Softmax<T>::moved(sm_m[w][n], top, c);
            const char* p = n < HALF ? tk[w] + n * DP * 4 : tv[w] + (n - HALF) * DP * 4;
            const float4 x = *reinterpret_cast<const float4*>(p + ((d / 4) ^ (n & KEY)) * 16);
            v[0] += x.x;
            v[1] += x.y;
            v[2] += x.z;
            v[3] += x.w;
        }
        if (used == 1) {
            const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] *= inv;
            store4n((T*)a.out + seq * a.ldo + (int64_t)(head0 + n) * a.D + d, v, a.D - d);
        } else {
            const int64_t at = ((int64_t)seq * a.heads + head0 + n) * a.splits + split;
            *reinterpret_cast<float4*>(a.part + at * DP + d) = make_float4(v[0], v[1], v[2], v[3]);
            if (d == 0) a.ml[at] = make_float2(top, l);
        }
    }
}

// Joins the workgroups of a sequence's head: their factors first, then their sums, several
// under way.
constexpr int64_t kMaxSplits = 512;   // of a sequence
template <class T, int DP>
__global__ __launch_bounds__(256) void k_attend_paged_join(const PagedArgs a) {
    constexpr int LANES = DP / 4, ROWS = 256 / LANES, DEEP = 4;   // ROWS splits at a time
    __shared__ float4 sm_v[256];
    __shared__ float factor[kMaxSplits], sm[2][4];
    const int seq = blockIdx.x / a.heads, head = blockIdx.x % a.heads;
    const int len = length_of(a, seq), chunk = chunk_of(a, len), used = max(1, (len + chunk - 1) / chunk);
    if (used == 1) return;
    const int64_t at = (int64_t)blockIdx.x * a.splits;
    const float c = a.scale * kLog2e;
    const int x = threadIdx.x % LANES, y = threadIdx.x / LANES, wave = threadIdx.x >> 6;
    static_assert(kMaxSplits == 2 * 256, "two splits a thread");
    float2 ml[2];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
        const int i = threadIdx.x + u * 256;
        ml[u] = i < used ? a.ml[at + i] : make_float2(-INFINITY, 0.f);
    }
    float top = lanes_max<64>(fmaxf(ml[0].x, ml[1].x));
    if ((threadIdx.x & 63) == 0) sm[0][wave] = top;
    __syncthreads();
    top = fmaxf(fmaxf(sm[0][0], sm[0][1]), fmaxf(sm[0][2], sm[0][3]));
    float l = 0.f;
#pragma unroll
    for (int u = 0; u < 2; ++u) {
        const float f = Softmax<T>::moved(ml[u].x, top, c);
        factor[threadIdx.x + u * 256] = f;
        l += ml[u].y * f;
    }
    l = lanes_sum<64>(l);
    if ((threadIdx.x & 63) == 0) sm[1][wave] = l;
    __syncthreads();
    l = (sm[1][0] + sm[1][1]) + (sm[1][2] + sm[1][3]);
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int i0 = y; y < ROWS && i0 < used; i0 += DEEP * ROWS) {
        float4 o[DEEP];
#pragma unroll
        for (int u = 0; u < DEEP; ++u) {
            const int i = i0 + u * ROWS;
            o[u] = i < used ? *reinterpret_cast<const float4*>(a.part + (at + i) * DP + x * 4)
                            : make_float4(0.f, 0.f, 0.f, 0.f);
        }
#pragma unroll
        for (int u = 0; u < DEEP; ++u) {
            const int i = i0 + u * ROWS;
            const float f = i < used ? factor[i] : 0.f;
            v.x = fmaf(o[u].x, f, v.x);
            v.y = fmaf(o[u].y, f, v.y);
            v.z = fmaf(o[u].z, f, v.z);
            v.w = fmaf(o[u].w, f, v.w);
        }
    }
    sm_v[threadIdx.x] = v;
    __syncthreads();
    if (threadIdx.x >= LANES) return;
    float r[4] = {};
    for (int i = 0; i < ROWS; ++i) {
        const float4 o = sm_v[i * LANES + x];
        r[0] += o.x;
        r[1] += o.y;
        r[2] += o.z;
        r[3] += o.w;
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
    for (int e = 0; e < 4; ++e) r[e] *= inv;
    store4n((T*)a.out + seq * a.ldo + (int64_t)head * a.D + x * 4, r, a.D - x * 4);
}

// Tokens of a sequence at most: counts past its end stay within 32 bits.
constexpr int64_t kMaxTokens = int64_t(1) << 30;
// Workgroups that a call is split to reach, by the number of its sequences alone, whose lengths the host does not
// know: a long one among very many short ones is split too little (256 sequences, one of 131072 tokens and
// the others of 500, 32 and 8 heads of 128 bf16: 3050 us; without it 107, it alone 121).
constexpr int64_t kGroups = 2048;

inline int64_t padded_dim(int64_t dim) { return (dim + 31) / 32 * 32; }

template <class T, int DP>
tt_status paged_launch(const PagedArgs& a) {
    const unsigned grid = (unsigned)((int64_t)a.seqs * a.splits * a.blocks * a.kv);
    const bool whole = a.D * sizeof(T) % 16 == 0 && (((uintptr_t)a.k | (uintptr_t)a.v) & 15) == 0;
    auto k = whole ? k_attend_paged<T, DP, true> : k_attend_paged<T, DP, false>;
    TT_LAUNCH(nullptr, "k_attend_paged", a.s, k, dim3(grid), dim3(kWaves * 64), 0, a.s, a);
    TT_LAUNCH_CHECK();
    if (a.splits > 1) {
        TT_LAUNCH(nullptr, "k_attend_paged_join", a.s, (k_attend_paged_join<T, DP>), dim3(a.seqs * a.heads), dim3(256), 0,
                  a.s, a);
        TT_LAUNCH_CHECK();
    }
    return TT_OK;
}

template <class T>
tt_status paged_by_dim(const PagedArgs& a) {
    if (a.D <= 32) return paged_launch<T, 32>(a);
    if (a.D <= 64) return paged_launch<T, 64>(a);
    if (a.D <= 96) return paged_launch<T, 96>(a);
    return paged_launch<T, 128>(a);
}

tt_status paged_sizes(int32_t dtype, int64_t seqs, int64_t heads, int64_t kv, int64_t dim) {
    if (!dtype_ok(dtype) || seqs < 0 || heads < 1 || kv < 1 || dim < 1 || heads % kv != 0) return TT_ERR_INVALID_ARG;
    if (dim > 128 || heads / kv > 256 || heads > (int64_t(1) << 20) || seqs > (int64_t(1) << 20) ||
        seqs * heads > int64_t(1) << 20)
        return TT_ERR_UNSUPPORTED;
    return TT_OK;
}

inline int64_t head_blocks(int64_t heads, int64_t kv) { return (heads / kv + kHeads - 1) / kHeads; }

}  // namespace
}  // namespace tt

using namespace tt;

extern "C" size_t tt_emb_attend_paged_workspace_bytes(int32_t dtype, int64_t seqs, int64_t heads, int64_t kv_heads,
                                                      int64_t dim) {
    if (paged_sizes(dtype, seqs, heads, kv_heads, dim) != TT_OK) return 0;
    // n sequences are cut into at most 1 + kGroups / (n kv_heads blocks) splits each, kMaxSplits at most
    const int64_t parts =
        heads * std::min(seqs * kMaxSplits, seqs + kGroups / (kv_heads * head_blocks(heads, kv_heads)));
    return std::max<size_t>(256, ((size_t)parts * (padded_dim(dim) + 2) * sizeof(float) + 511) & ~size_t(255));
}

extern "C" tt_status tt_emb_attend_paged(int32_t dtype, const void* q, int64_t ldq, const void* k_pages,
                                         const void* v_pages, int64_t pages, int64_t page_size, const int32_t* table,
                                         int64_t ldt, int64_t most_pages, const int64_t* lengths, void* out,
                                         int64_t ldo, int64_t seqs, int64_t heads, int64_t kv_heads, int64_t dim,
                                         float scale, void* workspace, size_t workspace_bytes, void* stream) {
    const tt_status st = paged_sizes(dtype, seqs, heads, kv_heads, dim);
    if (st != TT_OK) return st;
    if (pages < 0 || page_size < 1 || most_pages < 0 || ldt < most_pages || !scale_ok(scale))
        return TT_ERR_INVALID_ARG;
    if (ldq < heads * dim || ldo < heads * dim) return TT_ERR_INVALID_ARG;
    if (seqs > 0 && (!q || !out || !lengths || (most_pages > 0 && !table) || (pages > 0 && (!k_pages || !v_pages))))
        return TT_ERR_INVALID_ARG;
    if (page_size > INT32_MAX || most_pages > INT32_MAX || most_pages * page_size > kMaxTokens || pages > INT32_MAX)
        return TT_ERR_UNSUPPORTED;
    if (!workspace || ((uintptr_t)workspace & 255) != 0) return TT_ERR_INVALID_ARG;
    if (workspace_bytes < tt_emb_attend_paged_workspace_bytes(dtype, seqs, heads, kv_heads, dim))
        return TT_ERR_WORKSPACE;
    if (seqs == 0) return TT_OK;
    PagedArgs a{};
    a.q = q; a.k = k_pages; a.v = v_pages;
    a.ldq = ldq; a.pages = pages; a.ldt = ldt; a.ldo = ldo;
    a.table = table; a.lengths = lengths; a.out = out;
    a.page = (int)page_size; a.most = (int)(most_pages * page_size);
    a.seqs = (int)seqs; a.heads = (int)heads; a.kv = (int)kv_heads;
    a.group = (int)(heads / kv_heads); a.blocks = (int)head_blocks(heads, kv_heads);
    a.D = (int)dim;
    const int64_t n = seqs * kv_heads * a.blocks;
    const int64_t cuts = std::min(kMaxSplits, (kGroups + n - 1) / n);
    a.splits = (int)std::max<int64_t>(1, std::min<int64_t>(cuts, ((int64_t)a.most + kMinChunk - 1) / kMinChunk));
    a.scale = scale;
    a.part = (float*)workspace;
    a.ml = (float2*)(a.part + seqs * heads * a.splits * padded_dim(dim));
    a.s = (hipStream_t)stream;
    if (dtype == TT_F32) return paged_by_dim<float>(a);
    if (dtype == TT_BF16) return paged_by_dim<bf16>(a);
    return paged_by_dim<f16>(a);
}
