// The gated feed-forward block, forward and backward:
//
//   g = x Wg^T,  u = x Wu^T,  out = act(g) u            (x [M][K], Wg, Wu [H][K])
//   dg = dout u act'(g),  du = dout act(g)
//   dx = dg Wg + du Wu,  dWg = dg^T x,  dWu = du^T x
//
// Every product is D[m][n] = sum_k A(m, k) B(n, k) on the matrix cores. An
// operand lies in memory by rows (k contiguous: x and the weights in the
// forward, dg and du in dx) or by columns (m or n contiguous: the weights in
// dx, everything in dW); its tile keeps that layout in LDS, and the fragments
// of a tile by columns are read with the transposing LDS load, so that nothing
// is transposed in memory. The forward forms both projections in one launch
// and act(g) u in its epilogue; the backward's dg and du are formed once, by
// one pass over g, u and dout, into the workspace.
//
// Types. bf16 and f16 operands go to the matrix cores as they are; dg and du
// are rounded to them (half a step of 2^-8 or 2^-11, the size of the error that
// the rounding of dx, dWg and dWu themselves has: 2-norm errors of 0.0023 with it and
// 0.0017 without at 8192 x 4096 x 10240 bf16, where two bf16 parts of each would
// double the backward products' 2070 us). fp32 operands are cut into
// three bf16 planes, x = x0 + x1 + x2 exactly (8 digits each; down to 2^-110,
// where the last plane's digits end), and a product
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

// What a tensor of type T is on the matrix cores: elements E in P planes.
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
constexpr int kBK = 32;   // of the summed length, a step

// The planes of eight values.
__device__ __forceinline__ void cut_planes(const float (&f)[8], Raw8<bf16> (&out)[3]) {
    // values that 8 digits would round up to infinity start from the largest finite one
    constexpr float kTop = 3.38953139e38f;   // 0xFF 2^120
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float a = f[2 * i], b = f[2 * i + 1];
        out[0].w[i] = word_of<bf16>(__builtin_amdgcn_fmed3f(a, -kTop, kTop), __builtin_amdgcn_fmed3f(b, -kTop, kTop));
        a -= out[0].at(2 * i);
        b -= out[0].at(2 * i + 1);
        out[1].w[i] = word_of<bf16>(a, b);
        out[2].w[i] = word_of<bf16>(a - out[1].at(2 * i), b - out[1].at(2 * i + 1));
    }
}
// The six plane products, the smallest first.
__device__ constexpr int kPlaneA[6] = {2, 0, 1, 1, 0, 0}, kPlaneB[6] = {0, 2, 1, 0, 1, 0};

constexpr int kActs = 3;

// The hardware's 2^x and 1/x, each within a step of fp32, serve every type: what
// they leave out (results below 2^-126) is far below any sum it goes into.
__device__ __forceinline__ float sigmoid(float g) {
    return __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(-1.4426950408889634f * g));
}

// The normal distribution's function at g; e = e^(-g^2/2). With x = |g|/sqrt 2 it
// is erfc(x)/2 = e f(x)/2 or one less that, which keeps the small values' digits.
// f(x) = e^(x^2) erfc(x) as t times a polynomial in t = 1/(1 + x/2), fitted for the
// least largest relative error on [0, 10]: 3.1e-8 with these coefficients (at 0), 3e-7
// at most and 5e-8 on average evaluated in fp32. A third of erfcf's time: 32768 x
// 512 fp32 outputs took 34 us of the forward's vector time with that.
__device__ __forceinline__ float normal_cdf(float g, float& e) {
    const float t = __builtin_amdgcn_rcpf(fmaf(fabsf(g), 0.35355339059327376f, 1.f));
    e = __builtin_amdgcn_exp2f(-0.72134752044448170f * g * g);
    float f = 0.0122836372f;
    f = fmaf(f, t, -0.123252928f);
    f = fmaf(f, t, 0.428923279f);
    f = fmaf(f, t, -0.67001456f);
    f = fmaf(f, t, 0.421266973f);
    f = fmaf(f, t, -0.098313421f);
    f = fmaf(f, t, 0.225540325f);
    f = fmaf(f, t, 0.238645166f);
    f = fmaf(f, t, 0.282857001f);
    f = fmaf(f, t, 0.282064497f);
    const float tail = 0.5f * f * t * e;
    return g < 0.f ? tail : 1.f - tail;
}

__device__ __forceinline__ float act_of(int act, float g) {
    float e;
    if (act == TT_ACT_SILU) return g * sigmoid(g);
    if (act == TT_ACT_GELU) return g * normal_cdf(g, e);
    return g > 0.f ? g : g == g ? 0.f : g;   // NaN stays NaN
}
// The activation and its derivative.
__device__ __forceinline__ void act_grad(int act, float g, float& a, float& da) {
    if (act == TT_ACT_SILU) {
        const float s = sigmoid(g);
        a = g * s;
        da = s * (1.f + g * (1.f - s));
    } else if (act == TT_ACT_GELU) {
        float e;
        const float cdf = normal_cdf(g, e);
        a = g * cdf;
        da = cdf + g * (0.39894228040143268f * e);
    } else {
        a = g > 0.f ? g : g == g ? 0.f : g;
        da = g > 0.f ? 1.f : 0.f;
    }
}

// ---------------------------------------------------------------------------
// Elements of a line that lie together in an operand cut into panels: [panel]
// [line][kPanel]. A step's tile by rows is then one piece of memory.
constexpr int kPanel = 32;

// dg and du, into gu [2][Hp / panel][M][panel] (Hp: H up to a multiple of kPanel,
// zeros past H; panel: Hp for plain rows, or kPanel). A wave takes 16 rows of 32
// elements, which it reads as whole cache lines and writes as one piece.
// Bound by memory: 8192 x 10240 bf16, 1.17 GB in 221 us, 5.3 TB/s.
template <class T>
__global__ __launch_bounds__(256) void k_gate_grad(const float* __restrict__ gate, const float* __restrict__ up,
                                                   const T* __restrict__ dout, int64_t ldo, int64_t M, int H, int Hp,
                                                   int panel, int act, T* __restrict__ gu) {
    const int quads = (Hp / kPanel + 3) / 4;   // workgroups along a row
    const int64_t m = blockIdx.x / quads * 16 + (threadIdx.x & 63) / 4;
    const int h = (blockIdx.x % quads * 4 + threadIdx.x / 64) * kPanel + (threadIdx.x & 3) * 8, n = H - h;
    if (m >= M || h >= Hp) return;
    const Raw8<float> g = load8n(gate + m * H + h, n, 0.f), u = load8n(up + m * H + h, n, 0.f);
    const Raw8<T> d = load8n(dout + m * ldo + h, n, (T)0.f);
    float dg[8], du[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        float a, da;
        act_grad(act, g.at(e), a, da);
        const float o = d.at(e);
        dg[e] = e < n ? o * u.at(e) * da : 0.f;
        du[e] = e < n ? o * a : 0.f;
    }
    T* p = panel == kPanel ? gu + (h / kPanel * M + m) * kPanel + h % kPanel : gu + m * panel + h;
    store8n(p, dg, 8);
    store8n(p + M * Hp, du, 8);
}

// 16-bit operands whose rows do not start at whole 16-byte pieces, copied to
// rows that do, zeros past the last column: dst [cols up / panel][rows][panel],
// panel the whole row (a multiple of 8) or kPanel. Up to three operands in one
// launch (blockIdx.y); a wave takes 16 rows of 32 elements.
struct Align {
    const void* src[3];
    void* dst[3];
    int64_t ld[3], rows[3], first;   // first: of the rows of this launch
    int cols, up, panel;             // up: cols up to a multiple of kPanel
};
template <class T>
__global__ __launch_bounds__(256) void k_gate_align(const Align a) {
    const int z = blockIdx.y, quads = (a.up / kPanel + 3) / 4;
    const int64_t r = a.first + (int64_t)(blockIdx.x / quads) * 16 + (threadIdx.x & 63) / 4;
    const int c = (blockIdx.x % quads * 4 + threadIdx.x / 64) * kPanel + (threadIdx.x & 3) * 8;
    if (r >= a.rows[z] || c >= (a.panel == kPanel ? a.up : a.panel)) return;
    const Raw8<T> v = load8n((const T*)a.src[z] + r * a.ld[z] + c, a.cols - c, (T)0.f);
    *reinterpret_cast<Raw8<T>*>((T*)a.dst[z] + (a.panel == kPanel ? (c / kPanel * a.rows[z] + r) * kPanel + c % kPanel
                                                                  : r * a.panel + c)) = v;
}

// ---------------------------------------------------------------------------
// Tiles in LDS.
//
// By rows: ROWS rows of BK elements; a row's 16-byte pieces are stored in the
// order piece ^ key(row), so that the rows that lanes read together lie in
// different banks.
//
// By columns: BK rows (the summed index k) of ROWS elements; a row's 32-byte
// blocks are stored in the order block ^ (k & 3 | k >> 3 & 1): the transposing
// load of 16 lanes takes 32 bytes of four rows k, and four such groups are 8
// rows apart.

__device__ __forceinline__ int row_slot(int row, int piece) { return piece ^ ((row >> 1) & 3); }
__device__ __forceinline__ int col_key(int k) { return (k & 3) | (((k >> 3) & 1) << 2); }

// Byte offset of 16-byte piece `piece` of line `line` (a row, or a k).
template <bool COLS, int BK, int ROWS>
__device__ __forceinline__ int lds_piece(int line, int piece) {
    if (COLS) return line * (ROWS * 2) + ((piece >> 1) ^ col_key(line)) * 32 + (piece & 1) * 16;
    return line * (BK * 2) + row_slot(line, piece) * 16;
}

// The fragment of 16 rows (or columns) x 32 k, k in [32 h, 32 h + 32): lane l
// holds 8 consecutive k, from 8 (l / 16), of its row. By rows the lane's row
// is `row`; by columns the fragment's columns are row0 + 0..15.
template <class V, bool COLS, int BK, int ROWS>
__device__ __forceinline__ V fragment(const char* lds, int row, int row0, int h) {
    const int lane = threadIdx.x & 63, li = lane & 15, lk = lane >> 4;
    if constexpr (!COLS) {
        return *reinterpret_cast<const V*>(lds + lds_piece<false, BK, ROWS>(row, h * 4 + lk));
    } else {
        typedef short s16x4 __attribute__((ext_vector_type(4)));
        const int k = h * 32 + lk * 8 + (li >> 2);   // this lane's addresses: 4 columns of rows k and k + 4
        const char* p = lds + k * (ROWS * 2) + ((row0 >> 4) ^ col_key(k)) * 32 + (li & 3) * 8;
        auto at = [](const char* q) {
            return __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4*)q);
        };
        const s16x4 a = at(p), b = at(p + 4 * ROWS * 2);
        return __builtin_bit_cast(V, __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7));
    }
}

// ---------------------------------------------------------------------------
// The products.

enum Kind { FWD, DX, DW };
// FWD: A = x and B = both weights by rows; DX: A = [dg | du] by rows, B = the
// weights by columns, one after the other; DW: A = dg or du and B = x by columns.

struct Product {
    const void *a, *b, *b2;      // b2: the second weight (FWD, DX)
    int64_t lda, ldb;            // elements from line to line
    int64_t pa, pb;              // elements from panel to panel (kPanel elements of each line); kPanel: plain rows
    int64_t M;
    int N;
    int64_t K;                   // summed length; of each of two parts in DX
    int64_t a2;                  // elements from dg to du (DX, DW)
    void *out, *out2;            // out2: of du (DW)
    int64_t ldo;
    float *gate, *up;            // FWD: g and u [M][N], or null
    int act;
    float* part;                 // partial sums, when the summed length is split: [split][FWD: 2, DW: 2][M][N]
    int steps, split_steps;      // BK-steps in all, and of a split
    int mt, nt, splits;          // tiles
};

// A workgroup's part of a product: tile, split, and which of DW's two results.
struct Place {
    int tile, split, z;
};
__device__ __forceinline__ Place place_of(const Product& q, int block) {
    const int tiles = q.mt * q.nt, rest = block / tiles;
    return {block - rest * tiles, rest % q.splits, rest / q.splits};
}

// Tile of a workgroup: workgroups run on XCD index mod 8, so each XCD takes
// a run of consecutive tiles, and a run goes down bands of 8 rows of tiles,
// whose operands its L2 then holds.
__device__ __forceinline__ void tile_of(const Product& q, int index, int& tm, int& tn) {
    const int all = q.mt * q.nt, per = all / kXcds, rest = all % kXcds;
    const int x = index % kXcds;
    const int t = x * per + min(x, rest) + index / kXcds;
    const int band = t / (8 * q.nt), rows = min(8, q.mt - band * 8), in = t - band * 8 * q.nt;
    tm = band * 8 + in % rows;
    tn = in / rows;
}

// A tile's loads straight to LDS, 16 bytes a lane and 1024 an instruction. A
// lane's offsets within the tile stay; the buffer descriptor's base moves along
// the summed index. Rows and pieces past the operand's last are read as the
// last (their results are dropped); what lies past the summed length is given
// an offset outside the buffer, for which the load delivers zeros.
template <bool COLS, int BK, int ROWS, int WAVES>
struct DmaLoad {
    static constexpr int N = ROWS * BK * 2 / 1024 / WAVES;    // instructions of a wave
    static constexpr int PIECES = COLS ? ROWS / 8 : BK / 8;   // of a line
    static constexpr int LINES = 64 / PIECES;                 // of an instruction
    uint32_t off[N];
    int wave;
    __device__ __forceinline__ int line(int i) const { return (wave * N + i) * LINES + (threadIdx.x & 63) / PIECES; }
    __device__ __forceinline__ int piece(int i) const {
        const int l = line(i), s = (threadIdx.x & 63) % PIECES;
        return COLS ? ((s >> 1) ^ col_key(l)) * 2 + (s & 1) : row_slot(l, s);
    }
    // ld, panel: elements from line to line and from panel to panel; row0: the
    // tile's first row (column) of `rows`
    __device__ __forceinline__ void init(int64_t ld, int64_t panel, int64_t row0, int64_t rows) {
        wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
        const int64_t last = rows - 1 - row0;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            int l = line(i), p = piece(i);
            if (COLS) p = p < last / 8 ? p : (int)(last / 8);
            else l = l < last ? l : (int)last;
            off[i] = (uint32_t)((l * ld + p / (kPanel / 8) * panel) * 2 + p % (kPanel / 8) * 16);
        }
    }
    // Instruction i. base: the tile's first line at this step; left: of the
    // summed length
    __device__ __forceinline__ void load(int i, char* lds, const char* base, int left) const {
#ifdef __HIP_DEVICE_COMPILE__   // the descriptor's type is the device compiler's
        const auto rsrc = __builtin_amdgcn_make_buffer_rsrc((void*)base, 0, 0x7FFFFFFF, 0x00020000);
        const uint32_t o = (COLS ? line(i) : piece(i) * 8) < left ? off[i] : 0x80000000u;
        __builtin_amdgcn_raw_ptr_buffer_load_lds(
            rsrc, (__attribute__((address_space(3))) void*)(lds + (wave * N + i) * 1024), 16, o, 0, 0, 0);
#endif
    }
};

// Lambdas of the product's step are part of it, whatever their size.
#define TT_INLINE __attribute__((always_inline))

// f(0), .., f(N - 1) with constant arguments.
template <int N, class F, int I = 0>
__device__ __forceinline__ void each(F f) {
    if constexpr (I < N) {
        f(std::integral_constant<int, I>{});
        each<N, F, I + 1>(f);
    }
}

// The same tile of an fp32 operand through registers, cut into planes on its way
// to LDS.
template <class T, bool COLS, int BK, int ROWS, int THREADS>
struct RegLoad {
    static constexpr int N = ROWS * BK / 8 / THREADS;
    static constexpr int PIECES = COLS ? ROWS / 8 : BK / 8;
    Raw8<T> r[N];
    __device__ __forceinline__ void load(const T* __restrict__ p, int64_t ld, int64_t row0, int64_t rows, int64_t k0,
                                         int64_t K) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int id = i * THREADS + threadIdx.x, line = id / PIECES, piece = id % PIECES;
            const int64_t l = COLS ? k0 + line : row0 + line, e = (COLS ? row0 : k0) + piece * 8;
            const int64_t n = l < (COLS ? K : rows) ? (COLS ? rows : K) - e : 0;
            r[i] = load8n(p + l * ld + e, (int)(n < 8 ? n : 8), (T)0.f);
        }
    }
    __device__ __forceinline__ void store(char* lds) const {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int id = i * THREADS + threadIdx.x, line = id / PIECES, piece = id % PIECES;
            char* q = lds + lds_piece<COLS, BK, ROWS>(line, piece);
            float f[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) f[e] = r[i].at(e);
            Raw8<bf16> c[3];
            cut_planes(f, c);
#pragma unroll
            for (int s = 0; s < 3; ++s) *reinterpret_cast<Raw8<bf16>*>(q + s * ROWS * BK * 2) = c[s];
        }
    }
};

// What a kernel's waves and tiles are: WM x WN waves, FM x FN fragments each.
template <Kind KIND, int WM, int WN, int FM, int FN>
struct Shape {
    static constexpr int THREADS = WM * WN * 64, TM = WM * FM * 16, TN = WN * FN * 16;
    static constexpr bool AC = KIND == DW, BC = KIND != FWD;
    static constexpr int FH = KIND == FWD ? FN / 2 : FN;  // fragments of D's columns in a wave
    static constexpr int NB = KIND == FWD ? TN / 2 : TN;  // columns of D of a workgroup
    // (FWD: LDS rows [0, NB) of B are Wg's, [NB, TN) Wu's, and so are a wave's fragments)
};

// Orders this wave's LDS writes before its later LDS reads, and those before
// its later writes.
__device__ __forceinline__ void wave_sync() {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// Results of a wave: acc[i][j][r] is D[m][n], m = i * 16 + lane % 16 and
// n = j * 16 + lane / 16 * 4 + r; in FWD the first half of the fragments j is g,
// the second u. They pass through the wave's LDS, CI rows of fragments at a
// time: the first half's columns through x, the second's through y (16 CI rows
// of fp32 each). Memory then sees runs of 128 bytes and more, and the
// activation is a short loop: unrolled over the accumulators it would be more
// instructions than the instruction cache holds. The 16-byte pieces of a row lie
// in the order piece ^ row.
template <class T, Kind KIND, int CI, int FM, int FN>
__device__ __forceinline__ void put_out(const Product& q, Place place, char* x, char* y, const floatx4 (&acc)[FM][FN],
                                        int64_t m0, int n0) {
    constexpr int FH = FN / 2, PIECES = FH * 4, BYTES = PIECES * 16, LANES = PIECES / 2;   // lanes of 8 columns a row
    const int lane = threadIdx.x & 63, li = lane & 15, lk = lane >> 4;
    const int64_t MN = q.M * q.N;
    float *pg = q.gate, *pu = q.up;
    if (KIND == FWD && q.part) {
        pg = q.part + place.split * 2 * MN;
        pu = pg + MN;
    }
    float* part = q.part + (place.split * (KIND == DW ? 2 : 1) + place.z) * MN;
    T* out = (T*)(place.z ? q.out2 : q.out);
#pragma unroll
    for (int c = 0; c < FM; c += CI) {
        wave_sync();
#pragma unroll
        for (int i = 0; i < CI; ++i)
#pragma unroll
            for (int j = 0; j < FH; ++j) {
                const int at = (i * 16 + li) * BYTES + ((j * 4 + lk) ^ (li & (PIECES - 1))) * 16;
                *reinterpret_cast<floatx4*>(x + at) = acc[c + i][j];
                *reinterpret_cast<floatx4*>(y + at) = acc[c + i][j + FH];
            }
        wave_sync();
#pragma unroll 1
        for (int r = lane / LANES; r < CI * 16; r += 64 / LANES) {
            const int p = lane % LANES * 2, key = r & (PIECES - 1);
            float a[8], b[8];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int at = r * BYTES + ((p + h) ^ key) * 16;
                *reinterpret_cast<floatx4*>(a + h * 4) = *reinterpret_cast<const floatx4*>(x + at);
                *reinterpret_cast<floatx4*>(b + h * 4) = *reinterpret_cast<const floatx4*>(y + at);
            }
            const int64_t m = m0 + c * 16 + r;
            const int n = n0 + p * 4;
            if (m >= q.M) continue;
            const int64_t at = m * q.N + n;
            if constexpr (KIND == FWD) {
                const int left = q.N - n;
                if (left <= 0) continue;
                if (!q.part) {
                    float o[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) o[e] = act_of(q.act, a[e]) * b[e];
                    store8n((T*)q.out + m * q.ldo + n, o, left);
                }
                if (pg) {
                    store8n(pg + at, a, left);
                    store8n(pu + at, b, left);
                }
            } else if (q.part) {
                store8n(part + at, a, q.N - n);
                store8n(part + at + FH * 16, b, q.N - n - FH * 16);
            } else {
                store8n(out + m * q.ldo + n, a, q.N - n);
                store8n(out + m * q.ldo + n + FH * 16, b, q.N - n - FH * 16);
            }
        }
    }
}

// Waits until at most LEFT of this wave's loads to LDS are under way, and its LDS
// reads are done, then for the workgroup's other waves.
template <int LEFT>
__device__ __forceinline__ void landed_barrier() {
    // (fences for the compiler only: a workgroup fence would wait for every load under way)
    __atomic_signal_fence(__ATOMIC_SEQ_CST);
    __builtin_amdgcn_s_waitcnt((LEFT & 15) | 0x0070 | (LEFT >> 4) << 14);   // vmcnt(LEFT) lgkmcnt(0)
    __builtin_amdgcn_s_barrier();
    __atomic_signal_fence(__ATOMIC_SEQ_CST);
}

// c += b a, in place in the accumulation registers. (With all 256 of them in use
// the compiler's own choice moves accumulators to and fro, 100 moves a step.)
template <class T, class V>
__device__ __forceinline__ void mma_in_place(floatx4& c, const V& a, const V& b) {
    if constexpr (std::is_same<T, bf16>::value)
        asm volatile("v_mfma_f32_16x16x32_bf16 %0, %1, %2, %0" : "+a"(c) : "v"(b), "v"(a));
    else
        asm volatile("v_mfma_f32_16x16x32_f16 %0, %1, %2, %0" : "+a"(c) : "v"(b), "v"(a));
}

// Waits until the last two matrix instructions' results can be read (24 cycles;
// the earlier ones' can by then). It stands inside the loop, right behind them:
// the compiler does not know that they are matrix instructions, and may read or
// move accumulators anywhere after the loop.
__device__ __forceinline__ void mma_done(floatx4& last, floatx4& before) {
    asm volatile("s_nop 15\n\ts_nop 7" : "+a"(last), "+a"(before));
}

// 16-bit operands whose pieces are whole and aligned: tiles of 32 of the summed
// length go from memory straight to LDS, through a ring of four. While the
// matrix cores work on a step, whose fragments are in registers, the next
// step's fragments are read and the loads of the one four steps on are issued,
// both spread over the products: three steps are under way all the time, which
// covers the latency of the caches past L2. One barrier a step.
//
// The ring's tiles are separate objects, so that the compiler sees which loads a
// read depends on.
template <class T, Kind KIND, int WM, int WN, int FM, int FN>
__device__ __forceinline__ void mm(const Product& q, const Place place, char* sa0, char* sb0, char* sa1, char* sb1,
                                   char* sa2, char* sb2, char* sa3, char* sb3) {
    typedef Shape<KIND, WM, WN, FM, FN> S;
    typedef typename Frag<T>::V V;
    constexpr int BK = kBK, WAVES = WM * WN;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = wave / WN, wn = wave % WN, li = lane & 15;
    int tm, tn;
    tile_of(q, place.tile, tm, tn);
    const int64_t m0 = (int64_t)tm * S::TM;
    const int n0 = tn * S::NB;
    const int s0 = place.split * q.split_steps, s1 = min(q.steps, s0 + q.split_steps);

    DmaLoad<S::AC, BK, S::TM, WAVES> la;
    DmaLoad<S::BC, BK, S::NB, WAVES> lb;
    la.init(q.lda, q.pa, m0, q.M);
    lb.init(q.ldb, q.pb, n0, q.N);
    constexpr int LOADS = la.N + lb.N * (KIND == FWD ? 2 : 1);   // a wave's a step
    static_assert(BK == kPanel && S::TM % kPanel == 0 && S::NB % kPanel == 0, "tiles are whole panels");
    const int64_t ta = (S::AC ? m0 / kPanel * q.pa : m0 * q.lda) * 2 + (KIND == DW ? (int64_t)place.z * q.a2 * 2 : 0);
    const int64_t tb = (S::BC ? n0 / kPanel * q.pb : n0 * q.ldb) * 2;
    const int64_t da = (S::AC ? BK * q.lda : q.pa) * 2, db = (S::BC ? BK * q.ldb : q.pb) * 2;   // from step to step
    // DX: the steps of dg and Wg, then those of du and Wu
    const int half = KIND == DX ? q.steps / 2 : q.steps;
    const char *first_a, *first_b, *first_b2;   // of the step that is loaded next
    int left;                                   // of the summed length there; 0 past the last step
    auto start = [&](int step) TT_INLINE {
        const bool second = KIND == DX && step >= half;
        const int64_t k = second ? step - half : step;
        first_a = (const char*)q.a + ta + k * da + (second ? q.a2 * 2 : 0);
        first_b = (const char*)(second ? q.b2 : q.b) + tb + k * db;
        first_b2 = (const char*)q.b2 + tb + k * db;
        left = (int)(q.K - k * BK);
    };
    auto advance = [&](int step) TT_INLINE {   // to `step`
        if (KIND == DX && step == half) {
            start(step);
        } else {
            first_a += da;
            first_b += db;
            if (KIND == FWD) first_b2 += db;
            left -= BK;
        }
        if (step >= s1) left = 0;
    };
    // load x of the step that is loaded next
    auto load = [&](char* sa, char* sb, int x) TT_INLINE {
        if (x < la.N) la.load(x, sa, first_a, left);
        else if (x < la.N + lb.N) lb.load(x - la.N, sb, first_b, left);
        else lb.load(x - la.N - lb.N, sb + S::NB * BK * 2, first_b2, left);
    };

    floatx4 acc[FM][FN];
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j) acc[i][j] = floatx4{0.f, 0.f, 0.f, 0.f};

    // fragment x of a step: B's first, which every row of products needs, then A's
    V f0[FN + FM], f1[FN + FM];
    auto read = [&](V (&f)[FN + FM], const char* sa, const char* sb, int x) TT_INLINE {
        if (x < FN) {
            const int w = (wn * S::FH + x % S::FH) * 16;
            f[x] = fragment<V, S::BC, BK, S::NB>(sb + x / S::FH * S::NB * BK * 2, w + li, w, 0);
        } else {
            const int r = wm * FM * 16 + (x - FN) * 16;
            f[x] = fragment<V, S::AC, BK, S::TM>(sa, r + li, r, 0);
        }
    };
    // Step s: products of its fragments f; fragments g of step s + 1 from (ta, tb), early enough
    // that the last arrive before they are needed; loads of step s + 4 into (sa, sb), step s's own.
    // A matrix instruction takes 16 cycles, in which a wave can issue three others: reads and loads
    // stand one by one between them, never together.
    auto step = [&](int s, V (&f)[FN + FM], V (&g)[FN + FM], char* sa, char* sb, const char* ta,
                    const char* tb) TT_INLINE {
        landed_barrier<2 * LOADS>();   // step s + 1 is there, s + 2 and s + 3 may be under way
        constexpr int SLOTS = FM * FN, READ = SLOTS - FN;
        each<SLOTS>([&](auto slot) TT_INLINE {
            constexpr int t = slot;
            __builtin_amdgcn_sched_barrier(0);
            mma_in_place<T>(acc[t / FN][t % FN], f[FN + t / FN], f[t % FN]);
            if constexpr (t < READ)
                each<(t + 1) * (FN + FM) / READ - t * (FN + FM) / READ>(
                    [&](auto x) TT_INLINE { read(g, ta, tb, t * (FN + FM) / READ + x); });
            each<LOADS>([&](auto x) TT_INLINE {
                if constexpr (t == (2 * x + 1) * SLOTS / (2 * LOADS)) load(sa, sb, x);
            });
        });
        advance(s + 5);
    };
    if (s0 < s1) {
        start(s0);
        each<4>([&](auto d) TT_INLINE {
            char *sa = d == 0 ? sa0 : d == 1 ? sa1 : d == 2 ? sa2 : sa3, *sb = d == 0 ? sb0 : d == 1 ? sb1 : d == 2 ? sb2 : sb3;
            each<LOADS>([&](auto x) TT_INLINE { load(sa, sb, x); });
            advance(s0 + d + 1);
        });
        landed_barrier<3 * LOADS>();
        each<FN + FM>([&](auto x) TT_INLINE { read(f0, sa0, sb0, x); });
        for (int s = s0; s < s1; s += 4) {   // up to three steps of zeros at the end
            step(s, f0, f1, sa0, sb0, sa1, sb1);
            step(s + 1, f1, f0, sa1, sb1, sa2, sb2);
            step(s + 2, f0, f1, sa2, sb2, sa3, sb3);
            step(s + 3, f1, f0, sa3, sb3, sa0, sb0);
            mma_done(acc[FM - 1][FN - 1], acc[FM - 1][FN - 2]);
        }
    }
    landed_barrier<0>();   // no load to LDS is under way when the results pass through it
    static_assert(WAVES == 4 && FM / (FM > 4 ? 2 : 1) * 16 * (FN / 2) * 16 * 4 <= S::TM * BK * 2, "room for a wave's results");
    char* x = wave < 2 ? (wave == 0 ? sa0 : sa1) : (wave == 2 ? sa2 : sa3);
    char* y = wave < 2 ? (wave == 0 ? sb0 : sb1) : (wave == 2 ? sb2 : sb3);
    put_out<T, KIND, FM / (FM > 4 ? 2 : 1)>(q, place, x, y, acc, m0 + wm * FM * 16, n0 + wn * S::FH * 16);
}

#define TT_RING(SIZE_A, SIZE_B)                                                                                    \
    __shared__ __align__(16) char sa0[SIZE_A], sb0[SIZE_B], sa1[SIZE_A], sb1[SIZE_B], sa2[SIZE_A], sb2[SIZE_B],    \
        sa3[SIZE_A], sb3[SIZE_B]

template <class T, int WM, int WN, int FM, int FN>
__global__ __launch_bounds__(WM* WN * 64, FM * FN <= 32 ? 2 : 1) void k_gate_mm(const Product q) {
    TT_RING(WM * FM * 16 * kBK * 2, WN * FN * 16 * kBK * 2);
    mm<T, FWD, WM, WN, FM, FN>(q, place_of(q, blockIdx.x), sa0, sb0, sa1, sb1, sa2, sb2, sa3, sb3);
}

// The backward's products in one launch, dx's workgroups first: neither waits for
// the other, and their last workgroups fill the chip together.
template <class T, int WM, int WN, int FM, int FN>
__global__ __launch_bounds__(WM* WN * 64, FM * FN <= 32 ? 2 : 1) void k_gate_mm_back(const Product dx, const Product dw) {
    TT_RING(WM * FM * 16 * kBK * 2, WN * FN * 16 * kBK * 2);
    const int n = dx.mt * dx.nt * dx.splits, b = blockIdx.x;
    if (b < n) mm<T, DX, WM, WN, FM, FN>(dx, place_of(dx, b), sa0, sb0, sa1, sb1, sa2, sb2, sa3, sb3);
    else mm<T, DW, WM, WN, FM, FN>(dw, place_of(dw, b - n), sa0, sb0, sa1, sb1, sa2, sb2, sa3, sb3);
}

constexpr int kCutBytes = 3 * 128 * kBK * 2;   // of 128 rows' planes

// fp32 operands of any alignment: tiles pass through registers, where they are
// cut into planes, loaded while the matrix cores work on the step before.
template <class T, Kind KIND>
__device__ __forceinline__ void mm_cut(const Product& q, const Place place, char* sa, char* sb) {
    constexpr int FM = 4, FN = 4, WM = 2, WN = 2;
    typedef Shape<KIND, WM, WN, FM, FN> S;
    typedef typename Mat<T>::E E;
    typedef typename Frag<E>::V V;
    constexpr int BK = kBK, P = Mat<T>::P;
    constexpr int PA = S::TM * BK * 2, PB = S::NB * BK * 2;   // bytes of a plane
    static_assert(P * PA <= kCutBytes && (KIND == FWD ? 2 : 1) * P * PB <= kCutBytes, "room for the planes");
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = wave / WN, wn = wave % WN, li = lane & 15;
    int tm, tn;
    tile_of(q, place.tile, tm, tn);
    const int64_t m0 = (int64_t)tm * S::TM;
    const int n0 = tn * S::NB;
    const int s0 = place.split * q.split_steps, s1 = min(q.steps, s0 + q.split_steps);

    RegLoad<T, S::AC, BK, S::TM, 256> la;
    RegLoad<T, S::BC, BK, S::NB, 256> lb, lb2;
    const T* pa = (const T*)q.a + (KIND == DW ? (int64_t)place.z * q.a2 : 0);
    const int half = KIND == DX ? q.steps / 2 : q.steps;
    auto load = [&](int step) {
        const bool second = KIND == DX && step >= half;
        const int64_t k = (int64_t)(second ? step - half : step) * BK;
        la.load(pa + (second ? q.a2 : 0), q.lda, m0, q.M, k, q.K);
        lb.load((const T*)(second ? q.b2 : q.b), q.ldb, n0, q.N, k, q.K);
        if constexpr (KIND == FWD) lb2.load((const T*)q.b2, q.ldb, n0, q.N, k, q.K);
    };

    floatx4 acc[FM][FN];
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j) acc[i][j] = floatx4{0.f, 0.f, 0.f, 0.f};

    if (s0 < s1) load(s0);
    for (int s = s0; s < s1; ++s) {
        __syncthreads();
        la.store(sa);
        lb.store(sb);
        if constexpr (KIND == FWD) lb2.store(sb + P * PB);
        __syncthreads();
        if (s + 1 < s1) load(s + 1);
#pragma unroll
        for (int h = 0; h < BK / 32; ++h) {
            V fa[P][FM];
#pragma unroll
            for (int i = 0; i < FM; ++i)
#pragma unroll
                for (int p = 0; p < P; ++p) {
                    const int r = wm * FM * 16 + i * 16;
                    fa[p][i] = fragment<V, S::AC, BK, S::TM>(sa + p * PA, r + li, r, h);
                }
#pragma unroll
            for (int j = 0; j < FN; ++j) {
                V fb[P];
                const int w = (wn * S::FH + j % S::FH) * 16;
#pragma unroll
                for (int p = 0; p < P; ++p)
                    fb[p] = fragment<V, S::BC, BK, S::NB>(sb + (j / S::FH * P + p) * PB, w + li, w, h);
#pragma unroll
                for (int t = 0; t < 6; ++t)
#pragma unroll
                    for (int i = 0; i < FM; ++i)
                        acc[i][j] = Frag<E>::mma(fb[kPlaneB[t]], fa[kPlaneA[t]][i], acc[i][j]);
            }
        }
    }
    __syncthreads();
    put_out<T, KIND, 1>(q, place, sa + wave * 4096, sa + wave * 4096 + 2048, acc, m0 + wm * FM * 16,
                        n0 + wn * S::FH * 16);
}

template <class T>
__global__ __launch_bounds__(256, 2) void k_gate_mm_cut(const Product q) {
    __shared__ __align__(16) char sa[kCutBytes], sb[kCutBytes];
    mm_cut<T, FWD>(q, place_of(q, blockIdx.x), sa, sb);
}
template <class T>
__global__ __launch_bounds__(256, 2) void k_gate_mm_cut_back(const Product dx, const Product dw) {
    __shared__ __align__(16) char sa[kCutBytes], sb[kCutBytes];
    const int n = dx.mt * dx.nt * dx.splits, b = blockIdx.x;
    if (b < n) mm_cut<T, DX>(dx, place_of(dx, b), sa, sb);
    else mm_cut<T, DW>(dw, place_of(dw, b - n), sa, sb);
}

// The splits' partial sums, joined in their order. FWD: both projections of
// eight columns, then as the product's epilogue.
template <class T>
__global__ __launch_bounds__(256) void k_gate_join_fwd(const Product q) {
    const int per = (q.N + 7) / 8;
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x, m = i / per;
    const int n = (int)(i - m * per) * 8, left = q.N - n;
    if (m >= q.M) return;
    const int64_t MN = q.M * q.N, at = m * q.N + n;
    float g[8] = {}, u[8] = {}, o[8];
#pragma unroll 4
    for (int s = 0; s < q.splits; ++s) {
        const Raw8<float> a = load8n(q.part + s * 2 * MN + at, left, 0.f);
        const Raw8<float> b = load8n(q.part + (s * 2 + 1) * MN + at, left, 0.f);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            g[e] += a.at(e);
            u[e] += b.at(e);
        }
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) o[e] = act_of(q.act, g[e]) * u[e];
    store8n((T*)q.out + m * q.ldo + n, o, left);
    if (q.gate) {
        store8n(q.gate + at, g, left);
        store8n(q.up + at, u, left);
    }
}

// The backward's: dx's in the first dx_groups workgroups, then dWg's and dWu's.
template <class T>
__global__ __launch_bounds__(256) void k_gate_join(const Product dx, const Product dw, int dx_groups, int dw_groups) {
    const bool first = (int)blockIdx.x < dx_groups;
    const Product& q = first ? dx : dw;
    const int block = first ? blockIdx.x : blockIdx.x - dx_groups;
    const int z = first ? 0 : block / dw_groups, batch = first ? 1 : 2;
    const int per = (q.N + 7) / 8;
    const int64_t i = (int64_t)(block - z * dw_groups) * 256 + threadIdx.x, m = i / per;
    const int n = (int)(i - m * per) * 8, left = q.N - n;
    if (m >= q.M) return;
    const int64_t MN = q.M * q.N, at = m * q.N + n;
    float o[8] = {};
#pragma unroll 8
    for (int s = 0; s < q.splits; ++s) {
        const Raw8<float> a = load8n(q.part + (s * batch + z) * MN + at, left, 0.f);
#pragma unroll
        for (int e = 0; e < 8; ++e) o[e] += a.at(e);
    }
    store8n((T*)(z ? q.out2 : q.out) + m * q.ldo + n, o, left);
}

// ---------------------------------------------------------------------------
// The forward of a few rows: the weights' one pass through memory is all that
// counts. A workgroup takes 16 hidden units and its four waves a quarter of the
// summed length each; fragments go from memory to registers, without LDS, and
// the waves' sums meet at the end.
template <class T, int MF>
__global__ __launch_bounds__(256) void k_gate_few(const Product q) {
    typedef typename Mat<T>::E E;
    typedef typename Frag<E>::V V;
    constexpr int P = Mat<T>::P, DEEP = P == 1 ? 4 : 2;   // 32-steps under way
    __shared__ floatx4 sum[3][2 * MF][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, li = lane & 15, lk = lane >> 4;
    const int n0 = blockIdx.x * 16;
    const int64_t per = (((q.K + 31) / 32 + 3) / 4) * 32, k0 = wave * per, k1 = min(q.K, k0 + per);
    const int64_t n = min(n0 + li, q.N - 1);
    const T *pg = (const T*)q.b + n * q.ldb + lk * 8, *pu = (const T*)q.b2 + n * q.ldb + lk * 8;
    const T* px[MF];
#pragma unroll
    for (int i = 0; i < MF; ++i) px[i] = (const T*)q.a + min((int64_t)(i * 16 + li), q.M - 1) * q.lda + lk * 8;
    floatx4 acc[2][MF];
#pragma unroll
    for (int i = 0; i < MF; ++i) acc[0][i] = acc[1][i] = floatx4{0.f, 0.f, 0.f, 0.f};
    auto planes = [](const Raw8<T>& r, V (&v)[P]) {
        if constexpr (P == 1) {
            v[0] = __builtin_bit_cast(V, r);
        } else {
            float f[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) f[e] = r.at(e);
            Raw8<bf16> c[3];
            cut_planes(f, c);
#pragma unroll
            for (int p = 0; p < 3; ++p) v[p] = __builtin_bit_cast(V, c[p]);
        }
    };
    auto mma = [](const V (&b)[P], const V (&a)[P], floatx4 c) {
        if constexpr (P == 1) return Frag<E>::mma(b[0], a[0], c);
#pragma unroll
        for (int t = 0; t < (P == 1 ? 0 : 6); ++t) c = Frag<E>::mma(b[kPlaneB[t] % P], a[kPlaneA[t] % P], c);
        return c;
    };
    for (int64_t k = k0; k < k1; k += 32 * DEEP) {
        Raw8<T> rg[DEEP], ru[DEEP], rx[DEEP][MF];
#pragma unroll
        for (int d = 0; d < DEEP; ++d) {
            const int64_t kk = k + d * 32, left = k1 - kk - lk * 8;
            const int c = (int)(left < 8 ? left : 8);
            rg[d] = load8n(pg + kk, c, (T)0.f);
            ru[d] = load8n(pu + kk, c, (T)0.f);
#pragma unroll
            for (int i = 0; i < MF; ++i) rx[d][i] = load8n(px[i] + kk, c, (T)0.f);
        }
#pragma unroll
        for (int d = 0; d < DEEP; ++d) {
            V vg[P], vu[P];
            planes(rg[d], vg);
            planes(ru[d], vu);
#pragma unroll
            for (int i = 0; i < MF; ++i) {
                V vx[P];
                planes(rx[d][i], vx);
                acc[0][i] = mma(vg, vx, acc[0][i]);
                acc[1][i] = mma(vu, vx, acc[1][i]);
            }
        }
    }
    if (wave > 0) {
#pragma unroll
        for (int i = 0; i < MF; ++i) {
            sum[wave - 1][2 * i][lane] = acc[0][i];
            sum[wave - 1][2 * i + 1][lane] = acc[1][i];
        }
    }
    __syncthreads();
    if (wave > 0) return;
#pragma unroll
    for (int i = 0; i < MF; ++i) {
#pragma unroll
        for (int w = 0; w < 3; ++w) {
            acc[0][i] += sum[w][2 * i][lane];
            acc[1][i] += sum[w][2 * i + 1][lane];
        }
        const int64_t m = i * 16 + li;
        const int c = n0 + lk * 4, left = q.N - c;
        if (m >= q.M || left <= 0) continue;
        float g[4], u[4], o[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            g[r] = acc[0][i][r];
            u[r] = acc[1][i][r];
            o[r] = act_of(q.act, g[r]) * u[r];
        }
        store4n((T*)q.out + m * q.ldo + c, o, left);
        if (q.gate) {
            store4n(q.gate + m * q.N + c, g, left);
            store4n(q.up + m * q.N + c, u, left);
        }
    }
}

// ---------------------------------------------------------------------------
// Host side.

inline int64_t up_to(int64_t n, int64_t m) { return (n + m - 1) / m * m; }

// Rows the forward takes without tiles: 16, and 32 but for large 16-bit weights,
// whose tiles are many enough to keep memory busy by themselves (32 rows bf16:
// 4096 x 10240 46 us without tiles, 33 with them; 2048 x 8192 19 and 19.5; 512 x 1536
// 7.6 and 10.1; fp32 4096 x 10240 98 and 111).
bool few_rows(int32_t dtype, int64_t M, int64_t K, int64_t H) {
    return M <= 16 || (M <= 32 && (dtype == TT_F32 || K * H <= int64_t(1) << 24));
}

// How a launch's products are cut: tiles of 256 x 256 when these fill the chip, else
// of 128 x 128, two of which a CU takes. Summed lengths that are long beside what
// each of 512 workgroups would get are split into pieces of about that, eight steps
// or more (for large tiles 32: a partial sum of theirs is written and read again).
struct Cut {
    bool big;
    int mt, nt, steps, split_steps, splits;
};
struct Sum {   // D [M][N], N counting both projections; summed length in steps; how many of them
    int64_t M, N, steps, batch;
};
template <int N>
void cut_sums(int32_t dtype, const Sum (&p)[N], Cut (&c)[N]) {
    auto tiles = [&](int64_t t) {
        int64_t n = 0;
        for (int i = 0; i < N; ++i) {
            c[i].mt = (int)((p[i].M + t - 1) / t);
            c[i].nt = (int)((p[i].N + t - 1) / t);
            n += (int64_t)c[i].mt * c[i].nt * p[i].batch;
        }
        return n;
    };
    const bool big = dtype != TT_F32 && tiles(256) >= 256;
    if (!big) tiles(128);
    int64_t work = 0;
    for (int i = 0; i < N; ++i) work += (int64_t)c[i].mt * c[i].nt * p[i].batch * p[i].steps;
    const int64_t piece = std::max<int64_t>(big ? 32 : 8, (work + 511) / 512);
    for (int i = 0; i < N; ++i) {
        c[i].big = big;
        c[i].steps = (int)p[i].steps;
        const int64_t n = std::max<int64_t>(1, std::min<int64_t>(p[i].steps / piece, 64));
        c[i].split_steps = (int)std::max<int64_t>(1, (p[i].steps + n - 1) / n);
        c[i].splits = std::max(1, (c[i].steps + c[i].split_steps - 1) / c[i].split_steps);
    }
}

// Bytes that a launch's partial sums take at most, at these sizes and at any smaller M:
// a product that is split is split into pieces of work / 512 steps or more, so that the
// tiles and splits of all that are are 512 workgroups at most, and of eight steps or more.
template <int N>
size_t partial_bytes(int32_t dtype, const Sum (&p)[N]) {
    Cut c[N];
    cut_sums(dtype, p, c);
    const int64_t tile = c[0].big ? 256 : 128;
    int64_t sums = 0;
    for (int i = 0; i < N; ++i) {
        const int64_t n = std::min<int64_t>(p[i].steps / 8, 64);
        if (n > 1) sums += n * p[i].batch * p[i].M * p[i].N;
    }
    return sums ? up_to(std::min(sums, 512 * tile * tile) * sizeof(float), 256) + 256 * N : 0;   // each rounded up
}

// Where things lie in the workspace (bytes): x and the weights with aligned
// rows (16-bit types; used where the caller's are not), the backward's dg and
// du, partial sums. forward, backward: what a call of these sizes needs;
// most_forward, most: what a forward, or either, of these sizes or of fewer rows
// does (splits come and go with the rows, all else only grows).
struct GateSpace {
    int64_t Kp, Hp;
    Cut fwd[1], back[2];   // back: dx, dW
    size_t x, wg, wu, gu, part, part_dx, part_dw, forward, backward, most_forward, most;
    GateSpace(int32_t dtype, int64_t M, int64_t K, int64_t H) : Kp(up_to(K, kPanel)), Hp(up_to(H, kPanel)) {
        const int64_t k = (K + kBK - 1) / kBK, h = (H + kBK - 1) / kBK, m = (M + kBK - 1) / kBK;
        const Sum fwd_sums[1] = {{M, 2 * H, k, 1}}, back_sums[2] = {{M, K, 2 * h, 1}, {H, K, m, 2}};
        cut_sums(dtype, fwd_sums, fwd);
        cut_sums(dtype, back_sums, back);
        size_t at = 0;
        auto take = [&](size_t bytes) {
            const size_t o = at;
            at += up_to(bytes, 256);
            return o;
        };
        const bool copies = dtype != TT_F32;
        x = take(copies ? M * Kp * 2 : 0);
        wg = take(copies ? H * Kp * 2 : 0);
        wu = take(copies ? H * Kp * 2 : 0);
        gu = at;
        part = gu;
        const size_t few = 256;
        if (few_rows(dtype, M, K, H)) {   // (and any smaller M)
            forward = most_forward = few;
        } else {
            forward = std::max(few, at + (fwd[0].splits == 1 ? 0 : (size_t)fwd[0].splits * 2 * M * H * 4));
            most_forward = std::max(few, at + partial_bytes(dtype, fwd_sums));
        }
        take(M * 2 * Hp * (dtype == TT_F32 ? 4 : 2));
        const size_t parts = at;
        part_dx = take(back[0].splits == 1 ? 0 : (size_t)back[0].splits * M * K * 4);
        part_dw = take(back[1].splits == 1 ? 0 : (size_t)back[1].splits * 2 * H * K * 4);
        backward = std::max(few, at);
        most = std::max({few, most_forward, parts + partial_bytes(dtype, back_sums)});
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

void cut_product(Product& q, const Cut& c, char* part) {
    q.mt = c.mt;
    q.nt = c.nt;
    q.steps = c.steps;
    q.split_steps = c.split_steps;
    q.splits = c.splits;
    q.part = c.splits > 1 ? (float*)part : nullptr;
}

template <class T>
tt_status forward_product(const Product& q, bool big, hipStream_t s) {
    const dim3 grid((unsigned)(q.mt * q.nt * q.splits)), block(256);
    if constexpr (sizeof(T) == 4) {
        TT_LAUNCH(nullptr, "k_gate_mm_cut", s, (k_gate_mm_cut<T>), grid, block, 0, s, q);
    } else {
        auto k = big ? k_gate_mm<T, 2, 2, 8, 8> : k_gate_mm<T, 2, 2, 4, 4>;
        TT_LAUNCH(nullptr, "k_gate_mm", s, k, grid, block, 0, s, q);
    }
    TT_LAUNCH_CHECK();
    if (q.splits > 1) {
        const unsigned g = grid_for(q.M * ((q.N + 7) / 8), 256);
        TT_LAUNCH(nullptr, "k_gate_join_fwd", s, (k_gate_join_fwd<T>), dim3(g), dim3(256), 0, s, q);
        TT_LAUNCH_CHECK();
    }
    return TT_OK;
}

template <class T>
tt_status backward_products(const Product& dx, const Product& dw, bool big, hipStream_t s) {
    const dim3 grid((unsigned)(dx.mt * dx.nt * dx.splits + dw.mt * dw.nt * dw.splits * 2)), block(256);
    if constexpr (sizeof(T) == 4) {
        TT_LAUNCH(nullptr, "k_gate_mm_cut_back", s, (k_gate_mm_cut_back<T>), grid, block, 0, s, dx, dw);
    } else {
        auto k = big ? k_gate_mm_back<T, 2, 2, 8, 8> : k_gate_mm_back<T, 2, 2, 4, 4>;
        TT_LAUNCH(nullptr, "k_gate_mm_back", s, k, grid, block, 0, s, dx, dw);
    }
    TT_LAUNCH_CHECK();
    auto groups = [](const Product& q) { return q.splits > 1 ? (int)grid_for(q.M * ((q.N + 7) / 8), 256) : 0; };
    const int gx = groups(dx), gw = groups(dw);
    if (gx + gw > 0) {
        TT_LAUNCH(nullptr, "k_gate_join", s, (k_gate_join<T>), dim3((unsigned)(gx + 2 * gw)), dim3(256), 0, s, dx, dw,
                  gx, gw);
        TT_LAUNCH_CHECK();
    }
    return TT_OK;
}

// x and the weights as the products take them: as they are, or (16-bit types)
// copied to the workspace where a row does not start at a whole 16-byte piece.
// The copies are cut into panels for the forward, which reads them by rows: a
// step's tile is then one piece of memory instead of 64 bytes a row. That alone
// pays for copying aligned inputs too where a product is long enough beside its
// inputs, M H / (M + 2 H) from 2700 on (bf16 forward, copied and as they are, us):
// 8192 x 4096 x 10240 (2925) 1061 and 1122, 32768 x 1024 x 4096 (3276) 620 and 627,
// 16384 x 512 x 16384 (5461) 865 and 951, 16384 x 1024 x 4096 (2730) 316 and 316;
// but 6144 x 4096 x 10240 (2363) 836 and 819, 8192 x 4096 x 4096 (2048) 433 and 421,
// 4096 x 8192 x 16384 (1820) 1688 and 1609.
struct Inputs {
    const void *x, *wg, *wu;
    int64_t ldx, px, ldw, pw;   // from line to line, from panel to panel
};
template <class T>
tt_status aligned_inputs(Inputs& in, const GateArgs& a, const GateSpace& sp, bool panels) {
    in = Inputs{a.x, a.wg, a.wu, a.ldx, kPanel, a.K, kPanel};
    if constexpr (sizeof(T) == 4) {
        return TT_OK;
    } else {
        const bool pays = panels && a.M * a.H / (a.M + 2 * a.H) >= 2700;
        const bool x = pays || a.K % 8 != 0 || a.ldx % 8 != 0 || ((uintptr_t)a.x & 15) != 0;
        const bool w = pays || a.K % 8 != 0 || (((uintptr_t)a.wg | (uintptr_t)a.wu) & 15) != 0;
        Align c{};
        c.cols = (int)a.K;
        c.up = (int)sp.Kp;
        c.panel = panels ? kPanel : (int)up_to(a.K, 8);
        int n = 0;
        auto take = [&](const void*& p, int64_t ld, int64_t rows, size_t at) {
            c.src[n] = p;
            c.ld[n] = ld;
            c.rows[n] = rows;
            c.dst[n++] = a.ws + at;
            p = a.ws + at;
        };
        if (x && a.M > 0) {
            take(in.x, a.ldx, a.M, sp.x);
            in.ldx = c.panel;
            if (panels) in.px = a.M * kPanel;
        }
        if (w) {
            take(in.wg, a.K, a.H, sp.wg);
            take(in.wu, a.K, a.H, sp.wu);
            in.ldw = c.panel;
            if (panels) in.pw = a.H * kPanel;
        }
        if (n == 0) return TT_OK;
        // as many rows a launch as its threads allow, which must stay below 2^32 in all
        const int64_t rows = std::max(c.rows[0], c.rows[n - 1]), quads = (sp.Kp / kPanel + 3) / 4;
        const int64_t step = (int64_t(1) << 22) / quads * 16;
        for (c.first = 0; c.first < rows; c.first += step) {
            const int64_t groups = (std::min(step, rows - c.first) + 15) / 16 * quads;
            TT_LAUNCH(nullptr, "k_gate_align", a.s, (k_gate_align<T>), dim3((unsigned)groups, n), dim3(256), 0, a.s, c);
            TT_LAUNCH_CHECK();
        }
        return TT_OK;
    }
}

template <class T>
tt_status gate_forward(const GateArgs& a, const GateSpace& sp) {
    Product q{};
    q.a = a.x; q.b = a.wg; q.b2 = a.wu;
    q.lda = a.ldx; q.ldb = a.K;
    q.M = a.M; q.N = (int)a.H; q.K = a.K;
    q.out = a.out; q.ldo = a.ldout;
    q.gate = a.gate; q.up = a.up; q.act = a.act;
    if (few_rows(sizeof(T) == 4 ? TT_F32 : TT_BF16, a.M, a.K, a.H)) {
        auto k = a.M <= 16 ? k_gate_few<T, 1> : k_gate_few<T, 2>;
        TT_LAUNCH(nullptr, "k_gate_few", a.s, k, dim3(grid_for(a.H, 16)), dim3(256), 0, a.s, q);
        TT_LAUNCH_CHECK();
        return TT_OK;
    }
    Inputs in;
    const tt_status st = aligned_inputs<T>(in, a, sp, true);
    if (st != TT_OK) return st;
    q.a = in.x; q.b = in.wg; q.b2 = in.wu;
    q.lda = in.ldx; q.ldb = in.ldw;
    q.pa = in.px; q.pb = in.pw;
    cut_product(q, sp.fwd[0], a.ws + sp.part);
    return forward_product<T>(q, sp.fwd[0].big, a.s);
}

template <class T>
tt_status gate_backward(const GateArgs& a, const GateSpace& sp) {
    T* gu = (T*)(a.ws + sp.gu);
    const int panel = sizeof(T) == 2 ? kPanel : (int)sp.Hp;
    Inputs in;
    tt_status st = aligned_inputs<T>(in, a, sp, false);
    if (st != TT_OK) return st;
    Product q{};
    q.a = gu;
    q.lda = panel;
    q.pa = sizeof(T) == 2 ? a.M * kPanel : kPanel;
    q.pb = kPanel;
    q.a2 = a.M * sp.Hp;
    if (a.M > 0) {
        TT_LAUNCH(nullptr, "k_gate_grad", a.s, (k_gate_grad<T>),
                  dim3((unsigned)((a.M + 15) / 16 * ((sp.Hp / kPanel + 3) / 4))), dim3(256), 0, a.s, a.gate, a.up,
                  (const T*)a.dout, a.lddout, a.M, (int)a.H, (int)sp.Hp, panel, a.act, gu);
        TT_LAUNCH_CHECK();
    }
    Product dx = q, dw = q;
    dx.b = in.wg; dx.b2 = in.wu; dx.ldb = in.ldw;
    dx.M = a.M; dx.N = (int)a.K; dx.K = a.H;
    dx.out = a.dx; dx.ldo = a.lddx;
    cut_product(dx, sp.back[0], a.ws + sp.part_dx);
    dw.b = in.x; dw.ldb = in.ldx;
    dw.M = a.H; dw.N = (int)a.K; dw.K = a.M;
    dw.out = a.dwg; dw.out2 = a.dwu; dw.ldo = a.K;
    cut_product(dw, sp.back[1], a.ws + sp.part_dw);
    return backward_products<T>(dx, dw, sp.back[0].big, a.s);
}

tt_status gate_by_type(int32_t dtype, const GateArgs& a, size_t workspace_bytes, bool backward) {
    const GateSpace sp(dtype, a.M, a.K, a.H);
    if (workspace_bytes < (backward ? sp.backward : sp.forward)) return TT_ERR_WORKSPACE;
    if (!backward && a.M == 0) return TT_OK;
    if (dtype == TT_F32) return backward ? gate_backward<float>(a, sp) : gate_forward<float>(a, sp);
    if (dtype == TT_BF16) return backward ? gate_backward<bf16>(a, sp) : gate_forward<bf16>(a, sp);
    return backward ? gate_backward<f16>(a, sp) : gate_forward<f16>(a, sp);
}

constexpr int64_t kGateMaxWidth = 1 << 20;
constexpr int64_t kGateMaxRows = int64_t(1) << 22;   // 32-bit offsets from panel to panel within a tile

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
    return GateSpace(dtype, rows, dim, hidden).most;
}

extern "C" size_t tt_emb_gate_forward_workspace_bytes(int32_t dtype, int64_t rows, int64_t dim, int64_t hidden) {
    if (gate_check(dtype, rows, dim, hidden) != TT_OK) return 0;
    return GateSpace(dtype, rows, dim, hidden).most_forward;
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
    GateArgs a{};
    a.x = x; a.wg = w_gate; a.wu = w_up; a.out = out;
    a.ldx = ldx; a.ldout = ldout; a.M = rows; a.K = dim; a.H = hidden;
    a.gate = gate; a.up = up; a.act = act; a.ws = (char*)workspace; a.s = (hipStream_t)stream;
    return gate_by_type(dtype, a, workspace_bytes, false);
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
    GateArgs a{};
    a.x = x; a.wg = w_gate; a.wu = w_up; a.dout = dout; a.dx = dx; a.dwg = dw_gate; a.dwu = dw_up;
    a.ldx = ldx; a.lddout = lddout; a.lddx = lddx; a.M = rows; a.K = dim; a.H = hidden;
    a.gate = const_cast<float*>(gate); a.up = const_cast<float*>(up);
    a.act = act; a.ws = (char*)workspace; a.s = (hipStream_t)stream;
    return gate_by_type(dtype, a, workspace_bytes, true);
}
