// moe_route_backward: gradients of moe_route on the logits, the input and the
// weight.
//
// Mathematics. The routing weights are w_j = s_j / sum s over the picks, so
//   dl_j = w_j (1 - s_j) (dw_j - sum_i w_i dw_i)
// at the picks, to which the losses' gradient d_aux is added; then two matrix
// products of the [T,E] gradient G of the logits:
//   d_hidden = scale G W      (T x H, over E)
//   d_W      = scale G^T h    (E x H, over T)
//
// Both products run on the matrix cores as products of BF16 planes with FP32
// accumulation, as the projection does: an FP32 value is the sum of three
// BF16 planes, each the next 8 significant bits of what the previous ones
// missed (exact for magnitudes from 2^-100), and products of planes are exact in
// FP32. A BF16 input is its own single plane. The products kept are those of
// plane indices with sum <= 2 (the others are below 2^-23 of the largest), or
// <= 1 with two planes each where the result is rounded to BF16 anyway
// (2^-16 against its 2^-9).
//
// One kernel computes both: C[M,N] = A B with A the gradient and B a matrix
// whose rows are the summation index (W's experts, the input's tokens). A
// small kernel computes G and writes its planes twice as MFMA fragments, once
// per product; B is read in its own row-major layout, and each lane transposes
// eight rows of four columns in registers: the wave's columns are permuted (lane
// n of MFMA j holds column 4 n + j), which costs one v_perm per two elements and
// makes a lane's four results of a row adjacent in memory.
#include <cmath>

#include "launch.hpp"

namespace moe {
namespace {

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef float f32x16_t __attribute__((ext_vector_type(16)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

constexpr int kKStep = 16;            // summation index per MFMA
constexpr int kFrag = 1024;           // bytes of an A fragment: 32 rows x 16
constexpr size_t kZeroBytes = 1024;   // zeros standing for rows that do not count

__device__ __forceinline__ void split_pair(float x0, float x1, uint32_t& p0, uint32_t& p1, uint32_t& p2) {
    p0 = cvt_pk_bf16(x0, x1);
    const float r0 = x0 - bf16_lo(p0), r1 = x1 - bf16_hi(p0);
    p1 = cvt_pk_bf16(r0, r1);
    p2 = cvt_pk_bf16(r0 - bf16_lo(p1), r1 - bf16_hi(p1));
}

// ------------------------------------------------ gradient of the logits ----

constexpr int kPrepRows = 32, kPrepCols = 128, kPrepBlock = 256;
constexpr int kPrepStride = kPrepCols + 4;

// Eight values -> np planes of a fragment lane, plane p 64 lanes further on.
__device__ __forceinline__ void write_fragment(const float (&v)[8], int np, u32x4* __restrict__ out) {
    u32x4 q[3];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        uint32_t a, b, c;
        split_pair(v[2 * j], v[2 * j + 1], a, b, c);
        q[0][j] = a;
        q[1][j] = b;
        q[2][j] = c;
    }
#pragma unroll
    for (int p = 0; p < 3; ++p)
        if (p < np) out[p * kWave] = q[p];
}

// Block (x, y): tokens [32 x, +32), experts [128 y, +128). Fragments of a
// matrix with rows m and summation index c: [m / 32][c / 16][plane][lane], lane
// l holding row l % 32, c = 8 (l / 32) .. +8.
//   frag_h: rows tokens, summed over experts (np_h planes)
//   frag_w: rows experts, summed over tokens (three planes)
// row_bits: for every 16 tokens a word, one bit each, set for valid ones.
// d_aux may be d_logits: a block reads its tile before it writes it.
__global__ __launch_bounds__(kPrepBlock) void logits_gradient_kernel(
    const float* __restrict__ d_topk_w, const float* d_aux, const float* __restrict__ logits,
    const int32_t* __restrict__ ids, const float* __restrict__ topk_w, const uint8_t* __restrict__ mask, int T,
    int E, int k, float* d_logits, u32x4* __restrict__ frag_h, int np_h, u32x4* __restrict__ frag_w,
    uint32_t* __restrict__ row_bits, uint32_t* __restrict__ zeros) {
    __shared__ float tile[kPrepRows * kPrepStride];
    __shared__ int32_t pick_id[kPrepRows][MOE_MAX_TOPK];
    __shared__ float pick_v[kPrepRows][MOE_MAX_TOPK];
    const int tid = threadIdx.x;
    const int t0 = blockIdx.x * kPrepRows, e0 = blockIdx.y * kPrepCols;
    if (zeros && blockIdx.x == 0 && blockIdx.y == 0)
        for (int i = tid; i < static_cast<int>(kZeroBytes / 4); i += kPrepBlock) zeros[i] = 0;

    for (int i = tid; i < kPrepRows * kPrepCols; i += kPrepBlock) {
        const int r = i / kPrepCols, c = i - r * kPrepCols;
        const int t = t0 + r, e = e0 + c;
        float v = 0.f;
        if (d_aux && t < T && e < E && mask[t]) v = d_aux[static_cast<size_t>(t) * E + e];
        tile[r * kPrepStride + c] = v;
    }
    if (d_topk_w) {
        // eight threads a token
        const int r = tid >> 3, sub = tid & 7;
        const int t = t0 + r;
        const bool ok = t < T && mask[t] != 0;
        float s = 0.f;
        for (int j = sub; j < k; j += 8) {
            const size_t at = static_cast<size_t>(t) * k + j;
            int id = -1;
            if (ok) {
                id = ids[at];
                if (id < 0 || id >= E) id = -1;
            }
            pick_id[r][j] = id;
            if (id >= 0) s = __builtin_fmaf(topk_w[at], d_topk_w[at], s);
        }
        s = group_sum(s, 8);
        for (int j = sub; j < k; j += 8) {
            const int id = pick_id[r][j];
            float v = 0.f;
            if (id >= e0 && id < e0 + kPrepCols) {
                const size_t at = static_cast<size_t>(t) * k + j;
                // 1 - sigmoid(l) = 1 / (1 + exp(l))
                v = topk_w[at] * (d_topk_w[at] - s) / (1.f + expf(logits[static_cast<size_t>(t) * E + id]));
            }
            pick_v[r][j] = v;
        }
        __syncthreads();
        for (int j = sub; j < k; j += 8) {
            const int id = pick_id[r][j];
            if (id < e0 || id >= e0 + kPrepCols) continue;
            // the first pick of an expert adds every pick of it
            bool first = true;
            float v = pick_v[r][j];
            for (int i = 0; i < k; ++i) {
                if (i == j || pick_id[r][i] != id) continue;
                if (i < j) first = false;
                else v += pick_v[r][i];
            }
            if (first) tile[r * kPrepStride + id - e0] += v;
        }
    }
    __syncthreads();
    for (int i = tid; i < kPrepRows * kPrepCols; i += kPrepBlock) {
        const int r = i / kPrepCols, c = i - r * kPrepCols;
        const int t = t0 + r, e = e0 + c;
        if (t < T && e < E) d_logits[static_cast<size_t>(t) * E + e] = tile[r * kPrepStride + c];
    }
    if (row_bits && blockIdx.y == 0 && tid < kWave) {
        const bool ok = tid < kPrepRows && t0 + tid < T && mask[t0 + tid] != 0;
        const uint64_t b = ballot(ok);
        if (tid < 2) row_bits[blockIdx.x * 2 + tid] = static_cast<uint32_t>(b >> (16 * tid)) & 0xFFFFu;
    }
    const int lane = tid & 63;
    if (frag_h) {
        const int ks_n = (E + kKStep - 1) / kKStep;
        for (int f = tid / kWave; f < kPrepCols / kKStep; f += kPrepBlock / kWave) {
            const int ks = e0 / kKStep + f;
            if (ks >= ks_n) break;
            float v[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = tile[(lane & 31) * kPrepStride + f * kKStep + 8 * (lane >> 5) + j];
            write_fragment(v, np_h, frag_h + (static_cast<size_t>(blockIdx.x) * ks_n + ks) * np_h * kWave + lane);
        }
    }
    if (frag_w) {
        const int mt_n = (E + 31) / 32;
        const size_t ks_n = 2 * static_cast<size_t>(gridDim.x);
        for (int f = tid / kWave; f < 2 * (kPrepCols / 32); f += kPrepBlock / kWave) {
            const int mt = e0 / 32 + (f >> 1), half = f & 1;
            if (mt >= mt_n) break;
            float v[8];
#pragma unroll
            for (int j = 0; j < 8; ++j)
                v[j] = tile[(half * kKStep + 8 * (lane >> 5) + j) * kPrepStride + (f >> 1) * 32 + (lane & 31)];
            write_fragment(v, 3, frag_w + (mt * ks_n + 2 * blockIdx.x + half) * 3 * kWave + lane);
        }
    }
}

// FP32 rows [rows,H] -> np BF16 planes [np][rows][H]; rows whose mask byte is
// zero become zeros.
__global__ __launch_bounds__(256) void split_rows_kernel(const float* __restrict__ x, const uint8_t* __restrict__ mask,
                                                         int rows, int H, int np, uint16_t* __restrict__ planes) {
    const long long quads = static_cast<long long>(rows) * (H / 4);
    const size_t plane = static_cast<size_t>(rows) * H;
    for (long long i = blockIdx.x * 256ll + threadIdx.x; i < quads; i += gridDim.x * 256ll) {
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        if (!mask || mask[i / (H / 4)]) v = reinterpret_cast<const float4*>(x)[i];
        u32x2 q[3];
        uint32_t a, b, c;
        split_pair(v.x, v.y, a, b, c);
        q[0][0] = a;
        q[1][0] = b;
        q[2][0] = c;
        split_pair(v.z, v.w, a, b, c);
        q[0][1] = a;
        q[1][1] = b;
        q[2][1] = c;
#pragma unroll
        for (int p = 0; p < 3; ++p)
            if (p < np) reinterpret_cast<u32x2*>(planes + p * plane)[i] = q[p];
    }
}

// ------------------------------------------------------------- product ----

template <int N>
__device__ __forceinline__ void wait_vmcnt() {
    static_assert(N >= 0 && N < 64, "vmcnt range");
    __builtin_amdgcn_s_waitcnt((N & 0xF) | ((N >> 4) << 14) | (0x7 << 4) | (0xF << 8));
}

// Block tile 64 WM x 128 WN, one wave per 64 x 128 (2 x 4 accumulators of
// v_mfma_f32_32x32x16_bf16). Every K-step's A fragments and B rows go through
// a ring of LDS stages filled LOOK steps ahead by direct-to-LDS loads of 1 KB,
// the same number by every wave, so that waiting for all but the newest
// (LOOK - 1) groups means the step's own group has landed.
template <int NA, int NB, int WM, int WN>
struct ProductShape {
    static constexpr int WAVES = WM * WN;
    static constexpr int BLOCK = WAVES * kWave;
    static constexpr int BM = 64 * WM, BN = 128 * WN;
    static constexpr int LA = 2 * WM * NA;            // 1 KB loads of A per step
    static constexpr int LB = NB * 4 * WN;            // and of B: NB planes of 16 rows
    static constexpr int LOADS = (LA + LB) / WAVES;   // per wave
    static constexpr int STAGE = (LA + LB) * kFrag;
    static constexpr int SETS = 4 * STAGE <= 136 * 1024 ? 4 : 3;
    static constexpr int LOOK = SETS - 1;
    static constexpr size_t LDS = static_cast<size_t>(SETS) * STAGE;
    static_assert((LA + LB) % WAVES == 0, "every wave issues the same number of loads");
    static_assert(LDS <= 160 * 1024, "LDS of a CU");
    static_assert(BN * 2 <= static_cast<int>(kZeroBytes) && BN <= 512, "a row of zeros, a row per load");
};

struct ProductArgs {
    const u32x4* a;            // fragments [m / 32][K / 16][NA][64]
    const uint16_t* b;         // [NB][rows][n]
    size_t b_plane;            // elements between planes
    const uint32_t* row_bits;  // valid rows of each K-step, or NULL
    const uint16_t* zeros;     // kZeroBytes of zeros
    float scale;
    int m, n, rows, a_steps;   // a_steps: K-steps the fragments hold (>= steps)
    int steps, split_steps;    // K-steps in all, and of one split
    int tiles_m, tiles_n, nsplit;
    void* c;                   // [m,n]; with nsplit > 1 FP32 partial sums [nsplit,m,n]
};

template <int NA, int NB, int WM, int WN, bool BF16_OUT>
__global__ __launch_bounds__(WM* WN* kWave) void product_kernel(const ProductArgs p) {
    using S = ProductShape<NA, NB, WM, WN>;
    extern __shared__ __attribute__((aligned(16))) char lds[];
    // the blocks of an XCD (every eighth) take consecutive tiles: row tiles
    // of one column tile first, then column tiles, then K-splits
    const int total = p.tiles_m * p.tiles_n * p.nsplit;
    const int per_xcd = static_cast<int>(gridDim.x) / 8;
    const int idx = static_cast<int>(blockIdx.x % 8) * per_xcd + static_cast<int>(blockIdx.x / 8);
    if (idx >= total) return;
    const int split = idx / (p.tiles_m * p.tiles_n);
    const int tile = idx - split * (p.tiles_m * p.tiles_n);
    const int n_tile = tile / p.tiles_m, m_tile = tile - n_tile * p.tiles_m;
    const int m0 = m_tile * S::BM, n0 = n_tile * S::BN;
    const int s_beg = split * p.split_steps;
    const int nst = min(p.steps, s_beg + p.split_steps) - s_beg;

    const int lane = __lane_id();
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int wm = wave / WN, wn = wave % WN;

    f32x16_t acc[2][4];
#pragma unroll
    for (int mi = 0; mi < 2; ++mi)
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int i = 0; i < 16; ++i) acc[mi][j][i] = 0.f;

    const int m_last = (p.m + 31) / 32 - 1;
    // a B load covers 512 / BN rows; this lane's row within them and columns
    constexpr int kRowsPerLoad = 512 / S::BN;
    const int b_row = lane / (S::BN / 8);
    const int b_col = (lane % (S::BN / 8)) * 8;
    const int b_src_col = min(n0 + b_col, p.n - 8);   // columns past n repeat the last ones (never stored)

    auto issue = [&](int step, int set, uint32_t bits) {
        char* base = lds + set * S::STAGE;
        const int ks = s_beg + step;
#pragma unroll
        for (int i = 0; i < S::LOADS; ++i) {
            const int l = wave + i * S::WAVES;   // this load of the stage
            const void* src;
            if (l < S::LA) {
                const int mt = min(m0 / 32 + l / NA, m_last);
                src = p.a + ((static_cast<size_t>(mt) * p.a_steps + ks) * NA + l % NA) * kWave + lane;
            } else {
                const int lb = l - S::LA;
                const int pl = lb / (4 * WN);
                const int r = (lb - pl * 4 * WN) * kRowsPerLoad + b_row;
                const int row = ks * kKStep + r;
                const bool ok = row < p.rows && (bits >> r & 1);
                src = ok ? p.b + pl * p.b_plane + static_cast<size_t>(row) * p.n + b_src_col : p.zeros + b_col;
            }
            __builtin_amdgcn_global_load_lds(src, base + l * kFrag, 16, 0, 0);
        }
    };
    // through the constant address space: a scalar load, which the wait for the
    // vector loads does not count
    const auto* bits_at = (const __attribute__((address_space(4))) uint32_t*)(p.row_bits);
    auto bits_of = [&](int step) { return p.row_bits ? bits_at[s_beg + step] : 0xFFFFu; };

#pragma unroll
    for (int s = 0; s < S::LOOK; ++s) {
        issue(min(s, nst - 1), s, bits_of(min(s, nst - 1)));
        __builtin_amdgcn_sched_barrier(0);
    }
    uint32_t next_bits = bits_of(min(S::LOOK, nst - 1));
    int set = 0;
    for (int s = 0; s < nst; ++s) {
        __builtin_amdgcn_sched_barrier(0);
        wait_vmcnt<(S::LOOK - 1) * S::LOADS>();   // step s's loads have landed
        __builtin_amdgcn_s_barrier();             // ... in every wave, and step s - 1's stage is free
        __builtin_amdgcn_sched_barrier(0);
        const int refill = set == 0 ? S::SETS - 1 : set - 1;
        // past the last step the last one's loads are repeated, into a stage
        // that is not read again
        issue(min(s + S::LOOK, nst - 1), refill, next_bits);
        next_bits = bits_of(min(s + 1 + S::LOOK, nst - 1));
        __builtin_amdgcn_sched_barrier(0);
        const char* base = lds + set * S::STAGE;
        bf16x8_t a[NA][2];
#pragma unroll
        for (int pl = 0; pl < NA; ++pl)
#pragma unroll
            for (int mi = 0; mi < 2; ++mi)
                a[pl][mi] = *reinterpret_cast<const bf16x8_t*>(base + ((wm * 2 + mi) * NA + pl) * kFrag + lane * 16);
        bf16x8_t b[NB][4];
#pragma unroll
        for (int pl = 0; pl < NB; ++pl) {
            const char* src = base + S::LA * kFrag + (pl * kKStep + 8 * (lane >> 5)) * (S::BN * 2) + wn * 256 +
                              (lane & 31) * 8;
            u32x2 r[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) r[i] = *reinterpret_cast<const u32x2*>(src + i * (S::BN * 2));
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                u32x4 v;
#pragma unroll
                for (int d = 0; d < 4; ++d)
                    v[d] = __builtin_amdgcn_perm(r[2 * d + 1][j >> 1], r[2 * d][j >> 1],
                                                 j & 1 ? 0x07060302u : 0x05040100u);
                b[pl][j] = __builtin_bit_cast(bf16x8_t, v);
            }
        }
        // the products of planes (pa, pb) with pa + pb < max(NA, NB)
        constexpr int PMAX = NA > NB ? NA : NB;
#pragma unroll
        for (int pa = 0; pa < NA; ++pa)
#pragma unroll
            for (int pb = 0; pb < NB; ++pb) {
                if (pa + pb >= PMAX) continue;
#pragma unroll
                for (int mi = 0; mi < 2; ++mi)
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        acc[mi][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a[pa][mi], b[pb][j], acc[mi][j], 0, 0, 0);
            }
        set = set + 1 == S::SETS ? 0 : set + 1;
    }
    wait_vmcnt<0>();   // the repeated loads, before the block's LDS is given away

    // lane: columns 4 (lane % 32) + j of the wave's 128, rows
    // 8 (i / 4) + 4 (lane / 32) + i % 4 of each 32
    const int col = n0 + wn * 128 + 4 * (lane & 31);
    if (col >= p.n) return;
    const size_t part = p.nsplit > 1 ? static_cast<size_t>(split) * p.m : 0;
    const float scale = p.nsplit > 1 ? 1.f : p.scale;
#pragma unroll
    for (int mi = 0; mi < 2; ++mi)
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const int row = m0 + (wm * 2 + mi) * 32 + 8 * (i >> 2) + 4 * (lane >> 5) + (i & 3);
            if (row >= p.m) continue;
            const float v0 = acc[mi][0][i] * scale, v1 = acc[mi][1][i] * scale;
            const float v2 = acc[mi][2][i] * scale, v3 = acc[mi][3][i] * scale;
            const size_t at = (part + row) * p.n + col;
            if constexpr (BF16_OUT)
                *reinterpret_cast<u32x2*>(static_cast<uint16_t*>(p.c) + at) =
                    u32x2{cvt_pk_bf16(v0, v1), cvt_pk_bf16(v2, v3)};
            else
                *reinterpret_cast<float4*>(static_cast<float*>(p.c) + at) = make_float4(v0, v1, v2, v3);
        }
}

// out = scale * (sum of n partial arrays, in order); zeros without any.
__global__ __launch_bounds__(256) void sum_parts_kernel(const float4* __restrict__ parts, int n, long long quads,
                                                        float scale, float4* __restrict__ out) {
    for (long long i = blockIdx.x * 256ll + threadIdx.x; i < quads; i += gridDim.x * 256ll) {
        float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
        for (int q = 0; q < n; ++q) {
            const float4 v = parts[q * quads + i];
            s.x += v.x;
            s.y += v.y;
            s.z += v.z;
            s.w += v.w;
        }
        out[i] = make_float4(s.x * scale, s.y * scale, s.z * scale, s.w * scale);
    }
}

// -------------------------------------------------------------- planning ----

inline size_t round256(size_t b) { return (b + 255) / 256 * 256; }

struct ProductPlan {
    int wm;   // waves along the rows: block tile 64 wm x 256
    int tiles_m, tiles_n, steps, nsplit, split_steps;
};

// Row tiles of 64, 128 or 256 as the rows need. K is split where that shortens
// the product more than the partial sums, written and read once, cost: a step
// of a 256-row tile is taken as 1 us, partial sums as 4 TB/s.
inline ProductPlan plan_product(int m, int n, long long k, bool may_split) {
    ProductPlan p;
    p.wm = m <= 64 ? 1 : m <= 128 ? 2 : 4;
    p.tiles_m = ceil_div(m, 64 * p.wm);
    p.tiles_n = ceil_div(n, 256);
    p.steps = ceil_div(k, kKStep);
    p.nsplit = 1;
    p.split_steps = p.steps;
    if (!may_split) return p;
    const long long tiles = static_cast<long long>(p.tiles_m) * p.tiles_n;
    const int slots = p.wm == 4 ? 256 : 512;   // blocks resident at once
    double best = 0;
    for (int ns = 1; ns <= 32 && (ns == 1 || p.steps / ns >= 8); ++ns) {
        const int each = ceil_div(p.steps, ns);
        const int used = ceil_div(p.steps, each);
        const double rounds = static_cast<double>(ceil_div(tiles * used, slots));
        double us = rounds * each * (0.25 * p.wm);
        if (used > 1) us += 8e-6 * used * static_cast<double>(m) * n / 4.0;
        if (ns == 1 || us < best) {
            best = us;
            p.nsplit = used;
            p.split_steps = each;
        }
    }
    return p;
}

struct RouteBackwardPlan {
    int np_h;   // planes of each factor of d_hidden
    ProductPlan h, w;
    size_t zeros, bits, frag_h, frag_w, w_planes, x_planes, parts, bytes;
};

inline bool route_backward_shape_ok(int T, int H, int E) {
    return T >= 0 && T <= (1 << 30) && H >= 16 && H <= MOE_MAX_HIDDEN && H % 16 == 0 && E >= 1 &&
           E <= MOE_MAX_EXPERTS;
}

inline RouteBackwardPlan plan_route_backward(int T, int H, int E, int dtype) {
    RouteBackwardPlan p;
    const bool f32 = dtype == MOE_DTYPE_F32;
    p.np_h = f32 ? 3 : 2;
    p.h = plan_product(T, H, E, false);
    p.w = plan_product(E, H, T, true);
    const size_t t32 = ceil_div(T, 32), e16 = ceil_div(E, 16), e32 = ceil_div(E, 32);
    size_t at = 0;
    auto take = [&](size_t n) {
        const size_t here = at;
        at += round256(n);
        return here;
    };
    p.zeros = take(kZeroBytes);
    p.bits = take(t32 * 2 * sizeof(uint32_t));
    p.frag_h = take(t32 * e16 * p.np_h * kFrag);
    p.frag_w = take(e32 * t32 * 2 * 3 * kFrag);
    p.w_planes = take(static_cast<size_t>(p.np_h) * E * H * 2);
    p.x_planes = take(f32 ? 3ull * T * H * 2 : 0);
    p.parts = take(p.w.nsplit > 1 ? sizeof(float) * p.w.nsplit * E * H : 0);
    p.bytes = at;
    return p;
}

template <int NA, int NB, int WM, bool BF16_OUT>
int launch_product_as(const ProductArgs& a, void* stream) {
    using S = ProductShape<NA, NB, WM, 2>;
    const long long total = static_cast<long long>(a.tiles_m) * a.tiles_n * a.nsplit;
    return launch(product_kernel<NA, NB, WM, 2, BF16_OUT>, dim3(8 * ceil_div(total, 8)), dim3(S::BLOCK), S::LDS,
                  stream, a);
}

template <int NA, int NB, bool BF16_OUT>
int launch_product(const ProductPlan& p, ProductArgs a, void* stream) {
    a.steps = p.steps;
    a.split_steps = p.split_steps;
    a.tiles_m = p.tiles_m;
    a.tiles_n = p.tiles_n;
    a.nsplit = p.nsplit;
    return p.wm == 1   ? launch_product_as<NA, NB, 1, BF16_OUT>(a, stream)
           : p.wm == 2 ? launch_product_as<NA, NB, 2, BF16_OUT>(a, stream)
                       : launch_product_as<NA, NB, 4, BF16_OUT>(a, stream);
}

}  // namespace
}  // namespace moe

extern "C" size_t moe_route_backward_workspace_bytes(int T, int H, int E, int hidden_dtype, int logits_in) {
    using namespace moe;
    if (logits_in || !route_backward_shape_ok(T, H, E)) return 0;
    if (hidden_dtype != MOE_DTYPE_BF16 && hidden_dtype != MOE_DTYPE_F32) return 0;
    return T == 0 ? 0 : plan_route_backward(T, H, E, hidden_dtype).bytes;
}

extern "C" int moe_route_backward(const float* d_topk_w, const float* d_aux, const void* hidden, int hidden_dtype,
                                  const float* W, const float* logits, const int32_t* topk_ids, const float* topk_w,
                                  const uint8_t* token_mask, float scale, int T, int H, int E, int k,
                                  float* d_logits, void* d_hidden, float* d_W, void* workspace,
                                  size_t workspace_bytes, void* stream) {
    using namespace moe;
    const bool logits_in = hidden == nullptr && T > 0;
    if (!route_backward_shape_ok(T, logits_in ? 16 : H, E) || k < 1 || k > MOE_MAX_TOPK || k > E)
        return MOE_ERR_BAD_SHAPE;
    if (hidden_dtype != MOE_DTYPE_BF16 && hidden_dtype != MOE_DTYPE_F32) return MOE_ERR_BAD_DTYPE;
    if (!std::isfinite(scale)) return MOE_ERR_BAD_ARG;
    if (!all_aligned16(d_topk_w, d_aux, static_cast<const char*>(hidden), W, logits, topk_ids, topk_w, token_mask,
                       d_logits, static_cast<const char*>(d_hidden), d_W))
        return MOE_ERR_ALIGN;
    const long long w_quads = static_cast<long long>(E) * H / 4;
    auto grid_of = [](long long n) {
        const long long g = (n + 255) / 256;
        return dim3(static_cast<unsigned>(g < 2048 ? g : 2048));
    };
    if (T == 0)   // no token: the weight's gradient is zero
        return d_W ? launch(sum_parts_kernel, grid_of(w_quads), dim3(256), 0, stream, nullptr, 0, w_quads, 0.f,
                            reinterpret_cast<float4*>(d_W))
                   : MOE_OK;
    if (!token_mask || !d_logits || (!d_topk_w && !d_aux)) return MOE_ERR_NULL_ARG;
    if (d_topk_w && (!logits || !topk_ids || !topk_w)) return MOE_ERR_NULL_ARG;
    if (logits_in && (d_hidden || d_W)) return MOE_ERR_NULL_ARG;
    if (d_hidden && !W) return MOE_ERR_NULL_ARG;
    const bool f32 = hidden_dtype == MOE_DTYPE_F32;
    RouteBackwardPlan p{};
    char* ws = static_cast<char*>(workspace);
    if (!logits_in) {
        p = plan_route_backward(T, H, E, hidden_dtype);
        if (!workspace || workspace_bytes < p.bytes || (reinterpret_cast<uintptr_t>(workspace) & 255u) != 0)
            return MOE_ERR_WORKSPACE;
    }
    auto* frag_h = d_hidden ? reinterpret_cast<u32x4*>(ws + p.frag_h) : nullptr;
    auto* frag_w = d_W ? reinterpret_cast<u32x4*>(ws + p.frag_w) : nullptr;
    auto* bits = d_W ? reinterpret_cast<uint32_t*>(ws + p.bits) : nullptr;
    auto* zeros = logits_in ? nullptr : reinterpret_cast<uint32_t*>(ws + p.zeros);
    int st = launch(logits_gradient_kernel, dim3(ceil_div(T, kPrepRows), ceil_div(E, kPrepCols)), dim3(kPrepBlock), 0,
                    stream, d_topk_w, d_aux, logits, topk_ids, topk_w, token_mask, T, E, k, d_logits, frag_h, p.np_h,
                    frag_w, bits, zeros);
    if (st != MOE_OK) return st;
    ProductArgs a{};
    a.zeros = reinterpret_cast<const uint16_t*>(zeros);
    a.scale = scale;
    a.n = H;
    if (d_hidden) {
        auto* planes = reinterpret_cast<uint16_t*>(ws + p.w_planes);
        st = launch(split_rows_kernel, grid_of(w_quads), dim3(256), 0, stream, W, nullptr, E, H, p.np_h, planes);
        if (st != MOE_OK) return st;
        a.a = frag_h;
        a.b = planes;
        a.b_plane = static_cast<size_t>(E) * H;
        a.row_bits = nullptr;
        a.m = T;
        a.rows = E;
        a.a_steps = ceil_div(E, kKStep);
        a.c = d_hidden;
        st = f32 ? launch_product<3, 3, false>(p.h, a, stream) : launch_product<2, 2, true>(p.h, a, stream);
        if (st != MOE_OK) return st;
    }
    if (d_W) {
        a.a = frag_w;
        a.m = E;
        a.rows = T;
        a.a_steps = 2 * ceil_div(T, 32);
        a.c = p.w.nsplit > 1 ? static_cast<void*>(ws + p.parts) : static_cast<void*>(d_W);
        if (f32) {
            auto* planes = reinterpret_cast<uint16_t*>(ws + p.x_planes);
            st = launch(split_rows_kernel, grid_of(static_cast<long long>(T) * H / 4), dim3(256), 0, stream,
                        static_cast<const float*>(hidden), token_mask, T, H, 3, planes);
            if (st != MOE_OK) return st;
            a.b = planes;
            a.b_plane = static_cast<size_t>(T) * H;
            a.row_bits = nullptr;   // the planes hold zeros for invalid tokens
            st = launch_product<3, 3, false>(p.w, a, stream);
        } else {
            a.b = static_cast<const uint16_t*>(hidden);
            a.b_plane = 0;
            a.row_bits = bits;
            st = launch_product<3, 1, false>(p.w, a, stream);
        }
        if (st != MOE_OK) return st;
        if (p.w.nsplit > 1)
            st = launch(sum_parts_kernel, grid_of(w_quads), dim3(256), 0, stream,
                        reinterpret_cast<const float4*>(ws + p.parts), p.w.nsplit, w_quads, scale,
                        reinterpret_cast<float4*>(d_W));
    }
    return st;
}
