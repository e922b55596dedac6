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
//
// Bound by the matrix cores: six BF16 products of T E H for a BF16 input. Measured,
// 8192 tokens of 8192 x 256 (206 GFLOP): input's gradient 107-117 us, weight's 98-112
// (0.9-1.05 PFLOP/s, by the card's clock: the same loop runs at what its power
// allows, matrix cores 61-64% busy at 2.0-2.1 GHz), the gradient and planes 14,
// the partial sums' addition 13; 4001 tokens of 4096 x 2560 (503 GFLOP): 209-232
// and 217-246, 51 (270 MB: a copy's rate) and 27.
#include <cmath>
#include <type_traits>

#include "launch.hpp"

namespace moe {
namespace {

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef float f32x16_t __attribute__((ext_vector_type(16)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef int32_t i32x4 __attribute__((ext_vector_type(4)));

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
constexpr int kPrepLoads = kPrepRows * kPrepCols / 4 / kPrepBlock;   // 16-byte pieces of the tile per thread
constexpr int kSplitQuads = 4;                                       // 16-byte pieces of a row split per thread

// Four floats at any 4-byte aligned address (rows of an E that is not a
// multiple of four): still one 16-byte access.
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x4_any __attribute__((ext_vector_type(4), aligned(4)));

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

// FP32 rows to split into BF16 planes [np][rows][H].
struct SplitArgs {
    const float* x;        // NULL: nothing to split
    const uint8_t* mask;   // rows whose byte is zero become zeros; NULL: none
    int rows, np;
    uint16_t* planes;
};

struct PrepArgs {
    const float* d_topk_w;
    const float* d_aux;
    const float* logits;
    const int32_t* ids;
    const float* topk_w;
    const uint8_t* mask;
    int T, E, k, H;
    float scale;
    float* d_logits;
    u32x4* frag_h;        // fragments with rows tokens, summed over experts (np_h planes)
    int np_h;
    u32x4* frag_w;        // with rows experts, summed over tokens (three planes)
    uint32_t* row_bits;   // for every 16 tokens a word, one bit each, set for valid ones
    uint32_t* zeros;
    int tiles_t, tiles_e;   // blocks of the gradient; those behind them split rows
    SplitArgs split[2];     // W and an FP32 input
    long long split_blocks0;
};

__device__ __forceinline__ void split_rows(const SplitArgs& a, int H, long long block) {
    const long long per_row = H / 4;
    const long long quads = a.rows * per_row;
    const size_t plane = static_cast<size_t>(a.rows) * H;
    f32x4 v[kSplitQuads];
#pragma unroll
    for (int q = 0; q < kSplitQuads; ++q) {
        const long long i = (block * kSplitQuads + q) * kPrepBlock + threadIdx.x;
        v[q] = f32x4{0.f, 0.f, 0.f, 0.f};
        if (i < quads && (!a.mask || a.mask[i / per_row])) v[q] = reinterpret_cast<const f32x4*>(a.x)[i];
    }
#pragma unroll
    for (int q = 0; q < kSplitQuads; ++q) {
        const long long i = (block * kSplitQuads + q) * kPrepBlock + threadIdx.x;
        if (i >= quads) break;
        u32x2 o[3];
        uint32_t x, y, z;
        split_pair(v[q][0], v[q][1], x, y, z);
        o[0][0] = x;
        o[1][0] = y;
        o[2][0] = z;
        split_pair(v[q][2], v[q][3], x, y, z);
        o[0][1] = x;
        o[1][1] = y;
        o[2][1] = z;
#pragma unroll
        for (int p = 0; p < 3; ++p)
            if (p < a.np) reinterpret_cast<u32x2*>(a.planes + p * plane)[i] = o[p];
    }
}

// The picks of 32 tokens from t0 on, eight threads a token and up to four picks a
// thread, and what they add to the gradient of the logits in columns [e0, e1).
struct Picks {
    static constexpr int N = MOE_MAX_TOPK / 8;
    int id[N];
    float w[N], dw[N];

    // valid: bit r is set when token t0 + r is
    __device__ __forceinline__ void load(const PrepArgs& p, int t0, uint32_t valid) {
        const int r = threadIdx.x >> 3, sub = threadIdx.x & 7;
#pragma unroll
        for (int q = 0; q < N; ++q) {
            const int j = sub + 8 * q;
            const size_t at = static_cast<size_t>(t0 + r) * p.k + j;
            id[q] = -1;
            w[q] = dw[q] = 0.f;
            if (j < p.k && (valid >> r & 1)) {
                const int e = p.ids[at];
                if (e >= 0 && e < p.E) {
                    id[q] = e;
                    w[q] = p.topk_w[at];
                    dw[q] = p.d_topk_w[at];
                }
            }
        }
    }

    // w (1 - s) (dw - sum w dw) of each pick into LDS; a barrier must follow
    __device__ __forceinline__ void values(const PrepArgs& p, int t0, int e0, int e1,
                                           int32_t (*pick_id)[MOE_MAX_TOPK], float (*pick_v)[MOE_MAX_TOPK]) const {
        const int r = threadIdx.x >> 3, sub = threadIdx.x & 7;
        float l[N], s = 0.f;
#pragma unroll
        for (int q = 0; q < N; ++q) {
            s = __builtin_fmaf(w[q], dw[q], s);
            l[q] = 0.f;
            if (id[q] >= e0 && id[q] < e1) l[q] = p.logits[static_cast<size_t>(t0 + r) * p.E + id[q]];
        }
        s = group_sum(s, 8);
#pragma unroll
        for (int q = 0; q < N; ++q) {
            const int j = sub + 8 * q;
            pick_id[r][j] = id[q];   // -1 from k on
            pick_v[r][j] = w[q] * (dw[q] - s) / (1.f + expf(l[q]));   // 1 - sigmoid(l) = 1 / (1 + exp(l))
        }
    }

    // add(token, expert, value) for every expert that a token's picks name: the
    // first pick of an expert adds every pick of it, in order
    template <typename F>
    __device__ __forceinline__ void add(int e0, int e1, const int32_t (*pick_id)[MOE_MAX_TOPK],
                                        const float (*pick_v)[MOE_MAX_TOPK], F&& add) const {
        const int r = threadIdx.x >> 3, sub = threadIdx.x & 7;
        i32x4 all[MOE_MAX_TOPK / 4];
#pragma unroll
        for (int i = 0; i < MOE_MAX_TOPK / 4; ++i) all[i] = *reinterpret_cast<const i32x4*>(&pick_id[r][4 * i]);
#pragma unroll
        for (int q = 0; q < N; ++q) {
            if (id[q] < e0 || id[q] >= e1) continue;
            const int j = sub + 8 * q;
            uint32_t same = 0;
#pragma unroll
            for (int i = 0; i < MOE_MAX_TOPK; ++i) same |= static_cast<uint32_t>(all[i / 4][i % 4] == id[q]) << i;
            if (same & ((1u << j) - 1)) continue;
            float sum = pick_v[r][j];
            for (same &= same - 1; same; same &= same - 1) sum += pick_v[r][__builtin_ctz(same)];
            add(r, id[q], sum);
        }
    }
};

// Block x + tiles_t y: tokens [32 x, +32), experts [128 y, +128); the blocks
// behind them split W and an FP32 input into planes. Fragments of a matrix with
// rows m and summation index c: [m / 32][c / 16][plane][lane], lane l holding
// row l % 32, c = 8 (l / 32) .. +8; their values are scaled, d_logits is not.
// d_aux may be d_logits: a block reads its tile before it writes it.
__global__ __launch_bounds__(kPrepBlock) void logits_gradient_kernel(const PrepArgs p) {
    const int T = p.T, E = p.E;
    const long long grad_blocks = static_cast<long long>(p.tiles_t) * p.tiles_e;
    if (blockIdx.x >= grad_blocks) {
        const long long b = blockIdx.x - grad_blocks;
        if (b < p.split_blocks0) split_rows(p.split[0], p.H, b);
        else split_rows(p.split[1], p.H, b - p.split_blocks0);
        return;
    }
    __shared__ __attribute__((aligned(16))) float tile[kPrepRows * kPrepStride];
    __shared__ __attribute__((aligned(16))) int32_t pick_id[kPrepRows][MOE_MAX_TOPK];
    __shared__ float pick_v[kPrepRows][MOE_MAX_TOPK];
    const int tid = threadIdx.x, lane = tid & 63;
    const int by = static_cast<int>(blockIdx.x / p.tiles_t), bx = static_cast<int>(blockIdx.x - static_cast<long long>(by) * p.tiles_t);
    const int t0 = bx * kPrepRows, e0 = by * kPrepCols;
    if (p.zeros && blockIdx.x == 0)
        for (int i = tid; i < static_cast<int>(kZeroBytes / 4); i += kPrepBlock) p.zeros[i] = 0;

    const uint32_t valid = static_cast<uint32_t>(ballot(lane < kPrepRows && t0 + lane < T && p.mask[t0 + lane] != 0));
    if (p.row_bits && by == 0 && tid < 2) p.row_bits[bx * 2 + tid] = valid >> (16 * tid) & 0xFFFFu;
    Picks picks;
    if (p.d_topk_w) picks.load(p, t0, valid);
    // d_aux: piece i of the tile is row tid / 32 + 8 i, columns 4 (tid % 32) .. +4
    const int col = e0 + 4 * (tid & 31);
    f32x4 v[kPrepLoads];
#pragma unroll
    for (int i = 0; i < kPrepLoads; ++i) {
        const int r = (tid >> 5) + 8 * i;
        v[i] = f32x4{0.f, 0.f, 0.f, 0.f};
        if (p.d_aux && (valid >> r & 1)) {
            const float* src = p.d_aux + static_cast<size_t>(t0 + r) * E + col;
            if (col + 4 <= E) v[i] = *reinterpret_cast<const f32x4_any*>(src);
            else
                for (int c = 0; c < 4; ++c)
                    if (col + c < E) v[i][c] = src[c];
        }
    }
    if (p.d_topk_w) picks.values(p, t0, e0, e0 + kPrepCols, pick_id, pick_v);
#pragma unroll
    for (int i = 0; i < kPrepLoads; ++i)
        *reinterpret_cast<f32x4*>(&tile[((tid >> 5) + 8 * i) * kPrepStride + 4 * (tid & 31)]) = v[i];
    __syncthreads();
    if (p.d_topk_w) {
        picks.add(e0, e0 + kPrepCols, pick_id, pick_v,
                  [&](int r, int e, float v) { tile[r * kPrepStride + e - e0] += v; });
        __syncthreads();
    }
#pragma unroll
    for (int i = 0; i < kPrepLoads; ++i) {
        const int r = (tid >> 5) + 8 * i;
        if (t0 + r >= T) break;
        const f32x4 o = *reinterpret_cast<const f32x4*>(&tile[r * kPrepStride + 4 * (tid & 31)]);
        float* dst = p.d_logits + static_cast<size_t>(t0 + r) * E + col;
        if (col + 4 <= E) *reinterpret_cast<f32x4_any*>(dst) = o;
        else
            for (int c = 0; c < 4; ++c)
                if (col + c < E) dst[c] = o[c];
    }
    if (p.frag_h) {
        const int ks_n = (E + kKStep - 1) / kKStep;
#pragma unroll
        for (int q = 0; q < kPrepCols / kKStep / 4; ++q) {
            const int f = tid / kWave + 4 * q;
            const int ks = e0 / kKStep + f;
            if (ks >= ks_n) break;
            const f32x4* src = reinterpret_cast<const f32x4*>(&tile[(lane & 31) * kPrepStride + f * kKStep + 8 * (lane >> 5)]);
            const f32x4 lo = src[0] * p.scale, hi = src[1] * p.scale;
            const float x[8] = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
            write_fragment(x, p.np_h, p.frag_h + (static_cast<size_t>(bx) * ks_n + ks) * p.np_h * kWave + lane);
        }
    }
    if (p.frag_w) {
        const int mt_n = (E + 31) / 32;
        const size_t ks_n = 2 * static_cast<size_t>(p.tiles_t);
#pragma unroll
        for (int q = 0; q < kPrepCols / 32 / 2; ++q) {
            const int f = tid / kWave + 4 * q;
            const int mt = e0 / 32 + (f >> 1), half = f & 1;
            if (mt >= mt_n) break;
            float x[8];
#pragma unroll
            for (int j = 0; j < 8; ++j)
                x[j] = tile[(half * kKStep + 8 * (lane >> 5) + j) * kPrepStride + (f >> 1) * 32 + (lane & 31)] * p.scale;
            write_fragment(x, 3, p.frag_w + (mt * ks_n + 2 * bx + half) * 3 * kWave + lane);
        }
    }
}

// ---------------------------------------------------------- few tokens ----

constexpr int kFewTokens = 32;
constexpr int kFewCols = 32;                       // columns of H a block takes
constexpr int kFewGroups = kPrepBlock / kFewCols;   // groups of threads over the experts
constexpr int kFewValues = 16384;                  // TP E at most: the gradient of the logits in LDS, 64 KB
constexpr int kFewExperts = 1024;

// Both products of up to 32 tokens in FP32, without planes, fragments or a
// workspace, in one launch: a block computes the gradient of the logits itself
// (in LDS, [expert][token]) and takes 32 columns of H, a thread one column and
// every eighth expert. It reads W once and writes d_W once, which bounds it;
// each value of W meets the TP tokens' gradients from LDS. TP: T rounded up.
template <int TP, bool F32>
__global__ __launch_bounds__(kPrepBlock) void few_tokens_kernel(const PrepArgs p, const void* __restrict__ hidden,
                                                               const float* __restrict__ W, void* __restrict__ d_hidden,
                                                               float* __restrict__ d_W) {
    extern __shared__ __attribute__((aligned(16))) float grad[];   // [E][TP]
    __shared__ __attribute__((aligned(16))) int32_t pick_id[kPrepRows][MOE_MAX_TOPK];
    __shared__ float pick_v[kPrepRows][MOE_MAX_TOPK];
    __shared__ float part[kFewGroups][kFewCols][TP + 1];
    const int T = p.T, E = p.E, H = p.H;
    const int tid = threadIdx.x, lane = tid & 63;
    const uint32_t valid = static_cast<uint32_t>(ballot(lane < T && p.mask[lane] != 0));
    Picks picks;
    if (p.d_topk_w) picks.load(p, 0, valid);
    for (int i = tid; i < E * TP; i += kPrepBlock) {
        const int t = i / E, e = i - t * E;   // consecutive threads read consecutive experts
        grad[e * TP + t] = p.d_aux && t < T && (valid >> t & 1) ? p.d_aux[static_cast<size_t>(t) * E + e] : 0.f;
    }
    if (p.d_topk_w) picks.values(p, 0, 0, E, pick_id, pick_v);
    __syncthreads();
    if (p.d_topk_w) {
        picks.add(0, E, pick_id, pick_v, [&](int t, int e, float v) { grad[e * TP + t] += v; });
        __syncthreads();
    }
    if (p.d_logits && blockIdx.x == 0)
        for (int i = tid; i < E * T; i += kPrepBlock) {
            const int t = i / E, e = i - t * E;
            p.d_logits[i] = grad[e * TP + t];
        }
    const int c = tid % kFewCols, group = tid / kFewCols;
    const int col = static_cast<int>(blockIdx.x) * kFewCols + c;
    const bool mine = col < H;
    float h[TP], acc[TP];
#pragma unroll
    for (int t = 0; t < TP; ++t) {
        acc[t] = 0.f;
        h[t] = 0.f;
        if (mine && (valid >> t & 1)) {
            const size_t at = static_cast<size_t>(t) * H + col;
            if constexpr (F32) h[t] = static_cast<const float*>(hidden)[at];
            else h[t] = bf16_lo(static_cast<const uint16_t*>(hidden)[at]);
        }
    }
#pragma unroll 4
    for (int e = group; e < E; e += kFewGroups) {
        const float w = d_hidden && mine ? W[static_cast<size_t>(e) * H + col] : 0.f;
        float dw = 0.f;
#pragma unroll
        for (int t = 0; t < TP; t += 4) {
            const f32x4 g = *reinterpret_cast<const f32x4*>(&grad[e * TP + t]);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                acc[t + i] = __builtin_fmaf(g[i], w, acc[t + i]);
                dw = __builtin_fmaf(g[i], h[t + i], dw);
            }
        }
        if (d_W && mine) d_W[static_cast<size_t>(e) * H + col] = dw * p.scale;
    }
    if (!d_hidden) return;
#pragma unroll
    for (int t = 0; t < TP; ++t) part[group][c][t] = acc[t];
    __syncthreads();
    for (int i = tid; i < T * kFewCols; i += kPrepBlock) {
        const int t = i / kFewCols, q = i - t * kFewCols;
        const int at_col = static_cast<int>(blockIdx.x) * kFewCols + q;
        if (at_col >= H) continue;
        float s = part[0][q][t];
        for (int g = 1; g < kFewGroups; ++g) s += part[g][q][t];
        s = valid >> t & 1 ? s * p.scale : 0.f;   // W may hold infinities or NaN
        const size_t at = static_cast<size_t>(t) * H + at_col;
        if constexpr (F32) static_cast<float*>(d_hidden)[at] = s;
        else static_cast<uint16_t*>(d_hidden)[at] = static_cast<uint16_t>(f32_to_bf16_rne(s));
    }
}

// ------------------------------------------------------------- product ----

template <int N>
__device__ __forceinline__ void wait_vmcnt() {
    static_assert(N >= 0 && N < 64, "vmcnt range");
    __builtin_amdgcn_s_waitcnt((N & 0xF) | ((N >> 4) << 14) | (0x7 << 4) | (0xF << 8));
}

__device__ __forceinline__ void wait_lgkmcnt0() { __builtin_amdgcn_s_waitcnt(0xF | (0x3 << 14) | (0x7 << 4)); }

// Block tile 64 WM x 256, 2 WM waves of 64 x 128 (2 x 4 accumulators of
// v_mfma_f32_32x32x16_bf16). WM = 4, or 2 with three planes of each factor, whose
// operands take twice the registers (one wave a SIMD). Batches of fewer rows
// take the same tile, K split for more blocks: tiles of 64 or 128 rows have too
// few waves for a CU, two of them on a CU or more stages included (64 tokens of
// 8192 x 256: 34 us with 256 rows, 35 with 128, 43 with 64; 215 of 2624 x 235:
// 44, 58 and 60).
//
// Pipeline: every K-step's A fragments and B rows go through a ring of SETS LDS
// stages filled by direct-to-LDS loads of 1 KB, the same number by every wave;
// loads complete in issue order, so waiting for all but the newest (SETS - 2)
// groups means the next step's has landed. Step g issues the loads of step
// g + SETS into the stage that all waves have read, reads step g + 1's operands
// from LDS into the other register set and multiplies step g's, so that
// neither kind of load is waited for beside idle matrix cores. Blocks are
// persistent: the steps of a block's tiles form one sequence, and the loads of
// the next tile are in flight while the results of the last one are stored.
template <int NA, int NB>
struct ProductShape {
    static constexpr int WM = NB == 3 ? 2 : 4;
    static constexpr int WAVES = 2 * WM;
    static constexpr int BLOCK = WAVES * kWave;
    static constexpr int BM = 64 * WM, BN = 256;
    static constexpr int LA = 2 * WM * NA;      // 1 KB loads of A per step: NA per wave
    static constexpr int LB = 8 * NB;           // and of B: NB planes of 16 rows
    static constexpr int WB = LB / WAVES;       // per wave
    static constexpr int LOADS = NA + WB;
    static constexpr int STAGE = (LA + LB) * kFrag;
    static constexpr int SETS = 4 * STAGE <= 144 * 1024 ? 4 : 3;
    static constexpr size_t LDS = static_cast<size_t>(SETS) * STAGE;
    static constexpr int STORES = 32;           // of a wave per tile
    static_assert(LB % WAVES == 0, "every wave issues the same number of loads");
    static_assert(LDS <= 160 * 1024, "LDS of a CU");
    static_assert((SETS - 2) * LOADS + STORES < 64, "vmcnt range");
    static_assert(BN * 2 <= static_cast<int>(kZeroBytes), "a row of zeros");
};

struct ProductArgs {
    const u32x4* a;            // fragments [m / 32][K / 16][NA][64]
    const uint16_t* b;         // [NB][rows][n]
    size_t b_plane;            // elements between planes
    const uint32_t* row_bits;  // valid rows of each K-step; NULL: those below `rows`
    const uint32_t* out_bits;  // valid rows of c, 16 a word: the others get zeros; NULL: all
                               // (as many planes of each factor: the input's gradient)
    const uint16_t* zeros;     // kZeroBytes of zeros
    int m, n, rows, a_steps;   // a_steps: K-steps the fragments hold (>= steps)
    int steps, split_steps;    // K-steps in all, and of one split
    int tiles_m, tiles_n, nsplit;
    void* c;                   // [m,n]; with nsplit > 1 FP32 partial sums [nsplit,m,n]
};

// Operands of one K-step as a wave reads them from LDS: its A fragments, and
// eight rows of four columns of B.
template <int NA, int NB>
struct StepOperands {
    bf16x8_t a[NA][2];
    u32x2 b[NB][8];
};

template <int NA, int NB, bool BF16_OUT>
__global__ __launch_bounds__(NB == 3 ? 256 : 512, NB == 3 ? 1 : 2) void product_kernel(
    const ProductArgs p) {
#ifdef __HIP_DEVICE_COMPILE__   // the host pass only needs the kernel's handle
    using S = ProductShape<NA, NB>;
    extern __shared__ __attribute__((aligned(16))) char lds[];
    // The blocks of an XCD (every eighth) take a run of consecutive tiles: row
    // tiles of one column tile first, then column tiles, then K-splits.
    const int total = p.tiles_m * p.tiles_n * p.nsplit;
    const int per_xcd = (total + 7) / 8;
    const int xcd = static_cast<int>(blockIdx.x % 8);
    const int run_end = min(total, (xcd + 1) * per_xcd);
    const int stride = static_cast<int>(gridDim.x) / 8;
    const int first = xcd * per_xcd + static_cast<int>(blockIdx.x / 8);
    if (first >= run_end) return;

    const int lane = __lane_id();
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int wm = wave >> 1, wn = wave & 1;
    const int m_last = (p.m + 31) / 32 - 1;
    const int per_split = p.tiles_m * p.tiles_n;

    // ---- the loads' cursor: tile l_tile, K-step l_ks up to l_end
    int l_tile = first, l_ks = 0, l_end = 0;
    // wave-uniform parts of the sources (scalar registers); the lanes' offsets
    // are the same for every load of a tile
    const u32x4* a_src[NA];
    const uint16_t* b_src[S::WB];
    const int b_row = lane >> 5, b_col = (lane & 31) * 8;   // a B load covers two rows of 256 columns
    int b_lane = 0;
    auto load_tile = [&]() {
        const int split = l_tile / per_split;
        const int tile = l_tile - split * per_split;
        const int n_tile = tile / p.tiles_m, m_tile = tile - n_tile * p.tiles_m;
        l_ks = split * p.split_steps;
        l_end = min(p.steps, l_ks + p.split_steps);
#pragma unroll
        for (int i = 0; i < NA; ++i) {
            const int l = wave + i * S::WAVES;
            const int mt = min(m_tile * (S::BM / 32) + l / NA, m_last);
            a_src[i] = p.a + ((static_cast<size_t>(mt) * p.a_steps + l_ks) * NA + l % NA) * kWave;
        }
        const int n0 = n_tile * S::BN;
        b_lane = b_row * p.n + min(b_col, p.n - 8 - n0);   // columns past n repeat the last ones (never stored)
#pragma unroll
        for (int i = 0; i < S::WB; ++i) {
            const int l = wave + i * S::WAVES;
            const size_t row = static_cast<size_t>(l_ks) * kKStep + (l & 7) * 2;
            b_src[i] = p.b + (l >> 3) * p.b_plane + row * p.n + n0;
        }
    };
    // through the constant address space: scalar loads, which the waits for the
    // vector loads do not count
    using scalar_bits = const __attribute__((address_space(4))) uint32_t*;
    const auto bits_at = (scalar_bits)(p.row_bits), out_at = (scalar_bits)(p.out_bits);
    auto bits_of = [&](int ks) -> uint32_t {
        if (p.row_bits) return bits_at[ks];
        const int left = p.rows - ks * kKStep;
        return left >= kKStep ? 0xFFFFu : (1u << left) - 1u;
    };
    uint32_t l_bits;
    auto issue = [&](int set) {
        char* base = lds + set * S::STAGE;
#pragma unroll
        for (int i = 0; i < NA; ++i)
            __builtin_amdgcn_global_load_lds(a_src[i] + lane, base + (wave + i * S::WAVES) * kFrag, 16, 0, 0);
        if (l_bits == 0xFFFFu) {
#pragma unroll
            for (int i = 0; i < S::WB; ++i)
                __builtin_amdgcn_global_load_lds(b_src[i] + b_lane, base + (S::LA + wave + i * S::WAVES) * kFrag, 16, 0,
                                                 0);
        } else {
#pragma unroll
            for (int i = 0; i < S::WB; ++i) {
                const int l = wave + i * S::WAVES;
                const bool ok = l_bits >> ((l & 7) * 2 + b_row) & 1;
                const uint16_t* src = ok ? b_src[i] + b_lane : p.zeros + b_col;
                __builtin_amdgcn_global_load_lds(src, base + (S::LA + l) * kFrag, 16, 0, 0);
            }
        }
    };
    // on to the next step, or the next tile's first; behind the last tile the
    // last step is loaded again, into stages that nobody uses
    auto advance = [&]() {
        if (l_ks + 1 < l_end) {
            ++l_ks;
#pragma unroll
            for (int i = 0; i < NA; ++i) a_src[i] += NA * kWave;
#pragma unroll
            for (int i = 0; i < S::WB; ++i) b_src[i] += static_cast<size_t>(kKStep) * p.n;
        } else if (l_tile + stride < run_end) {
            l_tile += stride;
            load_tile();
        }
        l_bits = bits_of(l_ks);
    };
    // Piece i of a step's operands: first the pairs of B's rows, then the A
    // fragments.
    constexpr int kPieces = 4 * NB + 2 * NA;
    auto read_piece = [&](const char* base, StepOperands<NA, NB>& f, int i) {
        if (i < 4 * NB) {
            const int pl = i >> 2, r = (i & 3) * 2;
            const char* src = base + S::LA * kFrag + (pl * kKStep + 8 * (lane >> 5) + r) * (S::BN * 2) + wn * 256 +
                              (lane & 31) * 8;
            f.b[pl][r] = *reinterpret_cast<const u32x2*>(src);
            f.b[pl][r + 1] = *reinterpret_cast<const u32x2*>(src + S::BN * 2);
        } else if (i < kPieces) {
            const int mi = (i - 4 * NB) / NA, pl = (i - 4 * NB) % NA;
            f.a[pl][mi] = *reinterpret_cast<const bf16x8_t*>(base + ((wm * 2 + mi) * NA + pl) * kFrag + lane * 16);
        }
    };

    f32x16_t acc[2][4];
    auto clear = [&]() {
#pragma unroll
        for (int mi = 0; mi < 2; ++mi)
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int i = 0; i < 16; ++i) acc[mi][j][i] = 0.f;
    };
    // The products of planes (pa, pb) with pa + pb < max(NA, NB) of step f, and
    // the reads of the next step's operands spread between them, two pieces to
    // four MFMAs: issued in a run they would keep the matrix cores waiting for
    // the LDS queue.
    auto multiply = [&](const StepOperands<NA, NB>& f, const char* base, StepOperands<NA, NB>& next) {
        constexpr int PMAX = NA > NB ? NA : NB;
        int piece = 0;
#pragma unroll
        for (int pb = 0; pb < NB; ++pb) {
            bf16x8_t b[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                u32x4 v;
#pragma unroll
                for (int d = 0; d < 4; ++d)
                    v[d] = __builtin_amdgcn_perm(f.b[pb][2 * d + 1][j >> 1], f.b[pb][2 * d][j >> 1],
                                                 j & 1 ? 0x07060302u : 0x05040100u);
                b[j] = __builtin_bit_cast(bf16x8_t, v);
            }
#pragma unroll
            for (int pa = 0; pa < NA; ++pa) {
                if (pa + pb >= PMAX) continue;
#pragma unroll
                for (int mi = 0; mi < 2; ++mi) {
                    read_piece(base, next, piece);
                    read_piece(base, next, piece + 1);
                    piece += 2;
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        acc[mi][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(f.a[pa][mi], b[j], acc[mi][j], 0, 0, 0);
                    __builtin_amdgcn_sched_barrier(0);
                }
            }
        }
    };

    // Stores the tile's results; returns the stores that are certainly behind
    // the loads in flight (none at the matrix' edges, where some are skipped).
    // lane: columns 4 (lane % 32) + j of the wave's 128, rows 8 (i / 4) +
    // 4 (lane / 32) + i % 4 of each 32
    auto store_tile = [&](int t) {
        const int split = t / per_split;
        const int tile = t - split * per_split;
        const int n_tile = tile / p.tiles_m, m_tile = tile - n_tile * p.tiles_m;
        const int m0 = m_tile * S::BM + wm * 64 + 4 * (lane >> 5);
        const int col = n_tile * S::BN + wn * 128 + 4 * (lane & 31);
        const size_t part = p.nsplit > 1 ? static_cast<size_t>(split) * p.m : 0;
        // an invalid row's zeros met B's infinities and NaN, if it has any
        uint32_t valid[2] = {~0u, ~0u};
        if (NA == NB && p.out_bits) {
#pragma unroll
            for (int mi = 0; mi < 2; ++mi) {
                const int block = min(m_tile * (S::BM / 32) + wm * 2 + mi, m_last);
                valid[mi] = (out_at[2 * block] | out_at[2 * block + 1] << 16) >> (4 * (lane >> 5));
            }
        }
        auto put = [&](int mi, int i) {
            const int row = m0 + mi * 32 + 8 * (i >> 2) + (i & 3);
            const size_t at = (part + row) * p.n + col;
            const float v0 = acc[mi][0][i], v1 = acc[mi][1][i], v2 = acc[mi][2][i], v3 = acc[mi][3][i];
            const uint32_t keep = -(valid[mi] >> (8 * (i >> 2) + (i & 3)) & 1u);
            if constexpr (BF16_OUT)
                *reinterpret_cast<u32x2*>(static_cast<uint16_t*>(p.c) + at) =
                    u32x2{cvt_pk_bf16(v0, v1) & keep, cvt_pk_bf16(v2, v3) & keep};
            else if constexpr (NA == NB)
                *reinterpret_cast<u32x4*>(static_cast<float*>(p.c) + at) =
                    u32x4{__float_as_uint(v0) & keep, __float_as_uint(v1) & keep, __float_as_uint(v2) & keep,
                          __float_as_uint(v3) & keep};
            else
                *reinterpret_cast<float4*>(static_cast<float*>(p.c) + at) = make_float4(v0, v1, v2, v3);
        };
        const bool whole = (m_tile + 1) * S::BM <= p.m && (n_tile + 1) * S::BN <= p.n;
        if (whole) {
#pragma unroll
            for (int mi = 0; mi < 2; ++mi)
#pragma unroll
                for (int i = 0; i < 16; ++i) put(mi, i);
            return true;
        }
        if (col < p.n) {
#pragma unroll
            for (int mi = 0; mi < 2; ++mi)
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    if (m0 + mi * 32 + 8 * (i >> 2) + (i & 3) < p.m) put(mi, i);
        }
        return false;
    };

    // ---- the tile being computed
    int c_tile = first;
    auto tile_steps = [&](int t) {
        const int beg = t / per_split * p.split_steps;
        return min(p.steps, beg + p.split_steps) - beg;
    };
    int left = tile_steps(c_tile);
    int behind = 0;   // steps for which the last tile's stores are behind the loads waited for

    load_tile();
    l_bits = bits_of(l_ks);
#pragma unroll
    for (int s = 0; s < S::SETS; ++s) {
        issue(s);
        advance();
        __builtin_amdgcn_sched_barrier(0);
    }
    StepOperands<NA, NB> f0, f1;
    wait_vmcnt<(S::SETS - 1) * S::LOADS>();
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int i = 0; i < kPieces; ++i) read_piece(lds, f0, i);
    clear();
    int set = 0;
    // one step: f holds its operands, g takes the next step's; false behind the
    // last step of the last tile
    auto step = [&](const StepOperands<NA, NB>& f, StepOperands<NA, NB>& g) {
        __builtin_amdgcn_sched_barrier(0);
        // the next step's loads have landed ...
        if (behind > 0) {
            wait_vmcnt<(S::SETS - 2) * S::LOADS + S::STORES>();
            --behind;
        } else {
            wait_vmcnt<(S::SETS - 2) * S::LOADS>();
        }
        wait_lgkmcnt0();                // ... this step's operands are in registers ...
        __builtin_amdgcn_s_barrier();   // ... in every wave: its stage is free
        __builtin_amdgcn_sched_barrier(0);
        issue(set);
        set = set + 1 == S::SETS ? 0 : set + 1;
        __builtin_amdgcn_sched_barrier(0);
        multiply(f, lds + set * S::STAGE, g);
        advance();
        if (--left > 0) return true;
        __builtin_amdgcn_sched_barrier(0);
        behind = store_tile(c_tile) ? S::SETS - 1 : 0;
        __builtin_amdgcn_sched_barrier(0);
        c_tile += stride;
        if (c_tile >= run_end) return false;
        left = tile_steps(c_tile);
        clear();
        return true;
    };
    while (step(f0, f1) && step(f1, f0)) {}
    wait_vmcnt<0>();   // loads in flight, before the block's LDS is given away
#endif
}

// The sum of n partial arrays, in order; zeros without any.
template <bool BF16_OUT>
__global__ __launch_bounds__(256) void sum_parts_kernel(const float4* __restrict__ parts, int n, long long quads,
                                                        void* __restrict__ out) {
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
        if constexpr (BF16_OUT)
            static_cast<u32x2*>(out)[i] = u32x2{cvt_pk_bf16(s.x, s.y), cvt_pk_bf16(s.z, s.w)};
        else
            static_cast<float4*>(out)[i] = s;
    }
}

// -------------------------------------------------------------- planning ----

inline size_t round256(size_t b) { return (b + 255) / 256 * 256; }

struct ProductPlan {
    int tiles_m, tiles_n, steps, nsplit, split_steps;
};

// K is split in parts, whose sums a kernel of their own adds up, where a simple
// model makes that cheaper. Its figures are measured: a step of a block 1.4 us, a
// tile's first loads and results 5; partial sums read back, and half of their
// writing, at 4 TB/s, and 4 us for their kernel. It takes 256 CUs whatever the device has, so
// that the workspace query and the call agree.
inline ProductPlan plan_product(int m, int n, long long k, bool f32) {
    constexpr int kBlocks = 256;
    ProductPlan p;
    p.tiles_m = ceil_div(m, f32 ? ProductShape<3, 3>::BM : ProductShape<3, 1>::BM);
    p.tiles_n = ceil_div(n, 256);
    p.steps = ceil_div(k, kKStep);
    p.nsplit = 1;
    p.split_steps = p.steps;
    const long long tiles = static_cast<long long>(p.tiles_m) * p.tiles_n;
    double best = 0;
    for (int ns = 1; ns <= 32 && (ns == 1 || p.steps / ns >= 2); ++ns) {
        const int each = ceil_div(p.steps, ns);
        const int used = ceil_div(p.steps, each);
        double us = static_cast<double>((tiles * used + kBlocks - 1) / kBlocks) * (each * 1.4 + 5);
        if (used > 1) us += 4 + 6e-6 * used * static_cast<double>(m) * n / 4.0;
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

// Whether few_tokens_kernel takes the call. Its FP32 work grows with T E H and its
// threads walk the experts, while the general path's cost is its launches and
// latency: measured few / general, 16 tokens of 8192 x 256 experts 18 / 31 us, 32
// of 4096 x 512 43 / 31 (33 tokens), 32 of 8192 x 256 27 / 31, 8 of 1024 x 2560 72
// / 35, 4 of 8192 x 4096 116 / 113.
inline bool few_tokens(int T, int E) {
    const int tp = T <= 4 ? 4 : T <= 8 ? 8 : T <= 16 ? 16 : kFewTokens;
    return T <= kFewTokens && E <= kFewExperts && tp * E <= (tp < kFewTokens ? kFewValues : kFewValues / 2);
}

inline RouteBackwardPlan plan_route_backward(int T, int H, int E, int dtype) {
    RouteBackwardPlan p;
    const bool f32 = dtype == MOE_DTYPE_F32;
    p.np_h = f32 ? 3 : 2;
    p.h = plan_product(T, H, E, f32);
    p.w = plan_product(E, H, T, f32);
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
    // the products run one after the other, so their partial sums share the space
    const size_t parts_h = p.h.nsplit > 1 ? sizeof(float) * p.h.nsplit * T * H : 0;
    const size_t parts_w = p.w.nsplit > 1 ? sizeof(float) * p.w.nsplit * E * H : 0;
    p.parts = take(parts_h > parts_w ? parts_h : parts_w);
    p.bytes = at;
    return p;
}

template <int NA, int NB, bool BF16_OUT>
int launch_product(const ProductPlan& p, ProductArgs a, void* stream) {
    using S = ProductShape<NA, NB>;
    a.steps = p.steps;
    a.split_steps = p.split_steps;
    a.tiles_m = p.tiles_m;
    a.tiles_n = p.tiles_n;
    a.nsplit = p.nsplit;
    // one resident grid of persistent blocks, a multiple of the XCDs
    const long long grid = 8ll * ceil_div(static_cast<long long>(a.tiles_m) * a.tiles_n * a.nsplit, 8);
    const int most = device_cu_count() / 8 * 8;
    return launch(product_kernel<NA, NB, BF16_OUT>, dim3(static_cast<unsigned>(grid < most ? grid : most)),
                  dim3(S::BLOCK), S::LDS, stream, a);
}

}  // namespace
}  // namespace moe

extern "C" size_t moe_route_backward_workspace_bytes(int T, int H, int E, int hidden_dtype, int logits_in) {
    using namespace moe;
    if (logits_in || !route_backward_shape_ok(T, H, E)) return 0;
    if (hidden_dtype != MOE_DTYPE_BF16 && hidden_dtype != MOE_DTYPE_F32) return 0;
    return few_tokens(T, E) ? 0 : plan_route_backward(T, H, E, hidden_dtype).bytes;
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
        return d_W ? launch(sum_parts_kernel<false>, grid_of(w_quads), dim3(256), 0, stream, nullptr, 0, w_quads,
                            static_cast<void*>(d_W))
                   : MOE_OK;
    if (!token_mask || !d_logits || (!d_topk_w && !d_aux)) return MOE_ERR_NULL_ARG;
    if (d_topk_w && (!logits || !topk_ids || !topk_w)) return MOE_ERR_NULL_ARG;
    if (logits_in && (d_hidden || d_W)) return MOE_ERR_NULL_ARG;
    if (d_hidden && !W) return MOE_ERR_NULL_ARG;
    const bool f32 = hidden_dtype == MOE_DTYPE_F32;
    RouteBackwardPlan p{};
    char* ws = static_cast<char*>(workspace);
    const bool few = !logits_in && few_tokens(T, E);
    if (!logits_in && !few) {
        p = plan_route_backward(T, H, E, hidden_dtype);
        if (!workspace || workspace_bytes < p.bytes || (reinterpret_cast<uintptr_t>(workspace) & 255u) != 0)
            return MOE_ERR_WORKSPACE;
    }
    PrepArgs g{};
    g.d_topk_w = d_topk_w;
    g.d_aux = d_aux;
    g.logits = logits;
    g.ids = topk_ids;
    g.topk_w = topk_w;
    g.mask = token_mask;
    g.T = T;
    g.E = E;
    g.k = k;
    g.H = H;
    g.scale = scale;
    g.d_logits = d_logits;
    g.tiles_t = ceil_div(T, kPrepRows);
    g.tiles_e = ceil_div(E, kPrepCols);
    const long long grad_blocks = static_cast<long long>(g.tiles_t) * g.tiles_e;
    if (few && (d_hidden || d_W)) {
        if (d_aux == d_logits) {
            // in place: every block below reads all of d_aux, so the gradient
            // of the logits is written before
            const int st = launch(logits_gradient_kernel, dim3(static_cast<unsigned>(grad_blocks)), dim3(kPrepBlock), 0,
                                  stream, g);
            if (st != MOE_OK) return st;
            g.d_topk_w = nullptr;
            g.d_logits = nullptr;
        }
        auto run = [&](auto tp) {
            constexpr int TP = decltype(tp)::value;
            return launch(f32 ? few_tokens_kernel<TP, true> : few_tokens_kernel<TP, false>,
                          dim3(ceil_div(H, kFewCols)), dim3(kPrepBlock), sizeof(float) * TP * E, stream, g, hidden, W,
                          d_hidden, d_W);
        };
        return T <= 4    ? run(std::integral_constant<int, 4>())
               : T <= 8  ? run(std::integral_constant<int, 8>())
               : T <= 16 ? run(std::integral_constant<int, 16>())
                         : run(std::integral_constant<int, kFewTokens>());
    }
    g.frag_h = d_hidden ? reinterpret_cast<u32x4*>(ws + p.frag_h) : nullptr;
    g.np_h = p.np_h;
    g.frag_w = d_W ? reinterpret_cast<u32x4*>(ws + p.frag_w) : nullptr;
    g.row_bits = logits_in || few ? nullptr : reinterpret_cast<uint32_t*>(ws + p.bits);
    g.zeros = logits_in || few ? nullptr : reinterpret_cast<uint32_t*>(ws + p.zeros);
    auto* w_planes = reinterpret_cast<uint16_t*>(ws + p.w_planes);
    auto* x_planes = reinterpret_cast<uint16_t*>(ws + p.x_planes);
    long long blocks[2] = {0, 0};
    if (d_hidden) {
        g.split[0] = SplitArgs{W, nullptr, E, p.np_h, w_planes};
        blocks[0] = ceil_div(w_quads, kSplitQuads * kPrepBlock);
    }
    if (d_W && f32) {
        g.split[1] = SplitArgs{static_cast<const float*>(hidden), token_mask, T, 3, x_planes};
        blocks[1] = ceil_div(static_cast<long long>(T) * H / 4, kSplitQuads * kPrepBlock);
    }
    g.split_blocks0 = blocks[0];
    const long long grid = grad_blocks + blocks[0] + blocks[1];
    if (grid >= (1ll << 31)) return MOE_ERR_BAD_SHAPE;
    int st = launch(logits_gradient_kernel, dim3(static_cast<unsigned>(grid)), dim3(kPrepBlock), 0, stream, g);
    if (st != MOE_OK) return st;
    ProductArgs a{};
    a.zeros = reinterpret_cast<const uint16_t*>(g.zeros);
    a.n = H;
    if (d_hidden) {
        a.a = g.frag_h;
        a.b = w_planes;
        a.b_plane = static_cast<size_t>(E) * H;
        a.m = T;
        a.rows = E;
        a.a_steps = ceil_div(E, kKStep);
        a.out_bits = g.row_bits;
        const bool split = p.h.nsplit > 1;
        a.c = split ? static_cast<void*>(ws + p.parts) : d_hidden;
        st = f32     ? launch_product<3, 3, false>(p.h, a, stream)
             : split ? launch_product<2, 2, false>(p.h, a, stream)
                     : launch_product<2, 2, true>(p.h, a, stream);
        if (st != MOE_OK) return st;
        if (split) {
            const long long quads = static_cast<long long>(T) * H / 4;
            st = launch(f32 ? sum_parts_kernel<false> : sum_parts_kernel<true>, grid_of(quads), dim3(256), 0, stream,
                        reinterpret_cast<const float4*>(ws + p.parts), p.h.nsplit, quads, d_hidden);
            if (st != MOE_OK) return st;
        }
    }
    if (d_W) {
        a.a = g.frag_w;
        a.m = E;
        a.rows = T;
        a.a_steps = 2 * g.tiles_t;
        a.out_bits = nullptr;
        a.c = p.w.nsplit > 1 ? static_cast<void*>(ws + p.parts) : static_cast<void*>(d_W);
        if (f32) {   // the planes hold zeros for invalid tokens
            a.b = x_planes;
            a.b_plane = static_cast<size_t>(T) * H;
            st = launch_product<3, 3, false>(p.w, a, stream);
        } else {
            a.b = static_cast<const uint16_t*>(hidden);
            a.b_plane = 0;
            a.row_bits = g.row_bits;
            st = launch_product<3, 1, false>(p.w, a, stream);
        }
        if (st != MOE_OK) return st;
        if (p.w.nsplit > 1)
            st = launch(sum_parts_kernel<false>, grid_of(w_quads), dim3(256), 0, stream,
                        reinterpret_cast<const float4*>(ws + p.parts), p.w.nsplit, w_quads, static_cast<void*>(d_W));
    }
    return st;
}
