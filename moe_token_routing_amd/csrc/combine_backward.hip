// moe_combine_backward: gradients of moe_combine on the expert rows, the
// routing weights and the norm weight.
//
// Mathematics. With x the expert row of slot (t,j), g the gain, y the
// gradient of the token's output and rstd = 1 / sqrt(mean(x^2) + eps), the
// slot's share of the output is w z, z_i = x_i g_i rstd. Two sums over the row
// give everything: ss = sum x_i^2 and A = sum y_i g_i x_i.
//   dw   = rstd A
//   dx_i = w rstd (g_i y_i - x_i rstd (rstd A / H))
//   dg_i = sum over slots of w rstd x_i y_i
//
// Bound by HBM: every expert row is read once and its gradient written once,
// and y is read once per token. So one group of threads takes a token (a part of
// its picks, if the tokens are few), keeps y in registers for its k rows and each
// row in registers between the sums and the gradient. Measured: 8192 tokens of
// 8192, k 8, 420 us and 25 us for the rows kernel (2.28 GB: 5.1 TB/s, a large
// copy's rate); 16411 of 1032, k 22, 350 and 23 us (1.52 GB: 4.1 TB/s; rows of
// 2064 bytes in random order begin and end within lines of 128). Blocks are persistent over tokens, so that the gain's gradient
// is summed in registers and only one row of partial sums per block is
// written; a last kernel adds those in block order, beside the mending below.
//
// Rows and slots need not match one to one. The main kernel writes every named
// row's gradient and, for each row, a slot that names it (`owner`: any of them
// stays). The row kernel then finds the rows to mend: an owner that does not
// name its row is what the workspace held before, so no slot names the row and
// it gets zeros (checking the owner against the slots saves clearing it); a slot
// that is not the owner of its row says that several name it, and the row's
// gradient is computed anew as the sum over them in slot order.
#include <cmath>

#include "launch.hpp"
#include "rows.hpp"

namespace moe {
namespace {

constexpr int kSmallBlock = 256;
constexpr int kWideBlock = 512;   // rows of more than 1024 vectors

__device__ __forceinline__ float bf16_at(const u32x4& v, int e) {
    const uint32_t w = v[e >> 1];
    return e & 1 ? bf16_hi(w) : bf16_lo(w);
}

// Makes the compiler forget what it derived from a register, so that it unpacks
// a row again where it is used next instead of keeping the unpacked values.
__device__ __forceinline__ void keep_packed(u32x4& v) { asm volatile("" : "+v"(v)); }

// The block's row of partial gain gradients: its token groups' in order, each
// group's vectors tid + i tpt.
template <int VPT, int BLOCK>
__device__ __forceinline__ void store_gain_part(const float (&dgain)[VPT][8], int sub, int tid, int tpt, int H,
                                                float* lds, float* __restrict__ out) {
    const int nvec = H >> 3;
    if (tpt == BLOCK) {
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int v = tid + i * tpt;
            if (v < nvec) {
                float4* p = reinterpret_cast<float4*>(out) + 2 * v;
                p[0] = make_float4(dgain[i][0], dgain[i][1], dgain[i][2], dgain[i][3]);
                p[1] = make_float4(dgain[i][4], dgain[i][5], dgain[i][6], dgain[i][7]);
            }
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int v = tid + i * tpt;
        if (v < nvec)
#pragma unroll
            for (int e = 0; e < 8; ++e) lds[sub * H + v * 8 + e] = dgain[i][e];
    }
    __syncthreads();
    for (int c = threadIdx.x; c < H; c += BLOCK) {
        float s = lds[c];
        for (int q = 1; q < BLOCK / tpt; ++q) s += lds[q * H + c];
        out[c] = s;
    }
}

// Sums of N values over aligned groups of `width` lanes (a power of two) by
// register exchanges alone, the N interleaved: within fours, the mirrored halves
// of eights and sixteens, then rows of 16 lanes.
template <int CTRL>
__device__ __forceinline__ float dpp_f32(float v) {
    return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, 0xF, 0xF, false));
}
template <int N>
__device__ __forceinline__ void group_sums(float (&v)[N], int width) {
    if (width > 1)
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] += dpp_f32<0xB1>(v[i]);    // quad_perm [1,0,3,2]
    if (width > 2)
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] += dpp_f32<0x4E>(v[i]);    // quad_perm [2,3,0,1]
    if (width > 4)
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] += dpp_f32<0x141>(v[i]);   // row_half_mirror
    if (width > 8)
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] += dpp_f32<0x140>(v[i]);   // row_mirror
    if (width > 16)
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const uint32_t u = __float_as_uint(v[i]);
            const auto s = __builtin_amdgcn_permlane16_swap(u, u, false, false);
            v[i] = __uint_as_float(s[0]) + __uint_as_float(s[1]);
        }
}

constexpr int kNarrowRows = 4;   // rows of an item

// Rows of up to 32 vectors: tpt threads per item of a token's rows (a power of
// two), one vector each, several items in a wave.
__global__ __launch_bounds__(kSmallBlock) void combine_backward_narrow_kernel(
    const u32x4* __restrict__ d_out, const u32x4* __restrict__ expert_out, int R,
    const int32_t* __restrict__ slots, const float* __restrict__ topk_w, const float* __restrict__ norm_w,
    float gain_center, float eps, int T, int H, int k, int tpt, int32_t* __restrict__ owner,
    u32x4* __restrict__ d_rows, float* __restrict__ d_topk_w, float* __restrict__ part_gain) {
    constexpr int G = kNarrowRows;
    extern __shared__ float gain_lds[];
    const int groups = kSmallBlock / tpt;   // items of a block
    const int sub = static_cast<int>(threadIdx.x) / tpt;
    const int tid = static_cast<int>(threadIdx.x) - sub * tpt;
    const int nvec = H >> 3;
    const bool mine = tid < nvec;
    const float inv_h = 1.0f / static_cast<float>(H);
    float gain[8], dgain[1][8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        gain[e] = mine ? gain_center + norm_w[tid * 8 + e] : 0.f;
        dgain[0][e] = 0.f;
    }
    // Items of G picks of a token, item u by group u mod (groups of the grid): a
    // token's items go to neighbouring groups, whose sums for the gain meet in the
    // block's. An item's rows are loaded while the item before it is worked on, its
    // slots one item earlier still. ub, the block's first item, counts the turns,
    // so that every thread takes the same ones.
    const int per_token = (k + G - 1) / G;
    const long long items = static_cast<long long>(T) * per_token;
    const unsigned stride = gridDim.x * groups;
    const int step_t = static_cast<int>(stride / per_token), step_j = static_cast<int>(stride % per_token) * G;
    struct Place {
        long long t;
        int j;
    };
    auto advance = [&](Place& p) {
        p.t += step_t;
        p.j += step_j;
        if (p.j >= per_token * G) {
            p.j -= per_token * G;
            ++p.t;
        }
    };
    struct Item {
        int row[G];   // -1: none, or not to be read
        float w[G];
    };
    auto load_item = [&](const Place& at, Item& p) {
#pragma unroll
        for (int g = 0; g < G; ++g) {
            p.row[g] = -1;
            p.w[g] = 0.f;
            if (at.t < T && at.j + g < k) {
                p.row[g] = slots[at.t * k + at.j + g];
                p.w[g] = topk_w[at.t * k + at.j + g];
            }
        }
    };
    auto load_rows = [&](const Place& at, Item& p, u32x4 (&x)[G], u32x4& y) {
        y = at.t < T && mine ? d_out[at.t * nvec + tid] : u32x4{0, 0, 0, 0};
#pragma unroll
        for (int g = 0; g < G; ++g) {
            if (p.row[g] < 0 || p.row[g] >= R) p.row[g] = -1;
            x[g] = u32x4{0, 0, 0, 0};
            if (p.row[g] >= 0 && mine) x[g] = load_nt(&expert_out[static_cast<size_t>(p.row[g]) * nvec + tid]);
        }
    };
    long long ub = static_cast<long long>(blockIdx.x) * groups;
    const unsigned u = blockIdx.x * groups + sub;
    Place at = {u / per_token, static_cast<int>(u % per_token) * G};
    Place at1 = at;
    advance(at1);
    Place at2 = at1;
    Item item, next, after;
    u32x4 x[G], xn[G], y, yn;
    load_item(at, item);
    load_item(at1, next);
    load_rows(at, item, x, y);
    for (; ub < items; ub += stride) {
        advance(at2);
        load_item(at2, after);
        load_rows(at1, next, xn, yn);
        float sums[2 * G];
#pragma unroll
        for (int g = 0; g < G; ++g) {
            float ss = 0.f, a = 0.f;
#pragma unroll
            for (int q = 0; q < 4; ++q) ss = dot2_sq(x[g][q], ss);
#pragma unroll
            for (int e = 0; e < 8; ++e) a = __builtin_fmaf(bf16_at(x[g], e), bf16_at(y, e) * gain[e], a);
            sums[2 * g] = ss;
            sums[2 * g + 1] = a;
        }
        group_sums(sums, tpt);
        float acc[8] = {};   // sum over the item's picks of w rstd x
        bool named = false;
#pragma unroll
        for (int g = 0; g < G; ++g) {
            const int j = at.j + g;
            const bool ok = item.row[g] >= 0;
            const float rstd = 1.0f / sqrtf(sums[2 * g] * inv_h + eps);
            const float ra = ok ? rstd * sums[2 * g + 1] : 0.f;
            if (tid == 0 && at.t < T && j < k) {
                d_topk_w[at.t * k + j] = ra;
                if (ok) owner[item.row[g]] = static_cast<int32_t>(at.t * k + j);
            }
            if (!ok) continue;
            named = true;
            const float c = item.w[g] * rstd;
            const float d = rstd * (ra * inv_h);
            float o[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float xe = bf16_at(x[g], e);
                acc[e] = __builtin_fmaf(c, xe, acc[e]);
                o[e] = c * __builtin_fmaf(-xe, d, bf16_at(y, e) * gain[e]);
            }
            if (mine)
                store_nt(u32x4{cvt_pk_bf16(o[0], o[1]), cvt_pk_bf16(o[2], o[3]), cvt_pk_bf16(o[4], o[5]),
                               cvt_pk_bf16(o[6], o[7])},
                         &d_rows[static_cast<size_t>(item.row[g]) * nvec + tid]);
        }
        if (named)   // the output's gradient of a token without a slot may hold NaN
#pragma unroll
            for (int e = 0; e < 8; ++e) dgain[0][e] = __builtin_fmaf(bf16_at(y, e), acc[e], dgain[0][e]);
        at = at1;
        at1 = at2;
        item = next;
        next = after;
        y = yn;
#pragma unroll
        for (int g = 0; g < G; ++g) x[g] = xn[g];
    }
    if (part_gain)
        store_gain_part<1, kSmallBlock>(dgain, sub, tid, tpt, H, gain_lds, part_gain + static_cast<size_t>(blockIdx.x) * H);
}

// Rows a group of the kernel below: up to 32 registers of row data, and the next
// group's.
constexpr int row_group(int vpt) { return vpt <= 2 ? 4 : 2; }

// A token per wave (TPT = 64) or per block (TPT = BLOCK); of few tokens a part of
// its picks, kp of them, `parts` parts a token. Thread tid of a token owns vectors
// tid + i TPT of its rows, i < VPT. Lane j of every wave holds pick j's slot and
// weight (k <= 32), loaded one token ahead; the rows of the next G picks, the next
// token's first ones included, are in flight while the current ones are summed and
// written.
template <int VPT, int TPT, int BLOCK>
__global__ __launch_bounds__(BLOCK) __attribute__((amdgpu_waves_per_eu(2))) void combine_backward_kernel(
    const u32x4* __restrict__ d_out, const u32x4* __restrict__ expert_out, int R,
    const int32_t* __restrict__ slots, const float* __restrict__ topk_w, const float* __restrict__ norm_w,
    float gain_center, float eps, int T, int H, int k, int parts, int kp, int32_t* __restrict__ owner,
    u32x4* __restrict__ d_rows, float* __restrict__ d_topk_w, float* __restrict__ part_gain) {
    constexpr int G = row_group(VPT);
    // the sum over a token's slots of w rstd x, times y once per token; with
    // four vectors a thread there are no registers for it, and each slot's
    // product goes to the gain's gradient at once
    constexpr bool SUM = VPT < 4;
    constexpr int kBlockWaves = BLOCK / kWave;
    __shared__ float red[2][kBlockWaves][2 * G];
    extern __shared__ float gain_lds[];
    constexpr int groups = BLOCK / TPT;   // tokens of a block
    const int sub = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x) / TPT);
    const int tid = static_cast<int>(threadIdx.x) - sub * TPT;
    const int lane = __lane_id();
    const int wave = threadIdx.x / kWave;
    const int nvec = H >> 3;
    const float inv_h = 1.0f / static_cast<float>(H);

    float gain[VPT][8], dgain[VPT][8];
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int v = tid + i * TPT;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            gain[i][e] = v < nvec ? gain_center + norm_w[v * 8 + e] : 0.f;
            dgain[i][e] = 0.f;
        }
    }
    const long long units = static_cast<long long>(T) * parts;   // < 2^31, as T k is
    // unit u's token, and its first pick
    auto token_of = [&](long long u) { return parts == 1 ? u : static_cast<long long>(static_cast<uint32_t>(u) / parts); };
    auto pick_of = [&](long long u, long long t) { return parts == 1 ? 0 : static_cast<int>(u - t * parts) * kp; };
    auto load_picks = [&](long long u, int& r, float& w) {
        const long long t = token_of(u);
        const int j = pick_of(u, t) + lane;
        r = -1;
        w = 0.f;
        if (u < units && lane < kp && j < k) {
            r = slots[t * k + j];
            w = topk_w[t * k + j];
            if (r >= R) r = -1;
        }
    };
    auto load_token = [&](long long u, u32x4 (&y)[VPT]) {
        const u32x4* src = d_out + token_of(u) * nvec;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int v = tid + i * TPT;
            y[i] = u32x4{0, 0, 0, 0};
            if (u < units && v < nvec) y[i] = src[v];
        }
    };
    // lanes kp .. 63 hold slot -1, and j0 + G - 1 < 64
    auto load_rows = [&](int r, int j0, u32x4 (&x)[G][VPT]) {
#pragma unroll
        for (int g = 0; g < G; ++g) {
            const int row = __builtin_amdgcn_readlane(r, j0 + g);
#pragma unroll
            for (int i = 0; i < VPT; ++i) x[g][i] = u32x4{0, 0, 0, 0};
            if (row >= 0) {
                const u32x4* src = expert_out + static_cast<size_t>(row) * nvec;
#pragma unroll
                for (int i = 0; i < VPT; ++i) {
                    const int v = tid + i * TPT;
                    if (v < nvec) x[g][i] = load_nt(&src[v]);
                }
            }
        }
    };
    const long long stride = static_cast<long long>(gridDim.x) * groups;
    long long u = static_cast<long long>(blockIdx.x) * groups + sub;
    int pick_r, next_r;
    float pick_w, next_w;
    u32x4 y[VPT], x[G][VPT];
    load_picks(u, pick_r, pick_w);
    load_token(u, y);
    load_picks(u + stride, next_r, next_w);
    load_rows(pick_r, 0, x);
    int buf = 0;
    // the tokens of a block's groups start together, so that with a token per
    // block every thread takes the same turns
    for (; u < units; u += stride) {
        float acc[SUM ? VPT : 1][8] = {};
        u32x4 yn[VPT];
        float ra_of = 0.f;   // lane j: pick j's gradient
        for (int j0 = 0; j0 < kp; j0 += G) {
            u32x4 xn[G][VPT];
            if (j0 + G < kp) {
                load_rows(pick_r, j0 + G, xn);
            } else {
                load_token(u + stride, yn);
                load_rows(next_r, 0, xn);
            }
            float sums[2 * G];
#pragma unroll
            for (int g = 0; g < G; ++g) {
                float ss = 0.f, a = 0.f;
#pragma unroll
                for (int i = 0; i < VPT; ++i) {
#pragma unroll
                    for (int q = 0; q < 4; ++q) ss = dot2_sq(x[g][i][q], ss);
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        a = __builtin_fmaf(bf16_at(x[g][i], e), bf16_at(y[i], e) * gain[i][e], a);
                }
                sums[2 * g] = wave_sum(ss);
                sums[2 * g + 1] = wave_sum(a);
            }
            if constexpr (TPT == BLOCK) {
                if (lane == 0) {
#pragma unroll
                    for (int i = 0; i < 2 * G; ++i) red[buf][wave][i] = sums[i];
                }
                __syncthreads();
#pragma unroll
                for (int i = 0; i < 2 * G; ++i) {
                    sums[i] = red[buf][0][i];
                    for (int w = 1; w < kBlockWaves; ++w) sums[i] += red[buf][w][i];
                }
                buf ^= 1;   // the next group's sums go to the other buffer: one barrier a group
            }
#pragma unroll
            for (int i = 0; i < VPT; ++i) keep_packed(y[i]);
#pragma unroll
            for (int g = 0; g < G; ++g) {
                const int row = __builtin_amdgcn_readlane(pick_r, j0 + g);
                if (row < 0) continue;
#pragma unroll
                for (int i = 0; i < VPT; ++i) keep_packed(x[g][i]);
                const float w = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(pick_w), j0 + g));
                const float rstd = 1.0f / sqrtf(sums[2 * g] * inv_h + eps);
                const float ra = rstd * sums[2 * g + 1];
                if (lane == j0 + g) ra_of = ra;
                const float c = w * rstd;
                const float d = rstd * (ra * inv_h);
                u32x4* dst = d_rows + static_cast<size_t>(row) * nvec;
#pragma unroll
                for (int i = 0; i < VPT; ++i) {
                    const int v = tid + i * TPT;
                    float o[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const float xe = bf16_at(x[g][i], e);
                        if constexpr (SUM) acc[i][e] = __builtin_fmaf(c, xe, acc[i][e]);
                        else dgain[i][e] = __builtin_fmaf(c * xe, bf16_at(y[i], e), dgain[i][e]);
                        o[e] = c * __builtin_fmaf(-xe, d, bf16_at(y[i], e) * gain[i][e]);
                    }
                    if (v < nvec)
                        store_nt(u32x4{cvt_pk_bf16(o[0], o[1]), cvt_pk_bf16(o[2], o[3]), cvt_pk_bf16(o[4], o[5]),
                                       cvt_pk_bf16(o[6], o[7])},
                                 &dst[v]);
                }
            }
#pragma unroll
            for (int g = 0; g < G; ++g)
#pragma unroll
                for (int i = 0; i < VPT; ++i) x[g][i] = xn[g][i];
        }
        const long long t = token_of(u);
        const int j = pick_of(u, t) + tid;
        if (tid < kp && j < k) {   // the token's first wave; k <= 32
            d_topk_w[t * k + j] = ra_of;
            if (pick_r >= 0) owner[pick_r] = static_cast<int32_t>(t * k + j);
        }
        if constexpr (SUM) {
            if (ballot(pick_r >= 0))   // the output's gradient of other tokens may hold NaN
#pragma unroll
                for (int i = 0; i < VPT; ++i)
#pragma unroll
                    for (int e = 0; e < 8; ++e) dgain[i][e] = __builtin_fmaf(bf16_at(y[i], e), acc[i][e], dgain[i][e]);
        }
#pragma unroll
        for (int i = 0; i < VPT; ++i) y[i] = yn[i];
        pick_r = next_r;
        pick_w = next_w;
        load_picks(u + 2 * stride, next_r, next_w);
    }
    if (part_gain)
        store_gain_part<VPT, BLOCK>(dgain, sub, tid, TPT, H, gain_lds, part_gain + static_cast<size_t>(blockIdx.x) * H);
}

// The gradient of row r as the sum over the slots that name it, in slot order,
// by one wave. The slots are scanned for each 64 vectors of the row, twice: this
// is for the odd row that several slots name, not for speed.
__device__ __forceinline__ void repeated_row(const u32x4* __restrict__ d_out, const u32x4* __restrict__ expert_out,
                                             const int32_t* __restrict__ slots, const float* __restrict__ topk_w,
                                             const float* __restrict__ norm_w, float gain_center, float eps, int n,
                                             int H, int k, int r, u32x4* __restrict__ d_rows) {
    const int lane = __lane_id();
    const int nvec = H >> 3;
    const u32x4* src = expert_out + static_cast<size_t>(r) * nvec;
    u32x4* dst = d_rows + static_cast<size_t>(r) * nvec;
    // sum over the row's slots of w y for vector v
    auto gathered = [&](int v, float (&s)[8]) {
#pragma unroll
        for (int e = 0; e < 8; ++e) s[e] = 0.f;
        for (int f0 = 0; f0 < n; f0 = n - f0 > kWave ? f0 + kWave : n) {
            uint64_t hit = ballot(lane < n - f0 && slots[f0 + lane] == r);
            while (hit) {
                const int f = f0 + __builtin_ctzll(hit);
                hit &= hit - 1;
                const float w = topk_w[f];
                if (v < nvec) {
                    const u32x4 y = d_out[static_cast<size_t>(f / k) * nvec + v];
#pragma unroll
                    for (int e = 0; e < 8; ++e) s[e] = __builtin_fmaf(w, bf16_at(y, e), s[e]);
                }
            }
        }
    };
    float ss = 0.f, a = 0.f;
    for (int v0 = 0; v0 < nvec; v0 += kWave) {
        const int v = v0 + lane;
        float s[8];
        gathered(v, s);
        if (v < nvec) {
            const u32x4 x = src[v];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float xe = bf16_at(x, e);
                ss = __builtin_fmaf(xe, xe, ss);
                a = __builtin_fmaf(xe, s[e] * (gain_center + norm_w[v * 8 + e]), a);
            }
        }
    }
    ss = wave_sum(ss);
    a = wave_sum(a);
    const float inv_h = 1.0f / static_cast<float>(H);
    const float rstd = 1.0f / sqrtf(ss * inv_h + eps);
    const float d = rstd * (rstd * a * inv_h);
    for (int v0 = 0; v0 < nvec; v0 += kWave) {
        const int v = v0 + lane;
        float s[8];
        gathered(v, s);
        if (v < nvec) {
            const u32x4 x = src[v];
            float o[8];
#pragma unroll
            for (int e = 0; e < 8; ++e)
                o[e] = rstd * __builtin_fmaf(-bf16_at(x, e), d, s[e] * (gain_center + norm_w[v * 8 + e]));
            dst[v] = u32x4{cvt_pk_bf16(o[0], o[1]), cvt_pk_bf16(o[2], o[3]), cvt_pk_bf16(o[4], o[5]),
                           cvt_pk_bf16(o[6], o[7])};
        }
    }
}

constexpr int kGainCols = 16;
constexpr int kGainGroups = kSmallBlock / kGainCols;

// Columns [16 b, 16 b + 16) of the blocks' partial gain gradients, 16 groups of
// threads over them.
__device__ __forceinline__ void reduce_gain(const float* __restrict__ part, int rows, int H, int b,
                                            float* __restrict__ d_norm_w) {
    __shared__ float s[kGainGroups][kGainCols + 1];
    const int col = threadIdx.x % kGainCols, group = threadIdx.x / kGainCols;
    const int c = b * kGainCols + col;
    float v = 0.f;
    if (c < H)
        for_batches<16>(group, rows, kGainGroups, [&](int r) { return part[static_cast<size_t>(r) * H + c]; },
                        [&](float p) { v += p; });
    s[group][col] = v;
    __syncthreads();
    if (group == 0 && c < H) {
        for (int g = 1; g < kGainGroups; ++g) v += s[g][col];
        d_norm_w[c] = v;
    }
}

// The first gain_blocks blocks add up the gain's gradient. The others take rows
// and slots [8 w, 8 w + 8) by wave w: zeros for rows without a slot, the sum
// for rows with several. Eight, so that the unnamed rows at a dispatch's end
// spread over many waves. The first of a row's slots that finds another one as
// its owner claims the row by turning the owner into its complement; the
// complement still says who the owner is.
constexpr int kRowsPerWave = 8;

__global__ __launch_bounds__(kSmallBlock) void combine_backward_rows_kernel(
    const u32x4* __restrict__ d_out, const u32x4* __restrict__ expert_out, int R,
    const int32_t* __restrict__ slots, const float* __restrict__ topk_w, const float* __restrict__ norm_w,
    float gain_center, float eps, int n, int H, int k, int32_t* owner, u32x4* __restrict__ d_rows,
    const float* __restrict__ part_gain, int parts, int gain_blocks, float* __restrict__ d_norm_w) {
    if (static_cast<int>(blockIdx.x) < gain_blocks) {
        reduce_gain(part_gain, parts, H, blockIdx.x, d_norm_w);
        return;
    }
    const int lane = __lane_id();
    const int nvec = H >> 3;
    const long long items = R > n ? R : n;
    const long long block = static_cast<long long>(blockIdx.x) - gain_blocks;
    const long long stride = (static_cast<long long>(gridDim.x) - gain_blocks) * (kSmallBlock / kWave) * kRowsPerWave;
    for (long long i0 = (block * (kSmallBlock / kWave) + threadIdx.x / kWave) * kRowsPerWave;
         i0 < items; i0 += stride) {
        const long long i = i0 + lane;
        bool unnamed = false, repeated = false;
        int r = 0;
        if (lane < kRowsPerWave && i < R) {
            const int o = __hip_atomic_load(&owner[i], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            const int f = o < 0 ? ~o : o;
            unnamed = f >= n || slots[f] != i;
        }
        if (lane < kRowsPerWave && i < n) {
            r = slots[i];
            if (r >= 0 && r < R) {
                int o = __hip_atomic_load(&owner[r], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
                repeated = o >= 0 && o != i &&
                           __hip_atomic_compare_exchange_strong(&owner[r], &o, ~o, __ATOMIC_RELAXED, __ATOMIC_RELAXED,
                                                                __HIP_MEMORY_SCOPE_AGENT);
            }
        }
        uint64_t todo = ballot(unnamed);
        while (todo) {
            const long long row = i0 + __builtin_ctzll(todo);
            todo &= todo - 1;
            u32x4* dst = d_rows + row * nvec;
            for (int v = lane; v < nvec; v += kWave) store_nt(u32x4{0, 0, 0, 0}, &dst[v]);
        }
        todo = ballot(repeated);
        while (todo) {
            const int row = __builtin_amdgcn_readlane(r, __builtin_ctzll(todo));
            todo &= todo - 1;
            repeated_row(d_out, expert_out, slots, topk_w, norm_w, gain_center, eps, n, H, k, row, d_rows);
        }
    }
}

constexpr int kMostBlocks = 512;   // two a CU
// A token's picks are shared by several units while all units fit this many blocks
// (whole tokens / parts: 16 tokens of 2048, k 32, 41 / 12 us, 64 of 8192, k 8, 18 /
// 15; with up to 512 blocks 256 of 8192, k 8, took 33 us in all instead of 30: each
// block's partial sums of the gain are written and read).
constexpr int kSplitBlocks = 256;

struct CombineBackwardPlan {
    int tpt, vpt, block, groups, rows, grid;
    size_t owner, gain, bytes;
};

inline size_t round256(size_t b) { return (b + 255) / 256 * 256; }

// Depends on T, R and H alone (not on the device), so that the workspace query
// and the call agree.
inline CombineBackwardPlan plan_combine_backward(int T, int R, int H) {
    CombineBackwardPlan p;
    const int nvec = H / 8;
    p.block = kSmallBlock;
    if (nvec < kWave) {
        p.tpt = 1;
        while (p.tpt < nvec) p.tpt <<= 1;
    } else if (nvec <= 4 * kWave) {
        p.tpt = kWave;
    } else {
        if (nvec > 4 * kSmallBlock) p.block = kWideBlock;
        p.tpt = p.block;
    }
    p.vpt = ceil_div(nvec, p.tpt);
    p.groups = p.block / p.tpt;
    // at most a unit for every p.rows picks, of any k the workspace may be used with
    p.rows = p.tpt < kWave ? kNarrowRows : row_group(p.vpt);
    const long long need = (static_cast<long long>(T) * (MOE_MAX_TOPK / p.rows) + p.groups - 1) / p.groups;
    p.grid = static_cast<int>(need < kMostBlocks ? need : kMostBlocks);
    p.owner = 0;
    p.gain = round256(sizeof(int32_t) * static_cast<size_t>(R));
    p.bytes = p.gain + round256(sizeof(float) * static_cast<size_t>(p.grid) * H);
    if (p.bytes == 0) p.bytes = 256;
    return p;
}

inline bool combine_backward_shape_ok(int T, int R, int H) {
    return T >= 0 && R >= 0 && H >= 8 && H <= MOE_MAX_HIDDEN && H % 8 == 0;
}

}  // namespace
}  // namespace moe

extern "C" size_t moe_combine_backward_workspace_bytes(int T, int R, int H) {
    using namespace moe;
    return combine_backward_shape_ok(T, R, H) ? plan_combine_backward(T, R, H).bytes : 0;
}

extern "C" int moe_combine_backward(const uint16_t* d_out, const uint16_t* expert_out, int R, const int32_t* slots,
                                    const float* topk_w, const float* norm_w, float gain_center, float eps, int T,
                                    int H, int k, uint16_t* d_expert_out, float* d_topk_w, float* d_norm_w,
                                    void* workspace, size_t workspace_bytes, void* stream) {
    using namespace moe;
    if (!combine_backward_shape_ok(T, R, H) || k < 1 || k > MOE_MAX_TOPK) return MOE_ERR_BAD_SHAPE;
    if (static_cast<long long>(T) * k >= (1ll << 31) || static_cast<long long>(R) * (H / 8) >= (1ll << 40))
        return MOE_ERR_BAD_SHAPE;
    if (!std::isfinite(gain_center) || !std::isfinite(eps) || eps < 0.f) return MOE_ERR_BAD_ARG;
    if (T > 0 && (!d_out || !slots || !topk_w || !d_topk_w)) return MOE_ERR_NULL_ARG;
    if (!norm_w || (R > 0 && (!expert_out || !d_expert_out))) return MOE_ERR_NULL_ARG;
    if (!all_aligned16(d_out, expert_out, slots, topk_w, norm_w, d_expert_out, d_topk_w, d_norm_w))
        return MOE_ERR_ALIGN;
    CombineBackwardPlan p = plan_combine_backward(T, R, H);
    if (!workspace || workspace_bytes < p.bytes || !aligned16(workspace)) return MOE_ERR_WORKSPACE;
    // narrow rows: an item for every p.rows picks; else a token's picks in more
    // parts while those of all tokens fit a block a CU
    int kp = p.tpt < kWave ? p.rows : k;
    while (kp > p.rows && static_cast<long long>(T) * ceil_div(k, ceil_div(kp, 2 * p.rows) * p.rows) <= kSplitBlocks * p.groups)
        kp = ceil_div(kp, 2 * p.rows) * p.rows;
    const int parts = ceil_div(k, kp);
    const int need = ceil_div(static_cast<long long>(T) * parts, p.groups);
    if (need < p.grid) p.grid = need;
    auto* owner = reinterpret_cast<int32_t*>(static_cast<char*>(workspace) + p.owner);
    auto* part = d_norm_w ? reinterpret_cast<float*>(static_cast<char*>(workspace) + p.gain) : nullptr;
    const auto* y = reinterpret_cast<const u32x4*>(d_out);
    const auto* x = reinterpret_cast<const u32x4*>(expert_out);
    auto* dx = reinterpret_cast<u32x4*>(d_expert_out);
    int st;
    if (T > 0) {
        const size_t lds = p.groups > 1 ? sizeof(float) * static_cast<size_t>(p.groups) * H : 0;
        auto run = [&](auto kern) {
            return launch(kern, dim3(p.grid), dim3(p.block), lds, stream, y, x, R, slots, topk_w, norm_w, gain_center,
                          eps, T, H, k, parts, kp, owner, dx, d_topk_w, part);
        };
        if (p.tpt < kWave)
            st = launch(combine_backward_narrow_kernel, dim3(p.grid), dim3(p.block), lds, stream, y, x, R, slots,
                        topk_w, norm_w, gain_center, eps, T, H, k, p.tpt, owner, dx, d_topk_w, part);
        else if (p.tpt == kWave)
            st = p.vpt == 1   ? run(combine_backward_kernel<1, kWave, kSmallBlock>)
                 : p.vpt == 2 ? run(combine_backward_kernel<2, kWave, kSmallBlock>)
                 : p.vpt == 3 ? run(combine_backward_kernel<3, kWave, kSmallBlock>)
                              : run(combine_backward_kernel<4, kWave, kSmallBlock>);
        else if (p.block == kSmallBlock)
            st = p.vpt <= 2   ? run(combine_backward_kernel<2, kSmallBlock, kSmallBlock>)
                 : p.vpt == 3 ? run(combine_backward_kernel<3, kSmallBlock, kSmallBlock>)
                              : run(combine_backward_kernel<4, kSmallBlock, kSmallBlock>);
        else
            st = p.vpt <= 3 ? run(combine_backward_kernel<3, kWideBlock, kWideBlock>)
                            : run(combine_backward_kernel<4, kWideBlock, kWideBlock>);
        if (st != MOE_OK) return st;
    }
    if (R == 0 && !d_norm_w) return MOE_OK;
    const int n = T * k;
    const int gain_blocks = d_norm_w ? ceil_div(H, kGainCols) : 0;
    const long long blocks = R > 0 ? ceil_div(R > n ? R : n, kRowsPerWave * (kSmallBlock / kWave)) : 0;
    const long long most = 16ll * device_cu_count();
    return launch(combine_backward_rows_kernel,
                  dim3(gain_blocks + static_cast<unsigned>(blocks < most ? blocks : most)), dim3(kSmallBlock), 0, stream,
                  y, x, R, slots, topk_w, norm_w, gain_center, eps, n, H, k, owner, dx, part, T > 0 ? p.grid : 0,
                  gain_blocks, d_norm_w);
}
