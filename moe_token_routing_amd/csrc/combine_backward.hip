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
// and y is read once per token. So one group of threads takes a token, keeps y
// in registers for its k rows and each row in registers between the sums and
// the gradient. Blocks are persistent over tokens, so that the gain's gradient
// is summed in registers and only one row of partial sums per block is
// written; a last kernel adds those in block order.
//
// Rows and slots need not match one to one. The slots of each row are counted
// first (integer atomics); the main kernel writes the rows that one slot
// names, and the row kernel the others: zeros for none, and for several the
// sum over their slots in slot order.
#include <cmath>

#include "launch.hpp"
#include "rows.hpp"

namespace moe {
namespace {

constexpr int kSmallBlock = 256;
constexpr int kWideBlock = 512;   // rows of more than 1024 vectors

__global__ __launch_bounds__(kSmallBlock) void clear_kernel(int32_t* __restrict__ p, int n) {
    for (long long i = blockIdx.x * static_cast<long long>(kSmallBlock) + threadIdx.x; i < n;
         i += static_cast<long long>(gridDim.x) * kSmallBlock)
        p[i] = 0;
}

__global__ __launch_bounds__(kSmallBlock) void count_rows_kernel(const int32_t* __restrict__ slots, int n, int R,
                                                                 int32_t* __restrict__ named) {
    for (long long f = blockIdx.x * static_cast<long long>(kSmallBlock) + threadIdx.x; f < n;
         f += static_cast<long long>(gridDim.x) * kSmallBlock) {
        const int r = slots[f];
        if (r >= 0 && r < R) atomicAdd(&named[r], 1);
    }
}

__device__ __forceinline__ float bf16_at(const u32x4& v, int e) {
    const uint32_t w = v[e >> 1];
    return e & 1 ? bf16_hi(w) : bf16_lo(w);
}

// TPT threads per token: 0 for tpt < 64 (a power of two, so a wave holds
// several tokens), 64 (a token per wave), or BLOCK (a token per block). Thread
// tid of a token owns vectors tid + i tpt of its rows, i < VPT.
// Makes the compiler forget what it derived from a register, so that it unpacks
// a row again where it is used next instead of keeping the unpacked values.
__device__ __forceinline__ void keep_packed(u32x4& v) { asm volatile("" : "+v"(v)); }

template <int VPT, int TPT, int BLOCK>
__global__ __launch_bounds__(BLOCK) __attribute__((amdgpu_waves_per_eu(2))) void combine_backward_kernel(
    const u32x4* __restrict__ d_out, const u32x4* __restrict__ expert_out, int R,
    const int32_t* __restrict__ slots, const float* __restrict__ topk_w, const float* __restrict__ norm_w,
    float gain_center, float eps, int T, int H, int k, int tpt, const int32_t* __restrict__ named,
    u32x4* __restrict__ d_rows, float* __restrict__ d_topk_w, float* __restrict__ part_gain) {
    constexpr int G = VPT >= 3 ? 4 : 8;   // rows a group: up to 64 registers of row data
    constexpr int kBlockWaves = BLOCK / kWave;
    __shared__ float red[2][kBlockWaves][2 * G];
    extern __shared__ float gain_lds[];
    if (TPT != 0) tpt = TPT;
    const int groups = BLOCK / tpt;   // tokens of a block
    const int sub = TPT >= kWave ? __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x) / TPT)
                                 : static_cast<int>(threadIdx.x) / tpt;
    const int tid = static_cast<int>(threadIdx.x) - sub * tpt;
    const int lane = __lane_id();
    const int wave = threadIdx.x / kWave;
    const int nvec = H >> 3;
    const float inv_h = 1.0f / static_cast<float>(H);

    float gain[VPT][8], dgain[VPT][8];
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int v = tid + i * tpt;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            gain[i][e] = v < nvec ? gain_center + norm_w[v * 8 + e] : 0.f;
            dgain[i][e] = 0.f;
        }
    }
    int buf = 0;
    const long long stride = static_cast<long long>(gridDim.x) * groups;
    for (long long t0 = static_cast<long long>(blockIdx.x) * groups; t0 < T; t0 += stride) {
        const long long t = t0 + sub;
        const bool tok_ok = t < T;
        u32x4 y[VPT];
        float acc[VPT][8];   // sum over the slots of w rstd x
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int v = tid + i * tpt;
            y[i] = u32x4{0, 0, 0, 0};
            if (tok_ok && v < nvec) y[i] = d_out[t * nvec + v];
#pragma unroll
            for (int e = 0; e < 8; ++e) acc[i][e] = 0.f;
        }
        for (int j0 = 0; j0 < k; j0 += G) {
            u32x4 x[G][VPT];
            float wt[G], sums[2 * G];
            int row[G];
            bool ok[G], sole[G];
#pragma unroll
            for (int g = 0; g < G; ++g) {
                const int j = j0 + g;
                row[g] = -1;
                wt[g] = 0.f;
                if (tok_ok && j < k) {
                    row[g] = slots[t * k + j];
                    wt[g] = topk_w[t * k + j];
                }
                ok[g] = row[g] >= 0 && row[g] < R;
                sole[g] = false;
#pragma unroll
                for (int i = 0; i < VPT; ++i) x[g][i] = u32x4{0, 0, 0, 0};
                if (ok[g]) {
                    sole[g] = named[row[g]] == 1;
                    const u32x4* src = expert_out + static_cast<size_t>(row[g]) * nvec;
#pragma unroll
                    for (int i = 0; i < VPT; ++i) {
                        const int v = tid + i * tpt;
                        if (v < nvec) x[g][i] = load_nt(&src[v]);
                    }
                }
            }
#pragma unroll
            for (int g = 0; g < G; ++g) {
                float ss = 0.f, a = 0.f;
                if (ok[g]) {
#pragma unroll
                    for (int i = 0; i < VPT; ++i) {
#pragma unroll
                        for (int q = 0; q < 4; ++q) ss = dot2_sq(x[g][i][q], ss);
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            a = __builtin_fmaf(bf16_at(x[g][i], e), bf16_at(y[i], e) * gain[i][e], a);
                    }
                }
                sums[2 * g] = ss;
                sums[2 * g + 1] = a;
            }
            if constexpr (TPT == 0) {
#pragma unroll
                for (int i = 0; i < 2 * G; ++i) sums[i] = group_sum(sums[i], tpt);
            } else {
#pragma unroll
                for (int i = 0; i < 2 * G; ++i) sums[i] = wave_sum(sums[i]);
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
#pragma unroll
                for (int i = 0; i < VPT; ++i) keep_packed(x[g][i]);
                const int j = j0 + g;
                if (tok_ok && j < k && tid == 0 && !ok[g]) d_topk_w[t * k + j] = 0.f;
                if (!ok[g]) continue;
                const float rstd = 1.0f / sqrtf(sums[2 * g] * inv_h + eps);
                const float ra = rstd * sums[2 * g + 1];
                if (tid == 0) d_topk_w[t * k + j] = ra;
                const float c = wt[g] * rstd;
                const float d = rstd * (ra * inv_h);
                u32x4* dst = d_rows + static_cast<size_t>(row[g]) * nvec;
#pragma unroll
                for (int i = 0; i < VPT; ++i) {
                    const int v = tid + i * tpt;
                    float o[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const float xe = bf16_at(x[g][i], e);
                        acc[i][e] = __builtin_fmaf(c, xe, acc[i][e]);
                        o[e] = c * __builtin_fmaf(-xe, d, bf16_at(y[i], e) * gain[i][e]);
                    }
                    if (sole[g] && v < nvec) {
                        const u32x4 out = {cvt_pk_bf16(o[0], o[1]), cvt_pk_bf16(o[2], o[3]),
                                           cvt_pk_bf16(o[4], o[5]), cvt_pk_bf16(o[6], o[7])};
                        store_nt(out, &dst[v]);
                    }
                }
            }
        }
#pragma unroll
        for (int i = 0; i < VPT; ++i)
#pragma unroll
            for (int e = 0; e < 8; ++e) dgain[i][e] = __builtin_fmaf(bf16_at(y[i], e), acc[i][e], dgain[i][e]);
    }
    if (!part_gain) return;
    // the block's row of partial gain gradients: its token groups in order
    float* out = part_gain + static_cast<size_t>(blockIdx.x) * H;
    if constexpr (TPT == BLOCK) {
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int v = tid + i * tpt;
            if (v < nvec) {
                float4* p = reinterpret_cast<float4*>(out) + 2 * v;
                p[0] = make_float4(dgain[i][0], dgain[i][1], dgain[i][2], dgain[i][3]);
                p[1] = make_float4(dgain[i][4], dgain[i][5], dgain[i][6], dgain[i][7]);
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int v = tid + i * tpt;
            if (v < nvec)
#pragma unroll
                for (int e = 0; e < 8; ++e) gain_lds[sub * H + v * 8 + e] = dgain[i][e];
        }
        __syncthreads();
        for (int c = threadIdx.x; c < H; c += BLOCK) {
            float s = gain_lds[c];
            for (int q = 1; q < groups; ++q) s += gain_lds[q * H + c];
            out[c] = s;
        }
    }
}

// One wave per row that no slot or several slots name.
__global__ __launch_bounds__(kSmallBlock) void combine_backward_rows_kernel(
    const u32x4* __restrict__ d_out, const u32x4* __restrict__ expert_out, int R,
    const int32_t* __restrict__ slots, const float* __restrict__ topk_w, const float* __restrict__ norm_w,
    float gain_center, float eps, int T, int H, int k, const int32_t* __restrict__ named,
    u32x4* __restrict__ d_rows) {
    const int lane = __lane_id();
    const int nvec = H >> 3;
    const int waves = kSmallBlock / kWave;
    const long long n = static_cast<long long>(T) * k;
    for (long long r = static_cast<long long>(blockIdx.x) * waves + threadIdx.x / kWave; r < R;
         r += static_cast<long long>(gridDim.x) * waves) {
        const int count = __builtin_amdgcn_readfirstlane(named[r]);
        if (count == 1) continue;
        u32x4* dst = d_rows + r * nvec;
        if (count == 0) {
            for (int v = lane; v < nvec; v += kWave) store_nt(u32x4{0, 0, 0, 0}, &dst[v]);
            continue;
        }
        const u32x4* src = expert_out + r * nvec;
        // sum over the row's slots, in slot order, of w y for vector v
        auto gathered = [&](int v, float (&s)[8]) {
#pragma unroll
            for (int e = 0; e < 8; ++e) s[e] = 0.f;
            int left = count;
            for (long long f0 = 0; f0 < n && left > 0; f0 += kWave) {
                uint64_t hit = ballot(f0 + lane < n && slots[f0 + lane] == r);
                while (hit) {
                    const long long f = f0 + __builtin_ctzll(hit);
                    hit &= hit - 1;
                    --left;
                    const float w = topk_w[f];
                    if (v < nvec) {
                        const u32x4 y = d_out[(f / k) * nvec + v];
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
}

constexpr int kGainCols = 32;
constexpr int kGainGroups = 32;

// Columns [32 b, 32 b + 32) of the partial rows, 32 groups of threads over them.
__global__ __launch_bounds__(kGainCols* kGainGroups) void gain_reduce_kernel(const float* __restrict__ part, int rows,
                                                                              int H, float* __restrict__ d_norm_w) {
    __shared__ float s[kGainGroups][kGainCols + 1];
    const int col = threadIdx.x % kGainCols, group = threadIdx.x / kGainCols;
    const int c = blockIdx.x * kGainCols + col;
    float v = 0.f;
    if (c < H) {
#pragma unroll 4
        for (int r = group; r < rows; r += kGainGroups) v += part[static_cast<size_t>(r) * H + c];
    }
    s[group][col] = v;
    __syncthreads();
    if (group == 0 && c < H) {
        for (int g = 1; g < kGainGroups; ++g) v += s[g][col];
        d_norm_w[c] = v;
    }
}

struct CombineBackwardPlan {
    int tpt, vpt, block, groups, grid;
    size_t named, gain, bytes;
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
    const int need = ceil_div(T, p.groups);
    const int most = 512;   // two blocks a CU
    p.grid = need < most ? need : most;
    p.named = 0;
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
    const CombineBackwardPlan p = plan_combine_backward(T, R, H);
    if (!workspace || workspace_bytes < p.bytes || !aligned16(workspace)) return MOE_ERR_WORKSPACE;
    auto* named = reinterpret_cast<int32_t*>(static_cast<char*>(workspace) + p.named);
    auto* part = d_norm_w ? reinterpret_cast<float*>(static_cast<char*>(workspace) + p.gain) : nullptr;
    const auto* y = reinterpret_cast<const u32x4*>(d_out);
    const auto* x = reinterpret_cast<const u32x4*>(expert_out);
    auto* dx = reinterpret_cast<u32x4*>(d_expert_out);
    const int most = 8 * device_cu_count();
    auto grid_of = [&](long long n, int per) {
        const long long g = (n + per - 1) / per;
        return dim3(static_cast<unsigned>(g < most ? g : most));
    };
    int st;
    if (R > 0) {
        st = launch(clear_kernel, grid_of(R, kSmallBlock), dim3(kSmallBlock), 0, stream, named, R);
        if (st != MOE_OK) return st;
        if (T > 0) {
            st = launch(count_rows_kernel, grid_of(static_cast<long long>(T) * k, kSmallBlock), dim3(kSmallBlock), 0,
                        stream, slots, T * k, R, named);
            if (st != MOE_OK) return st;
        }
        st = launch(combine_backward_rows_kernel, grid_of(R, kSmallBlock / kWave), dim3(kSmallBlock), 0, stream, y,
                    x, R, slots, topk_w, norm_w, gain_center, eps, T, H, k, named, dx);
        if (st != MOE_OK) return st;
    }
    if (T > 0) {
#define MOE_CB_ARGS y, x, R, slots, topk_w, norm_w, gain_center, eps, T, H, k, p.tpt, named, dx, d_topk_w, part
        auto run = [&](auto kern) {
            const size_t lds = p.groups > 1 ? sizeof(float) * static_cast<size_t>(p.groups) * H : 0;
            return launch(kern, dim3(p.grid), dim3(p.block), lds, stream, MOE_CB_ARGS);
        };
        if (p.tpt < kWave) st = run(combine_backward_kernel<1, 0, kSmallBlock>);
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
#undef MOE_CB_ARGS
        if (st != MOE_OK) return st;
    }
    if (!d_norm_w) return MOE_OK;
    return launch(gain_reduce_kernel, dim3(ceil_div(H, kGainCols)), dim3(kGainCols * kGainGroups), 0, stream, part,
                  T > 0 ? p.grid : 0, H, d_norm_w);
}
