// A token's router logits held by one wave, and the router's distribution over
// them, for the losses on the logits.
//
// The row of E logits is spread over the wave in vectors of four: lane l owns
// columns 256 i + 4 l + (0..3) for i < NV (E <= 256 NV), so a load of the wave
// covers 1 KB of the row. Columns from E on hold -inf, which weighs zero.
#pragma once

#include "common.hpp"
#include "moe_training.h"

namespace moe {

// Four floats at any 4-byte aligned address (rows of an E that is not a
// multiple of four): still one 16-byte access.
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x4_any __attribute__((ext_vector_type(4), aligned(4)));

constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kNegInf = -__builtin_huge_valf();

// exp(x), x <= 0 or small: the product's rounding is |x| 2^-24, which stays
// near one ulp where the result counts.
__device__ __forceinline__ float exp_fast(float x) { return __builtin_amdgcn_exp2f(x * kLog2e); }

// Maximum over the wave (same exchanges as wave_sum). NaN is ignored unless
// every lane holds one.
__device__ __forceinline__ float wave_max(float v) {
    uint32_t u = __float_as_uint(v);
    const auto s32 = __builtin_amdgcn_permlane32_swap(u, u, false, false);
    v = fmaxf(__uint_as_float(s32[0]), __uint_as_float(s32[1]));
    u = __float_as_uint(v);
    const auto s16 = __builtin_amdgcn_permlane16_swap(u, u, false, false);
    v = fmaxf(__uint_as_float(s16[0]), __uint_as_float(s16[1]));
    v = fmaxf(v, __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x128, 0xF, 0xF, false)));
    v = fmaxf(v, __int_as_float(__builtin_amdgcn_ds_swizzle(__float_as_int(v), 0x101F)));
    v = fmaxf(v, __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x4E, 0xF, 0xF, false)));
    v = fmaxf(v, __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0xB1, 0xF, 0xF, false)));
    return v;
}

template <int NV>
__device__ __forceinline__ void load_row(const float* __restrict__ row, int E, int lane, float (&x)[NV][4]) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = i * 256 + lane * 4;
        if (c + 4 <= E) {
            const f32x4 v = *reinterpret_cast<const f32x4_any*>(row + c);
#pragma unroll
            for (int q = 0; q < 4; ++q) x[i][q] = v[q];
        } else {
#pragma unroll
            for (int q = 0; q < 4; ++q) x[i][q] = c + q < E ? row[c + q] : kNegInf;
        }
    }
}

// Writes the row, or adds it to what is there.
template <int NV>
__device__ __forceinline__ void store_row(float* __restrict__ row, int E, int lane, const float (&x)[NV][4],
                                          bool accumulate) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = i * 256 + lane * 4;
        if (c + 4 <= E) {
            f32x4_any* p = reinterpret_cast<f32x4_any*>(row + c);
            f32x4 v = {x[i][0], x[i][1], x[i][2], x[i][3]};
            if (accumulate) v += *p;
            *p = v;
        } else {
#pragma unroll
            for (int q = 0; q < 4; ++q)
                if (c + q < E) row[c + q] = accumulate ? row[c + q] + x[i][q] : x[i][q];
        }
    }
}

template <int NV>
__device__ __forceinline__ float row_max(const float (&x)[NV][4]) {
    float m = kNegInf;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int q = 0; q < 4; ++q) m = fmaxf(m, x[i][q]);
    return wave_max(m);
}

template <int NV>
__device__ __forceinline__ float row_sum(const float (&x)[NV][4]) {
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int q = 0; q < 4; ++q) s += x[i][q];
    return wave_sum(s);
}

// u = exp(x - max x), returning the maximum (0 for a row of -inf, whose u are
// then zero).
template <int NV>
__device__ __forceinline__ float softmax_weights(const float (&x)[NV][4], float (&u)[NV][4]) {
    float m = row_max(x);
    if (m == kNegInf) m = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int q = 0; q < 4; ++q) u[i][q] = exp_fast(x[i][q] - m);
    return m;
}

// The sigmoid s of x, relative to the row's largest: with e = exp(-|x|),
//   s = exp(min(x, 0)) / (1 + e),   1 - s = exp(-max(x, 0)) / (1 + e),
// u = exp(min(x, 0) - m) / (1 + e), m = max min(x, 0) <= 0, so that a row
// whose every s underflows keeps its proportions. Returns m (0 when a logit is
// positive, and then u = s with one exponential).
template <int NV, bool SLOPE>
__device__ __forceinline__ float sigmoid_weights(const float (&x)[NV][4], float (&u)[NV][4],
                                                 float (&slope)[SLOPE ? NV : 1][4]) {
    float m = fminf(row_max(x), 0.f);
    if (m == kNegInf) m = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const float v = x[i][q];
            const float e = exp_fast(-fabsf(v));
            const float r = __builtin_amdgcn_rcpf(1.f + e);
            const float er = e * r;
            u[i][q] = v > 0.f ? r : er;
            if constexpr (SLOPE) slope[i][q] = v > 0.f ? er : r;
            if (m < 0.f) u[i][q] = exp_fast(v - m) * r;   // every logit is negative
        }
    return m;
}

// log of the score of one logit (the sigmoid's, or the logit itself).
__device__ __forceinline__ float log_score(float x, int score) {
    if (score == MOE_SCORE_SOFTMAX) return x;
    return fminf(x, 0.f) - log1pf(expf(-fabsf(x)));
}

// ---- sequences of tokens ----------------------------------------------------

// Offset i of S + 1; without a table one sequence holds all T tokens.
__device__ __forceinline__ int seq_offset(const int32_t* __restrict__ off, int i, int T) {
    return off ? min(max(off[i], 0), T) : (i == 0 ? 0 : T);
}

// The sequence of token t (its offsets in begin, end), found by the whole wave
// in steps of 64 probes; -1 for a token in none.
__device__ __forceinline__ int find_sequence(const int32_t* __restrict__ off, int S, int T, int t, int& begin,
                                             int& end) {
    int lo = 0, len = S + 1;
    const int lane = __lane_id();
    while (true) {
        const int step = (len + kWave - 1) / kWave;
        const int i = lo + lane * step;
        const bool at = lane * step < len && seq_offset(off, i, T) <= t;
        const int n = __popcll(ballot(at));
        if (n == 0) return -1;
        lo += (n - 1) * step;
        if (step == 1) break;
        len = min(step, S + 1 - lo);
    }
    if (lo >= S) return -1;
    begin = seq_offset(off, lo, T);
    end = seq_offset(off, lo + 1, T);
    return t < end ? lo : -1;
}

// Picks NV for E experts and calls f with it as a constant.
template <typename F>
inline int with_row_vectors(int E, F&& f) {
    if (E <= 256) return f(std::integral_constant<int, 1>());
    if (E <= 512) return f(std::integral_constant<int, 2>());
    if (E <= 1024) return f(std::integral_constant<int, 4>());
    if (E <= 1536) return f(std::integral_constant<int, 6>());
    if (E <= 2048) return f(std::integral_constant<int, 8>());
    if (E <= 2560) return f(std::integral_constant<int, 10>());
    return f(std::integral_constant<int, 16>());
}

}  // namespace moe
