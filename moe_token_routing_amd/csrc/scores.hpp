// A token's router logits held by one wave or by several, and the router's
// distribution over them, for the losses on the logits.
//
// A row of E logits is spread over WPT waves in vectors of four: lane l of wave
// w owns columns 256 (WPT i + w) + 4 l + (0..3) for i < NV (E <= 256 NV WPT), so
// a load of a wave covers 1 KB of the row. Columns from E on hold -inf, which
// weighs zero. Narrow rows take one wave, which needs no barrier; wide ones all
// waves of a block, so that a row stays in few registers (with one wave for 4096
// columns, 64 registers for each array, the balance loss of 4096 tokens took 92
// us and its gradient 53; with four 17 and 22).
#pragma once

#include <type_traits>

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

// log(x) for x >= 1/2 or 0, by the hardware's base 2 logarithm.
__device__ __forceinline__ float log_fast(float x) { return __builtin_amdgcn_logf(x) * 0.693147180559945309417f; }

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

template <int NV, int WPT>
struct Row {
    float v[NV][4];

    static __device__ __forceinline__ int column(int i, int wave, int lane) {
        return (i * WPT + wave) * 256 + lane * 4;
    }

    __device__ __forceinline__ void fill(float f) {
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int q = 0; q < 4; ++q) v[i][q] = f;
    }

    __device__ __forceinline__ void scale(float f) {
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int q = 0; q < 4; ++q) v[i][q] *= f;
    }

    __device__ __forceinline__ void load(const float* __restrict__ row, int E, int wave, int lane) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = column(i, wave, lane);
            if (c + 4 <= E) {
                const f32x4 x = *reinterpret_cast<const f32x4_any*>(row + c);
#pragma unroll
                for (int q = 0; q < 4; ++q) v[i][q] = x[q];
            } else {
#pragma unroll
                for (int q = 0; q < 4; ++q) v[i][q] = c + q < E ? row[c + q] : kNegInf;
            }
        }
    }

    // Writes the row, or adds it to what is there.
    __device__ __forceinline__ void store(float* __restrict__ row, int E, int wave, int lane, bool accumulate) const {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = column(i, wave, lane);
            if (c + 4 <= E) {
                f32x4_any* p = reinterpret_cast<f32x4_any*>(row + c);
                f32x4 x = {v[i][0], v[i][1], v[i][2], v[i][3]};
                if (accumulate) x += *p;
                *p = x;
            } else {
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    if (c + q < E) row[c + q] = accumulate ? row[c + q] + v[i][q] : v[i][q];
            }
        }
    }

    // This lane's part of the maximum and the sum.
    __device__ __forceinline__ float max() const {
        float m = kNegInf;
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int q = 0; q < 4; ++q) m = fmaxf(m, v[i][q]);
        return m;
    }

    __device__ __forceinline__ float sum() const {
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int q = 0; q < 4; ++q) s += v[i][q];
        return s;
    }

    __device__ __forceinline__ float dot(const Row& o) const {
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int q = 0; q < 4; ++q) s = __builtin_fmaf(v[i][q], o.v[i][q], s);
        return s;
    }
};

// Reductions over a row's waves. With several the waves meet in LDS: every wave
// of the block calls, and two buffers alternate, so that a call costs one
// barrier.
template <int WPT>
struct RowReduce {
    float (*red)[WPT][4];   // [2][WPT][4] in LDS
    int wave;
    int buf = 0;

    __device__ __forceinline__ float max(float m) {
        m = wave_max(m);
        if constexpr (WPT > 1) {
            if (__lane_id() == 0) red[buf][wave][0] = m;
            __syncthreads();
            for (int w = 0; w < WPT; ++w) m = fmaxf(m, red[buf][w][0]);
            buf ^= 1;
        }
        return m;
    }

    // Sums of N values, the waves' in order.
    template <int N>
    __device__ __forceinline__ void sum(float (&v)[N]) {
        static_assert(N <= 4, "the buffer's width");
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = wave_sum(v[i]);
        if constexpr (WPT > 1) {
            if (__lane_id() == 0)
#pragma unroll
                for (int i = 0; i < N; ++i) red[buf][wave][i] = v[i];
            __syncthreads();
#pragma unroll
            for (int i = 0; i < N; ++i) {
                v[i] = red[buf][0][i];
                for (int w = 1; w < WPT; ++w) v[i] += red[buf][w][i];
            }
            buf ^= 1;
        }
    }
};

// The maximum that weights are taken relative to: 0 for a row of -inf, whose
// weights are then zero.
__device__ __forceinline__ float weight_origin(float m) { return m == kNegInf ? 0.f : m; }

// u = exp(x - m).
template <int NV, int WPT>
__device__ __forceinline__ void softmax_weights(const Row<NV, WPT>& x, float m, Row<NV, WPT>& u) {
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int q = 0; q < 4; ++q) u.v[i][q] = exp_fast(x.v[i][q] - m);
}

// The sigmoid s of x, relative to the row's largest: with e = exp(-|x|),
//   s = exp(min(x, 0)) / (1 + e),   1 - s = exp(-max(x, 0)) / (1 + e),
// u = exp(min(x, 0) - m) / (1 + e), m = min(max x, 0), so that a row whose every
// s underflows keeps its proportions. m = 0 when a logit is positive, and then
// u = s with one exponential; without the slope as 1 / (1 + exp(-x)), which is
// as exact and half the instructions. The branch is the wave's, not each lane's.
template <bool SLOPE, int NV, int WPT>
__device__ __forceinline__ void sigmoid_weights(const Row<NV, WPT>& x, float m, Row<NV, WPT>& u,
                                                Row<NV, WPT>& slope) {
    if (__int_as_float(__builtin_amdgcn_readfirstlane(__float_as_int(m))) < 0.f) {   // every logit is negative
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const float v = x.v[i][q];
                const float r = __builtin_amdgcn_rcpf(1.f + exp_fast(v));
                u.v[i][q] = exp_fast(v - m) * r;
                if constexpr (SLOPE) slope.v[i][q] = r;
            }
        return;
    }
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const float v = x.v[i][q];
            if constexpr (SLOPE) {
                const float e = exp_fast(-fabsf(v));
                const float r = __builtin_amdgcn_rcpf(1.f + e);
                const float er = e * r;
                u.v[i][q] = v > 0.f ? r : er;
                slope.v[i][q] = v > 0.f ? er : r;
            } else {
                u.v[i][q] = __builtin_amdgcn_rcpf(1.f + exp_fast(-v));
            }
        }
}

// log of the score of one logit (the sigmoid's, or the logit itself).
__device__ __forceinline__ float log_score(float x, int score) {
    if (score == MOE_SCORE_SOFTMAX) return x;
    // log(1 + e) with what 1 + e rounds off
    const float e = exp_fast(-fabsf(x)), y = 1.f + e;
    return fminf(x, 0.f) - __builtin_fmaf(e - (y - 1.f), __builtin_amdgcn_rcpf(y), log_fast(y));
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

// Calls f with the vectors per lane and the waves per row that E experts take.
// ONE_WAVE_MAX: the widest row for one wave, where what a pass keeps per column
// fits its registers.
template <int ONE_WAVE_MAX, typename F>
inline int with_row_shape(int E, F&& f) {
    using std::integral_constant;
    using one = integral_constant<int, 1>;
    if (E <= 256) return f(one(), one());
    if (E <= 512) return f(integral_constant<int, 2>(), one());
    if (E <= 1024) return f(integral_constant<int, 4>(), one());
    if constexpr (ONE_WAVE_MAX >= 2560) {
        if (E <= 1536) return f(integral_constant<int, 6>(), one());
        if (E <= 2560) return f(integral_constant<int, 10>(), one());
    } else {
        if (E <= 2048) return f(integral_constant<int, 2>(), integral_constant<int, 4>());
        if (E <= 2560) return f(integral_constant<int, 2>(), integral_constant<int, 5>());
    }
    return f(integral_constant<int, 4>(), integral_constant<int, 4>());
}

}  // namespace moe
