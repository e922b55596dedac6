// The losses on the router's logits: moe_balance_loss, moe_distill_loss and
// their gradients.
//
// All four are passes over the [T,E] logits with little else to move, so they
// are bound by reading the logits (and, backward, writing their gradient) once
// each. One wave takes a token: its row stays in registers through the
// maximum, the sums and the results (scores.hpp), and no pass reads it twice.
//
// Balance, forward: a block of four waves takes a chunk of tokens and, for
// every sequence that crosses it, sums the probabilities per expert in its
// lanes' registers (each lane owns fixed experts), counts the picks in LDS and
// writes one row of partial sums. Row b + s holds block b's part of sequence
// s: along the tokens either b or s grows, so no two parts share a row and
// nothing needs clearing. A second kernel adds each sequence's rows in block
// order and its last block, by a counter, forms the losses; only integers are
// added atomically, so results do not depend on timing.
#include <cmath>
#include <type_traits>

#include "launch.hpp"
#include "scores.hpp"

namespace moe {
namespace {

constexpr int kBlock = 256;
constexpr int kWaves = kBlock / kWave;
constexpr int kMaxChunk = 64;         // tokens of a block: one ballot holds their validity
constexpr int kTargetBlocks = 1024;   // four blocks a CU

// Tokens a block takes: as few as keep the grid within kTargetBlocks.
inline int chunk_tokens(int T) {
    int c = kWaves;
    while (c < kMaxChunk && ceil_div(T, c) > kTargetBlocks) c *= 2;
    return c;
}

// Bit i: token t0 + i (i < n) is valid.
__device__ __forceinline__ uint64_t valid_tokens(const uint8_t* __restrict__ mask, int t0, int n) {
    const int i = __lane_id();
    return ballot(i < n && mask[t0 + i] != 0);
}

// ------------------------------------------------------------- balance ----

template <int NV, bool SIGMOID>
__global__ __launch_bounds__(kBlock) void balance_partial_kernel(
    const float* __restrict__ logits, const int32_t* __restrict__ ids, const uint8_t* __restrict__ mask,
    const int32_t* __restrict__ seq_offsets, int T, int E, int k, int S, int chunk,
    float* __restrict__ part_probs, int32_t* __restrict__ part_counts, int32_t* __restrict__ part_n,
    float* __restrict__ part_z, int32_t* __restrict__ counter) {
    extern __shared__ float lds[];
    float* sum = lds;                                        // [E]
    int32_t* hist = reinterpret_cast<int32_t*>(lds + E);     // [E]
    __shared__ float zs[kWaves];
    const int lane = __lane_id();
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    if (blockIdx.x == 0 && threadIdx.x == 0) *counter = 0;   // for the kernel that follows
    const int t0 = static_cast<int>(blockIdx.x) * chunk;
    const int t1 = min(T, t0 + chunk);
    const uint64_t valid = valid_tokens(mask, t0, t1 - t0);

    int a = t0;
    while (a < t1) {
        int begin = 0, end = 0;
        const int s = find_sequence(seq_offsets, S, T, a, begin, end);
        if (s < 0) {
            // before the first sequence, or behind the last
            const int first = seq_offset(seq_offsets, 0, T);
            if (a >= first) break;
            a = first;
            continue;
        }
        const int b = min(end, t1);
        for (int c = threadIdx.x; c < E; c += kBlock) hist[c] = 0;
        __syncthreads();
        for (int f = (a - t0) * k + static_cast<int>(threadIdx.x); f < (b - t0) * k; f += kBlock) {
            if (valid >> (f / k) & 1) {
                const int id = ids[static_cast<size_t>(t0) * k + f];
                if (id >= 0 && id < E) atomicAdd(&hist[id], 1);
            }
        }
        float acc[NV][4];
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int q = 0; q < 4; ++q) acc[i][q] = 0.f;
        float z = 0.f;
        for (int t = a + wave; t < b; t += kWaves) {
            if (!(valid >> (t - t0) & 1)) continue;
            float x[NV][4], u[NV][4];
            load_row(logits + static_cast<size_t>(t) * E, E, lane, x);
            float m = softmax_weights(x, u);
            float total = row_sum(u);
            const float lse = m + logf(total);
            z += lse * lse;
            if constexpr (SIGMOID) {
                float none[1][4];
                sigmoid_weights<NV, false>(x, u, none);
                total = row_sum(u);
            }
            const float inv = total > 0.f ? 1.f / total : total == 0.f ? 0.f : total;
#pragma unroll
            for (int i = 0; i < NV; ++i)
#pragma unroll
                for (int q = 0; q < 4; ++q) acc[i][q] = __builtin_fmaf(u[i][q], inv, acc[i][q]);
        }
        if (lane == 0) zs[wave] = z;
        // the four waves' sums, in wave order
        for (int w = 0; w < kWaves; ++w) {
            if (wave == w) {
#pragma unroll
                for (int i = 0; i < NV; ++i)
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const int c = i * 256 + lane * 4 + q;
                        if (c < E) sum[c] = w == 0 ? acc[i][q] : sum[c] + acc[i][q];
                    }
            }
            __syncthreads();
        }
        const size_t row = static_cast<size_t>(blockIdx.x) + s;
        for (int c = threadIdx.x; c < E; c += kBlock) {
            part_probs[row * E + c] = sum[c];
            part_counts[row * E + c] = hist[c];
        }
        if (threadIdx.x == 0) {
            const uint64_t lo = valid >> (a - t0);
            part_n[row] = __popcll(b - a < 64 ? lo & ((1ull << (b - a)) - 1) : lo);
            float zt = zs[0];
            for (int w = 1; w < kWaves; ++w) zt += zs[w];
            part_z[row] = zt;
        }
        __syncthreads();
        a = b;
    }
}

constexpr int kReduceBlock = 1024;
constexpr int kReduceCols = 64;
constexpr int kReduceGroups = kReduceBlock / kReduceCols;

__device__ __forceinline__ float agent_load(const float* p) {
    return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ int32_t agent_load(const int32_t* p) {
    return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// Block sum of N doubles per thread, in a fixed order; thread 0 gets it.
template <int N>
__device__ __forceinline__ void block_sum(double (&v)[N], double* red) {
#pragma unroll
    for (int i = 0; i < N; ++i)
        for (int off = 32; off >= 1; off >>= 1) v[i] += __shfl_xor(v[i], off, kWave);
    const int wave = threadIdx.x / kWave, waves = blockDim.x / kWave;
    if (__lane_id() == 0)
#pragma unroll
        for (int i = 0; i < N; ++i) red[wave * N + i] = v[i];
    __syncthreads();
    if (threadIdx.x == 0)
#pragma unroll
        for (int i = 0; i < N; ++i) {
            v[i] = red[i];
            for (int w = 1; w < waves; ++w) v[i] += red[w * N + i];
        }
    __syncthreads();
}

// Block s * col_blocks + c: columns [64 c, 64 c + 64) of sequence s, sixteen
// groups of threads over its partial rows.
__global__ __launch_bounds__(kReduceBlock) void balance_reduce_kernel(
    const float* __restrict__ part_probs, const int32_t* __restrict__ part_counts,
    const int32_t* __restrict__ part_n, const float* __restrict__ part_z,
    const int32_t* __restrict__ seq_offsets, int T, int E, int k, int S, int chunk, int col_blocks,
    float* __restrict__ losses, int32_t* __restrict__ counts, float* __restrict__ probs,
    int32_t* __restrict__ tokens, float* __restrict__ seq_dot, float* __restrict__ seq_z,
    int32_t* __restrict__ counter) {
    __shared__ float sp[kReduceGroups][kReduceCols];
    __shared__ int32_t sc[kReduceGroups][kReduceCols];
    __shared__ double red[(kReduceBlock / kWave) * 4];
    __shared__ int last;
    const int s = blockIdx.x / col_blocks;
    const int cb = blockIdx.x - s * col_blocks;
    const int col = threadIdx.x % kReduceCols, group = threadIdx.x / kReduceCols;
    const int c = cb * kReduceCols + col;
    const int a = seq_offset(seq_offsets, s, T), b = seq_offset(seq_offsets, s + 1, T);
    const int b0 = a / chunk, b1 = a < b ? (b - 1) / chunk + 1 : b0;
    float p = 0.f;
    int32_t n = 0;
    if (c < E) {
#pragma unroll 4
        for (int r = b0 + group; r < b1; r += kReduceGroups) {
            const size_t at = (static_cast<size_t>(r) + s) * E + c;
            p += part_probs[at];
            n += part_counts[at];
        }
    }
    sp[group][col] = p;
    sc[group][col] = n;
    __syncthreads();
    if (group == 0) {
        for (int g = 1; g < kReduceGroups; ++g) {
            p += sp[g][col];
            n += sc[g][col];
        }
        if (c < E) {
            probs[static_cast<size_t>(s) * E + c] = p;
            counts[static_cast<size_t>(s) * E + c] = n;
        }
        const float dot = wave_sum(p * static_cast<float>(n));   // the 64 columns are one wave
        if (col == 0) seq_dot[static_cast<size_t>(s) * col_blocks + cb] = dot;
    } else if (group == 1 && cb == 0) {
        int32_t m = 0;
        float z = 0.f;
        for (int r = b0 + col; r < b1; r += kReduceCols) {
            m += part_n[r + s];
            z += part_z[r + s];
        }
        z = wave_sum(z);
        for (int off = 32; off >= 1; off >>= 1) m += __shfl_xor(m, off, kWave);
        if (col == 0) {
            tokens[s] = m;
            seq_z[s] = z;
        }
    }
    // the last block to get here has every sequence's sums before it
    __threadfence();
    __syncthreads();
    if (threadIdx.x == 0) last = atomicAdd(counter, 1) == S * col_blocks - 1;
    __syncthreads();
    if (!last) return;
    __threadfence();
    double v[4] = {0, 0, 0, 0};   // balance, z, tokens, sequences with a token
    for (int q = threadIdx.x; q < S; q += kReduceBlock) {
        const int32_t m = agent_load(&tokens[q]);
        if (m == 0) continue;
        double dot = 0;
        for (int i = 0; i < col_blocks; ++i) dot += agent_load(&seq_dot[static_cast<size_t>(q) * col_blocks + i]);
        v[0] += dot * E / (static_cast<double>(k) * m * m);
        v[1] += agent_load(&seq_z[q]);
        v[2] += m;
        v[3] += 1;
    }
    block_sum(v, red);
    if (threadIdx.x == 0) {
        losses[0] = v[3] > 0 ? static_cast<float>(v[0] / v[3]) : 0.f;
        losses[1] = v[2] > 0 ? static_cast<float>(v[1] / v[2]) : 0.f;
        tokens[S] = static_cast<int32_t>(v[2]);
        tokens[S + 1] = static_cast<int32_t>(v[3]);
    }
}

// Each wave takes the chunk's tokens in turn; the coefficients c_e of the
// current sequence stay in its registers.
template <int NV, bool SIGMOID>
__global__ __launch_bounds__(kBlock) void balance_backward_kernel(
    const float* __restrict__ d_losses, const float* __restrict__ logits, const uint8_t* __restrict__ mask,
    const int32_t* __restrict__ seq_offsets, const int32_t* __restrict__ counts,
    const int32_t* __restrict__ tokens, int T, int E, int k, int S, int chunk, int accumulate,
    float* __restrict__ d_logits) {
    const int lane = __lane_id();
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int t0 = static_cast<int>(blockIdx.x) * chunk;
    const int t1 = min(T, t0 + chunk);
    const uint64_t valid = valid_tokens(mask, t0, t1 - t0);
    const float n = static_cast<float>(max(tokens[S], 1));
    const float full = static_cast<float>(max(tokens[S + 1], 1));
    const float zg = 2.f * d_losses[1] / n;
    int s = -1, begin = 0, end = 0;
    float cf[NV][4] = {};
    for (int t = t0 + wave; t < t1; t += kWaves) {
        bool ok = valid >> (t - t0) & 1;
        if (ok && !(s >= 0 && t < end)) {
            s = find_sequence(seq_offsets, S, T, t, begin, end);
            if (s >= 0) {
                const float m = static_cast<float>(max(tokens[s], 1));
                const float w = d_losses[0] * static_cast<float>(E) / (static_cast<float>(k) * m * m * full);
#pragma unroll
                for (int i = 0; i < NV; ++i)
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const int c = i * 256 + lane * 4 + q;
                        cf[i][q] = c < E ? w * static_cast<float>(counts[static_cast<size_t>(s) * E + c]) : 0.f;
                    }
            }
        }
        ok = ok && s >= 0;
        float* out = d_logits + static_cast<size_t>(t) * E;
        float d[NV][4];
        if (!ok) {
            if (accumulate) continue;
#pragma unroll
            for (int i = 0; i < NV; ++i)
#pragma unroll
                for (int q = 0; q < 4; ++q) d[i][q] = 0.f;
            store_row(out, E, lane, d, false);
            continue;
        }
        float x[NV][4], u[NV][4];
        load_row(logits + static_cast<size_t>(t) * E, E, lane, x);
        // the z loss' part: (2 / n) lse softmax
        const float m = softmax_weights(x, u);
        float total = row_sum(u);
        const float inv = total > 0.f ? 1.f / total : total == 0.f ? 0.f : total;
        const float zc = zg == 0.f ? 0.f : zg * (m + logf(total)) * inv;
        if constexpr (SIGMOID) {
#pragma unroll
            for (int i = 0; i < NV; ++i)
#pragma unroll
                for (int q = 0; q < 4; ++q) d[i][q] = zc * u[i][q];
            float slope[NV][4];
            sigmoid_weights<NV, true>(x, u, slope);
            total = row_sum(u);
            const float pinv = total > 0.f ? 1.f / total : total == 0.f ? 0.f : total;
            float dot = 0.f;
#pragma unroll
            for (int i = 0; i < NV; ++i)
#pragma unroll
                for (int q = 0; q < 4; ++q) dot = __builtin_fmaf(u[i][q], cf[i][q], dot);
            dot = wave_sum(dot) * pinv;
#pragma unroll
            for (int i = 0; i < NV; ++i)
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    d[i][q] = __builtin_fmaf(u[i][q] * pinv * slope[i][q], cf[i][q] - dot, d[i][q]);
        } else {
            float dot = 0.f;
#pragma unroll
            for (int i = 0; i < NV; ++i)
#pragma unroll
                for (int q = 0; q < 4; ++q) dot = __builtin_fmaf(u[i][q], cf[i][q], dot);
            dot = wave_sum(dot) * inv;
#pragma unroll
            for (int i = 0; i < NV; ++i)
#pragma unroll
                for (int q = 0; q < 4; ++q) d[i][q] = u[i][q] * __builtin_fmaf(cf[i][q] - dot, inv, zc);
        }
        store_row(out, E, lane, d, accumulate);
    }
}

struct BalancePlan {
    int chunk, blocks, col_blocks;
    size_t rows, probs, counts, n, z, dot, seq_z, counter, bytes;   // byte offsets
};

inline size_t round256(size_t b) { return (b + 255) / 256 * 256; }

inline bool balance_shape_ok(int T, int E, int S) {
    return T >= 0 && T <= MOE_MAX_TOKENS && E >= 1 && E <= MOE_MAX_EXPERTS && S >= 1 && S <= MOE_MAX_SEQUENCES;
}

inline BalancePlan plan_balance(int T, int E, int S) {
    BalancePlan p;
    p.chunk = chunk_tokens(T);
    p.blocks = ceil_div(T, p.chunk);
    p.col_blocks = ceil_div(E, kReduceCols);
    p.rows = static_cast<size_t>(p.blocks) + S;
    size_t at = 0;
    auto take = [&](size_t n) {
        const size_t here = at;
        at += round256(n);
        return here;
    };
    p.probs = take(p.rows * E * sizeof(float));
    p.counts = take(p.rows * E * sizeof(int32_t));
    p.n = take(p.rows * sizeof(int32_t));
    p.z = take(p.rows * sizeof(float));
    p.dot = take(static_cast<size_t>(S) * p.col_blocks * sizeof(float));
    p.seq_z = take(static_cast<size_t>(S) * sizeof(float));
    p.counter = take(sizeof(int32_t));
    p.bytes = at;
    return p;
}

// ------------------------------------------------------------- distill ----

// Lane j < K: teacher entry j of token t, its share q of the entries' sum and
// log q; id -1 where there is none. Returns whether the token has an entry.
__device__ __forceinline__ bool teacher_shares(const int32_t* __restrict__ ids, const float* __restrict__ logits,
                                               size_t t, int K, int E, int score, float inv_temp, int& id,
                                               float& q, float& logq) {
    const int lane = __lane_id();
    id = -1;
    float z = kNegInf;
    if (lane < K) {
        id = ids[t * K + lane];
        z = logits[t * K + lane];
        if (id < 0 || id >= E || z == kNegInf) id = -1;
        z = id < 0 ? kNegInf : log_score(z * inv_temp, score);
    }
    if (ballot(id >= 0) == 0) return false;
    const float m = wave_max(z);
    const float e = id < 0 ? 0.f : expf(z - m);
    const float total = wave_sum(e);
    logq = id < 0 ? 0.f : (z - m) - logf(total);
    q = e / total;
    return true;
}

template <int NV>
__device__ __forceinline__ void scale_row(float (&x)[NV][4], float f) {
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int q = 0; q < 4; ++q) x[i][q] *= f;
}

template <int NV, bool SIGMOID>
__global__ __launch_bounds__(kBlock) void distill_kernel(
    const float* __restrict__ logits, const int32_t* __restrict__ t_ids, const float* __restrict__ t_logits,
    const uint8_t* __restrict__ mask, float inv_temp, float temp2, int T, int E, int K, int chunk,
    float* __restrict__ token_loss, float* __restrict__ part_loss, int32_t* __restrict__ part_n) {
    __shared__ float sl[kWaves];
    __shared__ int32_t sn[kWaves];
    constexpr int score = SIGMOID ? MOE_SCORE_SIGMOID : MOE_SCORE_SOFTMAX;
    const int lane = __lane_id();
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int t0 = static_cast<int>(blockIdx.x) * chunk;
    const int t1 = min(T, t0 + chunk);
    const uint64_t valid = valid_tokens(mask, t0, t1 - t0);
    float sum = 0.f;
    int32_t n = 0;
    for (int t = t0 + wave; t < t1; t += kWaves) {
        int id = -1;
        float q = 0.f, logq = 0.f, loss = 0.f;
        if ((valid >> (t - t0) & 1) &&
            teacher_shares(t_ids, t_logits, t, K, E, score, inv_temp, id, q, logq)) {
            const float* row = logits + static_cast<size_t>(t) * E;
            float x[NV][4], u[NV][4];
            load_row(row, E, lane, x);
            const float xp = id >= 0 ? row[id] * inv_temp : 0.f;
            scale_row(x, inv_temp);
            float m;
            if constexpr (SIGMOID) {
                float none[1][4];
                m = sigmoid_weights<NV, false>(x, u, none);
            } else {
                m = softmax_weights(x, u);
            }
            const float lse = m + logf(row_sum(u));
            const float term = id >= 0 && q > 0.f ? q * (logq - (log_score(xp, score) - lse)) : 0.f;
            loss = temp2 * wave_sum(term);
            sum += loss;
            ++n;
        }
        if (lane == 0) token_loss[t] = loss;
    }
    if (lane == 0) {
        sl[wave] = sum;
        sn[wave] = n;
    }
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int w = 1; w < kWaves; ++w) {
            sum += sl[w];
            n += sn[w];
        }
        part_loss[blockIdx.x] = sum;
        part_n[blockIdx.x] = n;
    }
}

__global__ __launch_bounds__(kBlock) void distill_reduce_kernel(const float* __restrict__ part_loss,
                                                                const int32_t* __restrict__ part_n, int blocks,
                                                                float* __restrict__ loss,
                                                                int32_t* __restrict__ tokens) {
    __shared__ double red[kWaves * 2];
    double v[2] = {0, 0};
    for (int b = threadIdx.x; b < blocks; b += kBlock) {
        v[0] += part_loss[b];
        v[1] += part_n[b];
    }
    block_sum(v, red);
    if (threadIdx.x == 0) {
        loss[0] = v[1] > 0 ? static_cast<float>(v[0] / v[1]) : 0.f;
        tokens[0] = static_cast<int32_t>(v[1]);
    }
}

// The teacher's shares reach the lanes that own their experts through a row of
// LDS per wave: zeros but for the entries, which are cleared again behind each
// token. LDS operations of one wave run in order, so no barrier is needed.
template <int NV, bool SIGMOID>
__global__ __launch_bounds__(kBlock) void distill_backward_kernel(
    const float* __restrict__ d_loss, const float* __restrict__ logits, const int32_t* __restrict__ t_ids,
    const float* __restrict__ t_logits, const uint8_t* __restrict__ mask, const int32_t* __restrict__ tokens,
    float inv_temp, float temp, int T, int E, int K, int chunk, int accumulate, float* __restrict__ d_logits) {
    extern __shared__ float lds[];
    constexpr int score = SIGMOID ? MOE_SCORE_SIGMOID : MOE_SCORE_SOFTMAX;
    const int lane = __lane_id();
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    float* share = lds + wave * (NV * 256);
#pragma unroll
    for (int i = 0; i < NV; ++i) *reinterpret_cast<f32x4*>(share + i * 256 + lane * 4) = f32x4{0.f, 0.f, 0.f, 0.f};
    const int t0 = static_cast<int>(blockIdx.x) * chunk;
    const int t1 = min(T, t0 + chunk);
    const uint64_t valid = valid_tokens(mask, t0, t1 - t0);
    const float g = d_loss[0] * temp / static_cast<float>(max(tokens[0], 1));
    for (int t = t0 + wave; t < t1; t += kWaves) {
        float* out = d_logits + static_cast<size_t>(t) * E;
        int id = -1;
        float q = 0.f, logq = 0.f;
        float d[NV][4];
        if (!((valid >> (t - t0) & 1) &&
              teacher_shares(t_ids, t_logits, t, K, E, score, inv_temp, id, q, logq))) {
            if (accumulate) continue;
#pragma unroll
            for (int i = 0; i < NV; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) d[i][j] = 0.f;
            store_row(out, E, lane, d, false);
            continue;
        }
        float x[NV][4], u[NV][4];
        load_row(logits + static_cast<size_t>(t) * E, E, lane, x);
        // an expert named twice: every entry that names it holds the sum
        float same = 0.f;
        for (int j = 0; j < K; ++j) {
            const int other = __builtin_amdgcn_readlane(id, j);
            const float oq = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(q), j));
            if (other == id) same += oq;
        }
        if (id >= 0) share[id] = same;
        scale_row(x, inv_temp);
        float slope[SIGMOID ? NV : 1][4];
        if constexpr (SIGMOID) sigmoid_weights<NV, true>(x, u, slope);
        else softmax_weights(x, u);
        const float total = row_sum(u);
        const float inv = total > 0.f ? 1.f / total : total == 0.f ? 0.f : total;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const f32x4 sq = *reinterpret_cast<const f32x4*>(share + i * 256 + lane * 4);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                d[i][j] = g * __builtin_fmaf(u[i][j], inv, -sq[j]);
                if constexpr (SIGMOID) d[i][j] *= slope[i][j];
            }
        }
        if (id >= 0) share[id] = 0.f;
        store_row(out, E, lane, d, accumulate);
    }
}

inline bool score_ok(int score) { return score == MOE_SCORE_SIGMOID || score == MOE_SCORE_SOFTMAX; }

}  // namespace
}  // namespace moe

extern "C" size_t moe_balance_loss_workspace_bytes(int T, int E, int S) {
    using namespace moe;
    return balance_shape_ok(T, E, S) ? plan_balance(T, E, S).bytes : 0;
}

extern "C" int moe_balance_loss(const float* logits, const int32_t* topk_ids, const uint8_t* token_mask,
                                const int32_t* seq_offsets, int score, int T, int E, int k, int S, float* losses,
                                int32_t* counts, float* probs, int32_t* tokens, void* workspace,
                                size_t workspace_bytes, void* stream) {
    using namespace moe;
    if (!balance_shape_ok(T, E, S) || k < 1 || k > MOE_MAX_TOPK || k > E) return MOE_ERR_BAD_SHAPE;
    if (static_cast<long long>(T) * k >= (1ll << 31)) return MOE_ERR_BAD_SHAPE;   // counts are int32
    if (!seq_offsets && S != 1) return MOE_ERR_NULL_ARG;
    if (!score_ok(score)) return MOE_ERR_BAD_ARG;
    if (!losses || !counts || !probs || !tokens) return MOE_ERR_NULL_ARG;
    if (T > 0 && (!logits || !topk_ids || !token_mask)) return MOE_ERR_NULL_ARG;
    if (!all_aligned16(logits, topk_ids, token_mask, seq_offsets, losses, counts, probs, tokens)) return MOE_ERR_ALIGN;
    const BalancePlan p = plan_balance(T, E, S);
    if (!workspace || workspace_bytes < p.bytes || !aligned16(workspace)) return MOE_ERR_WORKSPACE;
    char* ws = static_cast<char*>(workspace);
    auto* part_probs = reinterpret_cast<float*>(ws + p.probs);
    auto* part_counts = reinterpret_cast<int32_t*>(ws + p.counts);
    auto* part_n = reinterpret_cast<int32_t*>(ws + p.n);
    auto* part_z = reinterpret_cast<float*>(ws + p.z);
    auto* counter = reinterpret_cast<int32_t*>(ws + p.counter);
    int st = with_row_vectors(E, [&](auto nv) {
        constexpr int NV = decltype(nv)::value;
        auto kern = score == MOE_SCORE_SIGMOID ? balance_partial_kernel<NV, true> : balance_partial_kernel<NV, false>;
        return launch(kern, dim3(p.blocks > 0 ? p.blocks : 1), dim3(kBlock), 2 * sizeof(float) * E, stream, logits,
                      topk_ids, token_mask, seq_offsets, T, E, k, S, p.chunk, part_probs, part_counts, part_n,
                      part_z, counter);
    });
    if (st != MOE_OK) return st;
    return launch(balance_reduce_kernel, dim3(S * p.col_blocks), dim3(kReduceBlock), 0, stream, part_probs,
                  part_counts, part_n, part_z, seq_offsets, T, E, k, S, p.chunk, p.col_blocks, losses, counts, probs,
                  tokens, reinterpret_cast<float*>(ws + p.dot), reinterpret_cast<float*>(ws + p.seq_z), counter);
}

extern "C" int moe_balance_loss_backward(const float* d_losses, const float* logits, const uint8_t* token_mask,
                                         const int32_t* seq_offsets, const int32_t* counts, const int32_t* tokens,
                                         int score, int T, int E, int k, int S, int accumulate, float* d_logits,
                                         void* stream) {
    using namespace moe;
    if (!balance_shape_ok(T, E, S) || k < 1 || k > MOE_MAX_TOPK || k > E) return MOE_ERR_BAD_SHAPE;
    if (!seq_offsets && S != 1) return MOE_ERR_NULL_ARG;
    if (!score_ok(score)) return MOE_ERR_BAD_ARG;
    if (T == 0) return MOE_OK;
    if (!d_losses || !logits || !token_mask || !counts || !tokens || !d_logits) return MOE_ERR_NULL_ARG;
    if (!all_aligned16(d_losses, logits, token_mask, seq_offsets, counts, tokens, d_logits)) return MOE_ERR_ALIGN;
    const int chunk = chunk_tokens(T);
    return with_row_vectors(E, [&](auto nv) {
        constexpr int NV = decltype(nv)::value;
        auto kern = score == MOE_SCORE_SIGMOID ? balance_backward_kernel<NV, true> : balance_backward_kernel<NV, false>;
        return launch(kern, dim3(ceil_div(T, chunk)), dim3(kBlock), 0, stream, d_losses, logits, token_mask,
                      seq_offsets, counts, tokens, T, E, k, S, chunk, accumulate, d_logits);
    });
}

namespace moe {
namespace {

inline bool distill_shape_ok(int T, int E) {
    return T >= 0 && T <= MOE_MAX_TOKENS && E >= 1 && E <= MOE_MAX_EXPERTS;
}

}  // namespace
}  // namespace moe

extern "C" size_t moe_distill_loss_workspace_bytes(int T, int E) {
    using namespace moe;
    if (!distill_shape_ok(T, E)) return 0;
    const int blocks = ceil_div(T, chunk_tokens(T));
    return 2 * round256(sizeof(float) * (blocks > 0 ? blocks : 1));
}

extern "C" int moe_distill_loss(const float* logits, const int32_t* teacher_ids, const float* teacher_logits,
                                const uint8_t* token_mask, int score, float temperature, int T, int E, int K,
                                float* loss, float* token_loss, int32_t* tokens, void* workspace,
                                size_t workspace_bytes, void* stream) {
    using namespace moe;
    if (!distill_shape_ok(T, E) || K < 1 || K > MOE_MAX_TOPK) return MOE_ERR_BAD_SHAPE;
    if (!score_ok(score) || !std::isfinite(temperature) || !(temperature > 0.f)) return MOE_ERR_BAD_ARG;
    if (!loss || !tokens) return MOE_ERR_NULL_ARG;
    if (T > 0 && (!logits || !teacher_ids || !teacher_logits || !token_mask || !token_loss)) return MOE_ERR_NULL_ARG;
    if (!all_aligned16(logits, teacher_ids, teacher_logits, token_mask, loss, token_loss, tokens))
        return MOE_ERR_ALIGN;
    if (!workspace || workspace_bytes < moe_distill_loss_workspace_bytes(T, E) || !aligned16(workspace))
        return MOE_ERR_WORKSPACE;
    const int chunk = chunk_tokens(T);
    const int blocks = ceil_div(T, chunk);
    auto* part_loss = static_cast<float*>(workspace);
    auto* part_n = reinterpret_cast<int32_t*>(static_cast<char*>(workspace) + round256(sizeof(float) * (blocks > 0 ? blocks : 1)));
    if (T > 0) {
        const int st = with_row_vectors(E, [&](auto nv) {
            constexpr int NV = decltype(nv)::value;
            auto kern = score == MOE_SCORE_SIGMOID ? distill_kernel<NV, true> : distill_kernel<NV, false>;
            return launch(kern, dim3(blocks), dim3(kBlock), 0, stream, logits, teacher_ids, teacher_logits,
                          token_mask, 1.f / temperature, temperature * temperature, T, E, K, chunk, token_loss,
                          part_loss, part_n);
        });
        if (st != MOE_OK) return st;
    }
    return launch(distill_reduce_kernel, dim3(1), dim3(kBlock), 0, stream, part_loss, part_n, blocks, loss, tokens);
}

extern "C" int moe_distill_loss_backward(const float* d_loss, const float* logits, const int32_t* teacher_ids,
                                         const float* teacher_logits, const uint8_t* token_mask,
                                         const int32_t* tokens, int score, float temperature, int T, int E, int K,
                                         int accumulate, float* d_logits, void* stream) {
    using namespace moe;
    if (!distill_shape_ok(T, E) || K < 1 || K > MOE_MAX_TOPK) return MOE_ERR_BAD_SHAPE;
    if (!score_ok(score) || !std::isfinite(temperature) || !(temperature > 0.f)) return MOE_ERR_BAD_ARG;
    if (T == 0) return MOE_OK;
    if (!d_loss || !logits || !teacher_ids || !teacher_logits || !token_mask || !tokens || !d_logits)
        return MOE_ERR_NULL_ARG;
    if (!all_aligned16(d_loss, logits, teacher_ids, teacher_logits, token_mask, tokens, d_logits))
        return MOE_ERR_ALIGN;
    const int chunk = chunk_tokens(T);
    return with_row_vectors(E, [&](auto nv) {
        constexpr int NV = decltype(nv)::value;
        auto kern = score == MOE_SCORE_SIGMOID ? distill_backward_kernel<NV, true> : distill_backward_kernel<NV, false>;
        return launch(kern, dim3(ceil_div(T, chunk)), dim3(kBlock), sizeof(float) * kWaves * NV * 256, stream, d_loss,
                      logits, teacher_ids, teacher_logits, token_mask, tokens, 1.f / temperature, temperature, T, E,
                      K, chunk, accumulate, d_logits);
    });
}
