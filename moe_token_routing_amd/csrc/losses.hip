// The losses on the router's logits: moe_balance_loss, moe_distill_loss and
// their gradients.
//
// All four are passes over the [T,E] logits with little else to move, so they
// are bound by reading the logits (and, backward, writing their gradient) once
// each, and in small batches by the chain of dependent steps. A token's row
// stays in the registers of one wave (of a block's waves for wide rows,
// scores.hpp) through the maximum, the sums and the results; a wave's first row
// and picks are loaded before it knows whether its token is valid, so that
// these loads and the mask's are one wait.
//
// Balance, forward: a block takes a chunk of tokens and, for every sequence
// that crosses it, sums the probabilities per expert in its lanes' registers
// (each lane owns fixed experts), counts the picks in LDS and writes one row of
// partial sums. Row b + s holds block b's part of sequence s: along the tokens
// either b or s grows, so no two parts share a row and nothing needs clearing.
// A second kernel adds each sequence's rows in block order and its last block,
// by a counter, forms the losses; only integers are added atomically, so
// results do not depend on timing. A batch of up to kSmallTokens tokens takes
// one block of sixteen waves instead, which needs no second kernel and no
// workspace: at such sizes a launch costs more than the work.
//
// Measured (forward, its addition, backward): 8111 tokens of 254 experts in 13
// sequences 8.3, 7.2 and 8.8 us, a chain of dependent steps each (16 MB are 3 us at
// a copy's 5.1 TB/s); 32768 of 512 14.7 (4.6 TB/s), 8.8 and 23.5 us (5.7 TB/s);
// 16 tokens of 16 4.3 and 3.7 us. Distillation: 4093 tokens of 2560 11.1 (3.8
// TB/s), 3.1 and 16.5 us (5.1 TB/s); 8192 of 256 5.8, 2.2 and 7.5 us; one token of
// 64 2.5 and 2.4 us. The choices below were measured before the sigmoid and the
// logarithms took their present forms, which shortens both sides alike.
#include "launch.hpp"
#include "scores.hpp"

namespace moe {
namespace {

constexpr int kMaxChunk = 64;         // tokens of a block: one ballot holds their validity
constexpr int kGroups = 4;            // tokens of a block at a time where a wave takes a row
// Four such blocks a CU: with 512 / 1024 / 2048 of them, 32768 tokens of 512 experts
// took 15.9, 14.7 and 16.0 us, their parts' addition 9.4, 11.2 and 15.8, the
// gradient 24.5, 23.7 and 23.8.
constexpr int kTargetBlocks = 1024;
// Up to these a block takes one token of the balance loss: 500 tokens in 60
// sequences 4.3 us, by four tokens, with their sequences in turn, 6.5; in one
// sequence 4.3 and 4.2.
constexpr int kFewTokens = 512;
// By one block, if their rows take one wave, with up to kSmallSequences sequences in
// turn: one launch saves 3.5 us of an eager call, and its kernel takes no longer
// than the two others up to here (balance, 32 tokens of 64 experts 6.1 us against
// 4.1 + 5.5, of 1024 10.3 against 5.7 + 6.1, of 256 in four sequences 10.7 against
// 4.2 + 5.9; distillation of 16 4.9 against 4.1 + 2.1, of 32 8.2 against 4.4 + 1.8);
// 64 tokens of 1024 took 16.8 against 12.3, their distillation 21.2 against 6.9.
constexpr int kSmallGroups = 16;
constexpr int kSmallTokens = 32;
constexpr int kSmallExperts = 1024;
constexpr int kSmallSequences = 4;
// Widest rows that one wave takes; several waves need fewer registers each, but a
// barrier a sum. Balance, forward and gradient, one wave / several: 4096 tokens of
// 1500 experts 13.6 + 22.1 / 15.9 + 19.6 us, of 2560 21.2 + 46.3 / 19.9 + 27.9.
// Distillation keeps fewer arrays: of 1500 11.2 + 12.9 / 18.8 + 19.2, of 2560 15.3 +
// 20.8 / 25.4 + 27.3.
constexpr int kBalanceOneWave = 1024, kDistillOneWave = 2560;

inline bool small_batch(int T, int E) { return T <= kSmallTokens && E <= kSmallExperts; }

// Tokens a block takes: as few as keep the grid within `blocks`.
inline int chunk_tokens(int T, bool one_wave, int blocks) {
    int c = one_wave ? kGroups : 1;
    while (c < kMaxChunk && ceil_div(T, c) > blocks) c *= 2;
    return c;
}

// Bit i: token t0 + i (i < n) is valid.
__device__ __forceinline__ uint64_t valid_tokens(const uint8_t* __restrict__ mask, int t0, int n) {
    const int i = __lane_id();
    return ballot(i < n && mask[t0 + i] != 0);
}

// Bits [a, b) of a chunk's 64.
__device__ __forceinline__ uint64_t bit_range(int a, int b) {
    const uint64_t below_b = b >= 64 ? ~0ull : (1ull << b) - 1;
    return below_b & ~((1ull << a) - 1);
}

// The place of a wave in a block that takes GROUPS tokens at a time with WPT
// waves each (one of the two is 1): its token group and its part of the row.
template <int WPT, int GROUPS>
struct Place {
    static_assert(WPT == 1 || GROUPS == 1, "a token per wave, or the block's");
    static constexpr int WAVES = WPT * GROUPS;
    static constexpr int BLOCK = WAVES * kWave;
    int lane, wave, group, part;
    __device__ __forceinline__ Place() {
        lane = __lane_id();
        wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
        group = WPT == 1 ? wave : 0;
        part = WPT == 1 ? 0 : wave;
    }
    // the bits of the chunk's tokens that fall to this wave's group
    __device__ __forceinline__ uint64_t share() const {
        return GROUPS == 1 ? ~0ull : (GROUPS == 4 ? 0x1111111111111111ull : 0x0001000100010001ull) << group;
    }
};

// Calls body(t, row) for the tokens whose bits are set, in order, t relative to
// the chunk. x holds row `have` already; the next token's row is loaded while
// the current one is worked on, if two of them fit the registers.
template <int NV, int WPT, typename F>
__device__ __forceinline__ void for_rows(uint64_t bits, const float* __restrict__ logits, int E, int part, int lane,
                                         Row<NV, WPT>& x, int have, F&& body) {
    while (bits) {
        const int t = __builtin_ctzll(bits);
        bits &= bits - 1;
        if (t != have) x.load(logits + static_cast<size_t>(t) * E, E, part, lane);
        have = -1;
        if constexpr (NV <= 4) {
            Row<NV, WPT> row = x;
            if (bits) {
                have = __builtin_ctzll(bits);
                x.load(logits + static_cast<size_t>(have) * E, E, part, lane);
            }
            body(t, row);
        } else {
            body(t, x);
        }
    }
}

// 1 / total, or 0 for a row whose every weight is zero.
__device__ __forceinline__ float inverse(float total) { return total == 0.f ? 0.f : 1.f / total; }

// Sum of a double over the wave by register exchanges alone: within fours, the
// mirrored halves of eights and sixteens, then rows of 16 and 32 lanes (64-bit
// shuffles go through LDS, two a step).
template <int CTRL>
__device__ __forceinline__ double dpp_f64(double v) {
    const uint64_t b = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = __builtin_amdgcn_update_dpp(0, static_cast<int>(b), CTRL, 0xF, 0xF, false);
    const uint32_t hi = __builtin_amdgcn_update_dpp(0, static_cast<int>(b >> 32), CTRL, 0xF, 0xF, false);
    return __builtin_bit_cast(double, static_cast<uint64_t>(hi) << 32 | lo);
}
__device__ __forceinline__ double wave_sum_f64(double v) {
    v += dpp_f64<0xB1>(v);    // quad_perm [1,0,3,2]
    v += dpp_f64<0x4E>(v);    // quad_perm [2,3,0,1]
    v += dpp_f64<0x141>(v);   // row_half_mirror
    v += dpp_f64<0x140>(v);   // row_mirror
    auto halves = [](const auto& lo, const auto& hi) {
        return __builtin_bit_cast(double, static_cast<uint64_t>(hi[0]) << 32 | lo[0]) +
               __builtin_bit_cast(double, static_cast<uint64_t>(hi[1]) << 32 | lo[1]);
    };
    uint64_t b = __builtin_bit_cast(uint64_t, v);
    uint32_t lo = static_cast<uint32_t>(b), hi = static_cast<uint32_t>(b >> 32);
    v = halves(__builtin_amdgcn_permlane16_swap(lo, lo, false, false), __builtin_amdgcn_permlane16_swap(hi, hi, false, false));
    b = __builtin_bit_cast(uint64_t, v);
    lo = static_cast<uint32_t>(b);
    hi = static_cast<uint32_t>(b >> 32);
    return halves(__builtin_amdgcn_permlane32_swap(lo, lo, false, false), __builtin_amdgcn_permlane32_swap(hi, hi, false, false));
}

// Block sum of N doubles per thread, in a fixed order; the first wave gets it.
// The waves' sums meet in one wave's lanes: added up by a thread in turn they
// took 3 us of the sixteen waves' reductions.
template <int N, int BLOCK>
__device__ __forceinline__ void block_sum(double (&v)[N], double* red) {
    constexpr int WAVES = BLOCK / kWave;
    static_assert(WAVES * N <= kWave && (WAVES & (WAVES - 1)) == 0 && (N & (N - 1)) == 0, "one wave's lanes");
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = wave_sum_f64(v[i]);
    const int wave = threadIdx.x / kWave;
    if (__lane_id() == 0)
#pragma unroll
        for (int i = 0; i < N; ++i) red[wave * N + i] = v[i];
    __syncthreads();
    if (wave == 0) {
        double s = red[__lane_id() % (WAVES * N)];
#pragma unroll
        for (int off = N; off < WAVES * N; off <<= 1) s += __shfl_xor(s, off, kWave);
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = __shfl(s, i, kWave);
    }
    __syncthreads();
}

// ------------------------------------------------------------- balance ----

// Sums of one sequence's part of a block's tokens, [a, b) of the chunk at
// `logits`: picks into hist[E] and, with a token per wave, each wave's
// probabilities into sums[wave][E] (else they stay in acc, each wave's columns),
// the token groups' sums of lse^2 into zs. Complete behind the last barrier.
template <bool SIGMOID, int NV, int WPT, int GROUPS>
__device__ __forceinline__ void balance_part(const Place<WPT, GROUPS>& at, const float* __restrict__ logits,
                                             const int32_t* __restrict__ ids, uint64_t valid, int a, int b, int E,
                                             int k, Row<NV, WPT>& first, int have, RowReduce<WPT>& reduce,
                                             Row<NV, WPT>& acc, float* sums, int32_t* hist, float* zs) {
    constexpr int BLOCK = Place<WPT, GROUPS>::BLOCK;
    for (int c = threadIdx.x; c < E; c += BLOCK) hist[c] = 0;
    __syncthreads();
    for (int f = a * k + static_cast<int>(threadIdx.x); f < b * k; f += BLOCK) {
        const int id = ids[f];
        if ((valid >> (f / k) & 1) && id >= 0 && id < E) atomicAdd(&hist[id], 1);
    }
    acc.fill(0.f);
    float z = 0.f;
    for_rows(valid & bit_range(a, b) & at.share(), logits, E, at.part, at.lane, first, have,
             [&](int, Row<NV, WPT>& x) {
        Row<NV, WPT> u;
        const float m = weight_origin(reduce.max(x.max()));
        softmax_weights(x, m, u);
        float total[2] = {u.sum(), 0.f};
        if constexpr (SIGMOID) {
            sigmoid_weights<false>(x, fminf(m, 0.f), u, u);
            total[1] = u.sum();
        }
        reduce.sum(total);
        const float lse = total[0] == 0.f ? 0.f : m + log_fast(total[0]);   // a row of -inf adds nothing
        z += lse * lse;
        const float inv = inverse(total[SIGMOID ? 1 : 0]);
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int q = 0; q < 4; ++q) acc.v[i][q] = __builtin_fmaf(u.v[i][q], inv, acc.v[i][q]);
    });
    if (at.lane == 0 && at.part == 0) zs[at.group] = z;
    if constexpr (WPT == 1) acc.store(sums + at.wave * E, E, 0, at.lane, false);
    __syncthreads();
}

// Column c of the waves' sums, in wave order.
template <int GROUPS>
__device__ __forceinline__ float column_sum(const float* sums, int E, int c) {
    float s = sums[c];
#pragma unroll
    for (int w = 1; w < GROUPS; ++w) s += sums[w * E + c];
    return s;
}

template <int NV, int WPT, int GROUPS, bool SIGMOID>
__global__ __launch_bounds__(WPT* GROUPS* kWave) void balance_partial_kernel(
    const float* __restrict__ logits, const int32_t* __restrict__ ids, const uint8_t* __restrict__ mask,
    const int32_t* __restrict__ seq_offsets, int T, int E, int k, int S, int chunk,
    float* __restrict__ part_probs, int32_t* __restrict__ part_counts, int32_t* __restrict__ part_n,
    float* __restrict__ part_z, int32_t* __restrict__ counter) {
    using P = Place<WPT, GROUPS>;
    extern __shared__ float lds[];
    int32_t* hist = reinterpret_cast<int32_t*>(lds);   // [E]
    float* sums = lds + E;                             // [GROUPS][E] with a token per wave
    __shared__ float zs[GROUPS];
    __shared__ float red[2][WPT][4];
    const P at;
    RowReduce<WPT> reduce{red, at.part};
    if (blockIdx.x == 0 && threadIdx.x == 0) *counter = 0;   // for the kernel that follows
    const int t0 = static_cast<int>(blockIdx.x) * chunk;
    const int t1 = min(T, t0 + chunk);
    Row<NV, WPT> first, acc;
    int have = -1;
    if (t0 + at.group < t1) {
        have = at.group;
        first.load(logits + static_cast<size_t>(t0 + at.group) * E, E, at.part, at.lane);
    }
    const uint64_t valid = valid_tokens(mask, t0, t1 - t0);
    int a = t0;
    while (a < t1) {
        int begin = 0, end = 0;
        const int s = find_sequence(seq_offsets, S, T, a, begin, end);
        if (s < 0) {
            // before the first sequence, or behind the last
            const int start = seq_offset(seq_offsets, 0, T);
            if (a >= start) break;
            a = start;
            continue;
        }
        const int b = min(end, t1);
        balance_part<SIGMOID>(at, logits + static_cast<size_t>(t0) * E, ids + static_cast<size_t>(t0) * k, valid,
                              a - t0, b - t0, E, k, first, have, reduce, acc, sums, hist, zs);
        have = -1;
        const size_t row = static_cast<size_t>(blockIdx.x) + s;
        for (int c = threadIdx.x; c < E; c += P::BLOCK) {
            part_counts[row * E + c] = hist[c];
            if constexpr (WPT == 1) part_probs[row * E + c] = column_sum<GROUPS>(sums, E, c);
        }
        if constexpr (WPT > 1) acc.store(part_probs + row * E, E, at.part, at.lane, false);
        if (threadIdx.x == 0) {
            part_n[row] = __popcll(valid & bit_range(a - t0, b - t0));
            float zt = zs[0];
            for (int w = 1; w < GROUPS; ++w) zt += zs[w];
            part_z[row] = zt;
        }
        __syncthreads();
        a = b;
    }
}

// A batch of up to kSmallTokens tokens, its sequences in turn.
template <int NV, bool SIGMOID>
__global__ __launch_bounds__(kSmallGroups* kWave) void balance_small_kernel(
    const float* __restrict__ logits, const int32_t* __restrict__ ids, const uint8_t* __restrict__ mask,
    const int32_t* __restrict__ seq_offsets, int T, int E, int k, int S, float* __restrict__ losses,
    int32_t* __restrict__ counts, float* __restrict__ probs, int32_t* __restrict__ tokens) {
    using P = Place<1, kSmallGroups>;
    static_assert(P::BLOCK >= kSmallExperts, "a thread per expert");
    extern __shared__ float sums[];   // [kSmallGroups][E]
    __shared__ int32_t hist[kSmallExperts];
    __shared__ float zs[kSmallGroups];
    __shared__ double red[kSmallGroups];
    const P at;
    RowReduce<1> reduce{nullptr, 0};
    Row<NV, 1> first, acc;
    int have = -1;
    if (at.group < T) {
        have = at.group;
        first.load(logits + static_cast<size_t>(at.group) * E, E, 0, at.lane);
    }
    const uint64_t valid = valid_tokens(mask, 0, T);
    const int c = threadIdx.x;
    double balance = 0, z = 0;   // thread 0's
    int n = 0, full = 0;
    for (int s = 0; s < S; ++s) {
        const int a = seq_offset(seq_offsets, s, T), b = seq_offset(seq_offsets, s + 1, T);
        const int m = a < b ? __popcll(valid & bit_range(a, b)) : 0;
        if (c == 0) tokens[s] = m;
        float p = 0.f;
        int32_t h = 0;
        if (m > 0) {
            balance_part<SIGMOID>(at, logits, ids, valid, a, b, E, k, first, have, reduce, acc, sums, hist, zs);
            have = -1;
            if (c < E) {
                p = column_sum<kSmallGroups>(sums, E, c);
                h = hist[c];
            }
            double v[1] = {static_cast<double>(p * static_cast<float>(h))};
            block_sum<1, P::BLOCK>(v, red);
            if (c == 0) {
                balance += v[0] * E / (static_cast<double>(k) * m * m);
                for (int w = 0; w < kSmallGroups; ++w) z += zs[w];
            }
            n += m;
            ++full;
            __syncthreads();
        }
        if (c < E) {
            probs[static_cast<size_t>(s) * E + c] = p;
            counts[static_cast<size_t>(s) * E + c] = h;
        }
    }
    if (c == 0) {
        losses[0] = full > 0 ? static_cast<float>(balance / full) : 0.f;
        losses[1] = n > 0 ? static_cast<float>(z / n) : 0.f;
        tokens[S] = n;
        tokens[S + 1] = full;
    }
}

constexpr int kReduceBlock = 1024;

struct PartSum {
    float f;
    int32_t n;
};

template <typename V>
__device__ __forceinline__ V agent_load(const V* p) {
    return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
// Publishes a value to the whole device: written through to where agent_load
// reads, and waited for (wait_stores). A __threadfence per block would write
// back its XCD's L2 instead (the reduction 26 -> 10 us with 52 blocks).
template <typename V>
__device__ __forceinline__ void agent_store(V* p, V v) {
    __hip_atomic_store(p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ void wait_stores() { __builtin_amdgcn_s_waitcnt(0); }

// Block s * col_blocks + c: columns [COLS c, COLS c + COLS) of sequence s,
// 1024 / COLS groups of threads over its partial rows. Few columns spread one
// sequence's sums over many CUs, many keep the blocks of many sequences few: the
// fewest columns with up to 256 blocks (16 and 64 columns: 13 sequences of 254
// experts 9.4 and 10.8 us, 40 of 256 14.9 and 10.3, 8 of 1024 14.9 and 12.9).
template <int COLS>
__global__ __launch_bounds__(kReduceBlock) void balance_reduce_kernel(
    const float* __restrict__ part_probs, const int32_t* __restrict__ part_counts,
    const int32_t* __restrict__ part_n, const float* __restrict__ part_z,
    const int32_t* __restrict__ seq_offsets, int T, int E, int k, int S, int chunk, int col_blocks,
    float* __restrict__ losses, int32_t* __restrict__ counts, float* __restrict__ probs,
    int32_t* __restrict__ tokens, float* __restrict__ seq_dot, float* __restrict__ seq_z,
    int32_t* __restrict__ counter) {
    constexpr int kReduceGroups = kReduceBlock / COLS;
    __shared__ float sp[kReduceGroups][COLS];
    __shared__ int32_t sc[kReduceGroups][COLS];
    __shared__ double red[(kReduceBlock / kWave) * 4];
    __shared__ int last;
    const int s = blockIdx.x / col_blocks;
    const int cb = blockIdx.x - s * col_blocks;
    const int col = threadIdx.x % COLS, group = threadIdx.x / COLS;
    const int c = cb * COLS + col;
    const int a = seq_offset(seq_offsets, s, T), b = seq_offset(seq_offsets, s + 1, T);
    const int b0 = a / chunk, b1 = a < b ? (b - 1) / chunk + 1 : b0;
    float p = 0.f;
    int32_t n = 0;
    if (c < E)
        for_batches<8>(b0 + group, b1, kReduceGroups,
                       [&](int r) {
                           const size_t at = (static_cast<size_t>(r) + s) * E + c;
                           return PartSum{part_probs[at], part_counts[at]};
                       },
                       [&](const PartSum& v) {
                           p += v.f;
                           n += v.n;
                       });
    sp[group][col] = p;
    sc[group][col] = n;
    if (threadIdx.x >= kReduceBlock - kWave && cb == 0) {
        int32_t m = 0;
        float z = 0.f;
        const int i = threadIdx.x - (kReduceBlock - kWave);
        for_batches<8>(b0 + i, b1, kWave, [&](int r) { return PartSum{part_z[r + s], part_n[r + s]}; },
                       [&](const PartSum& v) {
                           m += v.n;
                           z += v.f;
                       });
        z = wave_sum(z);
        for (int off = 32; off >= 1; off >>= 1) m += __shfl_xor(m, off, kWave);
        if (i == 0) {
            agent_store(&tokens[s], m);
            agent_store(&seq_z[s], z);
        }
    }
    __syncthreads();
    // sixteen lanes a column add its groups, four columns a wave at a time
    const int l16 = threadIdx.x % 16;
    for (int q = threadIdx.x / 16; q < COLS; q += kReduceBlock / 16) {
        p = 0.f;
        n = 0;
        for (int g = l16; g < kReduceGroups; g += 16) {
            p += sp[g][q];
            n += sc[g][q];
        }
        p = group_sum(p, 16);
        for (int off = 8; off >= 1; off >>= 1) n += __shfl_xor(n, off, kWave);
        if (l16 == 0) {
            const int e = cb * COLS + q;
            if (e < E) {
                probs[static_cast<size_t>(s) * E + e] = p;
                counts[static_cast<size_t>(s) * E + e] = n;
            }
            sp[0][q] = p * static_cast<float>(n);   // this column's first group: read above by these lanes alone
        }
    }
    __syncthreads();
    if (threadIdx.x < kWave) {
        float dot = 0.f;
        for (int q = threadIdx.x; q < COLS; q += kWave) dot += sp[0][q];
        dot = wave_sum(dot);
        if (threadIdx.x == 0) agent_store(&seq_dot[static_cast<size_t>(s) * col_blocks + cb], dot);
    }
    // the last block to count itself finds every block's values published
    wait_stores();
    __syncthreads();
    if (threadIdx.x == 0)
        last = __hip_atomic_fetch_add(counter, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == S * col_blocks - 1;
    __syncthreads();
    if (!last) return;
    double v[4] = {0, 0, 0, 0};   // balance, z, tokens, sequences with a token
    for (int i = threadIdx.x; i < S * col_blocks; i += kReduceBlock) {
        const float dot = agent_load(&seq_dot[i]);
        const double m = agent_load(&tokens[i / col_blocks]);
        if (m > 0) v[0] += dot * static_cast<double>(E) / (k * m * m);
    }
    for (int q = threadIdx.x; q < S; q += kReduceBlock) {
        const int32_t m = agent_load(&tokens[q]);
        v[1] += agent_load(&seq_z[q]);
        v[2] += m;
        v[3] += m > 0;
    }
    block_sum<4, kReduceBlock>(v, red);
    if (threadIdx.x == 0) {
        losses[0] = v[3] > 0 ? static_cast<float>(v[0] / v[3]) : 0.f;
        losses[1] = v[2] > 0 ? static_cast<float>(v[1] / v[2]) : 0.f;
        tokens[S] = static_cast<int32_t>(v[2]);
        tokens[S + 1] = static_cast<int32_t>(v[3]);
    }
}

// The chunk's tokens in turn; the coefficients c_e of the current sequence stay
// in registers.
template <int NV, int WPT, bool SIGMOID>
__global__ __launch_bounds__((WPT > 1 ? WPT : kGroups) * kWave) void balance_backward_kernel(
    const float* __restrict__ d_losses, const float* __restrict__ logits, const uint8_t* __restrict__ mask,
    const int32_t* __restrict__ seq_offsets, const int32_t* __restrict__ counts,
    const int32_t* __restrict__ tokens, int T, int E, int k, int S, int chunk, int accumulate,
    float* __restrict__ d_logits) {
    using P = Place<WPT, WPT == 1 ? kGroups : 1>;
    __shared__ float red[2][WPT][4];
    const P at;
    RowReduce<WPT> reduce{red, at.part};
    const int t0 = static_cast<int>(blockIdx.x) * chunk;
    const int len = min(chunk, T - t0);
    const float* rows = logits + static_cast<size_t>(t0) * E;
    float* out = d_logits + static_cast<size_t>(t0) * E;
    Row<NV, WPT> first;
    if (at.group < len) first.load(rows + static_cast<size_t>(at.group) * E, E, at.part, at.lane);
    const uint64_t valid = valid_tokens(mask, t0, len);
    const uint64_t share = at.share() & bit_range(0, len);
    const float n = static_cast<float>(max(tokens[S], 1));
    const float full = static_cast<float>(max(tokens[S + 1], 1));
    const float zg = 2.f * d_losses[1] / n;
    int s = -1, begin = 0, end = 0;
    Row<NV, WPT> cf;
    cf.fill(0.f);
    for_rows(valid & share, rows, E, at.part, at.lane, first, at.group, [&](int t, Row<NV, WPT>& x) {
        if (!(s >= 0 && t0 + t < end)) {
            s = find_sequence(seq_offsets, S, T, t0 + t, begin, end);
            if (s >= 0) {
                const float m = static_cast<float>(max(tokens[s], 1));
                const float w = d_losses[0] * static_cast<float>(E) / (static_cast<float>(k) * m * m * full);
#pragma unroll
                for (int i = 0; i < NV; ++i)
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const int c = cf.column(i, at.part, at.lane) + q;
                        cf.v[i][q] = c < E ? w * static_cast<float>(counts[static_cast<size_t>(s) * E + c]) : 0.f;
                    }
            }
        }
        Row<NV, WPT> d;
        if (s < 0) {   // in no sequence: as invalid
            d.fill(0.f);
            if (!accumulate) d.store(out + static_cast<size_t>(t) * E, E, at.part, at.lane, false);
            return;
        }
        Row<NV, WPT> u;
        const float m = weight_origin(reduce.max(x.max()));
        softmax_weights(x, m, u);
        if constexpr (SIGMOID) {
            d = u;
            Row<NV, WPT> slope;
            sigmoid_weights<true>(x, fminf(m, 0.f), u, slope);
            float v[3] = {d.sum(), u.sum(), u.dot(cf)};
            reduce.sum(v);
            // the z loss' part: (2 / n) lse softmax
            const float zc = zg == 0.f || v[0] == 0.f ? 0.f : zg * (m + log_fast(v[0])) * inverse(v[0]);
            const float inv = inverse(v[1]), dot = v[2] * inv;
#pragma unroll
            for (int i = 0; i < NV; ++i)
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    d.v[i][q] = __builtin_fmaf(u.v[i][q] * inv * slope.v[i][q], cf.v[i][q] - dot, zc * d.v[i][q]);
        } else {
            float v[2] = {u.sum(), u.dot(cf)};
            reduce.sum(v);
            const float inv = inverse(v[0]), dot = v[1] * inv;
            const float zc = zg == 0.f || v[0] == 0.f ? 0.f : zg * (m + log_fast(v[0])) * inv;
#pragma unroll
            for (int i = 0; i < NV; ++i)
#pragma unroll
                for (int q = 0; q < 4; ++q) d.v[i][q] = u.v[i][q] * __builtin_fmaf(cf.v[i][q] - dot, inv, zc);
        }
        d.store(out + static_cast<size_t>(t) * E, E, at.part, at.lane, accumulate);
    });
    if (accumulate) return;
    Row<NV, WPT> zero;
    zero.fill(0.f);
    for (uint64_t bits = ~valid & share; bits; bits &= bits - 1)
        zero.store(out + static_cast<size_t>(__builtin_ctzll(bits)) * E, E, at.part, at.lane, false);
}

struct BalancePlan {
    int chunk, blocks, cols, col_blocks;
    size_t rows, probs, counts, n, z, dot, seq_z, counter, bytes;   // byte offsets
};

inline size_t round256(size_t b) { return (b + 255) / 256 * 256; }

inline bool balance_shape_ok(int T, int E, int S) {
    return T >= 0 && T <= MOE_MAX_TOKENS && E >= 1 && E <= MOE_MAX_EXPERTS && S >= 1 && S <= MOE_MAX_SEQUENCES;
}

inline bool balance_small(int T, int E, int S) { return small_batch(T, E) && S <= kSmallSequences; }

inline BalancePlan plan_balance(int T, int E, int S) {
    BalancePlan p;
    p.chunk = T <= kFewTokens ? 1 : chunk_tokens(T, E <= kBalanceOneWave, kTargetBlocks);
    p.blocks = ceil_div(T, p.chunk);
    p.cols = 16;
    while (p.cols < 256 && static_cast<long long>(S) * ceil_div(E, p.cols) > 256) p.cols *= 4;
    p.col_blocks = ceil_div(E, p.cols);
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

constexpr int kDistillBlocks = 2 * kTargetBlocks;   // no partial rows to add up: a token per wave sooner

// Lane j < K: teacher entry j of token t; id -1 where there is none.
struct Entry {
    int id = -1;
    float z = kNegInf;
};

__device__ __forceinline__ Entry teacher_entry(const int32_t* __restrict__ ids, const float* __restrict__ logits,
                                               size_t t, int K) {
    Entry e;
    const int lane = __lane_id();
    if (lane < K) {
        e.id = ids[t * K + lane];
        e.z = logits[t * K + lane];
    }
    return e;
}

// The entry's share q of the entries' sum and log q; id -1 where there is none.
// Returns whether the token has an entry.
__device__ __forceinline__ bool teacher_shares(const Entry& e, int E, int score, float inv_temp, int& id, float& q,
                                               float& logq) {
    id = e.id < 0 || e.id >= E || e.z == kNegInf ? -1 : e.id;
    if (ballot(id >= 0) == 0) return false;
    const float z = id < 0 ? kNegInf : log_score(e.z * inv_temp, score);
    const float m = wave_max(z);
    const float w = id < 0 ? 0.f : exp_fast(z - m);
    const float total = wave_sum(w);
    logq = id < 0 ? 0.f : (z - m) - logf(total);
    q = w / total;
    return true;
}

// GROUPS = kSmallGroups: one block for a batch of up to kSmallTokens tokens,
// which writes the loss itself; else one partial sum per block.
template <int NV, int WPT, int GROUPS, bool SIGMOID>
__global__ __launch_bounds__(WPT* GROUPS* kWave) void distill_kernel(
    const float* __restrict__ logits, const int32_t* __restrict__ t_ids, const float* __restrict__ t_logits,
    const uint8_t* __restrict__ mask, float inv_temp, float temp2, int T, int E, int K, int chunk,
    float* __restrict__ token_loss, float* __restrict__ part_loss, int32_t* __restrict__ part_n) {
    __shared__ float sl[GROUPS];
    __shared__ int32_t sn[GROUPS];
    __shared__ float red[2][WPT][4];
    constexpr int score = SIGMOID ? MOE_SCORE_SIGMOID : MOE_SCORE_SOFTMAX;
    const Place<WPT, GROUPS> at;
    RowReduce<WPT> reduce{red, at.part};
    const int t0 = static_cast<int>(blockIdx.x) * chunk;
    const int len = min(chunk, T - t0);
    const float* rows = logits + static_cast<size_t>(t0) * E;
    Row<NV, WPT> first;
    Entry entry;
    if (at.group < len) {
        first.load(rows + static_cast<size_t>(at.group) * E, E, at.part, at.lane);
        entry = teacher_entry(t_ids, t_logits, static_cast<size_t>(t0) + at.group, K);
    }
    const uint64_t valid = valid_tokens(mask, t0, len);
    const uint64_t share = at.share() & bit_range(0, len);
    const bool writes = at.lane == 0 && at.part == 0;
    float sum = 0.f;
    int32_t n = 0;
    int have = at.group;   // the token that entry belongs to
    for_rows(valid & share, rows, E, at.part, at.lane, first, at.group, [&](int t, Row<NV, WPT>& x) {
        const size_t tok = static_cast<size_t>(t0) + t;
        if (t != have) entry = teacher_entry(t_ids, t_logits, tok, K);
        float xp = 0.f;   // the student's logit of the entry
        if (entry.id >= 0 && entry.id < E) xp = logits[tok * E + entry.id] * inv_temp;
        const Entry mine = entry;
        have = t + GROUPS;   // the group's next token, likely valid
        if (have < len) entry = teacher_entry(t_ids, t_logits, static_cast<size_t>(t0) + have, K);
        int id = -1;
        float q = 0.f, logq = 0.f, loss = 0.f;
        if (teacher_shares(mine, E, score, inv_temp, id, q, logq)) {
            Row<NV, WPT> u;
            x.scale(inv_temp);
            float m = weight_origin(reduce.max(x.max()));
            if constexpr (SIGMOID) {
                m = fminf(m, 0.f);
                sigmoid_weights<false>(x, m, u, u);
            } else {
                softmax_weights(x, m, u);
            }
            float total[1] = {u.sum()};
            reduce.sum(total);
            // an expert that the student masks is infinitely far, in a row of -inf too
            const float ls = log_score(xp, score);
            const float logp = ls == kNegInf ? kNegInf : (ls - m) - logf(total[0]);
            const float term = id >= 0 && q > 0.f ? q * (logq - logp) : 0.f;
            loss = temp2 * wave_sum(term);
            sum += loss;
            ++n;
        }
        if (writes) token_loss[tok] = loss;
    });
    for (uint64_t bits = ~valid & share; bits; bits &= bits - 1)
        if (writes) token_loss[static_cast<size_t>(t0) + __builtin_ctzll(bits)] = 0.f;
    if (writes) {
        sl[at.group] = sum;
        sn[at.group] = n;
    }
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int w = 1; w < GROUPS; ++w) {
            sum += sl[w];
            n += sn[w];
        }
        part_loss[blockIdx.x] = GROUPS != kSmallGroups ? sum : n > 0 ? sum / static_cast<float>(n) : 0.f;
        part_n[blockIdx.x] = n;
    }
}

constexpr int kDistillReduceBlock = 256;

__global__ __launch_bounds__(kDistillReduceBlock) void distill_reduce_kernel(const float* __restrict__ part_loss,
                                                                             const int32_t* __restrict__ part_n,
                                                                             int blocks, float* __restrict__ loss,
                                                                             int32_t* __restrict__ tokens) {
    __shared__ double red[kDistillReduceBlock / kWave * 2];
    double v[2] = {0, 0};
    for_batches<8>(threadIdx.x, blocks, kDistillReduceBlock, [&](int b) { return PartSum{part_loss[b], part_n[b]}; },
                   [&](const PartSum& p) {
                       v[0] += p.f;
                       v[1] += p.n;
                   });
    block_sum<2, kDistillReduceBlock>(v, red);
    if (threadIdx.x == 0) {
        loss[0] = v[1] > 0 ? static_cast<float>(v[0] / v[1]) : 0.f;
        tokens[0] = static_cast<int32_t>(v[1]);
    }
}

// The teacher's shares reach the lanes that own their experts through a row of
// LDS per wave: zeros but for the entries, which are cleared again behind each
// token. Each wave keeps its own columns; LDS
// operations of one wave run in order, so no barrier is needed.
template <int NV, int WPT, bool SIGMOID>
__global__ __launch_bounds__((WPT > 1 ? WPT : kGroups) * kWave) void distill_backward_kernel(
    const float* __restrict__ d_loss, const float* __restrict__ logits, const int32_t* __restrict__ t_ids,
    const float* __restrict__ t_logits, const uint8_t* __restrict__ mask, const int32_t* __restrict__ tokens,
    float inv_temp, float temp, int T, int E, int K, int chunk, int accumulate, float* __restrict__ d_logits) {
    extern __shared__ float lds[];
    __shared__ float red[2][WPT][4];
    constexpr int score = SIGMOID ? MOE_SCORE_SIGMOID : MOE_SCORE_SOFTMAX;
    const Place<WPT, WPT == 1 ? kGroups : 1> at;
    RowReduce<WPT> reduce{red, at.part};
    // a wave's columns, 256 at a time: column c of the row is at
    // 256 (c / (256 WPT)) + c % 256 of the wave c / 256 % WPT that owns it
    float* shares = lds + at.wave * (NV * 256);
    auto place = [&](int c) { return (c / (256 * WPT)) * 256 + c % 256; };
#pragma unroll
    for (int i = 0; i < NV; ++i)
        *reinterpret_cast<f32x4*>(shares + i * 256 + at.lane * 4) = f32x4{0.f, 0.f, 0.f, 0.f};
    const int t0 = static_cast<int>(blockIdx.x) * chunk;
    const int len = min(chunk, T - t0);
    const float* rows = logits + static_cast<size_t>(t0) * E;
    float* out = d_logits + static_cast<size_t>(t0) * E;
    Row<NV, WPT> first;
    Entry entry;
    if (at.group < len) {
        first.load(rows + static_cast<size_t>(at.group) * E, E, at.part, at.lane);
        entry = teacher_entry(t_ids, t_logits, static_cast<size_t>(t0) + at.group, K);
    }
    const uint64_t valid = valid_tokens(mask, t0, len);
    const uint64_t share = at.share() & bit_range(0, len);
    const float g = d_loss[0] * temp / static_cast<float>(max(tokens[0], 1));
    int have = at.group;   // the token that entry belongs to
    for_rows(valid & share, rows, E, at.part, at.lane, first, at.group, [&](int t, Row<NV, WPT>& x) {
        if (t != have) entry = teacher_entry(t_ids, t_logits, static_cast<size_t>(t0) + t, K);
        const Entry now = entry;
        have = t + (WPT > 1 ? 1 : kGroups);   // the group's next token, likely valid
        if (have < len) entry = teacher_entry(t_ids, t_logits, static_cast<size_t>(t0) + have, K);
        int id = -1;
        float q = 0.f, logq = 0.f;
        if (!teacher_shares(now, E, score, inv_temp, id, q, logq)) {
            x.fill(0.f);
            if (!accumulate) x.store(out + static_cast<size_t>(t) * E, E, at.part, at.lane, false);
            return;
        }
        // an expert named twice: every entry that names it holds the sum
        float same = 0.f;
        for (int j = 0; j < K; ++j) {
            const int other = __builtin_amdgcn_readlane(id, j);
            const float oq = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(q), j));
            if (other == id) same += oq;
        }
        const bool mine = id >= 0 && (WPT == 1 || id / 256 % WPT == at.part);
        if (mine) shares[place(id)] = same;
        Row<NV, WPT> u, slope;
        x.scale(inv_temp);
        const float m = weight_origin(reduce.max(x.max()));
        if constexpr (SIGMOID) sigmoid_weights<true>(x, fminf(m, 0.f), u, slope);
        else softmax_weights(x, m, u);
        float total[1] = {u.sum()};
        reduce.sum(total);
        const float inv = inverse(total[0]);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const f32x4 sq = *reinterpret_cast<const f32x4*>(shares + i * 256 + at.lane * 4);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                u.v[i][j] = g * __builtin_fmaf(u.v[i][j], inv, -sq[j]);
                if constexpr (SIGMOID) u.v[i][j] *= slope.v[i][j];
            }
        }
        if (mine) shares[place(id)] = 0.f;
        u.store(out + static_cast<size_t>(t) * E, E, at.part, at.lane, accumulate);
    });
    if (accumulate) return;
    Row<NV, WPT> zero;
    zero.fill(0.f);
    for (uint64_t bits = ~valid & share; bits; bits &= bits - 1)
        zero.store(out + static_cast<size_t>(__builtin_ctzll(bits)) * E, E, at.part, at.lane, false);
}

inline bool distill_shape_ok(int T, int E) {
    return T >= 0 && T <= MOE_MAX_TOKENS && E >= 1 && E <= MOE_MAX_EXPERTS;
}

// The temperature's square and reciprocal, and logits times it, stay normal.
inline bool temperature_ok(float t) { return t >= 1e-6f && t <= 1e6f; }

inline bool score_ok(int score) { return score == MOE_SCORE_SIGMOID || score == MOE_SCORE_SOFTMAX; }

}  // namespace
}  // namespace moe

extern "C" size_t moe_balance_loss_workspace_bytes(int T, int E, int S) {
    using namespace moe;
    return balance_shape_ok(T, E, S) && !balance_small(T, E, S) ? plan_balance(T, E, S).bytes : 0;
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
    const bool sigmoid = score == MOE_SCORE_SIGMOID;
    if (balance_small(T, E, S))
        return with_row_shape<kBalanceOneWave>(E, [&](auto nv, auto wpt) {
            if constexpr (decltype(wpt)::value == 1) {
                constexpr int NV = decltype(nv)::value;
                auto kern = sigmoid ? balance_small_kernel<NV, true> : balance_small_kernel<NV, false>;
                return launch(kern, dim3(1), dim3(kSmallGroups * kWave), sizeof(float) * kSmallGroups * E, stream, logits,
                              topk_ids, token_mask, seq_offsets, T, E, k, S, losses, counts, probs, tokens);
            } else {
                return static_cast<int>(MOE_ERR_BAD_SHAPE);
            }
        });
    const BalancePlan p = plan_balance(T, E, S);
    if (!workspace || workspace_bytes < p.bytes || !aligned16(workspace)) return MOE_ERR_WORKSPACE;
    char* ws = static_cast<char*>(workspace);
    auto* part_probs = reinterpret_cast<float*>(ws + p.probs);
    auto* part_counts = reinterpret_cast<int32_t*>(ws + p.counts);
    auto* part_n = reinterpret_cast<int32_t*>(ws + p.n);
    auto* part_z = reinterpret_cast<float*>(ws + p.z);
    auto* counter = reinterpret_cast<int32_t*>(ws + p.counter);
    const int st = with_row_shape<kBalanceOneWave>(E, [&](auto nv, auto wpt) {
        constexpr int NV = decltype(nv)::value, WPT = decltype(wpt)::value;
        constexpr int GROUPS = WPT > 1 ? 1 : kGroups;
        const int groups = p.chunk == 1 ? 1 : GROUPS;
        auto kern = groups == 1 ? (sigmoid ? balance_partial_kernel<NV, WPT, 1, true> : balance_partial_kernel<NV, WPT, 1, false>)
                                : (sigmoid ? balance_partial_kernel<NV, WPT, GROUPS, true>
                                           : balance_partial_kernel<NV, WPT, GROUPS, false>);
        return launch(kern, dim3(p.blocks > 0 ? p.blocks : 1), dim3(WPT * groups * kWave),
                      sizeof(float) * E * (WPT > 1 ? 1 : 1 + groups), stream, logits, topk_ids, token_mask, seq_offsets, T, E, k,
                      S, p.chunk, part_probs, part_counts, part_n, part_z, counter);
    });
    if (st != MOE_OK) return st;
    auto reduce = p.cols == 16   ? balance_reduce_kernel<16>
                  : p.cols == 64 ? balance_reduce_kernel<64>
                                 : balance_reduce_kernel<256>;
    return launch(reduce, dim3(S * p.col_blocks), dim3(kReduceBlock), 0, stream, part_probs,
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
    const int chunk = chunk_tokens(T, E <= kBalanceOneWave, kTargetBlocks);
    return with_row_shape<kBalanceOneWave>(E, [&](auto nv, auto wpt) {
        constexpr int NV = decltype(nv)::value, WPT = decltype(wpt)::value;
        auto kern = score == MOE_SCORE_SIGMOID ? balance_backward_kernel<NV, WPT, true>
                                               : balance_backward_kernel<NV, WPT, false>;
        return launch(kern, dim3(ceil_div(T, chunk)), dim3((WPT > 1 ? WPT : kGroups) * kWave), 0, stream, d_losses,
                      logits, token_mask, seq_offsets, counts, tokens, T, E, k, S, chunk, accumulate, d_logits);
    });
}

extern "C" size_t moe_distill_loss_workspace_bytes(int T, int E) {
    using namespace moe;
    if (!distill_shape_ok(T, E) || small_batch(T, E)) return 0;
    const int blocks = ceil_div(T, chunk_tokens(T, E <= kDistillOneWave, kDistillBlocks));
    return 2 * round256(sizeof(float) * (blocks > 0 ? blocks : 1));
}

extern "C" int moe_distill_loss(const float* logits, const int32_t* teacher_ids, const float* teacher_logits,
                                const uint8_t* token_mask, int score, float temperature, int T, int E, int K,
                                float* loss, float* token_loss, int32_t* tokens, void* workspace,
                                size_t workspace_bytes, void* stream) {
    using namespace moe;
    if (!distill_shape_ok(T, E) || K < 1 || K > MOE_MAX_TOPK) return MOE_ERR_BAD_SHAPE;
    if (!score_ok(score) || !temperature_ok(temperature)) return MOE_ERR_BAD_ARG;
    if (!loss || !tokens) return MOE_ERR_NULL_ARG;
    if (T > 0 && (!logits || !teacher_ids || !teacher_logits || !token_mask || !token_loss)) return MOE_ERR_NULL_ARG;
    if (!all_aligned16(logits, teacher_ids, teacher_logits, token_mask, loss, token_loss, tokens))
        return MOE_ERR_ALIGN;
    const bool sigmoid = score == MOE_SCORE_SIGMOID;
    const float inv_temp = 1.f / temperature, temp2 = temperature * temperature;
    if (small_batch(T, E))
        return with_row_shape<kDistillOneWave>(E, [&](auto nv, auto wpt) {
            if constexpr (decltype(wpt)::value == 1) {
                constexpr int NV = decltype(nv)::value <= 4 ? decltype(nv)::value : 4;   // up to kSmallExperts
                auto kern = sigmoid ? distill_kernel<NV, 1, kSmallGroups, true> : distill_kernel<NV, 1, kSmallGroups, false>;
                return launch(kern, dim3(1), dim3(kSmallGroups * kWave), 0, stream, logits, teacher_ids,
                              teacher_logits, token_mask, inv_temp, temp2, T, E, K, kSmallTokens, token_loss, loss,
                              tokens);
            } else {
                return static_cast<int>(MOE_ERR_BAD_SHAPE);
            }
        });
    if (!workspace || workspace_bytes < moe_distill_loss_workspace_bytes(T, E) || !aligned16(workspace))
        return MOE_ERR_WORKSPACE;
    const int chunk = chunk_tokens(T, E <= kDistillOneWave, kDistillBlocks);
    const int blocks = ceil_div(T, chunk);
    auto* part_loss = static_cast<float*>(workspace);
    auto* part_n = reinterpret_cast<int32_t*>(static_cast<char*>(workspace) + round256(sizeof(float) * (blocks > 0 ? blocks : 1)));
    if (T > 0) {
        const int st = with_row_shape<kDistillOneWave>(E, [&](auto nv, auto wpt) {
            constexpr int NV = decltype(nv)::value, WPT = decltype(wpt)::value, GROUPS = WPT > 1 ? 1 : kGroups;
            auto kern = sigmoid ? distill_kernel<NV, WPT, GROUPS, true> : distill_kernel<NV, WPT, GROUPS, false>;
            return launch(kern, dim3(blocks), dim3(WPT * GROUPS * kWave), 0, stream, logits, teacher_ids,
                          teacher_logits, token_mask, inv_temp, temp2, T, E, K, chunk, token_loss, part_loss, part_n);
        });
        if (st != MOE_OK) return st;
    }
    return launch(distill_reduce_kernel, dim3(1), dim3(kDistillReduceBlock), 0, stream, part_loss, part_n, blocks,
                  loss, tokens);
}

extern "C" int moe_distill_loss_backward(const float* d_loss, const float* logits, const int32_t* teacher_ids,
                                         const float* teacher_logits, const uint8_t* token_mask,
                                         const int32_t* tokens, int score, float temperature, int T, int E, int K,
                                         int accumulate, float* d_logits, void* stream) {
    using namespace moe;
    if (!distill_shape_ok(T, E) || K < 1 || K > MOE_MAX_TOPK) return MOE_ERR_BAD_SHAPE;
    if (!score_ok(score) || !temperature_ok(temperature)) return MOE_ERR_BAD_ARG;
    if (T == 0) return MOE_OK;
    if (!d_loss || !logits || !teacher_ids || !teacher_logits || !token_mask || !tokens || !d_logits)
        return MOE_ERR_NULL_ARG;
    if (!all_aligned16(d_loss, logits, teacher_ids, teacher_logits, token_mask, tokens, d_logits))
        return MOE_ERR_ALIGN;
    const int chunk = chunk_tokens(T, E <= kDistillOneWave, kDistillBlocks);
    return with_row_shape<kDistillOneWave>(E, [&](auto nv, auto wpt) {
        constexpr int NV = decltype(nv)::value, WPT = decltype(wpt)::value, WAVES = WPT > 1 ? WPT : kGroups;
        auto kern = score == MOE_SCORE_SIGMOID ? distill_backward_kernel<NV, WPT, true>
                                               : distill_backward_kernel<NV, WPT, false>;
        return launch(kern, dim3(ceil_div(T, chunk)), dim3(WAVES * kWave), sizeof(float) * WAVES * NV * 256, stream,
                      d_loss, logits, teacher_ids, teacher_logits, token_mask, tokens, 1.f / temperature, temperature,
                      T, E, K, chunk, accumulate, d_logits);
    });
}
