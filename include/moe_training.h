/*
 * moe_training.h — C ABI of the router's training operators on MI355X
 * (gfx950): the losses on the router's logits and the backward passes of
 * moe_route and moe_combine (moe_routing.h).
 *
 *   moe_balance_loss       per-sequence expert counts and probability sums, the
 *                          balance loss and the z loss
 *   moe_balance_loss_backward
 *                          their gradient on the logits
 *   moe_distill_loss       Kullback-Leibler divergence of the router's
 *                          distribution from a teacher's top logits
 *   moe_distill_loss_backward
 *                          its gradient on the logits
 *   moe_route_backward     gradients of moe_route on logits, input and weight
 *   moe_combine_backward   gradients of moe_combine on expert rows, routing
 *                          weights and norm weight
 *
 * One training step's use of them: moe_combine_backward gives d_topk_w; the
 * two losses' backward calls write and accumulate into one [T,E] gradient of
 * the logits; moe_route_backward takes both.
 *
 * The conventions of moe_routing.h hold (device pointers, row-major,
 * contiguous, 16-byte aligned; caller-owned memory; no allocation, no
 * synchronisation, nothing kept between calls; checks before any work; status
 * codes), with these differences:
 *   - T == 0 is valid; outputs whose size does not depend on T are then
 *     written (zero losses, counts and gradients).
 *   - A workspace belongs to one call at a time: two calls that may overlap
 *     (two streams, two captured graphs replayed together) need one each.
 *   - Results are deterministic: every sum has a fixed order.
 *   - Outputs overlap neither inputs nor each other, except where a call says
 *     that they may.
 *   - A token is valid when its token_mask byte is nonzero. The logits and
 *     input of other tokens are never inspected (they may hold NaN); their
 *     gradients are zero.
 */
#ifndef MOE_TRAINING_H
#define MOE_TRAINING_H

#include "moe_routing.h"

#ifdef __cplusplus
extern "C" {
#endif

/* The router's score of an expert, and with it the distribution over the
 * experts of a token:
 *   MOE_SCORE_SIGMOID  s_e = sigmoid(l_e), p_e = s_e / sum s   (moe_route's)
 *   MOE_SCORE_SOFTMAX  p = softmax(l)
 * Both are softmax(log score); the sigmoid form is evaluated so that it holds
 * where every s_e underflows. A row whose every score is zero (all logits
 * -inf) has p = 0; it counts as a token, adds nothing to the balance and z
 * losses and has no gradient of them. */
enum moe_score {
    MOE_SCORE_SIGMOID = 0,
    MOE_SCORE_SOFTMAX = 1
};

#define MOE_MAX_SEQUENCES 65536
#define MOE_MAX_TOKENS (1 << 30)

/*
 * moe_balance_loss — balance loss and z loss of the router's logits, with the
 * per-expert counts they need.
 *
 * Sequence s is the valid tokens t of [seq_offsets[s], seq_offsets[s+1]), n_s
 * of them; n is their total and S+ the number of sequences with n_s > 0.
 *   counts[s,e] = picks (t,j) of the sequence with topk_ids[t,j] == e
 *   probs[s,e]  = sum_t p[t,e]
 *   losses[0]   = 1/S+ sum_s E sum_e (counts[s,e] / (k n_s)) (probs[s,e] / n_s)
 *   losses[1]   = 1/n sum_t (log sum_e exp(l[t,e]))^2
 *   tokens      = n_0 .. n_{S-1}, n, S+
 * Each is 0 where it has no token. Tokens outside every sequence (behind the
 * last one) count as invalid.
 *
 * counts, probs and tokens are sums over tokens: ranks that hold parts of a
 * batch may add theirs up, take losses[0] from the sums and pass summed
 * counts and tokens to the backward call.
 *
 *   logits       [T,E] FP32.     topk_ids [T,k] int32 (entries outside [0,E)
 *                count nowhere). token_mask [T] u8.
 *   seq_offsets  [S+1] int32, ascending, within [0,T]; NULL: one sequence of
 *                all tokens (S must be 1). Values out of range are clamped.
 *   score        MOE_SCORE_*.
 *   0 <= T <= MOE_MAX_TOKENS, T k < 2^31, 1 <= E <= MOE_MAX_EXPERTS,
 *   1 <= k <= min(E, MOE_MAX_TOPK), 1 <= S <= MOE_MAX_SEQUENCES.
 *   losses [2] FP32, counts [S,E] int32, probs [S,E] FP32, tokens [S+2] int32:
 *                outputs.
 *   workspace    at least moe_balance_loss_workspace_bytes(T, E, S) bytes
 *                (0: a batch too small to need any, or a size out of range).
 * Errors: NULL_ARG, BAD_SHAPE, BAD_ARG (score), ALIGN, WORKSPACE, HIP.
 */
size_t moe_balance_loss_workspace_bytes(int T, int E, int S);

int moe_balance_loss(const float* logits, const int32_t* topk_ids, const uint8_t* token_mask,
                     const int32_t* seq_offsets, int score, int T, int E, int k, int S,
                     float* losses, int32_t* counts, float* probs, int32_t* tokens,
                     void* workspace, size_t workspace_bytes, void* stream);

/*
 * moe_balance_loss_backward — d_logits = d_losses[0] dlosses[0]/dl +
 * d_losses[1] dlosses[1]/dl, the counts taken as constants:
 *   c_e     = d_losses[0] E counts[s,e] / (k n_s^2 S+)
 *   slope_e = 1 - s_e (sigmoid) or 1 (softmax)
 *   dl[t,e] = p_e slope_e (c_e - sum_i p_i c_i)
 *             + d_losses[1] (2/n) lse_t softmax(l)_e
 *
 *   d_losses  [2] FP32 on the device.
 *   counts, tokens: moe_balance_loss's outputs (or their sums over ranks).
 *   accumulate 0: d_logits [T,E] FP32 is written (zeros for invalid tokens);
 *             1: added to (rows of invalid tokens are left as they are).
 * The other arguments are the forward call's.
 * Errors: NULL_ARG, BAD_SHAPE, BAD_ARG, ALIGN, HIP.
 */
int moe_balance_loss_backward(const float* d_losses, const float* logits, const uint8_t* token_mask,
                              const int32_t* seq_offsets, const int32_t* counts, const int32_t* tokens,
                              int score, int T, int E, int k, int S, int accumulate,
                              float* d_logits, void* stream);

/*
 * moe_distill_loss — distillation of the router from a teacher's top logits.
 *
 * Token t takes part when it is valid and has a teacher entry j with
 * 0 <= teacher_ids[t,j] < E and teacher_logits[t,j] != -inf; n tokens do.
 *   q[t,:]        the teacher's distribution over its entries: the score's, of
 *                 teacher_logits / temperature, normalised over the entries
 *                 (with MOE_SCORE_SIGMOID and temperature 1 the topk_w of a
 *                 moe_route call); an expert named twice gets both shares
 *   p[t,:]        the distribution over all E experts of logits / temperature
 *   token_loss[t] = temperature^2 sum_j q_j (log q_j - log p[id_j])
 *   loss[0]       = 1/n sum_t token_loss[t]
 *   tokens[0]     = n
 * Tokens that take no part have token_loss 0; loss is 0 when n is. An expert
 * with q > 0 whose student logit is -inf makes the loss infinite; the gradient
 * is finite there.
 *
 *   logits [T,E] FP32 (the student's). teacher_ids, teacher_logits [T,K]
 *   int32 / FP32. token_mask [T] u8. 1e-6 <= temperature <= 1e6; a quotient
 *   outside FP32's range counts as infinite.
 *   0 <= T <= MOE_MAX_TOKENS, 1 <= E <= MOE_MAX_EXPERTS, 1 <= K <= MOE_MAX_TOPK
 *   (K may exceed E).
 *   loss [1], token_loss [T] FP32, tokens [1] int32: outputs.
 *   workspace    at least moe_distill_loss_workspace_bytes(T, E) bytes (0: a
 *                batch too small to need any, or a size out of range).
 * Errors: NULL_ARG, BAD_SHAPE, BAD_ARG (score, temperature), ALIGN, WORKSPACE,
 * HIP.
 */
size_t moe_distill_loss_workspace_bytes(int T, int E);

int moe_distill_loss(const float* logits, const int32_t* teacher_ids, const float* teacher_logits,
                     const uint8_t* token_mask, int score, float temperature, int T, int E, int K,
                     float* loss, float* token_loss, int32_t* tokens,
                     void* workspace, size_t workspace_bytes, void* stream);

/*
 * moe_distill_loss_backward — gradient of the loss on the student's logits:
 *   dl[t,e] = d_loss (temperature / n) slope_e (p_e - q_e)
 * with slope as in moe_balance_loss_backward, at logits / temperature.
 *   d_loss [1] FP32 on the device; tokens [1]: the forward call's n (or its
 *   sum over ranks); accumulate as in moe_balance_loss_backward (rows of
 *   tokens that take no part count as invalid).
 * Errors: NULL_ARG, BAD_SHAPE, BAD_ARG, ALIGN, HIP.
 */
int moe_distill_loss_backward(const float* d_loss, const float* logits, const int32_t* teacher_ids,
                              const float* teacher_logits, const uint8_t* token_mask, const int32_t* tokens,
                              int score, float temperature, int T, int E, int K, int accumulate,
                              float* d_logits, void* stream);

/*
 * moe_route_backward — gradients of moe_route.
 *
 * The picks are constants and the bias only selects, so it has no gradient.
 * For a valid token, over its picks j with 0 <= id_j < E (s = sigmoid(l)):
 *   dl[t,id_j] = w_j (1 - s_{id_j}) (d_topk_w[t,j] - sum_i w_i d_topk_w[t,i])
 *   d_logits   = d_aux + those        (an expert named twice gets both)
 *   d_hidden[t,:] = scale sum_e d_logits[t,e] W[e,:]
 *   d_W[e,:]      = scale sum_t d_logits[t,e] hidden[t,:]
 * Rows of invalid tokens: d_logits and d_hidden are zero and nothing of them
 * reaches d_W.
 *
 * Numerics: products of BF16 planes on the matrix cores with FP32
 * accumulation. d_W and an FP32 d_hidden keep every product above 2^-23 of
 * the largest; a BF16 d_hidden keeps those above 2^-16 of it, well under its
 * own rounding.
 *
 *   d_topk_w   [T,k] FP32, or NULL: only d_aux's gradient.
 *   d_aux      [T,E] FP32 gradient on the logits from elsewhere (the losses),
 *              or NULL. At least one of the two is required.
 *   hidden     [T,H] in hidden_dtype as given to moe_route, or NULL:
 *              logits-in mode, d_logits is the only output.
 *   W          [E,H] FP32 (unused in logits-in mode or without d_hidden).
 *   logits     [T,E] FP32, topk_ids [T,k] int32, topk_w [T,k] FP32: moe_route's
 *              outputs (unused when d_topk_w is NULL). token_mask [T] u8.
 *   T, H, E, k, scale as in moe_route.
 *   d_logits   [T,E] FP32 output (may be d_aux itself).
 *   d_hidden   [T,H] output in hidden_dtype, or NULL: not wanted.
 *   d_W        [E,H] FP32 output, or NULL: not wanted.
 *   workspace  at least moe_route_backward_workspace_bytes(T, H, E,
 *              hidden_dtype, logits_in) bytes, 256-byte aligned (may be NULL
 *              when that is 0: logits-in mode, or too few tokens to need any).
 * Errors: NULL_ARG, BAD_SHAPE, BAD_DTYPE, BAD_ARG (non-finite scale), ALIGN,
 * WORKSPACE, HIP.
 */
size_t moe_route_backward_workspace_bytes(int T, int H, int E, int hidden_dtype, int logits_in);

int moe_route_backward(const float* d_topk_w, const float* d_aux, const void* hidden, int hidden_dtype,
                       const float* W, const float* logits, const int32_t* topk_ids, const float* topk_w,
                       const uint8_t* token_mask, float scale, int T, int H, int E, int k,
                       float* d_logits, void* d_hidden, float* d_W,
                       void* workspace, size_t workspace_bytes, void* stream);

/*
 * moe_combine_backward — gradients of moe_combine.
 *
 * The roundings to BF16 inside moe_combine count as the identity. For slot
 * (t,j) with r = slots[t,j] in [0,R), x = expert_out[r,:], g = gain_center +
 * norm_w, rstd = 1 / sqrt(mean(x^2) + eps) and A = sum_i d_out[t,i] g_i x_i:
 *   d_topk_w[t,j]     = rstd A                      (0 for an invalid slot)
 *   d_expert_out[r,i] = w rstd (g_i d_out[t,i] - x_i rstd^2 A / H)
 *   d_norm_w[i]       = sum_{t,j} w rstd x_i d_out[t,i]
 * A row named by several slots gets the sum of their gradients; a row that no
 * slot names gets zeros and is never read. moe_dispatch names every row once,
 * and the call is made for that: each row named more than once costs a scan of
 * all slots by one wave. d_out and topk_w of a token whose slots are all
 * invalid may hold anything.
 *
 *   d_out [T,H] BF16 bits; expert_out [R,H] BF16 bits (may be NULL only if R ==
 *   0); slots [T,k] int32; topk_w [T,k] FP32; norm_w [H] FP32; ranges as in
 *   moe_combine.
 *   d_expert_out [R,H] BF16 bits, d_topk_w [T,k] FP32, d_norm_w [H] FP32 or
 *   NULL (not wanted): outputs.
 *   workspace  at least moe_combine_backward_workspace_bytes(T, R, H) bytes.
 * Errors: NULL_ARG, BAD_SHAPE, BAD_ARG, ALIGN, WORKSPACE, HIP.
 */
size_t moe_combine_backward_workspace_bytes(int T, int R, int H);

int moe_combine_backward(const uint16_t* d_out, const uint16_t* expert_out, int R, const int32_t* slots,
                         const float* topk_w, const float* norm_w, float gain_center, float eps,
                         int T, int H, int k, uint16_t* d_expert_out, float* d_topk_w, float* d_norm_w,
                         void* workspace, size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_TRAINING_H */
