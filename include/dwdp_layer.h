/*
 * dwdp_layer.h -- C ABI of what stands around the MoE block of dwdp.h in a pre-norm layer:
 *
 *   dwdp_route_gate            router GEMM and a model's gate: softmax or sigmoid scores, a balance
 *                              bias, group-limited top-k, (renormalised) scaled weights
 *   dwdp_gate_topk             the gate alone, from logits
 *   dwdp_add_rmsnorm           residual addition and RMS norm of the block's input, in the layer's
 *                              activation type and / or as E4M3 codes with 1x128 scales
 *   dwdp_combine_add_rmsnorm   the boundary between two layers: the block's weighted unpermute and
 *                              shared expert, the residual addition, and the next layer's norm
 *   dwdp_branch_add_rmsnorm, dwdp_combine_branch_add_rmsnorm
 *                              the same two for layers whose blocks end in a norm of their own, a gate
 *                              and a scale; int8 codes too
 *   dwdp_quantize_int8         rows (tokens, or weights by channel) as int8 codes with one scale each
 *   dwdp_balance_loss          per-expert counts, the balance loss and the z loss of each sequence
 *   dwdp_gate_backward         the logits' gradient of a gate's weights and of both losses
 *
 * They take the place of, or feed, the entry points of dwdp.h: route_gate writes the topk_idx and
 * topk_w that dwdp_permute and dwdp_combine read, the norms write the tokens (and, for fp8, the codes
 * and scales of dwdp_quantize_tokens_fp8) that dwdp_moe_grouped_ffn_tokens reads, and
 * combine_add_rmsnorm replaces dwdp_combine.  dwdp.h's conventions (ownership, streams, errors,
 * determinism, T == 0) hold here too; every matrix is dense and row-major.
 */
#ifndef DWDP_LAYER_H_
#define DWDP_LAYER_H_

#include "dwdp.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    DWDP_SCORE_SOFTMAX = 0,
    DWDP_SCORE_SIGMOID = 1
} dwdp_score;

/* A model's gate.  For the logits l of one token over E experts:
 *   scores   s_e = softmax(l)_e, or sigmoid(l_e) each by itself
 *   choice   c_e = s_e + balance_bias[e] (the bias steers the choice only, never the weights)
 *   groups   the experts are n_groups runs of E / n_groups; a group's value is the sum of its
 *            group_top largest choices (of its largest alone if group_top is 1), and only the experts
 *            of the topk_groups groups of largest value stay.  n_groups 1: no groups.
 *   top-k    the k largest choices, in slot order from the largest down
 *   weights  w_j = s of slot j's expert, divided by the sum over the chosen if renormalize, times scale
 * Equal choices go to the lower expert, equal groups to the lower group.
 * Choices are compared as if computed in fp64 from the fp32 logits (without a balance bias scores are
 * ordered as their logits, which is the same order); weights are fp32.
 * Experts that cannot be chosen: a logit of NaN or -inf, or a balance bias of NaN or -inf (an expert
 * out of service; its logit still counts in the softmax).  They add nothing to their group's value, and
 * a group of none other is kept last.  A NaN or -inf logit has score 0.  Logits of +inf share the whole
 * softmax.  A slot for which no expert is left holds index -1 and weight 0 (dwdp_permute drops it, and
 * dwdp_combine skips it); renormalised weights are those of the limit, so they sum to `scale` even where
 * every chosen score underflows.
 * 1 <= E <= 1024; 1 <= k <= min(E, 32); n_groups divides E; 1 <= topk_groups <= n_groups;
 * k <= topk_groups * E / n_groups; group_top 1 or 2; scale finite. */
typedef struct {
    int32_t score;              /* dwdp_score */
    int32_t k;
    int32_t n_groups;
    int32_t topk_groups;
    int32_t group_top;
    int32_t renormalize;        /* 0 or 1 */
    float scale;
} dwdp_gate;

/* Router: logits = x * w_router^T + bias as in dwdp_route_topk (fp32 accumulation), then the gate.
 *   x [T,H], w_router [E,H]: DWDP_F32 or DWDP_BF16 (in_dtype), 16-byte aligned.
 *   bias [E] fp32 or NULL (part of the logits); balance_bias [E] fp32 or NULL.
 *   H % 64 == 0 (bf16) or H % 16 == 0 (f32).  `gate` is host memory, read during the call.
 *   logits_out [T,E] fp32 (written, bias included), topk_idx [T,k] int32, topk_w [T,k] fp32.
 *   ws: dwdp_route_gate_workspace_bytes(...) bytes of device scratch, 16-byte aligned (NULL if 0); its
 *   contents need no preparation and mean nothing after the call.  Calls that may run at the same time
 *   need a workspace each.  The size is that of exactly these T, H, E and in_dtype, whatever the gate: a larger T
 *   may need less, or none.  It is never more than DWDP_ROUTE_GATE_WORKSPACE_MAX, and a larger ws is taken, so one
 *   buffer of that size serves every batch of a stream.
 *   No output, nor ws, may overlap another buffer.  T is limited by one launch of the product: more than 10^8
 *   tokens of 256 experts (f32 with H % 32 != 0: 8 * 10^6); larger batches are refused. */
int dwdp_route_gate(const void* x, const void* w_router, int in_dtype, const float* bias,
                    const float* balance_bias, int64_t T, int H, int E, const dwdp_gate* gate,
                    float* logits_out, int32_t* topk_idx, float* topk_w, void* ws, size_t ws_bytes,
                    void* stream);

/* Device scratch dwdp_route_gate needs (0 where it needs none, and for arguments it rejects). */
#define DWDP_ROUTE_GATE_WORKSPACE_MAX ((size_t)32 << 20)
size_t dwdp_route_gate_workspace_bytes(int64_t T, int H, int E, int in_dtype);

/* The gate alone: logits [T,E] fp32 -> topk_idx [T,k], topk_w [T,k], neither of which may overlap another buffer. */
int dwdp_gate_topk(const float* logits, const float* balance_bias, int64_t T, int E, const dwdp_gate* gate,
                   int32_t* topk_idx, float* topk_w, void* stream);

/* Residual addition and RMS norm, row by row:
 *   z = x + residual (x alone where residual is NULL), in fp32
 *   sum_out = z rounded to dtype                                   (NULL: not written)
 *   n = z / sqrt(mean(z^2) + eps) * weight, in fp32 from the unrounded z
 *   y = n rounded to dtype                                         (NULL: not written)
 *   q, q_scale = n quantised like dwdp_quantize_tokens_fp8 quantises a row, from the unrounded n: per
 *   128 columns scale = amax/448 (1 when amax is 0, 2^-126 where amax/448 is less), code = E4M3(n/scale)
 *   (NULL, both: not written)
 * At least one of y and q is given.  Non-finite values follow IEEE arithmetic; a NaN in a 128-column
 * group makes its scale and its codes NaN.  The sum of z^2 has fp32's range: rows whose sum of squares passes
 * 3.4e38 norm to zero, and with eps 0 a row whose squares all underflow norms to infinities and NaN.
 *   x, residual, sum_out, y [T,H] of dtype (DWDP_F32 or DWDP_BF16); weight [H] of w_dtype (DWDP_F32 or
 *   DWDP_BF16).  Any H >= 1 and any element-aligned pointers; rows are read fastest where
 *   H % 8 == 0 and all pointers are 16-byte aligned.  q [T,H] (8-byte aligned) with q_scale [T,H/128]
 *   fp32 needs dtype DWDP_BF16, H % 128 == 0 and 16-byte aligned x, residual, weight, sum_out and y.
 *   eps >= 0, finite.
 *   In place: sum_out and y may each be x or residual (the same address), but not each other; other
 *   overlaps of an output with any buffer are refused. */
int dwdp_add_rmsnorm(const void* x, const void* residual, int dtype, const void* weight, int w_dtype, float eps,
                     int64_t T, int H, void* sum_out, void* y, void* q, float* q_scale, void* stream);

/* The boundary between two layers: dwdp_combine's sum, the residual, and the next layer's norm.
 *   z[t] = sum_{j<k} topk_w[t,j] * y_perm[inv_perm[t,j]] (+ y_perm[T*k + t] when shared) + residual[t]
 * summed in fp32 in that order (residual NULL: none), then sum_out, y, q and q_scale from z as in
 * dwdp_add_rmsnorm.  Slots with inv_perm < 0 or >= T*k + shared*T contribute nothing.  Without y and q
 * (the last layer of a model) only sum_out is written and weight may be NULL; at least one of sum_out,
 * y and q is given.
 *   T >= 0, T*(k + shared) < 2^31, 1 <= k <= 64, H % 8 == 0 (H % 128 == 0 and DWDP_BF16 with q); y_perm [T*k + shared*T, H],
 *   residual, sum_out, y [T,H] of dtype, weight [H] of w_dtype, all 16-byte aligned (q: 8-byte).
 *   In place: sum_out or y may be residual (the same address); other overlaps of an output with any buffer
 *   are refused. */
int dwdp_combine_add_rmsnorm(const void* y_perm, const int32_t* inv_perm, const float* topk_w, int64_t T, int k,
                             int shared, int H, int dtype, const void* residual, const void* weight, int w_dtype,
                             float eps, void* sum_out, void* y, void* q, float* q_scale, void* stream);

/* What a layer makes of its block's output u before the residual addition:
 *   n[c] = u[c] / sqrt(mean(u^2) + eps) * norm[c]        (u[c] where norm is NULL)
 *   z[c] = residual_scale * residual[c] + scale * token_gate[t] * gate[c] * n[c]
 * in fp32.  gate NULL: 1 for every channel; token_gate (an argument of the calls, since it belongs to a
 * batch) NULL: 1 for every token; residual NULL: none.  norm [H] of norm_dtype and gate [H] of gate_dtype
 * are DWDP_F32 or DWDP_BF16 device arrays; eps >= 0; eps, scale and residual_scale finite. */
typedef struct {
    const void* norm;
    const void* gate;
    int32_t norm_dtype;
    int32_t gate_dtype;
    float eps;
    float scale;
    float residual_scale;
} dwdp_branch;

/* dwdp_add_rmsnorm with a branch: u = x, z as above, then sum_out, y and codes from z as there.
 *   branch: host memory, read during the call; NULL is a branch without norm and gate whose scales are 1.
 *   token_gate [T] fp32 or NULL.
 *   q [T,H] (8-byte aligned) with q_scale, of q_dtype (ignored without q):
 *     DWDP_FP8_E4M3  as in dwdp_add_rmsnorm: q_scale [T,H/128], dtype DWDP_BF16, H % 128 == 0
 *     DWDP_INT8      as dwdp_quantize_int8 quantises a row, from the unrounded norm: q_scale [T], any
 *                    dtype, H % 8 == 0
 *     both need 16-byte aligned x, residual, weight, sum_out, y, norm and gate.
 *   Without y and q only sum_out is written and weight may be NULL; at least one of them is given.
 *   Other sizes, types, alignments, and what may be in place: as in dwdp_add_rmsnorm. */
int dwdp_branch_add_rmsnorm(const void* x, const void* residual, int dtype, const dwdp_branch* branch,
                            const float* token_gate, const void* weight, int w_dtype, float eps, int64_t T, int H,
                            void* sum_out, void* y, void* q, int q_dtype, float* q_scale, void* stream);

/* dwdp_combine_add_rmsnorm with a branch: u[t] = sum_{j<k} topk_w[t,j] * y_perm[inv_perm[t,j]]
 * (+ y_perm[T*k + t] when shared) in fp32 in that order, z as above, then the outputs from z.
 * branch, token_gate, q, q_dtype and q_scale as in dwdp_branch_add_rmsnorm (norm and gate 16-byte aligned);
 * everything else as in dwdp_combine_add_rmsnorm. */
int dwdp_combine_branch_add_rmsnorm(const void* y_perm, const int32_t* inv_perm, const float* topk_w, int64_t T, int k,
                                    int shared, int H, int dtype, const void* residual, const dwdp_branch* branch,
                                    const float* token_gate, const void* weight, int w_dtype, float eps, void* sum_out,
                                    void* y, void* q, int q_dtype, float* q_scale, void* stream);

/* Rows of x [rows, cols] (DWDP_F32 or DWDP_BF16) as int8 codes with one fp32 scale each: tokens for the
 * grouped FFN's DWDP_INT8 path, or a weight matrix [out, in] by output channel.
 *   scale = amax/127 (1 when amax is 0, 2^-126 where amax/127 is less), code = value/scale rounded to
 *   nearest even, in [-127, 127].  A row with an infinity or a NaN has the scale NaN and codes 0.
 *   x 16-byte aligned, q [rows, cols] 8-byte aligned, scale [rows]; cols % 8 == 0; rows < 2^31.  No output
 *   may overlap another buffer. */
int dwdp_quantize_int8(const void* x, int dtype, int64_t rows, int cols, void* q, float* scale, void* stream);

/* How evenly a batch's sequences load the experts, from the gate's logits [T,E] and choice topk_idx [T,k].
 * Sequence s holds the N_s tokens [seq_offsets[s], seq_offsets[s+1]).  Over them
 *   p        softmax(l), or for DWDP_SCORE_SIGMOID sigmoid(l) divided by its sum over the experts
 *   counts   counts[s,e] = how many (token, slot) chose expert e
 *   probs    probs[s,e] = mean of p[e]
 *   balance  balance[s] = sum_e f_e * probs[s,e],  f_e = counts[s,e] * E / (k * N_s); 1 for an even load
 *   z        z[s] = mean of logsumexp(l)^2                                     (NULL: not written)
 * in fp32 (logits of NaN or -inf have p = 0; a token of none other adds nothing; a logit of +inf shares
 * p with its like and makes z infinite).  Entries of topk_idx outside [0, E) are not counted.  An empty
 * sequence has zeros.  Losses of a whole batch, e.g. their mean, are the caller's to form.
 *   seq_offsets [S+1] int32, device memory, ascending from >= 0 to <= T; tokens outside belong to no
 *   sequence.  NULL: one sequence of all T tokens (S = 1).  Descending offsets give undefined values.
 *   1 <= E <= 1024, 1 <= k <= min(E, 32), 1 <= S <= 2^20, T * k < 2^31.  T == 0 writes zeros.
 *   counts [S,E] int32, probs [S,E], balance [S], z [S] fp32.
 *   ws: dwdp_balance_loss_workspace_bytes(T, E, S) bytes of device scratch, 16-byte aligned; its contents
 *   need no preparation.  Calls that may run at the same time need a workspace each.  A larger one, e.g.
 *   that of a larger T, E or S, is taken.  No output, nor ws, may overlap another buffer. */
int dwdp_balance_loss(const float* logits, const int32_t* topk_idx, int64_t T, int E, int k, int score,
                      const int32_t* seq_offsets, int S, int32_t* counts, float* probs, float* balance, float* z,
                      void* ws, size_t ws_bytes, void* stream);

/* Device scratch of dwdp_balance_loss (0 for arguments it rejects); it grows with each of T, E and S. */
size_t dwdp_balance_loss_workspace_bytes(int64_t T, int E, int S);

/* The gradient with respect to the logits of
 *   sum_tj d_w[t,j] * topk_w[t,j]  +  sum_s d_balance[s] * balance[s]  +  sum_s d_z[s] * z[s]
 * with topk_w the gate's weights of the choice topk_idx (dwdp_gate_topk; score, k, renormalize and scale of
 * `gate`), and balance and z as in dwdp_balance_loss.  The choice itself, and so counts, is constant.  Per
 * token, with sg_i = sigmoid(l_i), h_i = 1 - sg_i for DWDP_SCORE_SIGMOID and 1 for DWDP_SCORE_SOFTMAX:
 *   balance   d_balance/N_s * p_i h_i (f_i - sum_e f_e p_e)
 *   z         d_z/N_s * 2 logsumexp(l) softmax(l)_i
 *   weights   renormalised, a_j = score_j / sum over the chosen: to the logit of slot j's expert
 *                 scale a_j h_j (d_w_j - sum_m d_w_m a_m)
 *             not renormalised: scale d_w_j score_j h_j to the logit of slot j's expert; for softmax also
 *                 - softmax(l)_i sum_j scale d_w_j score_j to every logit
 * An expert that several slots of a token name takes the sum of theirs.  Slots outside [0, E) and logits of
 * NaN or -inf take no part and get 0; a logit of +inf makes the z loss's gradient of its token (d_z not 0) NaN.
 *   d_w [T,k], d_balance [S], d_z [S] fp32, each NULL if there is none of it (not all three).
 *   counts [S,E]: dwdp_balance_loss's (needed with d_balance).  seq_offsets, S: as there; tokens of no
 *   sequence get the gradient of their weights alone.  d_logits [T,E] fp32 (written, not added to).
 *   Limits of T, E, k and S as there, but T == 0 is a no-op; d_logits may overlap no other buffer. */
int dwdp_gate_backward(const float* logits, const int32_t* topk_idx, int64_t T, int E, const dwdp_gate* gate,
                       const float* d_w, const int32_t* seq_offsets, int S, const int32_t* counts,
                       const float* d_balance, const float* d_z, float* d_logits, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* DWDP_LAYER_H_ */
