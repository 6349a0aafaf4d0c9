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

#ifdef __cplusplus
}
#endif

#endif /* DWDP_LAYER_H_ */
