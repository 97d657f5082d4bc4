/*
 * moe_block.h - C ABI of the operators around the expert layer of moe.h, for GB300 (sm_103a):
 *
 *     moe_add_rmsnorm  ->  (gate product)  ->  moe_route_topk  ->  moe_dispatch ... moe_combine
 *                                                              or  moe_forward_w4
 *
 * The layer takes rows, expert ids and routing weights; these calls make the rows (residual
 * addition and root-mean-square norm, bf16 and e4m3) and the ids and weights (router), and
 * compute the routed experts of a small batch from 4-bit weights.  The first two have their
 * gradients here too.
 *
 * The conventions of moe.h hold: *_dev pointers are device pointers of the current device,
 * the caller owns all memory, calls are stream-ordered and asynchronous, the return value is
 * MOE_OK or a negative moe_error, and host-detected errors return before anything is queued.
 * Rows are bf16 unless a dtype says otherwise; strides count elements, and 0 means packed.
 */
#ifndef COMBINE_TOPK_IDS_MOE_BLOCK_H
#define COMBINE_TOPK_IDS_MOE_BLOCK_H

#include "moe.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum { MOE_DTYPE_BF16 = 0, MOE_DTYPE_FP32 = 1 } moe_dtype;

/* ---- residual addition and RMS norm ---------------------------------------------------- */

typedef struct {
    int32_t num_tokens, hidden;
    int32_t residual_dtype; /* moe_dtype of residual and sum (backward: of h, dsum and dx)  */
    int32_t weight_dtype;   /* moe_dtype of weight                                          */
    float eps;
    int64_t x_stride, residual_stride, sum_stride, out_stride; /* row strides in elements   */
} moe_norm;

/*
 * moe_add_rmsnorm - for every row t:
 *     h = x + residual;  rstd = 1 / sqrt(mean(h^2) + eps);  y = h * rstd * weight
 *   x_dev            bf16 [num_tokens, hidden]
 *   residual_dev     NULL: h = x
 *   weight_dev       [hidden]
 *   sum_dev          h (the residual stream of the next block), rounded to residual_dtype;
 *                    NULL: not written.  May be residual_dev (with the same stride).
 *   out_dev          bf16 y, or NULL.  May be x_dev (with the same stride).
 *   out_fp8_dev, scales_dev   e4m3 codes of y [num_tokens, hidden] (packed) with one float32
 *                    scale per 128 columns [num_tokens, hidden / 128], by the rule of
 *                    MOE_QUANT_FP8_E4M3, or both NULL.  moe_dispatch_fp8 takes them as they are.
 *   rstd_dev         float32 [num_tokens] for the gradient, or NULL
 *   All sums are float32; y is rounded once, from float32, for each output.
 *   Errors: MOE_ERR_INVALID_ARGUMENT (a NULL x or weight, no output, codes without scales, a
 *   stride below hidden, a bad dtype, eps below 0 or not a number), MOE_ERR_HIDDEN_ALIGNMENT
 *   (codes with hidden % 128 != 0), MOE_ERR_LIMIT (hidden above MOE_MAX_HIDDEN),
 *   MOE_ERR_MISALIGNED (an array off its element's alignment, codes off 16 bytes).
 */
int moe_add_rmsnorm(const moe_norm *n, const void *x_dev, const void *residual_dev, const void *weight_dev,
                    void *sum_dev, void *out_dev, void *out_fp8_dev, float *scales_dev, float *rstd_dev,
                    void *stream);

/*
 * moe_add_rmsnorm_backward - with g = dout * weight and xhat = h * rstd:
 *     dx = rstd * (g - xhat * mean(g * xhat)) + dsum;   dweight = sum over rows of dout * xhat
 *   dx is the gradient of x and of residual alike (both enter h).
 *   dout_dev bf16 (stride x_stride), h_dev the forward's sum (residual_stride), dsum_dev the
 *   gradient that reaches h from the residual stream or NULL (sum_stride), dx_dev
 *   (out_stride; may be dsum_dev with the same stride); h, dsum and dx are of residual_dtype.
 *   rstd_dev float32 [num_tokens]; dweight_dev float32 [hidden].
 *   workspace_dev holds the row blocks' partial sums of dweight; they are added in a fixed
 *   order, so equal inputs give equal bits.
 *   Errors as moe_add_rmsnorm, and MOE_ERR_WORKSPACE_TOO_SMALL.
 */
int moe_add_rmsnorm_workspace_size(const moe_norm *n, size_t *bytes);
int moe_add_rmsnorm_backward(const moe_norm *n, const void *dout_dev, const void *h_dev, const void *weight_dev,
                             const float *rstd_dev, const void *dsum_dev, void *dx_dev, float *dweight_dev,
                             void *workspace_dev, size_t workspace_bytes, void *stream);

/*
 * moe_dispatch_fp8 - moe_dispatch for an FP8 geometry (MOE_QUANT_FP8_E4M3) and rows that are
 *   quantised already: x_codes_dev [num_tokens, hidden] and x_scales_dev [num_tokens,
 *   hidden / 128], as moe_add_rmsnorm writes them.  They are copied as they are; everything
 *   else, the handle among it, is as after moe_dispatch.
 *   Errors: those of moe_dispatch, and MOE_ERR_INVALID_ARGUMENT for a bf16 geometry or NULL scales.
 */
int moe_dispatch_fp8(const moe_geom *g, const uint8_t *x_codes_dev, const float *x_scales_dev,
                     const void *topk_ids_dev, int ids_dtype, const float *topk_weights_dev,
                     const int32_t *active_ranks_dev, void *workspace_dev, size_t workspace_bytes,
                     moe_handle *handle, void *stream);

/* ---- router ----------------------------------------------------------------------------- */

typedef enum { MOE_SCORE_SOFTMAX = 0, MOE_SCORE_SIGMOID = 1 } moe_score;
typedef enum { MOE_GROUP_MAX = 0, MOE_GROUP_TOP2 = 1 } moe_group_score;

#define MOE_MAX_GROUPS 32

typedef struct {
    int32_t num_experts, top_k;
    int32_t score;        /* moe_score                                                      */
    int32_t groups;       /* equal runs of experts (1: none)                                */
    int32_t top_groups;   /* groups whose experts may be picked                             */
    int32_t group_score;  /* moe_group_score: a group's largest key, or its two largest, added */
    int32_t renormalize;  /* divide the picked scores by their sum                          */
    int32_t logits_dtype; /* moe_dtype of logits (backward: and of dlogits)                 */
    float scale;          /* factor of every routing weight                                 */
    int64_t logits_stride;/* row stride in elements                                         */
} moe_router;

/*
 * moe_route_topk - expert ids and routing weights from the gate's logits, for every token:
 *     s_e = softmax(logits)_e or 1 / (1 + exp(-logit_e));   key_e = s_e + bias_e
 *     keep the top_groups best groups; pick the top_k largest keys in them;
 *     weight_j = scale * s_{e_j} / (renormalize ? sum of the picked s : 1)
 *   bias_dev  float32 [num_experts], for the picking alone (load balance), or NULL.
 *   Without a bias, and without groups or with MOE_GROUP_MAX, the experts are picked by their
 *   logits (both scores rise with the logit).  Picks are in falling order of their keys; equal
 *   keys go to the lowest index, equal groups to the lowest group.
 *   An expert whose logit is -infinity or not a number is absent: it has score 0 and is never
 *   picked.  One whose bias is -infinity or not a number is never picked either; its logit still
 *   counts in a softmax's sum.  Picks that find no expert get id -1 and weight 0, which moe_dispatch
 *   and moe_forward_w4 skip.  Where the picked scores' sum is 0 the weights are 0 (scores are
 *   float32: one below 2^-126, of a softmax before its division, counts as 0).  A score's relative
 *   error is at most (1.2 |v| + 48) 2^-23, v the logit (sigmoid) or how far it lies below the row's
 *   largest (softmax).
 *   topk_ids_dev int32 or int64 [num_tokens, top_k]; topk_weights_dev float32.
 *   Errors: MOE_ERR_INVALID_ARGUMENT (NULL, a bad enum, a stride below num_experts, groups
 *   that do not divide num_experts, top_groups outside [1, groups]), MOE_ERR_TOPK (top_k
 *   outside [1, min(MOE_MAX_TOPK, the kept groups' experts)]), MOE_ERR_LIMIT (num_experts
 *   above MOE_MAX_EXPERTS, groups above MOE_MAX_GROUPS), MOE_ERR_IDS_DTYPE,
 *   MOE_ERR_MISALIGNED.
 */
int moe_route_topk(const moe_router *r, int32_t num_tokens, const void *logits_dev, const float *bias_dev,
                   void *topk_ids_dev, int ids_dtype, float *topk_weights_dev, void *stream);

/*
 * moe_route_topk_backward - dlogits [num_tokens, num_experts] (packed, of logits_dtype) from
 *   dweights float32 [num_tokens, top_k]: the gradient of topk_weights in the logits with the
 *   picks held fixed.  Every element is written.  Picks of id -1 (and ids outside
 *   [0, num_experts), and absent experts) take no part; the bias has no gradient.
 */
int moe_route_topk_backward(const moe_router *r, int32_t num_tokens, const void *logits_dev,
                            const void *topk_ids_dev, int ids_dtype, const float *dweights_dev,
                            void *dlogits_dev, void *stream);

/* ---- routed experts with 4-bit weights ---------------------------------------------------- */

/*
 * A weight matrix [rows, cols] is held as codes uint8 [rows, cols / 2] (the even column in the
 * low four bits) and bf16 scales [rows, cols / group]: weight = (code - 8) * scale.
 */
typedef struct {
    int32_t num_tokens, hidden, num_experts, top_k, intermediate;
    int32_t group;          /* 32, 64 or 128 inputs per scale                               */
} moe_w4_geom;

/*
 * moe_quantize_w4 - bf16 [rows, cols] to codes and scales: scale = bf16(amax / 7) over each
 *   group, code = 8 + clamp(rint(w / scale), -8, 7); a group of zeros gets scale 0, code 8.
 *   A group with an infinity or NaN among its weights gets scale NaN, code 8: its weights are NaN.
 *   cols % group == 0, rows * cols < 2^62.
 */
int moe_quantize_w4(int64_t rows, int64_t cols, int32_t group, const void *w_dev, uint8_t *codes_dev,
                    void *scales_dev, void *stream);

/*
 * moe_prepare_weights_w4 - one-time order of codes and scales for moe_forward_w4.
 *   w1 [num_experts, 2 * intermediate, hidden] (gate rows, then up rows) and
 *   w2 [num_experts, hidden, intermediate], as codes and scales; the prepared arrays have the
 *   same sizes and may not overlap the given ones.  num_tokens and top_k play no part.
 */
int moe_prepare_weights_w4(const moe_w4_geom *g, const uint8_t *w1_codes_dev, const void *w1_scales_dev,
                           const uint8_t *w2_codes_dev, const void *w2_scales_dev, uint8_t *w1_prepared_dev,
                           void *w1_scales_prepared_dev, uint8_t *w2_prepared_dev, void *w2_scales_prepared_dev,
                           void *stream);

/*
 * moe_forward_w4 - the routed experts' SwiGLU FFN of a decode batch:
 *     out[t] = sum over picks j of topk_weights[t, j] * W2_e (silu(Wg_e x[t]) * (Wu_e x[t]))
 *   The same function as moe_dispatch -> moe_expert_ffn -> moe_combine, for batches with few
 *   rows for each expert, whose time is that of reading the picked experts' weights.  Weights
 *   enter the products exactly (integers, scaled in float32), and so does x where the values of
 *   each aligned run of 64 lie within 2^32 of each other (smaller ones to 2^-39 of the run's largest);
 *   the activation is rounded to the eleven bits of f16 (with a power of two for each 64 values
 *   of a row, so that its size does not matter), where moe_expert_ffn's default holds a pair of
 *   bf16; sums are float32; out is rounded once.  An infinity in a row of x makes the token's
 *   out not a number.
 *   x_dev, out_dev bf16 [num_tokens, hidden]; topk_ids_dev [num_tokens, top_k]: -1 is a masked
 *   pick, an id outside [-1, num_experts) is dropped and sets MOE_STATUS_BAD_EXPERT_ID.
 *   status_dev: one int32, written by the call (0: clean).  workspace_dev: 256-byte aligned.
 *   Errors: those of moe_workspace_size's geometry, MOE_ERR_INVALID_ARGUMENT (group, NULL),
 *   MOE_ERR_IDS_DTYPE, MOE_ERR_MISALIGNED, MOE_ERR_WORKSPACE_TOO_SMALL.
 */
int moe_forward_w4_workspace_size(const moe_w4_geom *g, size_t *bytes);
int moe_forward_w4(const moe_w4_geom *g, const void *x_dev, const void *topk_ids_dev, int ids_dtype,
                   const float *topk_weights_dev, const uint8_t *w1_prepared_dev,
                   const void *w1_scales_prepared_dev, const uint8_t *w2_prepared_dev,
                   const void *w2_scales_prepared_dev, void *out_dev, int32_t *status_dev,
                   void *workspace_dev, size_t workspace_bytes, void *stream);

#ifdef __cplusplus
}
#endif
#endif /* COMBINE_TOPK_IDS_MOE_BLOCK_H */
