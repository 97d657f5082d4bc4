/*
 * moe_grouped.h - C ABI of the operators on expert-grouped rows, for GB300 (sm_103a):
 *
 *     moe_sort_picks, moe_sort_rows  ->  moe_product_fp8  ->  moe_swiglu_fp8  ->  moe_product_fp8
 *                                    ->  moe_unsort_rows
 *
 * moe.h runs the whole expert layer in its own receive layouts; these calls give its steps to a
 * caller who computes on the experts' rows: the rows packed in expert order and back (with their
 * gradients, the routing weights' among them, which moe_route_topk_backward takes), and the FP8
 * products and quantisations between.  A product with one weight matrix serves what stands beside
 * the routed experts: the shared expert and dense layers, on the e4m3 rows that moe_add_rmsnorm
 * writes.
 *
 * The conventions of moe.h hold: *_dev pointers are device pointers of the current device, the
 * caller owns all memory, calls are stream-ordered and asynchronous, the return value is MOE_OK or
 * a negative moe_error, and host-detected errors return before anything is queued.  Strides count
 * elements, and 0 means packed.  e4m3 codes and scales follow the rule of MOE_QUANT_FP8_E4M3.
 */
#ifndef COMBINE_TOPK_IDS_MOE_GROUPED_H
#define COMBINE_TOPK_IDS_MOE_GROUPED_H

#include "moe_block.h"

#ifdef __cplusplus
extern "C" {
#endif

#define MOE_DTYPE_E4M3 2 /* beside moe_dtype: e4m3 codes with one float32 scale per 128 columns */

/* ---- rows in expert order and back ------------------------------------------------------- */

typedef struct {
    int32_t num_tokens, num_experts, top_k;
} moe_sort;

/*
 * moe_sort_picks - the order of a batch's picks (t, j) by (expert, token, pick):
 *   topk_ids_dev  int32 or int64 [num_tokens, top_k]; -1 is a masked pick, an id outside
 *                 [-1, num_experts) is dropped and sets MOE_STATUS_BAD_EXPERT_ID.  A token may name
 *                 an expert more than once.
 *   offsets_dev   int32 [num_experts + 1]: expert e has the rows [offsets[e], offsets[e + 1])
 *   position_dev  int32 [num_tokens, top_k]: the pick's row, or -1
 *   source_dev    int32 [num_tokens * top_k]: t * top_k + j of each row, -1 behind the last one;
 *                 or NULL
 *   status_dev    one int32, written by the call (0: clean), or NULL
 *   workspace_dev 16-byte aligned
 * Positions follow from counts alone: equal inputs give equal outputs.
 * Errors: MOE_ERR_INVALID_ARGUMENT (NULL, a negative size), MOE_ERR_TOPK (top_k outside
 * [1, MOE_MAX_TOPK]), MOE_ERR_LIMIT (num_experts above MOE_MAX_EXPERTS, num_tokens * top_k above
 * 2^31 - 1024), MOE_ERR_IDS_DTYPE, MOE_ERR_MISALIGNED, MOE_ERR_WORKSPACE_TOO_SMALL.
 */
int moe_sort_picks_workspace_size(const moe_sort *g, size_t *bytes);
int moe_sort_picks(const moe_sort *g, const void *topk_ids_dev, int ids_dtype, int32_t *offsets_dev,
                   int32_t *position_dev, int32_t *source_dev, int32_t *status_dev, void *workspace_dev,
                   size_t workspace_bytes, void *stream);

typedef struct {
    int32_t num_tokens, top_k, hidden;
    int32_t num_rows;       /* rows that the sorted matrices have: num_tokens * top_k holds any batch */
    int32_t rows_dtype;     /* of the sorted rows (and, in moe_sort_rows, of x)                   */
    int32_t tokens_dtype;   /* of out and dout (moe_sort_rows: unused)                            */
    int64_t rows_stride, drows_stride, tokens_stride; /* row strides in elements                  */
} moe_rows;

/*
 * For all four calls: position_dev int32 [num_tokens, top_k] as moe_sort_picks writes it; a pick
 * whose position is outside [0, num_rows) takes no part.  No two picks share a position.  Rows that
 * no pick has are neither read nor written.  The matrices do not overlap.
 *
 * moe_sort_rows - rows[position[t, j]] = x[t]; with MOE_DTYPE_E4M3 codes (packed, 16-byte aligned,
 *   hidden % 128 == 0) and scales [.., hidden / 128] alike.  x has tokens_stride.
 * moe_sort_rows_backward - dx[t] = sum over j of drows[position[t, j]], of bf16 or float32 rows:
 *   moe_unsort_rows without weights.
 * moe_unsort_rows - out[t] = sum over j ascending of weights[t, j] * rows[position[t, j]], float32
 *   sums, rounded once; weights_dev float32 [num_tokens, top_k] or NULL (all 1).  A token without
 *   picks gets zeros.  A masked pick's weight does not matter.
 * moe_unsort_rows_backward - drows[position[t, j]] = weights[t, j] * dout[t] and
 *   dweights[t, j] = <dout[t], rows[position[t, j]]>, 0 for masked picks; drows (of rows_dtype,
 *   drows_stride) or dweights (float32 [num_tokens, top_k]) may be NULL, and so may rows without
 *   dweights and weights (then 1).
 * Errors: MOE_ERR_INVALID_ARGUMENT (NULL, a negative size, a bad dtype, a stride below hidden),
 * MOE_ERR_TOPK, MOE_ERR_LIMIT (hidden above MOE_MAX_HIDDEN), MOE_ERR_HIDDEN_ALIGNMENT (codes with
 * hidden % 128 != 0), MOE_ERR_MISALIGNED.
 */
int moe_sort_rows(const moe_rows *g, const void *x_dev, const float *x_scales_dev, const int32_t *position_dev,
                  void *rows_dev, float *rows_scales_dev, void *stream);
int moe_sort_rows_backward(const moe_rows *g, const void *drows_dev, const int32_t *position_dev, void *dx_dev,
                           void *stream);
int moe_unsort_rows(const moe_rows *g, const void *rows_dev, const float *weights_dev, const int32_t *position_dev,
                    void *out_dev, void *stream);
int moe_unsort_rows_backward(const moe_rows *g, const void *dout_dev, const void *rows_dev,
                             const float *weights_dev, const int32_t *position_dev, void *drows_dev,
                             float *dweights_dev, void *stream);

/* ---- quantisation ------------------------------------------------------------------------- */

typedef struct {
    int32_t matrices;       /* of num_rows rows each, one behind the other                       */
    int32_t num_rows, cols; /* cols: of the codes, a multiple of 128                             */
    int32_t block_rows;     /* rows of a matrix that share a scale: 1, or 128 (weights)          */
    int32_t x_dtype;        /* moe_dtype                                                          */
    int64_t x_stride;
} moe_quantize;

/*
 * moe_quantize_fp8 - x [matrices, num_rows, cols] to e4m3 codes (packed) and scales [matrices,
 *   ceil(num_rows / block_rows), cols / 128].  A value that is not a number gets the code of NaN and does not touch
 *   its block's scale; an infinity makes its whole block NaN.
 * moe_swiglu_fp8 - v = silu(gate) * up of gate_up [matrices, num_rows, 2 * cols] (the gate in the first half
 *   of the columns) in float32, quantised the same way (block_rows 1).  silu(g) = g / (1 + exp(-g)); where
 *   1 / (1 + exp(-g)) is below 2^-126, the smallest normal float32 (finite g below -126 ln 2 = -87.34), silu is 0.  At
 *   g = -infinity the formula is not a number, which marks that column's code alone.
 * live_rows_dev: one int32 in device memory, or NULL: only the first that many rows are taken,
 *   the outputs of those behind are left as they were (with moe_sort_picks: &offsets[num_experts]).
 *   It has to be NULL with block_rows 128 or several matrices.
 * The outputs do not overlap the inputs.
 * Errors: MOE_ERR_INVALID_ARGUMENT, MOE_ERR_HIDDEN_ALIGNMENT (cols % 128 != 0), MOE_ERR_LIMIT
 * (cols above MOE_MAX_HIDDEN), MOE_ERR_MISALIGNED (codes off 16 bytes, others off their element).
 */
int moe_quantize_fp8(const moe_quantize *q, const void *x_dev, const int32_t *live_rows_dev, uint8_t *codes_dev,
                     float *scales_dev, void *stream);
int moe_swiglu_fp8(const moe_quantize *q, const void *gate_up_dev, const int32_t *live_rows_dev, uint8_t *codes_dev,
                   float *scales_dev, void *stream);

/* ---- block-scaled FP8 products ------------------------------------------------------------ */

typedef struct {
    int32_t num_rows;       /* rows of a and out                                                 */
    int32_t n, k;           /* columns of out; inner dimension, a multiple of 128                */
    int32_t groups;         /* weight matrices; 0: one, for all rows (offsets_dev is NULL)       */
    int32_t out_dtype;      /* moe_dtype                                                         */
    int64_t a_stride;       /* a multiple of 16                                                  */
    int64_t out_stride;
} moe_product;

/*
 * moe_product_fp8 - for every row m of group g:
 *     out[m, n] = sum over blocks b of 128 inner columns of
 *                 a_scales[m, b] * b_scales[g, n / 128, b] * (sum over i in b of a[m, i] * b[g, n, i])
 *   a_dev        e4m3 [num_rows, k]; a_scales_dev float32 [num_rows, k / 128]
 *   b_dev        e4m3 [groups, n, k] (packed); b_scales_dev float32 [groups, ceil(n / 128), k / 128]
 *   offsets_dev  int32 [groups + 1]: group g has the rows [offsets[g], offsets[g + 1]), ascending, as
 *                moe_sort_picks writes them (values are taken as if clamped to [0, num_rows]; where
 *                they do not ascend, what out holds afterwards is undefined); rows of no group are left
 *                as they were in out and do not matter in a
 *   out_dev      bf16 or float32 [num_rows, n]; does not overlap the inputs
 *   status_dev   one int32 into which MOE_STATUS_TIMEOUT is or-ed where a wait of the kernel gave up, and
 *                out is then not valid; or NULL, and that cannot be seen.  The caller clears it: one
 *                word serves a chain of calls, which moe_sort_picks writes and the products add to
 * Products of codes are exact, sums are float32, and so are the scales' products; out is rounded
 * once.  The order of the sums depends on the sizes alone, so equal inputs give equal bits.
 * The gradient of a is the same product on the transposed codes and block scales of b.
 * Errors: MOE_ERR_INVALID_ARGUMENT, MOE_ERR_HIDDEN_ALIGNMENT (k % 128 != 0), MOE_ERR_LIMIT (k or n
 * above MOE_MAX_HIDDEN, groups above MOE_MAX_EXPERTS), MOE_ERR_MISALIGNED (a and b off 16 bytes,
 * others off their element).
 */
int moe_product_fp8(const moe_product *p, const uint8_t *a_dev, const float *a_scales_dev, const uint8_t *b_dev,
                    const float *b_scales_dev, const int32_t *offsets_dev, void *out_dev, int32_t *status_dev,
                    void *stream);

#ifdef __cplusplus
}
#endif
#endif /* COMBINE_TOPK_IDS_MOE_GROUPED_H */
