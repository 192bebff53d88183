/*
 * moe_train.h -- training operators of the experts: products grouped by
 * expert in the three directions of a linear layer, and activations kept in
 * 8 bits between the forward and the backward pass.
 *
 * The pages describe the forward pass of the block only; every operator here
 * is the derivative of, or a storage format for, a step of moe_experts.h:
 * the expert MLP w2(silu(w1 x) * w3 x) of the moe-init excerpt of
 * "DeepSeek-V3.2-Exp · Mixture of experts", applied to rows grouped by
 * expert as moe_dispatch_build groups them.
 *
 * Conventions beyond those of moe_common.h:
 *  - Rows are expert-contiguous: group g owns the rows
 *    offsets[g] .. offsets[g+1]-1 of every row buffer (offsets from
 *    moe_dispatch_build, or any non-decreasing list within [0, rows]).
 *    Groups may be empty.  Rows outside offsets[0] .. offsets[groups] are
 *    neither read into a result nor written.
 *  - Offsets that decrease or leave [0, rows] are clamped on the device, so
 *    that no access leaves a buffer and no row is in two groups;
 *    MOE_ERR_RANGE goes to dev_status and the outputs of that call are
 *    unspecified.
 *  - Operands are MOE_BF16 or MOE_F32, both operands of a product the same.
 *    Sums are fp32 and rounded once at the end.
 *  - No atomics: results do not depend on the order in which blocks run.
 *  - bf16 operands whose rows are multiples of 16 bytes and whose addresses
 *    are 16-byte aligned run on the tcgen05 tensor cores as they are.  Other
 *    products of some size do through copies in the workspace: bf16 rows
 *    padded, fp32 operands split into three bf16 terms (results as exact as
 *    fp32 sums of operands that are multiples of 2^-133, as all above 2^-110
 *    are; a result that depends on an infinite fp32 operand may be NaN).
 *    The copies are of whole operands, the weights of groups without rows
 *    included: as many bytes again for bf16, one and a half times as many for
 *    fp32.  Small products, and any without a workspace, run on the CUDA cores
 *    with fp32 multiply-adds.
 *  - Each *_workspace_size takes `aligned`: 1 when every operand of the call
 *    is 16-byte aligned, as fresh allocations are; 0 asks for enough for any,
 *    aligned ones too.
 *  - Outputs share no memory with operands.
 */
#ifndef MOE_TRAIN_H
#define MOE_TRAIN_H
#include "moe_common.h"
#ifdef __cplusplus
extern "C" {
#endif

/* groups weights of [n, k], and rows rows grouped by offsets [groups + 1].
 * Limits: 1 <= groups <= 1024, 0 <= rows < 2^31, n, k in [1, 2^20]. */
typedef struct {
  int32_t groups, n, k;
  int64_t rows;
} moe_grouped_shape;

/*
 * y[p,:] = x[p,:] w[g]^T for every row p of every group g.
 *   x [rows, k], w [groups, n, k] of type dt; y [rows, n] of type y_dt
 *   ws  moe_grouped_linear_workspace_size bytes, 16-byte aligned; may be NULL
 *       (then the CUDA cores do what would have been copied)
 * Rows of y outside the groups are left as they were.
 * Device errors: MOE_ERR_RANGE (offsets), MOE_ERR_TIMEOUT (a pipeline wait
 * expired; outputs unspecified).  The same for the calls below.
 */
size_t moe_grouped_linear_workspace_size(const moe_grouped_shape *s, moe_dtype dt,
                                         int32_t aligned);
moe_status moe_grouped_linear(const moe_grouped_shape *s, const void *x, moe_dtype dt,
                              const void *w, const int32_t *offsets, void *y, moe_dtype y_dt,
                              void *ws, size_t ws_bytes, int32_t *dev_status,
                              moe_stream_t stream);

/*
 * The input gradient: dx[p,:] = dy[p,:] w[g] (+ dy2[p,:] w2[g]).
 *   dy, dy2 [rows, n]; w, w2 [groups, n, k]; dx [rows, k] of type dx_dt
 * dy2 and w2 (both or neither NULL) add a second product in the same fp32
 * sum: w1 and w3 share their input, so its gradient is the sum of two.
 */
size_t moe_grouped_linear_dx_workspace_size(const moe_grouped_shape *s, moe_dtype dt,
                                            int32_t two, int32_t aligned); /* two: with dy2 */
moe_status moe_grouped_linear_dx(const moe_grouped_shape *s, const void *dy, moe_dtype dt,
                                 const void *w, const void *dy2, const void *w2,
                                 const int32_t *offsets, void *dx, moe_dtype dx_dt, void *ws,
                                 size_t ws_bytes, int32_t *dev_status, moe_stream_t stream);

/*
 * The weight gradient: dw[g] = sum over the rows p of group g of
 * dy[p,:]^T x[p,:], added to dw when accumulate is 1.
 *   dy [rows, n], x [rows, k] of type dt; dw [groups, n, k] of type dw_dt
 * A group without rows has a zero gradient (accumulate 0) or leaves its part
 * of dw as it was (accumulate 1).  The addition to dw is one more rounding of
 * the sum in fp32 (fp32 sums below 2^-126 may become zero in it).
 */
size_t moe_grouped_linear_dw_workspace_size(const moe_grouped_shape *s, moe_dtype dt,
                                            int32_t aligned);
moe_status moe_grouped_linear_dw(const moe_grouped_shape *s, const void *dy, moe_dtype dt,
                                 const void *x, const int32_t *offsets, void *dw,
                                 moe_dtype dw_dt, int32_t accumulate, void *ws, size_t ws_bytes,
                                 int32_t *dev_status, moe_stream_t stream);

/*
 * The 8-bit format: a row of k values is stored as k e4m3 codes and
 * ceil(k / 32) scales, one for each 32 consecutive values.  A scale is the
 * power of two 2^(e - 127) of a biased exponent byte e, the smallest with
 * which the block's largest finite magnitude is at most 448 codes (not below
 * 2^-127; e = 0 for a block of zeros); a code is e4m3(v / scale), rounded to
 * nearest even.  A decoded value, code * scale, is exact in bf16 down to
 * 2^-133.  Infinities and NaN are stored as NaN: e4m3 has no infinity, and a
 * finite stand-in would hide a diverged activation.
 *
 * moe_checkpoint_rows stores src [rows, k] (MOE_BF16 or MOE_F32) into
 *   codes [rows, k] uint8 and exps [rows, ceil(k / 32)] uint8.
 * moe_restore_rows writes row index[i] of the stored rows to out [n, k]
 *   (i < n; index NULL: row i itself), rounded once to out_dt.  An index
 *   outside [0, rows) gives a row of zeros and MOE_ERR_RANGE in dev_status.
 * Limits: rows, n < 2^31, k in [1, 2^20].
 */
moe_status moe_checkpoint_rows(const void *src, moe_dtype dt, int64_t rows, int32_t k,
                               uint8_t *codes, uint8_t *exps, moe_stream_t stream);
moe_status moe_restore_rows(const uint8_t *codes, const uint8_t *exps, int64_t rows, int32_t k,
                            const int32_t *index, int64_t n, void *out, moe_dtype out_dt,
                            int32_t *dev_status, moe_stream_t stream);

/*
 * The experts' first matmul with its checkpoint: a = x w1[g]^T,
 * u = x w3[g]^T, h = silu(a) * u, with a and u stored in the 8-bit format
 * straight from their fp32 sums (s->n is the hidden width, s->k the model's).
 *   x [rows, k], w1, w3 [groups, n, k] of type dt; h [rows, n] of type dt
 *   codes_a, codes_u [rows, n], exps_a, exps_u [rows, ceil(n / 32)] uint8
 *   ws  moe_swiglu_checkpoint_workspace_size bytes, 16-byte aligned (NULL if
 *       that is 0); operands: x, w1, w3
 */
size_t moe_swiglu_checkpoint_workspace_size(const moe_grouped_shape *s, moe_dtype dt,
                                            int32_t aligned);
moe_status moe_swiglu_checkpoint(const moe_grouped_shape *s, const void *x, moe_dtype dt,
                                 const void *w1, const void *w3, const int32_t *offsets, void *h,
                                 uint8_t *codes_a, uint8_t *exps_a, uint8_t *codes_u,
                                 uint8_t *exps_u, void *ws, size_t ws_bytes,
                                 int32_t *dev_status, moe_stream_t stream);

/*
 * The backward pass of o[p,:] = gate[p] * (h[p,:] w2[g]^T) down to the
 * projections, from the stored a and u.  With dh = dy[p,:] w2[g],
 * s = sigmoid(a) and h = a * s * u of the decoded values:
 *   dgate[p] = sum_i dh_i h_i                     (fp32)
 *   da = gate * dh * u * s * (1 + a * (1 - s))    (type dt)
 *   du = gate * dh * a * s                        (type dt)
 *   hg = gate * h                                 (type dt)
 * hg is the operand of w2's gradient, grouped_linear_dw(dy, hg).
 *   dy [rows, k], w2 [groups, k, n] of type dt (s->n the hidden width)
 *   gate [rows] fp32 or NULL (1); da, du, hg [rows, n]; dgate [rows] fp32
 *   ws  moe_swiglu_backward_workspace_size bytes, 16-byte aligned; operands:
 *       dy, w2
 */
size_t moe_swiglu_backward_workspace_size(const moe_grouped_shape *s, moe_dtype dt,
                                          int32_t aligned);
moe_status moe_swiglu_backward(const moe_grouped_shape *s, const void *dy, moe_dtype dt,
                               const void *w2, const uint8_t *codes_a, const uint8_t *exps_a,
                               const uint8_t *codes_u, const uint8_t *exps_u, const float *gate,
                               const int32_t *offsets, void *da, void *du, void *hg,
                               float *dgate, void *ws, size_t ws_bytes, int32_t *dev_status,
                               moe_stream_t stream);

/*
 * Row lists of the experts' training pass for T tokens: the T * topk routed
 * rows in the order of moe_dispatch_build, then, when n_shared is 1, one row
 * per token for the shared expert, which becomes the last group.
 *   offsets [n_routed + 1], sorted_token [T * topk], slot_of [T, topk] from
 *   moe_dispatch_build, weights [T, topk] from moe_router_forward
 *   row_token [R] int32, row_gate [R] fp32 out, R = T * (topk + n_shared):
 *     the token of each row and its gate (1 for the shared expert)
 *   group_offsets [n_routed + n_shared + 1] int32 out
 * Limits: n_shared <= 1, R < 2^31.  A token or slot out of range is reported
 * (MOE_ERR_RANGE) and not written.
 */
moe_status moe_training_rows(const moe_cfg *cfg, int64_t T, const int32_t *offsets,
                             const int32_t *sorted_token, const int32_t *slot_of,
                             const float *weights, int32_t *row_token, float *row_gate,
                             int32_t *group_offsets, int32_t *dev_status, moe_stream_t stream);

/*
 * out[i,:] = src[index[i],:] for i < n, converted to out_dt (rounded once).
 *   src [rows, k] of type dt, index [n] int32, out [n, k] of type out_dt
 * An index outside [0, rows) gives a row of zeros and MOE_ERR_RANGE.
 * Limits: rows, n < 2^31, k in [1, 2^20].
 */
moe_status moe_gather_rows(const void *src, moe_dtype dt, int64_t rows, int32_t k,
                           const int32_t *index, int64_t n, void *out, moe_dtype out_dt,
                           int32_t *dev_status, moe_stream_t stream);

#ifdef __cplusplus
}
#endif
#endif
