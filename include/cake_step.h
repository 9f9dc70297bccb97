/*
 * cake_step.h -- C ABI of the training-step operators around the RMSNorm:
 * the sandwich norm (forward and backward), the global gradient norm and
 * clipping over many tensors, and the embedding lookup with its gradient by
 * sorted tokens.  Same library and conventions as cake_rmsnorm.h: device
 * pointers owned by the caller, no allocation, no host synchronisation, every
 * launch asynchronous on `stream`, host-side validation with a cake_status.
 *
 * These operators have no counterpart in the pages that cake_rmsnorm.h cites:
 * they are additions of this library.
 *
 * Workspaces here hold nothing between calls: they need no initialisation
 * (and none after an error), must be 256-byte aligned, share no memory with
 * the call's tensors, and may be shared by calls that are ordered on one
 * stream.  Every result is bitwise reproducible for equal inputs and shapes.
 * Waits inside the kernels (for staged copies, for a row's sums, and for the
 * flag that the embedding gradient's zeroing starts at) are bounded and report
 * through cake_rmsnorm_device_status(); the CTAs of a thread-block cluster meet
 * at hardware barriers besides, which every thread reaches.  A first call on a device looks up addresses
 * and sets kernel attributes: make it before any stream capture.
 */
#ifndef CAKE_STEP_H
#define CAKE_STEP_H

#include "cake_rmsnorm.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ---- sandwich norm -------------------------------------------------------
 *
 * The norms after one block and before the next, with the gate, the residual
 * scale and the residual addition between them, per row of H elements:
 *
 *   forward   rstd_post = 1 / sqrt(mean_j(z_j^2) + eps)       z: block output
 *             n_j   = z_j * rstd_post * w_post_j
 *             h_j   = bf16(x_j + scale * g * n_j)             x: residual stream
 *             rstd_pre = 1 / sqrt(mean_j(h_j^2) + eps)        of the rounded h
 *             y_j   = bf16(h_j * rstd_pre * w_pre_j)          next block's input
 *   backward  a_j = dy_j * w_pre_j, hh_j = h_j * rstd_pre, c2 = mean_j(a_j * hh_j)
 *             t_j = rstd_pre * (a_j - hh_j * c2) [+ dh_j],    dx_j = bf16(t_j)
 *             dn_j = scale * g * t_j, zh_j = z_j * rstd_post,
 *             c1 = mean_j(dn_j * w_post_j * zh_j)
 *             dz_j = bf16(rstd_post * (dn_j * w_post_j - zh_j * c1))
 *             dw_pre_j  = sum over all rows of dy_j * hh_j    FP32
 *             dw_post_j = sum over all rows of dn_j * zh_j    FP32
 *             dgate = scale * sum_j t_j * n_j (a value per row), or
 *                     bf16(scale * t_j * n_j) (a value per element)
 *
 * The gate g is none (gate_rows and gate both NULL), one FP32 value per row
 * (gate_rows, [T*nh], rows in (t, k) order) or one BF16 value per element
 * (gate, a tensor of the rows' shape); giving both is CAKE_ERR_INVALID.  It
 * multiplies as it is given: an activation before it is the caller's.
 * Shapes, strides, alignment and sharing of memory as for cake_rmsnorm_fwd
 * and cake_rmsnorm_bwd: an output of the forward may be exactly an input view
 * (y or h_new in place of z, x or gate), and nothing else that a call writes
 * may share memory with any other tensor of it.  (Tensors that are columns of
 * one buffer share none; they are told apart where their rows are equally
 * spaced, and alike.)  w_post and w_pre have a dtype each.
 */
cake_status cake_sandwich_fwd(const cake_shape *shape, const cake_tensor *z, const cake_tensor *x,
                              const void *w_post, cake_dtype w_post_dtype, const void *w_pre,
                              cake_dtype w_pre_dtype, const float *gate_rows, const cake_tensor *gate,
                              float scale, float eps, const cake_tensor *y, const cake_tensor *h_new,
                              float *rstd_post, float *rstd_pre, cake_stream_t stream);

/* Bytes of workspace cake_sandwich_bwd needs for this shape (0 for T = 0). */
size_t cake_sandwich_bwd_workspace_size(const cake_shape *shape);

/*
 * dh: NULL, or the gradient that reaches h_new directly.  dx is the gradient
 * of h_new as a whole, which is that of x.  dgate_rows goes with gate_rows
 * and dgate with gate; NULL leaves that gradient out.  dw_post, dw_pre: [H]
 * FP32, 16-byte aligned, overwritten.  T = 0: both are zero-filled.
 */
cake_status cake_sandwich_bwd(const cake_shape *shape, const cake_tensor *dy, const cake_tensor *dh,
                              const cake_tensor *h_new, const cake_tensor *z, const float *rstd_post,
                              const float *rstd_pre, const void *w_post, cake_dtype w_post_dtype,
                              const void *w_pre, cake_dtype w_pre_dtype, const float *gate_rows,
                              const cake_tensor *gate, float scale, const cake_tensor *dx,
                              const cake_tensor *dz, float *dw_post, float *dw_pre, float *dgate_rows,
                              const cake_tensor *dgate, void *workspace, size_t workspace_bytes,
                              cake_stream_t stream);

/* ---- gradient norm and clipping --------------------------------------------
 *
 *   norm = sqrt(sum over all values of all tensors of g^2)        FP32
 *   coef = min(1, max_norm / (norm + eps)),   out = round(g * coef)
 *
 * n tensors: data[i] is a device pointer (aligned to its element size) to
 * counts[i] contiguous values of dtypes[i]; BF16 and FP32 may be mixed.  The
 * arrays themselves are HOST memory, read before the call returns.  norm: one
 * FP32 device value, in none of the tensors (CAKE_ERR_INVALID).  Squares whose FP32 sum would overflow or vanish are
 * summed again in FP64, so norm is within 6 half-steps of FP32 (2^-24 of the
 * value each) over the whole range of the types.  A NaN or infinity gives a NaN or infinite norm, and
 * clipping then follows the formula (infinite: coef is 0, and infinity * 0 is
 * NaN; NaN: everything becomes NaN).
 *
 * cake_grad_clip writes g * coef, rounded once to out_dtypes[i], to outs[i];
 * outs NULL (out_dtypes NULL too) clips in place, and then writes nothing
 * where coef is 1.  An output may be exactly its own input or share no memory
 * with any tensor of the call; inputs may share memory with each other only
 * where they are not written (CAKE_ERR_INVALID).  max_norm >= 0 (infinity is allowed), eps >= 0; coef is 1 where
 * norm + eps is 0.  n at most 1000000; n = 0: norm is 0.
 */
size_t cake_grad_norm_workspace_size(int64_t n);

cake_status cake_grad_norm(const void *const *data, const int64_t *counts, const int32_t *dtypes,
                           int64_t n, float *norm, void *workspace, size_t workspace_bytes,
                           cake_stream_t stream);

cake_status cake_grad_clip(void *const *data, const int64_t *counts, const int32_t *dtypes,
                           void *const *outs, const int32_t *out_dtypes, int64_t n, float max_norm,
                           float eps, float *norm, void *workspace, size_t workspace_bytes,
                           cake_stream_t stream);

/* ---- embedding ---------------------------------------------------------------
 *
 *   y_t = bf16(scale * table[ids_t])                                BF16 rows
 *   dtable_v = [dtable_v +] scale * sum over t with ids_t = v of dy_t
 *
 * ids: [T] int32 (ids_int64 = 0) or int64.  A negative id means no token: its
 * row of y is zero and it adds nothing to dtable.  An id >= vocab does the
 * same and sets the device status (cake_rmsnorm_device_status) to
 * CAKE_ERR_INVALID.  padding_idx (-1: none): that id adds nothing to dtable.
 * table, dtable: [vocab, H] BF16 or FP32, row strides in elements, 16-byte
 * aligned rows; y, dy: BF16 rows [T, H].  H a multiple of 8, at most
 * CAKE_MAX_HIDDEN; T and vocab below 2^31.  What is written shares memory with
 * no other tensor of the call.
 *
 * The gradient sorts the tokens by id (stably) and sums each id's rows in
 * FP32 in an order that depends on the ids alone, so it is bitwise
 * reproducible.  accumulate = 0 writes every row of dtable (zeros for ids
 * without a token); accumulate = 1 adds to the rows with tokens, the sum
 * rounded once to dtable's type, and leaves the others alone.
 */
cake_status cake_embedding_fwd(const void *ids, int ids_int64, int64_t tokens, const void *table,
                               cake_dtype table_dtype, int64_t vocab, int64_t hidden,
                               int64_t table_stride, float scale, const cake_tensor *y,
                               cake_stream_t stream);

size_t cake_embedding_bwd_workspace_size(int64_t tokens, int64_t vocab, int64_t hidden);

cake_status cake_embedding_bwd(const cake_tensor *dy, const void *ids, int ids_int64, int64_t tokens,
                               int64_t vocab, int64_t hidden, float scale, int64_t padding_idx,
                               void *dtable, cake_dtype dtable_dtype, int64_t dtable_stride,
                               int accumulate, void *workspace, size_t workspace_bytes,
                               cake_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* CAKE_STEP_H */
