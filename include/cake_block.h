/*
 * cake_block.h -- C ABI of a training block's operators between the norms:
 * the gated feed-forward block, the per-head norm of queries and keys with
 * rotary positions, and dropout from a counter-based generator (alone, and
 * with the residual addition and the norm after it); each forward and
 * backward.  Same library and conventions as cake_rmsnorm.h and cake_step.h:
 * device pointers owned by the caller, no allocation, no host synchronisation,
 * every launch asynchronous on `stream`, host-side validation with a
 * cake_status.
 *
 * These operators have no counterpart in the pages that cake_rmsnorm.h cites:
 * they are additions of this library.
 *
 * Workspaces hold nothing between calls: they need no initialisation, must be
 * 256-byte aligned, share no memory with the call's tensors, and may be shared
 * by calls that are ordered on one stream.  What a call writes shares no
 * memory with any other tensor of it, except where an operator says so.
 * (Tensors that are columns of one buffer share none.)  Every result is
 * bitwise reproducible for equal inputs and shapes.  Waits inside the kernels
 * are bounded and report through cake_rmsnorm_device_status(); the CTAs of a
 * thread-block cluster meet at hardware barriers besides, which every thread
 * reaches.  A first call on a device looks up addresses and sets kernel
 * attributes: make it before any stream capture.
 */
#ifndef CAKE_BLOCK_H
#define CAKE_BLOCK_H

#include "cake_rmsnorm.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ---- gated feed-forward block --------------------------------------------
 *
 *   forward   g = x Wg^T, u = x Wu^T (FP32 sums), h = bf16(act(g) * u)
 *   backward  dg = dh * u * act'(g), du = dh * act(g)
 *             dx = bf16(dg Wg + du Wu), dWg = bf16(dg^T x), dWu = bf16(du^T x)
 *
 * act: v * sigmoid(v) (CAKE_ACT_SILU), or
 * v * (1 + tanh(sqrt(2 / pi) (v + 0.044715 v^3))) / 2 (CAKE_ACT_GELU).
 * x, dx: BF16 [tokens, hidden]; Wg, Wu, dWg, dWu: BF16 [ffn, hidden]; h, g, u,
 * dh: BF16 [tokens, ffn].  hidden and ffn are multiples of 8, at most
 * CAKE_MAX_BLOCK_WIDTH.  Of a cake_tensor here, stride_token is the row
 * stride: a multiple of 8 elements, no less than a row; data is 16-byte
 * aligned.  Wg and Wu may be halves of one matrix.
 *
 * The forward writes bf16(g) and bf16(u) too where g and u are given (both or
 * neither); h is computed from the FP32 sums.  The backward takes them as
 * they were written.  dg and du are rounded to BF16 because the tensor cores
 * multiply BF16: an error of the result's norm of 2.3e-3 where exact ones would
 * leave the 1.7e-3 of its own rounding.  With at most 64 tokens what this
 * rounding leaves is multiplied too, so that they are good to 2^-16.  Sums are
 * FP32, those of a split sum added in a fixed order.
 * dx NULL leaves it out, and dw_gate and dw_up NULL (both or neither) those.
 */
typedef enum { CAKE_ACT_SILU = 0, CAKE_ACT_GELU = 1 } cake_act;

#define CAKE_MAX_BLOCK_WIDTH 131072

cake_status cake_gated_fwd(int64_t tokens, int64_t hidden, int64_t ffn, const cake_tensor *x,
                           const cake_tensor *w_gate, const cake_tensor *w_up, cake_act act,
                           const cake_tensor *h, const cake_tensor *g, const cake_tensor *u,
                           cake_stream_t stream);

size_t cake_gated_bwd_workspace_size(int64_t tokens, int64_t hidden, int64_t ffn);

cake_status cake_gated_bwd(int64_t tokens, int64_t hidden, int64_t ffn, const cake_tensor *dh,
                           const cake_tensor *x, const cake_tensor *g, const cake_tensor *u,
                           const cake_tensor *w_gate, const cake_tensor *w_up, cake_act act,
                           const cake_tensor *dx, const cake_tensor *dw_gate, const cake_tensor *dw_up,
                           void *workspace, size_t workspace_bytes, cake_stream_t stream);

/* ---- per-head norm and rotary positions ------------------------------------
 *
 * Per token t and head, over D = hidden elements, for queries and keys:
 *
 *   forward   rstd = 1 / sqrt(mean_j(v_j^2) + eps),  n_j = v_j * rstd * w_j
 *             y = bf16(rotated n)
 *   backward  d = dy rotated back,  a_j = d_j * w_j,  vh_j = v_j * rstd
 *             dv_j = bf16(rstd * (a_j - vh_j * mean_j(a_j * vh_j)))
 *             dw_j = sum over tokens and heads of d_j * vh_j        FP32
 *
 * Pair i of `pairs` (a, b) becomes (a cos - b sin, b cos + a sin) with the
 * angle 2 pi * turns[i] * position[axis[i]][t] / 2^64.  It is columns i and
 * pairs + i (CAKE_ROTARY_HALF) or 2 i and 2 i + 1 (CAKE_ROTARY_ADJACENT); the
 * columns from 2 * pairs on are not rotated.  turns is a frequency's share of a
 * turn in units of 2^-64; whole turns drop out of the product modulo 2^64 and
 * nothing else does, so an angle is off by the position times the error of its
 * turns (2^-65 of a turn where that is rounded once), and 2^-32 of a turn.
 *
 * q, k: BF16 [tokens, heads, hidden] views of the same tokens and hidden (k
 * with k_heads = 0: none).  hidden is a multiple of 16, at most 512; pairs is a
 * multiple of 8, at most hidden / 2 (0: no rotation).  positions: int32 or
 * int64, that of axis a and token t at positions[a * axis_stride + t *
 * token_stride]; negative ones turn backwards.  axis: NULL where axes is 1, or
 * int32 [pairs]; one outside [0, axes) leaves its pair unrotated and sets the
 * device status to CAKE_ERR_INVALID.  w_q and w_k NULL (both, or without keys
 * w_q): no norm, y is v rotated, and rstd, dw and the backward's q and k are
 * not used.  rstd_q, rstd_k: FP32 [tokens * heads] in (t, head) order.
 *
 * q_out may be exactly q and k_out exactly k (of the backward, dq_out dq and
 * dk_out dk).  dw_q, dw_k: [hidden] FP32, overwritten (dw_k, where it is given
 * without keys, with zeros).
 */
typedef enum { CAKE_ROTARY_HALF = 0, CAKE_ROTARY_ADJACENT = 1 } cake_rotary_style;

typedef struct {
    int64_t pairs, axes;
    const uint64_t *turns;     /* [pairs] device */
    const int32_t *axis;       /* [pairs] device, or NULL */
    const void *positions;     /* device */
    int positions_int64;
    int64_t axis_stride, token_stride; /* elements, >= 0 */
    int style;                 /* cake_rotary_style */
} cake_rotary;

cake_status cake_rotary_fwd(int64_t tokens, int64_t q_heads, int64_t k_heads, int64_t hidden,
                            const cake_tensor *q, const cake_tensor *k, const cake_rotary *rotary,
                            const void *w_q, cake_dtype w_q_dtype, const void *w_k, cake_dtype w_k_dtype,
                            float eps, const cake_tensor *q_out, const cake_tensor *k_out, float *rstd_q,
                            float *rstd_k, cake_stream_t stream);

size_t cake_rotary_bwd_workspace_size(int64_t tokens, int64_t q_heads, int64_t k_heads, int64_t hidden);

cake_status cake_rotary_bwd(int64_t tokens, int64_t q_heads, int64_t k_heads, int64_t hidden,
                            const cake_tensor *dq, const cake_tensor *dk, const cake_rotary *rotary,
                            const cake_tensor *q, const cake_tensor *k, const float *rstd_q,
                            const float *rstd_k, const void *w_q, cake_dtype w_q_dtype, const void *w_k,
                            cake_dtype w_k_dtype, const cake_tensor *dq_out, const cake_tensor *dk_out,
                            float *dw_q, float *dw_k, void *workspace, size_t workspace_bytes,
                            cake_stream_t stream);

/* ---- dropout ------------------------------------------------------------------
 *
 * The factor m of element e (e counts a tensor's elements row by row, rows in
 * (t, k) order) is 0, or 65536 / (65536 - cut) where the element is kept:
 * cut = p * 65536 rounded to the nearest whole number, and the element is kept
 * where its 16 random bits are at least cut.  They are bits 16 (e % 8) on of
 * the 128-bit Philox4x32-10 block (Salmon, Moraes, Dror and Shaw, "Parallel
 * random numbers: as easy as 1, 2, 3", 2011) of the counter
 * (low, high word of e / 8; low, high word of offset) and the key (low, high
 * word of seed).  No mask is stored: the backward computes it again.  rng
 * NULL: seed and offset as given; else a device pointer to two uint64, the
 * seed and a number that is added to offset, read when the kernel runs.
 *
 *   cake_dropout       y = bf16(m * x [+ residual]); its own gradient without residual
 *   cake_dropout_norm  h_j = bf16(residual_j + m * x_j)
 *                      rstd = 1 / sqrt(mean_j(h_j^2) + eps)  of the rounded h
 *                      y_j = bf16(h_j * rstd * w_j)
 *   backward           a_j = dy_j * w_j, hh_j = h_j * rstd
 *                      t_j = rstd * (a_j - hh_j * mean_j(a_j * hh_j)) [+ dh_j]
 *                      dresidual_j = bf16(t_j), dx_j = bf16(m * t_j)
 *                      dw_j = sum over all rows of dy_j * hh_j     FP32
 *
 * Shapes, strides and alignment as for cake_rmsnorm_fwd.  A dropped element
 * adds 0, also where x is infinite or NaN.  y may be exactly x or residual,
 * and of cake_dropout_norm_fwd y and h_new may be exactly an input view.
 */
cake_status cake_dropout(const cake_shape *shape, const cake_tensor *x, const cake_tensor *residual, double p,
                         uint64_t seed, uint64_t offset, const uint64_t *rng, const cake_tensor *y,
                         cake_stream_t stream);

cake_status cake_dropout_norm_fwd(const cake_shape *shape, const cake_tensor *x, const cake_tensor *residual,
                                  const void *w, cake_dtype w_dtype, double p, uint64_t seed, uint64_t offset,
                                  const uint64_t *rng, float eps, const cake_tensor *y,
                                  const cake_tensor *h_new, float *rstd, cake_stream_t stream);

size_t cake_dropout_norm_bwd_workspace_size(const cake_shape *shape);

/* dh: NULL, or the gradient that reaches h_new directly. */
cake_status cake_dropout_norm_bwd(const cake_shape *shape, const cake_tensor *dy, const cake_tensor *dh,
                                  const cake_tensor *h_new, const float *rstd, const void *w,
                                  cake_dtype w_dtype, double p, uint64_t seed, uint64_t offset,
                                  const uint64_t *rng, const cake_tensor *dx, const cake_tensor *dresidual,
                                  float *dw, void *workspace, size_t workspace_bytes, cake_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* CAKE_BLOCK_H */
