/*
 * tide_ops.h -- C ABI of libtide's training-block operators: what a rank
 * computes between the all-gather of a group's parameters (tide_ag_place) and
 * the reduce-scatter of their gradients (tide_rs_reduce).
 *
 *   RMS norm with the residual's addition, forward and backward
 *   linear layer: bias, activation, residual; input, weight and bias gradients
 *   activation checkpoints in 8 bits, and their use in the backward pass
 *
 * Conventions, beside those of tide.h:
 *   - Every matrix is row-major with a row stride (ld...) in elements, at
 *     least its number of columns; elements of a row are contiguous.  Base
 *     pointers are aligned to their element size; no other alignment is asked
 *     for (16-byte aligned rows are faster).
 *   - All calls enqueue work on `stream` of the current device, allocate
 *     nothing and can be captured into a CUDA graph (after a first call of
 *     the kind, which loads its kernels).  A call with nothing to write
 *     returns TIDE_OK.
 *   - Arithmetic is fp32 whatever the tensors' type; each output is rounded
 *     once, to nearest even, when it is stored.  Results do not depend on
 *     timing: the same call gives the same bits.
 *   - `workspace` is caller-owned device scratch, 16-byte aligned, of at least
 *     the bytes the matching ..._workspace() query returns; its contents are
 *     overwritten.  NULL is fine where the query returns 0.  Calls that may
 *     overlap on the GPU need workspaces of their own.
 *   - Outputs must not overlap inputs or each other, except where said.
 *   - Errors: INVALID_ARG (null pointer, negative size, stride shorter than a
 *     row, unknown type or activation, workspace too small), ALIGNMENT,
 *     OVERFLOW (a matrix beyond int64 bytes), UNIMPLEMENTED (a size outside
 *     what is built), CUDA.
 */
#ifndef TIDE_OPS_H
#define TIDE_OPS_H

#include "tide.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum tide_dtype { TIDE_BF16 = 0, TIDE_F32 = 1 } tide_dtype;

/* Activations f and the derivatives f' the backward calls use.
 *   RELU      max(z, 0); f' = 1 for z > 0, else 0
 *   GELU      tanh form: z / (1 + exp(-2u)), u = sqrt(2/pi) (z + 0.044715 z^3)
 *   GELU_ERF  z * (1 + erf(z / sqrt(2))) / 2
 *   SILU      z / (1 + exp(-z))
 * At -inf the last three and their derivatives give 0, at +inf z and 1; NaN
 * stays NaN.  Values and derivatives below 2^-119 in magnitude, where the
 * exponentials leave fp32, may come out as 0. */
typedef enum tide_act {
  TIDE_ACT_NONE = 0,
  TIDE_ACT_RELU = 1,
  TIDE_ACT_GELU = 2,
  TIDE_ACT_GELU_ERF = 3,
  TIDE_ACT_SILU = 4
} tide_act;

/* Synchronise the current device and report whether a kernel of these operators
 * gave up a bounded wait there (TIDE_ERR_TIMEOUT) since the calling thread's last
 * check of that device, or since the library was loaded if this is its first.
 * Every thread that checks learns of it, whichever thread made the call.  Such a
 * call's outputs are undefined.  Errors: CUDA. */
tide_status tide_ops_check(void);

/* Options.
 *   TIDE_OPS_OPT_WAIT_LIMIT_NS   bound, in nanoseconds, on every wait inside
 *                                the operators' kernels (default 2e9), for the
 *                                whole process
 *   TIDE_OPS_OPT_TEST_DROP_LOAD  test hook, for the calling thread's own calls
 *                                alone: a product's CTAs withhold the
 *                                loads of the given block of 64 of the summed
 *                                axis, and the norm's backward pass the
 *                                copies of the given turn of rows (counted per
 *                                CTA from 0), so a bounded wait runs out; -1
 *                                (default) disables
 * Errors: INVALID_ARG. */
typedef enum tide_ops_option { TIDE_OPS_OPT_WAIT_LIMIT_NS = 1, TIDE_OPS_OPT_TEST_DROP_LOAD = 2 } tide_ops_option;
tide_status tide_ops_set_option(int32_t option, int64_t value);

/* ---- 8-bit checkpoints ----------------------------------------------------
 * A matrix kept in 8 bits: `codes` [rows, cols] e4m3 bytes (row stride
 * ld_codes bytes) and `scales` [rows, ceil(cols/32)] bytes (row stride
 * ld_scales), one for each block of 32 columns (the last may be shorter).
 * Value = e4m3(code) * 2^(scale - 127).  The scale is the smallest power of
 * two, at least 2^-127, that puts the block's largest finite magnitude at or
 * below 448 (so nothing finite saturates below 1.875 * 2^127; larger values
 * are kept as that); codes round to nearest even.  A value that is not finite
 * is kept as NaN and leaves the rest of its block as it is.  The values have
 * 4 significant bits, so bf16 holds them exactly (scales above 2^-124). */

/* x [rows, cols] of `dtype` -> codes, scales. */
tide_status tide_checkpoint_store(int64_t rows, int64_t cols, int32_t dtype, const void* x, int64_t ldx, uint8_t* codes,
                                  int64_t ld_codes, uint8_t* scales, int64_t ld_scales, void* stream);

/* out [rows, cols] of `dtype`: f(value) of every kept value, or, with grad
 * not NULL ([rows, cols] of `dtype`), grad * f'(value) (grad itself for
 * TIDE_ACT_NONE).  out may be grad. */
tide_status tide_checkpoint_load(int64_t rows, int64_t cols, const uint8_t* codes, int64_t ld_codes,
                                 const uint8_t* scales, int64_t ld_scales, int32_t act, int32_t dtype, const void* grad,
                                 int64_t ld_grad, void* out, int64_t ld_out, void* stream);

/* ---- RMS norm with the residual's addition --------------------------------
 * s = x + residual (fp32; residual may be NULL), r = (mean(s^2) + eps)^(-1/2)
 * per row, out: h = s, y = s * r * weight, rstd = r, and y again as an 8-bit
 * checkpoint (codes, scales) made from its fp32 values.  All matrices and
 * weight [cols] are of `dtype`; rstd [rows] is fp32.  h, y, rstd and codes may
 * each be NULL (scales goes with codes).  h or y may be x or residual.
 * cols at most 16384 (UNIMPLEMENTED beyond). */
tide_status tide_rms_norm(int64_t rows, int64_t cols, int32_t dtype, const void* x, int64_t ldx, const void* residual,
                          int64_t ldr, const void* weight, float eps, void* h, int64_t ldh, void* y, int64_t ldy,
                          float* rstd, uint8_t* codes, int64_t ld_codes, uint8_t* scales, int64_t ld_scales,
                          void* stream);

/* The gradient: with n = h * rstd and g = dy * weight,
 *   dx = rstd * (g - n * mean(g * n)) + dres,   dweight = sum over rows of dy * n.
 * dx is the gradient of x and of residual alike; dres (may be NULL) is what
 * reaches h past the norm.  h is given in `dtype` (h, ldh) or, with h NULL, as
 * an 8-bit checkpoint (codes, scales).  dx and dweight [cols] are of `dtype`;
 * either may be NULL.  dx may be dy or dres.  No rows: dweight is zero. */
int64_t tide_rms_norm_backward_workspace(int64_t rows, int64_t cols);
tide_status tide_rms_norm_backward(int64_t rows, int64_t cols, int32_t dtype, const void* dy, int64_t lddy,
                                   const void* h, int64_t ldh, const uint8_t* codes, int64_t ld_codes,
                                   const uint8_t* scales, int64_t ld_scales, const void* weight, const float* rstd,
                                   const void* dres, int64_t ld_dres, void* dx, int64_t lddx, void* dweight,
                                   void* workspace, int64_t workspace_bytes, void* stream);

/* ---- Linear layer ---------------------------------------------------------
 * All matrices, bias included, are bf16; products accumulate in fp32. */

/* z = x W^T + bias, y = f(z) + residual.  x [rows, inner], w [outer, inner],
 * bias [outer] or NULL, residual [rows, outer] or NULL, y [rows, outer].
 * z [rows, outer] (or NULL) receives z in bf16, codes/scales (or NULL) z as an
 * 8-bit checkpoint; both are made from the fp32 z.  y may be residual. */
int64_t tide_linear_workspace(int64_t rows, int64_t inner, int64_t outer, const void* x, int64_t ldx, const void* w,
                              int64_t ldw);
tide_status tide_linear(int64_t rows, int64_t inner, int64_t outer, const void* x, int64_t ldx, const void* w,
                        int64_t ldw, const void* bias, int32_t act, const void* residual, int64_t ldr, void* y,
                        int64_t ldy, void* z, int64_t ldz, uint8_t* codes, int64_t ld_codes, uint8_t* scales,
                        int64_t ld_scales, void* workspace, int64_t workspace_bytes, void* stream);

/* dx = (dy W) * f'(z): dy [rows, outer], w [outer, inner], dx [rows, inner].
 * z [rows, inner] is the pre-activation whose f(z) was this layer's input, in
 * bf16 (z) or as an 8-bit checkpoint (codes, scales); with TIDE_ACT_NONE
 * neither is read and dx = dy W. */
int64_t tide_linear_grad_input_workspace(int64_t rows, int64_t inner, int64_t outer, const void* dy, int64_t lddy,
                                         const void* w, int64_t ldw);
tide_status tide_linear_grad_input(int64_t rows, int64_t inner, int64_t outer, const void* dy, int64_t lddy,
                                   const void* w, int64_t ldw, int32_t act, const void* z, int64_t ldz,
                                   const uint8_t* codes, int64_t ld_codes, const uint8_t* scales, int64_t ld_scales,
                                   void* dx, int64_t lddx, void* workspace, int64_t workspace_bytes, void* stream);

/* dw = dy^T X, db = sum over rows of dy (may be NULL): dy [rows, outer],
 * dw [outer, inner], db [outer].  X [rows, inner] is x in bf16, or, with x
 * NULL, f(value) of an 8-bit checkpoint rounded to bf16, as the forward pass
 * rounded it (exact for TIDE_ACT_NONE).  With x given, act must be
 * TIDE_ACT_NONE.  No rows: dw and db are zero.  with_db: whether db is asked
 * for. */
int64_t tide_linear_grad_weight_workspace(int64_t rows, int64_t inner, int64_t outer, const void* dy, int64_t lddy,
                                          const void* x, int64_t ldx, int32_t with_db);
tide_status tide_linear_grad_weight(int64_t rows, int64_t inner, int64_t outer, const void* dy, int64_t lddy,
                                    const void* x, int64_t ldx, const uint8_t* codes, int64_t ld_codes,
                                    const uint8_t* scales, int64_t ld_scales, int32_t act, void* dw, int64_t lddw,
                                    void* db, void* workspace, int64_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* TIDE_OPS_H */
