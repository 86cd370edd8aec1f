/*
 * block_train.h -- C ABI of the GB300 (sm_103a) entry points for a block's boundary in a
 * training step: the norm behind a block, its gate, the residual add with its scales, and the
 * norm before the next block, in one pass each way.  Built into the same library as
 * rmsnorm_train.h (whose status codes and conventions apply here too).
 *
 * The operation, on rows of H values (r1, r2 FP32, one a row; all arithmetic FP32, each output
 * rounded once):
 *
 *   r1 = 1 / sqrt(mean(x^2) + eps),  p = x * r1 * w_post        (no norm behind: p = x)
 *   h  = residual_scale * residual + scale * gate * p           (no gate: 1), written rounded
 *   r2 = 1 / sqrt(mean(h^2) + eps),  y = h * r2 * w_pre         of h before its rounding
 *
 * w_post, the gate and w_pre are optional; at least one norm is there.  The gate is [N, H] with
 * R a multiple of N: rows n * R/N to (n+1) * R/N - 1 (a sample's) take row n; N = 1 is one gate
 * for every row.
 *
 *   backward  t  = r2 * (dy * w_pre - hhat * mean(dy * w_pre * hhat)) + dh,   hhat = h * r2
 *                  (no norm before: t = dh)
 *             dresidual = residual_scale * t
 *             m  = scale * gate * w_post * t,  xhat = x * r1
 *             dx = r1 * (m - xhat * mean(m * xhat))             (no norm behind: scale * gate * t)
 *             S_n = sum of t * xhat over sample n's rows        (no norm behind: xhat = x)
 *             dgate_n = scale * w_post * S_n,  dw_post = scale * sum over n of gate_n * S_n
 *             dw_pre = sum over rows of dy * hhat               (the last four FP32)
 *
 * What the backward reads of the forward is h (with a norm before), x (with a norm behind or a
 * gate), and the r's.  x and h may be kept in 8 bits (act8_train.h): the forward packs the x it
 * reads and the h it writes.
 */
#ifndef BLOCK_TRAIN_H
#define BLOCK_TRAIN_H

#include <stddef.h>
#include <stdint.h>

#include "act8_train.h" /* ACT8_BF16, ACT8_FP32, ACT8_FP16; RMSN_* */

#ifdef __cplusplus
extern "C" {
#endif

/*
 * Forward.
 *   x, residual    dtype ACT8_BF16 or ACT8_FP16, row r at element r * s_x, r * s_res
 *   w_pre, w_post  [H], both of w_dtype (ACT8_BF16, ACT8_FP32 or ACT8_FP16); NULL: no such norm
 *   gate           [N, H] of gate_dtype (as w_dtype), or NULL (N is then 1)
 *   y              [R, H] out of x's type; NULL iff w_pre is
 *   h              [R, H] out of x's type
 *   rstd_pre, rstd_post  FP32 [R] out; NULL iff the norm's weight is
 *   x8, h8         [R, act8_train_row_bytes(H)] out: x and h in 8 bits, or NULL.  Either both of
 *                  those that the backward reads are given, or neither
 *   scale, residual_scale  finite
 *   eps            finite, >= 0
 * H a multiple of 8, 8 <= H <= 8192; s_x and s_res multiples of 8; pointers 16-byte aligned (the
 * r's 4-byte); N >= 1, R a multiple of N, 0 <= R <= 2^31 - 2^16.  R == 0: nothing enqueued, row
 * tensors may be NULL.
 */
int rmsnorm_block_train_fwd(const void* x, const void* residual, int dtype, const void* w_pre,
                            const void* w_post, int w_dtype, const void* gate, int gate_dtype,
                            int64_t N, void* y, void* h, float* rstd_pre, float* rstd_post,
                            void* x8, void* h8, int64_t R, int32_t H, int64_t s_x, int64_t s_res,
                            float scale, float residual_scale, float eps, void* stream);

/*
 * Bytes of device workspace of rmsnorm_block_train_bwd, enough for every combination of norms and
 * gate; 0 on invalid sizes and for R == 0.
 */
size_t rmsnorm_block_train_bwd_workspace_bytes(int64_t R, int32_t H, int64_t N);

/*
 * Backward.
 *   dy           [R, H], contiguous; NULL iff w_pre is
 *   dh           [R, H], contiguous, the gradient of h; may be NULL with a norm before
 *   x            with a norm behind or a gate: the forward's x (row r at element r * s_x), or, with
 *                packed = 1, its x8; else ignored
 *   h            with a norm before: the forward's h, or its h8; else ignored
 *   dx, dresidual  [R, H] out of dtype
 *   dw_pre, dw_post  FP32 [H] out, with their norms (else NULL)
 *   dgate        FP32 [N, H] out, with a gate (else NULL)
 *   workspace    rmsnorm_block_train_bwd_workspace_bytes(R, H, N) bytes, 16-byte aligned, no initial
 *                contents, clobbered; one for each of two calls that may overlap
 * Everything else as the forward.  dw_pre, dw_post and dgate are summed as rmsnorm_act8_train_bwd's
 * dw.  Bit-reproducible: the order of every sum is a function of R, H,
 * N and of which arguments are given.  R == 0: dw_pre, dw_post and dgate become 0.
 */
int rmsnorm_block_train_bwd(const void* dy, const void* dh, const void* x, const void* h,
                            int packed, int dtype, const float* rstd_pre, const float* rstd_post,
                            const void* w_pre, const void* w_post, int w_dtype, const void* gate,
                            int gate_dtype, int64_t N, void* dx, void* dresidual, float* dw_pre,
                            float* dw_post, float* dgate, void* workspace, size_t workspace_bytes,
                            int64_t R, int32_t H, int64_t s_x, float scale, float residual_scale,
                            void* stream);

/*
 * The launch plan of a kernel: for tests and diagnostics.  No device access.  `kernel` is a sum of
 * the flags below; 0 is the forward with both norms, BLOCK_PLAN_BACKWARD the backward with both
 * norms, a gate and dh.  packed: the backward from 8 bits.  out receives min(n_out, BLOCK_PLAN_FIELDS)
 * values: 16-byte vectors a thread, threads a row, teams a CTA, rows a ring slot, slots a team,
 * threads a CTA, CTAs, dynamic shared memory bytes.  R >= 1; sizes as above; N = 1 without a gate.
 */
#define BLOCK_PLAN_FIELDS 8
#define BLOCK_PLAN_BACKWARD 1
#define BLOCK_PLAN_NO_NORM_BEHIND 2 /* w_post NULL */
#define BLOCK_PLAN_NO_NORM_BEFORE 4 /* w_pre NULL */
#define BLOCK_PLAN_NO_GATE 8        /* gate NULL */
#define BLOCK_PLAN_ONE_INPUT 16     /* dh NULL; in rmsnorm_act8_train_fwd residual NULL */
#define BLOCK_PLAN_ACT8_NORM 32     /* rmsnorm_act8_train_fwd or _bwd (packed = 1) */
int rmsnorm_block_train_launch_plan(int64_t R, int32_t H, int64_t N, int kernel, int packed,
                                    int64_t* out, int n_out);

/*
 * Reads (and, if reset != 0, clears) the error word of these kernels' and of
 * rmsnorm_act8_train_*'s bounded waits on the current device into *flags (host pointer), as
 * rmsnorm_train_device_error.  Synchronizes the device.
 */
int rmsnorm_block_train_device_error(unsigned int* flags, int reset);

#ifdef __cplusplus
}
#endif

#endif /* BLOCK_TRAIN_H */
