/*
 * act8_train.h -- C ABI of the GB300 (sm_103a) entry points that keep activations in 8 bits
 * between a training step's forward and backward, built into the same library as
 * rmsnorm_train.h (whose status codes and conventions -- device pointers, caller-owned buffers,
 * no allocation or synchronization, everything enqueued on `stream`, outputs that do not
 * overlap inputs -- apply here too).
 *
 * The format.  A row's values are taken in blocks of 32 consecutive ones (the last block may be
 * shorter).  A block is held as 8-bit two's complement numbers q and one power of two:
 *
 *   value = q * 2^(e-6),  q = the whole number nearest to x * 2^(6-e), ties to even
 *   e     = the smallest exponent from -120 to 127 with max|x| * 2^(6-e) < 127.5
 *
 * so |q| <= 127, and a value is off by at most 2^(e-7), half a number: at most 1/127 of the
 * block's greatest magnitude above 2^-120.  (At e = 127, magnitudes from 127.5 * 2^121 on, the last
 * 0.4 % of FP32's and BF16's range, take |q| = 127 and are off by up to a whole number.)  The
 * sign of zero is not kept.  A block that holds an infinity or a NaN is NaN as a whole.  A value
 * has at most 7 significant bits: exact in BF16.
 *
 * A packed row is act8_train_row_bytes(H) bytes: H numbers, padded to a multiple of 16 bytes;
 * then a byte e + 127 for each block (255: a NaN block, whose numbers are 0), padded to a multiple
 * of 16.  Padding is zero, so equal activations have equal bytes.  Rows are back to back and
 * start at a 16-byte boundary.
 */
#ifndef ACT8_TRAIN_H
#define ACT8_TRAIN_H

#include <stddef.h>
#include <stdint.h>

#include "rmsnorm_train.h" /* RMSN_OK, RMSN_ERR_* */

#ifdef __cplusplus
extern "C" {
#endif

#define ACT8_BF16 0
#define ACT8_FP32 1
#define ACT8_FP16 2

/* Bytes of a packed row of H values; 0 unless 1 <= H <= 2^30.  Host-only. */
int64_t act8_train_row_bytes(int64_t H);

/*
 * Packs R rows of H values.
 *   x       dtype ACT8_*, row r at element r * s_row, aligned to its elements (memory is read
 *           in whole 16-byte vectors that hold an element of the row)
 *   packed  [R, act8_train_row_bytes(H)] out, 16-byte aligned
 * H <= 2^30, R * act8_train_row_bytes(H) <= 2^42 (RMSN_ERR_UNSUPPORTED above).  R == 0 returns RMSN_OK with
 * nothing enqueued (pointers may then be NULL).
 */
int act8_train_pack(const void* x, int dtype, void* packed, int64_t R, int64_t H, int64_t s_row,
                    void* stream);

/*
 * The values of R packed rows, into y [R, H], contiguous, in dtype (rounded to nearest even where
 * it has too few bits; in FP16, finite values past its range become its largest).
 */
int act8_train_unpack(const void* packed, void* y, int dtype, int64_t R, int64_t H, void* stream);

/*
 * rmsnorm_train_fwd that also keeps what its backward reads, the normalized input, in 8 bits:
 *   [residual] h = round(x + residual) (written),  else h = x
 *   rstd = 1 / sqrt(mean(h^2) + eps),  y = round(h * rstd * w),  packed = the rows of h in 8 bits
 *
 *   x, residual   dtype ACT8_BF16 or ACT8_FP16, row r at element r * s_x (r * s_res); residual
 *                 may be NULL
 *   w             [H], w_dtype ACT8_BF16, ACT8_FP32 or ACT8_FP16
 *   y, h_out      [R, H] out, of x's type; h_out NULL iff residual is
 *   rstd          FP32 [R] out
 *   packed        [R, act8_train_row_bytes(H)] out
 *   eps           finite, >= 0
 * H a multiple of 8, 8 <= H <= 8192; s_x and s_res multiples of 8; every pointer 16-byte aligned,
 * rstd 4-byte; 0 <= R <= 2^31 - 2^16.  R == 0: nothing enqueued, row tensors may be NULL.
 */
int rmsnorm_act8_train_fwd(const void* x, const void* residual, int dtype, const void* w,
                           int w_dtype, void* y, void* h_out, float* rstd, void* packed,
                           int64_t R, int32_t H, int64_t s_x, int64_t s_res, float eps,
                           void* stream);

/* Bytes of device workspace of rmsnorm_act8_train_bwd; 0 on invalid sizes and for R == 0. */
size_t rmsnorm_act8_train_bwd_workspace_bytes(int64_t R, int32_t H);

/*
 * Its backward: with xhat = (the packed values) * rstd and g = dy * w,
 *   dx = round(rstd * (g - xhat * mean(g * xhat)) [+ dh]),  dw = sum over rows of dy * xhat (FP32)
 * dy, dh (may be NULL) and dx are [R, H], contiguous, dtype ACT8_BF16 or ACT8_FP16.  workspace as
 * rmsnorm_train_bwd's: no initial contents, clobbered, one for each of two calls that may overlap.
 * dw is an FP32 sum, of a thread's rows in plain additions (past 64 rows in two levels, runs of them and
 * the runs' sums), from there on with the additions' errors carried; rmsnorm_train_bwd carries them
 * throughout.  Bit-reproducible: the order of every sum is a function of R, H and of whether dh is
 * given.  R == 0: dw = 0.
 */
int rmsnorm_act8_train_bwd(const void* packed, const void* dy, const void* dh, int dtype,
                           const float* rstd, const void* w, int w_dtype, void* dx, float* dw,
                           void* workspace, size_t workspace_bytes, int64_t R, int32_t H,
                           void* stream);

#ifdef __cplusplus
}
#endif

#endif /* ACT8_TRAIN_H */
