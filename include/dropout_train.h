/*
 * dropout_train.h -- C ABI of the GB300 (sm_103a) dropout entry points, built into the same
 * library as rmsnorm_train.h (whose status codes, weight dtypes and conventions -- device
 * pointers, caller-owned buffers, no allocation or synchronization, everything enqueued on
 * `stream`, outputs that do not overlap inputs -- apply here too).
 *
 * The operation: every element is kept or dropped by a number drawn from a counter-based
 * generator; the keep mask is a function of (seed, offset + *step, p, element index) alone
 * and is never stored -- the backward draws it again:
 *
 *   forward   y_i = [residual_i +] (keep_i ? x_i * scale : 0)
 *   backward  dx_i = keep_i ? dy_i * scale : 0         (the residual's gradient is dy)
 *   t = floor(65536 p + 1/2),  scale = 65536 / (65536 - t),  keep_i = (u_i >= t)
 *
 * The probability is thus p rounded to a multiple of 2^-16 (scale uses the rounded one, so
 * the expectation is exact; p below 2^-17 drops nothing, p = 1 drops everything).  A dropped
 * element contributes zero whatever its value: infinities and NaN there do not pass.
 * Arithmetic is FP32 with one rounding to the output type.
 *
 * u_i: element i (of the flattened contiguous tensor) takes 16 bits of a Philox4x32-10 block
 * (Salmon, Moraes, Dror and Shaw, "Parallel random numbers: as easy as 1, 2, 3", SC 2011):
 * the block of counter words (q low, q high, c low, c high) with q = i / 8 and
 * c = offset + *step modulo 2^64, key words (seed low, seed high); element i takes half
 * (i & 1) (0: the low half) of output word (i >> 1) & 3.  Calls whose masks have to be
 * independent need different seeds or different c: a step that owns several dropouts gives
 * each an offset and advances `step` by their number.
 *
 *   step    device pointer to one uint64 (8-byte aligned), or NULL (0): added to `offset` when
 *           the kernel runs, so that a captured graph draws new masks at each replay after
 *           the program has advanced it on the stream.  The backward has to see the value
 *           that its forward saw.
 */
#ifndef DROPOUT_TRAIN_H
#define DROPOUT_TRAIN_H

#include <stddef.h>
#include <stdint.h>

#include "rmsnorm_train.h" /* RMSN_OK, RMSN_ERR_*, RMSN_W_BF16, RMSN_W_FP32 */

#ifdef __cplusplus
extern "C" {
#endif

#define DROPOUT_BF16 0
#define DROPOUT_FP32 1
#define DROPOUT_FP16 2

/*
 * Forward over n contiguous elements.
 *   x         [n], dtype DROPOUT_*
 *   residual  [n] of the same dtype, or NULL
 *   y         [n] of the same dtype, out
 *   p         0 <= p <= 1
 * Pointers 16-byte aligned; 0 <= n < 2^40 (RMSN_ERR_UNSUPPORTED above).  n == 0 returns
 * RMSN_OK with nothing enqueued (x, residual and y may then be NULL).
 */
int dropout_train_fwd(const void* x, const void* residual, void* y, int dtype, int64_t n,
                      double p, uint64_t seed, uint64_t offset, const uint64_t* step,
                      void* stream);

/* Backward: dx from dy, with the forward's dtype, n, p, seed, offset and step value. */
int dropout_train_bwd(const void* dy, void* dx, int dtype, int64_t n, double p, uint64_t seed,
                      uint64_t offset, const uint64_t* step, void* stream);

/*
 * The residual form of rmsnorm_train_fwd with dropout on the added branch, in one pass:
 *   h = BF16(residual + dropout(x)),  rstd = 1 / sqrt(mean(h^2) + eps),  y = BF16(h * rstd * w)
 * Element (t, head, j) of the logical [T, nh, H] tensor has mask index (t * nh + head) * H + j,
 * whatever the strides.  Arguments, layouts and limits as rmsnorm_train_fwd (residual and
 * h_out required), then dropout_train_fwd's.  When T == 0 the row tensors may be NULL.
 */
int rmsnorm_dropout_train_fwd(const void* x, const void* residual, const void* w, int w_dtype,
                              void* y, void* h_out, float* rstd, int64_t T, int32_t nh,
                              int32_t H, int64_t s_tok, int64_t s_head, float eps, double p,
                              uint64_t seed, uint64_t offset, const uint64_t* step,
                              void* stream);

/*
 * Its backward.  With total = the gradient of h (the norm's, plus dh):
 *   dresidual = BF16(total),  dx = BF16(keep * scale * total)  (each rounded once from FP32)
 *   h          BF16 [T, nh, H], contiguous: the forward's h_out
 *   dy, dh     BF16 [T, nh, H]; dh (the upstream gradient of h_out) may be NULL
 *   dx, dresidual  BF16 [T, nh, H] out, both required
 *   workspace  rmsnorm_train_bwd_workspace_bytes(T, nh, H, deterministic) bytes
 * Everything else as rmsnorm_train_bwd: dw, the two modes, and the determinism contract.
 * When T == 0 the row tensors may be NULL.
 */
int rmsnorm_dropout_train_bwd(const void* h, const void* dy, const void* dh, const float* rstd,
                              const void* w, int w_dtype, void* dx, void* dresidual, float* dw,
                              void* workspace, size_t workspace_bytes, int64_t T, int32_t nh,
                              int32_t H, double p, uint64_t seed, uint64_t offset,
                              const uint64_t* step, int deterministic, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* DROPOUT_TRAIN_H */
