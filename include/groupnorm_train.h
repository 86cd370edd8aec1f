/*
 * groupnorm_train.h -- C ABI of the GB300 (sm_103a) group norm for training, channels last,
 * with an activation behind it; built into the same library as rmsnorm_train.h (whose status
 * codes and conventions -- device pointers, caller-owned buffers, no allocation or
 * synchronization, everything enqueued on `stream`, outputs that do not overlap inputs --
 * apply here too).
 *
 * The operation, on x [N, S, C] (S: the places of a sample, all spatial axes as one) with the
 * C channels in G groups of C/G neighbours; m = S * C/G values a (sample, group):
 *
 *   forward   mean = (1/m) sum x,  var = (1/m) sum (x - mean)^2,  rstd = 1/sqrt(var + eps)
 *             z = (x - mean) * rstd * w_c + b_c,   y = act(z)
 *   backward  xhat = (x - mean) * rstd,  dz = dy * act'(z),  g = dz * w_c
 *             dx = rstd * (g - mean(g) - xhat * mean(g * xhat))       (means over the group)
 *             dw_c = sum over n, s of dz * xhat,   db_c = sum over n, s of dz
 *   act       identity; SiLU z / (1 + exp(-z)); GELU z * Phi(z) (the exact form;
 *             for the 16-bit types Phi is within 2e-7, for FP32 Phi(z), z < 0, within 1e-6 of
 *             itself, so its tail is kept)
 *
 * Statistics, sums and arithmetic are FP32, with one rounding to the output type.  The variance
 * is formed from values shifted by one of their own, so a mean far from zero costs it nothing
 * beyond what FP32 holds of mean itself.  Every order of summation is a function of the shape
 * and dtype alone: results are bit-reproducible run to run and on GPUs of any SM count.  A group's
 * sum of squared deviations has to stay within FP32's range, and its variance, where eps is 0,
 * within FP32's normal numbers; the backward takes any finite rstd.
 *
 * Layout: x is read through strides (elements): place s of sample n starts at n*s_n + s*s_s,
 * its C channels side by side.  y, dy and dx are contiguous [N, S, C]; mean and rstd [N, G]
 * FP32; w, b [C] of one dtype; dw, db [C] FP32.
 * Alignment: x, y, dy, dx 16-byte aligned, and so every place of x (strides in multiples of
 * 8 elements for BF16 and FP16, 4 for FP32); mean, rstd, dw, db 4-byte; w, b by their type.
 * Limits: C a multiple of 8 and of G, C <= 4096, and the fewest neighbouring groups that make
 * whole 16-byte vectors hold at most 512 vectors (met by every G at C <= 2048);
 * N * S * C < 2^40, N and S < 2^31 (RMSN_ERR_UNSUPPORTED otherwise).
 */
#ifndef GROUPNORM_TRAIN_H
#define GROUPNORM_TRAIN_H

#include <stddef.h>
#include <stdint.h>

#include "rmsnorm_train.h" /* RMSN_OK, RMSN_ERR_* */

#ifdef __cplusplus
extern "C" {
#endif

#define GROUPNORM_BF16 0
#define GROUPNORM_FP32 1
#define GROUPNORM_FP16 2

#define GROUPNORM_ACT_NONE 0
#define GROUPNORM_ACT_SILU 1
#define GROUPNORM_ACT_GELU 2

/*
 * Bytes of device workspace groupnorm_train_fwd / _bwd need for a shape and activation dtype:
 * a function of these alone.  0 on invalid sizes, for no elements, and where a forward keeps
 * its samples on chip.  At most 1.125 times the activation's bytes and 20 KB a channel, where a
 * sample's groups have 32 values or more.
 */
size_t groupnorm_train_fwd_workspace_bytes(int dtype, int64_t N, int64_t S, int32_t C, int32_t G);
size_t groupnorm_train_bwd_workspace_bytes(int dtype, int64_t N, int64_t S, int32_t C, int32_t G);

/*
 * Forward.
 *   x         dtype (GROUPNORM_BF16 / _FP32 / _FP16), read through (s_n, s_s)
 *   w, b      [C] each, both of dtype wb_dtype (the same codes)
 *   y         [N, S, C] of dtype, out
 *   mean, rstd  FP32 [N, G] out
 *   workspace   16-byte aligned, no initial contents, clobbered (may be NULL when its size
 *               is 0); calls that may overlap on the GPU need separate ones
 *   eps       finite, >= 0;  act: GROUPNORM_ACT_*
 * N == 0 returns RMSN_OK with nothing enqueued (tensors but w and b may be NULL); S is at least
 * 1 unless N is 0.
 */
int groupnorm_train_fwd(const void* x, int dtype, const void* w, const void* b, int wb_dtype,
                        void* y, float* mean, float* rstd, void* workspace,
                        size_t workspace_bytes, int64_t N, int64_t S, int32_t C, int32_t G,
                        int64_t s_n, int64_t s_s, float eps, int act, void* stream);

/*
 * Backward.  x, w, b, act as the forward's; mean, rstd as it returned them.
 *   dy        [N, S, C] of dtype
 *   dx        [N, S, C] of dtype, out
 *   dw, db    FP32 [C] out, overwritten; zero-filled when N == 0
 */
int groupnorm_train_bwd(const void* x, const void* dy, int dtype, const float* mean,
                        const float* rstd, const void* w, const void* b, int wb_dtype, void* dx,
                        float* dw, float* db, void* workspace, size_t workspace_bytes, int64_t N,
                        int64_t S, int32_t C, int32_t G, int64_t s_n, int64_t s_s, int act,
                        void* stream);

/*
 * How the library runs a shape (host-only): writes min(n_out, GROUPNORM_PLAN_FIELDS) values to
 * `out` (host memory): 1 if samples stay on chip between the statistics and the output (one
 * pass over memory; else a cooperative grid streams them, twice), channels a CTA
 * takes (its slab), threads a CTA, CTAs a cluster, CTAs of the launch at most, its dynamic
 * shared memory bytes, units -- slabs of samples -- taken at a time, chunks a unit's places are
 * split into (1 on chip).  backward: 0 or 1.
 */
#define GROUPNORM_PLAN_FIELDS 8
int groupnorm_train_launch_plan(int dtype, int64_t N, int64_t S, int32_t C, int32_t G,
                                int backward, int64_t* out, int n_out);

#ifdef __cplusplus
}
#endif

#endif /* GROUPNORM_TRAIN_H */
