/*
 * lnorm.h -- C ABI of layer norm and its gradient (part of libmoebound.so),
 * for AMD Instinct MI355X (gfx950).
 *
 * Per row x [H]:
 *   mean = sum_h x_h / H,   rstd = 1 / sqrt(sum_h (x_h - mean)^2 / H + eps)
 *   xh_h = (x_h - mean) rstd,   y_h = xh_h gamma_h + beta_h
 * and for an upstream gradient dy, with d_h = dy_h gamma_h:
 *   dx_h     = rstd (d_h - sum_j d_j / H - xh_h sum_j d_j xh_j / H)
 *   dgamma_h = sum over rows of dy_h xh_h,   dbeta_h = sum over rows of dy_h
 * The variance is summed from the centred row (no cancellation between large
 * means), every sum is fp32, and y and dx are rounded once.  Every output is
 * deterministic: sums run in a fixed order, without atomics.
 *
 * Conventions: as moebound.h (row-major contiguous device tensors, caller-
 * owned memory and workspace, no allocation or synchronisation, work enqueued
 * on `stream`, enum moe_status returns, host-side argument checks before
 * anything is enqueued, finite inputs: a row with NaN or Inf spoils that row
 * and the two sums over rows, nothing else).
 *   dtype MOE_BF16: X, Y, dY, dX bfloat16; MOE_F32: fp32.  gamma, beta, mean,
 *   rstd, dgamma, dbeta are fp32 always.
 */
#ifndef LNORM_H
#define LNORM_H

#include <stddef.h>
#include <stdint.h>

#include "moebound.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Filled by lnorm_plan; passed unchanged to the other calls. */
typedef struct lnorm_plan {
    uint32_t magic;              /* set by lnorm_plan                      */
    int32_t dtype;               /* enum moe_dtype                         */
    int64_t N;                   /* rows                                   */
    int32_t H;                   /* row width                              */
    float eps;
    int64_t bwd_workspace_bytes; /* workspace lnorm_backward needs         */
} lnorm_plan_t;

/*
 * lnorm_plan -- host only, pure.  N = 0 is valid (forward is a no-op, backward
 * zeroes dgamma and dbeta).
 * Errors: MOE_EINVAL if out is NULL, N < 0, H < 1, dtype unknown, or eps not a
 *   finite number above 0.  MOE_EUNSUPPORTED if H > 65536 or N >= 2^31.
 */
int lnorm_plan(int64_t N, int32_t H, int32_t dtype, float eps, lnorm_plan_t* out);

/*
 * lnorm_forward -- Y, and the row statistics lnorm_backward needs.
 * Inputs (device): X [N][H]; gamma [H]; beta [H] or NULL (0).
 * Outputs (device, overwritten): Y [N][H] (may be X itself, if the backward
 *   pass is not wanted); mean, rstd [N].
 * Errors: MOE_EINVAL (plan not from lnorm_plan, a required pointer NULL with
 *   N > 0), MOE_EHIP (enqueue failed).  Nothing is enqueued on the first.
 */
int lnorm_forward(const lnorm_plan_t* plan, const void* X, const float* gamma,
                  const float* beta, void* Y, float* mean, float* rstd, void* stream);

/*
 * lnorm_backward -- gradients of <Y, dY>.
 * Inputs (device): X, gamma as in lnorm_forward; dY [N][H]; mean, rstd [N] as
 *   it returned them.
 * Outputs (device, overwritten): dX [N][H] (may be dY itself); dgamma [H];
 *   dbeta [H] or NULL (not wanted).
 * workspace: at least plan->bwd_workspace_bytes bytes, 256-byte aligned;
 *   contents on entry do not matter.  It holds the partial sums over rows.
 * Errors: as lnorm_forward; MOE_EINVAL also for a workspace that is not
 *   256-byte aligned, MOE_EWORKSPACE for one that is too small.
 */
int lnorm_backward(const lnorm_plan_t* plan, const void* X, const float* gamma,
                   const void* dY, const float* mean, const float* rstd, void* dX,
                   float* dgamma, float* dbeta, void* workspace, size_t workspace_bytes,
                   void* stream);

#ifdef __cplusplus
}
#endif

#endif /* LNORM_H */
