/*
 * rms.h -- C ABI of root-mean-square norm with the residual's addition, and its
 * gradient (part of libmoebound.so), for AMD Instinct MI355X (gfx950).
 *
 * Per row, with x [H] and a residual row r [H] (or none):
 *   s = x + r (rounded to the rows' type: s is the residual stream from here on)
 *   rstd = 1 / sqrt(sum_h s_h^2 / H + eps),   y_h = s_h rstd gamma_h
 * and for upstream gradients dy (of y) and ds (of s, where it goes on; or none),
 * with xh_h = s_h rstd and d_h = dy_h gamma_h:
 *   dx_h     = ds_h + rstd (d_h - xh_h sum_j d_j xh_j / H)   (dr = dx)
 *   dgamma_h = sum over rows of dy_h xh_h
 * The sum of squares is fp32 within 16 lanes (512 columns at most) and 64 bits from
 * there on, of rows past 16,384 columns 64 bits throughout; the backward pass's sums
 * are fp32.  y and dx are rounded once.  y can come as rows of 8 bits with scales
 * (q8.h): formed in fp32, and again in 64 bits where that lies next to where e4m3 or
 * a scale turn, so that it is rounded to 8 bits as the 64-bit value of that sum is.
 * Every output is deterministic: sums run in a fixed order, without atomics.
 *
 * Conventions: as moebound.h (row-major contiguous device tensors, caller-
 * owned memory and workspace, no allocation or synchronisation, work enqueued
 * on `stream`, enum moe_status returns, host-side argument checks before
 * anything is enqueued, finite inputs: a row with NaN or Inf, or whose sum of
 * squares passes fp32's range, spoils that row and the sum over rows, nothing
 * else).
 *   dtype MOE_BF16: X, residual, S, Y, dY, dS, dX bfloat16; MOE_F32: fp32.
 *   gamma, rstd, dgamma are fp32 always.
 */
#ifndef RMS_H
#define RMS_H

#include <stddef.h>
#include <stdint.h>

#include "moebound.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Filled by rms_plan; passed unchanged to the other calls. */
typedef struct rms_plan {
    uint32_t magic;              /* set by rms_plan                          */
    int32_t dtype;               /* enum moe_dtype                           */
    int64_t N;                   /* rows                                     */
    int32_t H;                   /* row width                                */
    float eps;
    int32_t row_pitch;           /* of an 8-bit output, as in q8.h           */
    int32_t scale_pitch;
    int64_t bwd_workspace_bytes; /* workspace rms_backward needs             */
} rms_plan_t;

/*
 * rms_plan -- host only, pure.  N = 0 is valid (forward is a no-op, backward
 * zeroes dgamma).
 * Errors: MOE_EINVAL if out is NULL, N < 0, H < 1, dtype unknown, or eps not a
 *   finite number above 0.  MOE_EUNSUPPORTED if H > 65536 or N >= 2^31.
 */
int rms_plan(int64_t N, int32_t H, int32_t dtype, float eps, rms_plan_t* out);

/*
 * rms_forward -- Y, the sum S, and the statistic rms_backward needs.
 * Inputs (device): X [N][H]; residual [N][H] or NULL (none); gamma [H].
 * Outputs (device, overwritten): S [N][H], wanted with a residual and NULL
 *   without (S is then X); it may be X or the residual itself.  Y [N][H], which
 *   may be X itself where S is not.  rstd [N].
 * Errors: MOE_EINVAL (plan not from rms_plan, a required pointer NULL with
 *   N > 0, S without a residual or a residual without S), MOE_EHIP (enqueue
 *   failed).  Nothing is enqueued on the first.
 */
int rms_forward(const rms_plan_t* plan, const void* X, const void* residual, const float* gamma,
                void* S, void* Y, float* rstd, void* stream);

/*
 * rms_forward_q8 -- the same with Y as rows of 8 bits.
 * Outputs: Yq [N][row_pitch], 16-byte aligned, Ys [N][scale_pitch], 4-byte
 *   aligned (padding written too); S, rstd as in rms_forward.
 * Errors: as rms_forward, MOE_EINVAL also for Yq or Ys not aligned.
 */
int rms_forward_q8(const rms_plan_t* plan, const void* X, const void* residual,
                   const float* gamma, void* S, void* Yq, void* Ys, float* rstd, void* stream);

/*
 * rms_backward -- gradients of <Y, dY> + <S, dS>.
 * Inputs (device): S [N][H] and rstd [N] as rms_forward returned them; gamma;
 *   dY [N][H]; dS [N][H] or NULL (none).  For an 8-bit Y the gradient is that of
 *   the unrounded one.
 * Outputs (device, overwritten): dX [N][H], the gradient of X and of the
 *   residual alike (may be dY or dS itself); dgamma [H].
 * workspace: at least plan->bwd_workspace_bytes bytes, 256-byte aligned;
 *   contents on entry do not matter.  It holds the partial sums over rows, and
 *   serves one call at a time: calls that may overlap each take their own.
 * Errors: as rms_forward; MOE_EINVAL also for a workspace that is not
 *   256-byte aligned, MOE_EWORKSPACE for one that is too small.
 */
int rms_backward(const rms_plan_t* plan, const void* S, const float* gamma, const void* dY,
                 const float* rstd, const void* dS, void* dX, float* dgamma, void* workspace,
                 size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* RMS_H */
