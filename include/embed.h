/*
 * embed.h -- C ABI of token embedding with scaling and its gradient (part of
 * libmoebound.so), for AMD Instinct MI355X (gfx950).
 *
 *   Y[t] = scale W[ids[t]]                      (fp32 product, rounded once)
 *   dW[v] = scale sum over t with ids[t] = v, t ascending, of dY[t]
 * An id outside [0, V) marks a padded position, as a target outside [0, V)
 * does in cce.h: its row of Y is 0 and it has no gradient.
 *
 * W [V][H] is laid out as cce.h's projection (one row per vocabulary entry),
 * so tied weights are one matrix; embed_backward then adds its gradient onto
 * the dW that cce_backward or kd_backward has written (accumulate).
 * The gradient sorts the positions by id, keeping their order within an id,
 * and sums each id's rows in fp32 over runs whose bounds depend on the sorted
 * ids alone: every output is deterministic, and no sum uses atomics.
 *
 * Conventions: as moebound.h (row-major contiguous device tensors, caller-
 * owned memory and workspace, no allocation or synchronisation, work enqueued
 * on `stream`, enum moe_status returns, host-side argument checks before
 * anything is enqueued, finite inputs).
 *   dtype MOE_BF16: W, Y, dY bfloat16; MOE_F32: fp32.  dW is fp32 always; ids
 *   are int32.
 */
#ifndef EMBED_H
#define EMBED_H

#include <stddef.h>
#include <stdint.h>

#include "moebound.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Filled by embed_plan; passed unchanged to the other calls. */
typedef struct embed_plan {
    uint32_t magic;              /* set by embed_plan                      */
    int32_t dtype;               /* enum moe_dtype                         */
    int64_t N;                   /* positions                              */
    int64_t V;                   /* vocabulary entries                     */
    int32_t H;                   /* row width                              */
    float scale;
    int64_t bwd_workspace_bytes; /* workspace embed_backward needs         */
} embed_plan_t;

/*
 * embed_plan -- host only, pure.  N = 0 is valid (forward is a no-op, backward
 * zeroes dW unless it accumulates).
 * Errors: MOE_EINVAL if out is NULL, N < 0, V < 1, H < 1, dtype unknown or
 *   scale not finite.  MOE_EUNSUPPORTED if N >= 2^26, V >= 2^30 or H > 65536.
 */
int embed_plan(int64_t N, int64_t V, int32_t H, int32_t dtype, float scale, embed_plan_t* out);

/*
 * embed_forward -- Inputs (device): W [V][H], ids [N].  Output (device,
 * overwritten): Y [N][H].
 * Errors: MOE_EINVAL (plan not from embed_plan, a required pointer NULL with
 *   N > 0), MOE_EHIP (enqueue failed).  Nothing is enqueued on the first.
 */
int embed_forward(const embed_plan_t* plan, const void* W, const int32_t* ids, void* Y,
                  void* stream);

/*
 * embed_backward -- Inputs (device): ids [N] as in embed_forward, dY [N][H].
 * Output (device): dW [V][H] fp32: overwritten whole, zeros for ids that do
 *   not occur; with accumulate != 0 the rows of ids that do occur are added to
 *   (each in one fp32 addition) and the others left as they are.
 * workspace: at least plan->bwd_workspace_bytes bytes, 256-byte aligned;
 *   contents on entry do not matter.  It holds the sort's keys and positions
 *   and the sums of runs that were split.
 * Errors: as embed_forward; MOE_EINVAL also for a workspace that is not
 *   256-byte aligned, MOE_EWORKSPACE for one that is too small.
 */
int embed_backward(const embed_plan_t* plan, const int32_t* ids, const void* dY, float* dW,
                   int32_t accumulate, void* workspace, size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* EMBED_H */
