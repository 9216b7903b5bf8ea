/*
 * distill.h -- C ABI of distillation from a teacher's top logits through the
 * vocabulary projection, computed over vocabulary strips (part of
 * libmoebound.so), for AMD Instinct MI355X (gfx950).
 *
 * The student's logits over the vocabulary never exist as a whole: the strips
 * are cce.h's.  Per token t with hidden row x_t, temperature T, and the
 * teacher's list of K entries (index i_j, logit t_j):
 *   y_tv  = x_t W[v]                                student logits
 *   lse_t = log sum_v exp(y_tv / T),   q_v = exp(y_tv / T - lse_t)
 *   p     = softmax of t_j / T over the list's entries
 *   loss_t = T^2 sum_j p_j (log p_j - log q_{i_j})
 * and, for an upstream gradient dloss_t,
 *   dy_tv = dloss_t T (q_v - sum of p_j over j with i_j = v)
 *   dX    = dy W,   dW = dy^T X.
 * An entry with an index outside [0, V), or a logit of -inf or NaN, is no
 * part of the list (lists may so be of different lengths); a token whose list
 * is empty is ignored: loss 0 and no gradient, lse still computed.  An index
 * that occurs twice counts twice, each entry by itself.  The teacher gets no
 * gradient.
 *
 * The forward pass takes the logits' statistics as cce_forward does, over
 * strips of its own that depend on N, V and H alone (it keeps no logits, and
 * v_chunk does not bear on it), and then forms the list entries' logits as K
 * products of rows, so its cost does not grow with K V.
 * The backward pass recomputes each strip's logits, stores the strip's share
 * of dy in bf16 (the only strip-sized buffer), corrects the list entries that
 * fall into the strip, and consumes it in the dX and dW products.  That
 * rounding, up to 2^-8 of an entry of dy, limits dX and dW, also where dW is
 * fp32.  A small batch would fill few of the GPU's units with one strip of
 * v_chunk entries, so its strips are as many times v_chunk as fit that buffer
 * into KD_STRIP_BYTES, and its dX is summed over ranges of the vocabulary that
 * run side by side, in at most 64 MiB of sums (one sum: 4 N H bytes).  Every
 * output is deterministic, and bitwise independent of v_chunk as cce.h's are.
 *
 * lse is fp32 and y / T is formed in fp32, so q is off by up to |y / T| 2^-22
 * of itself: temperatures that take y / T towards 2^22 leave nothing of it.
 *
 * Conventions: as cce.h.  X [N][H] and W [V][H] are bfloat16; t_idx [N][K]
 * int32, t_logit [N][K] fp32; loss, lse, dloss [N] and y_top [N][K] fp32; dX
 * [N][H] bfloat16; dW [V][H] fp32 or bfloat16, as the plan says.
 */
#ifndef DISTILL_H
#define DISTILL_H

#include <stddef.h>
#include <stdint.h>

#include "moebound.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Strips wider than v_chunk keep the strip buffer within this. */
#define KD_STRIP_BYTES (64u << 20)

/* Filled by kd_plan; passed unchanged to the other calls. */
typedef struct kd_plan {
    uint32_t magic;               /* set by kd_plan                           */
    int32_t dtype;                /* enum moe_dtype (MOE_BF16)                */
    int64_t N;                    /* tokens                                   */
    int64_t V;                    /* vocabulary entries                       */
    int32_t H;                    /* hidden width                             */
    int32_t v_chunk;              /* least strip width                        */
    int32_t K;                    /* entries of a teacher's list              */
    float temperature;
    int32_t dw_dtype;             /* enum moe_dtype of dW                     */
    int32_t S;                    /* strips, ceil(V / strip); 0 if N = 0      */
    int32_t strip;                /* strip width: v_chunk, or a multiple with
                                     strip_bound_bytes <= KD_STRIP_BYTES      */
    int32_t reserved0;
    int64_t strip_bound_bytes;    /* N * min(strip, V) * 2                    */
    int64_t fwd_workspace_bytes;  /* workspace kd_forward needs               */
    int64_t bwd_workspace_bytes;  /* workspace kd_backward needs              */
} kd_plan_t;

/*
 * kd_plan -- strip plan and workspace sizing.  Host only, pure.  N = 0 is
 * valid (S = 0; the calls are no-ops, except that kd_backward zeroes dW).
 * Errors: MOE_EINVAL if out is NULL, N < 0, V < 1, H < 1, v_chunk < 1, K < 1,
 *   temperature not a finite number above 0 with a finite fp32 reciprocal, or a
 *   dtype unknown.
 *   MOE_EUNSUPPORTED if dtype is not MOE_BF16, H is not a multiple of 128,
 *   v_chunk is not a multiple of 256, N*H, N*v_chunk or v_chunk*H reach 2^30,
 *   V >= 2^31, or K > 256.
 */
int kd_plan(int64_t N, int32_t H, int64_t V, int32_t v_chunk, int32_t K, float temperature,
            int32_t dtype, int32_t dw_dtype, kd_plan_t* out);

/*
 * kd_forward -- per-token loss and the state kd_backward needs.
 * Inputs (device): X, W, t_idx, t_logit.
 * Outputs (device, overwritten): loss [N], lse [N], y_top [N][K] (the
 *   student's logits at the list's entries; 0 where an entry is no part of it).
 * workspace: at least plan->fwd_workspace_bytes bytes, 256-byte aligned;
 *   contents on entry do not matter.
 * Errors: MOE_EINVAL (plan not from kd_plan, a required pointer NULL with
 *   N > 0, workspace not 256-byte aligned, X or W (kd_backward: dX or dW) not
 *   16-byte aligned), MOE_EWORKSPACE (too small),
 *   MOE_EHIP (enqueue failed).  Nothing is enqueued on the first two.
 */
int kd_forward(const kd_plan_t* plan, const void* X, const void* W, const int32_t* t_idx,
               const float* t_logit, float* loss, float* lse, float* y_top, void* workspace,
               size_t workspace_bytes, void* stream);

/*
 * kd_backward -- gradients of sum_t dloss_t loss_t.
 * Inputs (device): X, W, t_idx, t_logit as in kd_forward; lse, y_top as it
 *   returned them; dloss [N].
 * Outputs (device, overwritten): dX [N][H] bf16 (rounded once from the fp32
 *   sum over the vocabulary); dW [V][H], fp32 or rounded once to bf16.
 * workspace: at least plan->bwd_workspace_bytes bytes, 256-byte aligned.
 * Errors: as kd_forward, against bwd_workspace_bytes.
 */
int kd_backward(const kd_plan_t* plan, const void* X, const void* W, const int32_t* t_idx,
                const float* t_logit, const float* lse, const float* y_top, const float* dloss,
                void* dX, void* dW, void* workspace, size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* DISTILL_H */
