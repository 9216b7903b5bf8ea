/*
 * route.h -- C ABI of routing by scores and of the layer under a given
 * routing (part of libmoebound.so), for AMD Instinct MI355X (gfx950).
 *
 * moe_bounded_forward routes by the softmax of its own router's logits.  The
 * operators here take the logits from the caller and serve the other rules in
 * use: softmax or sigmoid scores, a bias per expert that steers the selection
 * only (load balance), selection limited to the best groups of experts,
 * gates renormalised over the selection or not, and a common factor.
 *
 * Per token, from its logits l_e (e < E):
 *   s_e   = softmax(l)_e            (ROUTE_SOFTMAX)
 *         = 1 / (1 + exp(-l_e))     (ROUTE_SIGMOID)
 *   v_e   = s_e + bias_e; without a bias experts rank by l_e, whose order is
 *           the scores'
 *   A logit of -inf (or NaN) masks its expert: s_e = 0, and it ranks behind
 *   every other expert.
 *   With n_group > 1 the experts are n_group runs of E / n_group.  A group's
 *   strength is the sum of its group_top (1 or 2) largest v_e over experts
 *   that are not masked, -inf if there are none; the topk_group strongest
 *   groups are kept, and only their experts can be selected.
 *   S     = the k experts that rank highest, slot s holding the s-th
 *   g_s   = scale * s_e / (renorm ? sum over S of s : 1),  e = S[s]; 0 where
 *           s_e is 0
 * Every order is by value descending, then index ascending.  Scores that
 * decide an order are compared in 64 bits wherever 32 bits could get it wrong,
 * so topk_idx is the definition's wherever fp64 tells the values apart: values
 * of different logits or biases, and sums of two, that are equal but for fp64's
 * rounding may come in either order.  The bias has no gradient.
 *
 * For an upstream gradient dg_s of the gates, with w_s = g_s / scale:
 *   sigmoid:            dl_e = w_s (1 - s_e) (scale dg_s - [renorm] sum_j g_j dg_j)
 *   softmax, renorm:    dl_e = w_s (scale dg_s - sum_j g_j dg_j)
 *   softmax, no renorm: dl_e = [e in S] g_s dg_s - s_e sum_j g_j dg_j   (all e)
 * and 0 for every other expert in the first two.
 *
 * Conventions: as moebound.h (row-major contiguous device tensors, caller-
 * owned memory, no allocation or synchronisation, work enqueued on `stream`,
 * enum moe_status returns, host-side argument checks before anything is
 * enqueued).  Logits, gates and their gradients are fp32.  A logit of +inf
 * gives unspecified gates; topk_idx still holds k distinct experts.
 */
#ifndef ROUTE_H
#define ROUTE_H

#include <stddef.h>
#include <stdint.h>

#include "moebound.h"

#ifdef __cplusplus
extern "C" {
#endif

enum route_score { ROUTE_SOFTMAX = 0, ROUTE_SIGMOID = 1 };

/* Filled by route_plan; passed unchanged to the other calls. */
typedef struct route_plan {
    uint32_t magic;      /* set by route_plan                             */
    int32_t score;       /* enum route_score                              */
    int64_t N;           /* tokens                                        */
    int32_t E, k;        /* experts, experts selected per token           */
    int32_t n_group;     /* groups of experts; 1: no group limit          */
    int32_t topk_group;  /* groups kept per token                         */
    int32_t group_top;   /* values summed into a group's strength, 1 or 2 */
    int32_t renorm;      /* 1: gates sum to scale                         */
    float scale;         /* factor on every gate                          */
    int32_t reserved0;
} route_plan_t;

/*
 * route_plan -- host only, pure.  N = 0 is valid (the calls are no-ops).
 * Errors: MOE_EINVAL if out is NULL, N < 0, E < 1, k < 1, k > E, score
 *   unknown, n_group < 1, E not a multiple of n_group, topk_group outside
 *   [1, n_group], k > topk_group * (E / n_group), group_top not 1 or 2,
 *   renorm not 0 or 1, or scale not a finite number above 0.
 *   MOE_EUNSUPPORTED if E > 1024, k > 64, n_group > 64 or N >= 2^26.
 */
int route_plan(int64_t N, int32_t E, int32_t k, int32_t score, int32_t n_group,
               int32_t topk_group, int32_t group_top, int32_t renorm, float scale,
               route_plan_t* out);

/*
 * route_forward -- the selection and its gates.
 * Inputs (device): logits [N][E] fp32; bias [E] fp32 (finite) or NULL.
 * Outputs (device, overwritten): topk_idx [N][k] int32, gates [N][k] fp32, in
 *   slot order, as moe_routed_forward takes them.
 * Errors: MOE_EINVAL (plan not from route_plan, a required pointer NULL with
 *   N > 0), MOE_EHIP (enqueue failed).  Nothing is enqueued on the first.
 */
int route_forward(const route_plan_t* plan, const float* logits, const float* bias,
                  int32_t* topk_idx, float* gates, void* stream);

/*
 * route_backward -- gradient of the logits with the selection held constant.
 * Inputs (device): logits as in route_forward; topk_idx [N][k] as it returned
 *   them (an entry outside [0, E) counts as an expert with s = 0); dgates
 *   [N][k] fp32, as moe_routed_backward returns them.
 * Output (device, overwritten): dlogits [N][E] fp32; it must not overlap
 *   logits.
 * Errors: as route_forward.
 */
int route_backward(const route_plan_t* plan, const float* logits, const int32_t* topk_idx,
                   const float* dgates, float* dlogits, void* stream);

/*
 * moe_routed_forward -- the layer's expert pass under a given routing:
 * moe_bounded_forward without its router.  plan is a moe_plan_t
 * (moe_plan_chunks); topk_idx [N][k] int32 must hold experts in [0, E),
 * distinct within a row; gates [N][k] fp32 may be any finite values.  Same
 * chunk schedule, buffers, workspace size, numerics and stats as
 * moe_bounded_forward; with that call's topk_idx and gates, Y is bitwise its Y.
 * Errors: as moe_bounded_forward; MOE_EINVAL also where N > 0 and X, a weight
 *   matrix or Y is not 16-byte aligned.
 */
int moe_routed_forward(const moe_plan_t* plan, const void* X, const void* W_gate,
                       const void* W_up, const void* W_down, const int32_t* topk_idx,
                       const float* gates, void* Y, void* workspace, size_t workspace_bytes,
                       void* stream, moe_stats_t* stats);

/*
 * moe_routed_backward -- gradients of <Y, dY> for moe_routed_forward:
 * moe_bounded_backward without its router.  Outputs (device, overwritten):
 * dX [N][H] through the experts only (the caller adds its router's share);
 * dW_gate, dW_up, dW_down fp32 and dgates [N][k] fp32, bitwise
 * moe_bounded_backward's.  MOE_PLAN_EXACT_DW plans are served.
 * Errors: as moe_bounded_backward; MOE_EINVAL also where N > 0 and X, dY, dX, a
 *   weight matrix or its gradient is not 16-byte aligned.
 */
int moe_routed_backward(const moe_plan_t* plan, const void* X, const void* W_gate,
                        const void* W_up, const void* W_down, const void* dY,
                        const int32_t* topk_idx, const float* gates, void* dX, float* dW_gate,
                        float* dW_up, float* dW_down, float* dgates, void* workspace,
                        size_t workspace_bytes, void* stream, moe_stats_t* stats);

#ifdef __cplusplus
}
#endif

#endif /* ROUTE_H */
