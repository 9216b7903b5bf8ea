/*
 * gmm.h -- C ABI of matrix products grouped by expert, with ragged sizes, in
 * bfloat16 and in 8 bits (part of libmoebound.so), for AMD Instinct MI355X
 * (gfx950).
 *
 * Rows that belong to expert e stand together: rows offsets[e] .. offsets[e+1]-1
 * of an [R]-row matrix.  With X_e, dY_e these rows of X [R][K] and dY [R][N]:
 *   forward       Y_e  = X_e W[e]           W [E][K][N]
 *   backward, dX  dX_e = dY_e W[e]^T
 *   backward, dW  dW[e] = X_e^T dY_e        (zeros for an expert without rows)
 * The layer (moebound.h) runs such products inside; these are for experts of
 * another form than SwiGLU, for projections, and for training in 8 bits.  With
 * E = 1 and offsets NULL they are plain products of R rows.
 *
 * In 8 bits (q8.h) X is e4m3 with a scale per row and 128 columns, W e4m3 with a
 * scale per 128 x 128 block, its rows along the axis that is summed over:
 *   gmm8_forward      Y_e = X_e Wt[e]^T       Wt [E][N][K to 128]
 *   gmm8_backward_dw  dW[e] = X_e^T dY_e      X in 8 bits, as a checkpoint of the
 *                     forward pass's operand, dY bfloat16
 * dX in 8 bits is gmm8_forward of a plan (R, N, K, E) on dY's rows in 8 bits and
 * on W in 8 bits along N (q8_pack_weights gives both orientations).
 *
 * Y and dX are rounded once to bfloat16, dW is fp32.  Every output is
 * deterministic: sums run in a fixed order, without atomics; the order is the
 * call's (R, K, N, E), so a row has other bits in a call of other sizes, never by
 * what other rows hold.
 * Sums are fp32, but for one: gmm8_forward of more than four rows sums by the
 * matrix instruction for e4m3, which adds eight products at a time, each cut 2^13
 * below the largest of the eight, before they reach the fp32 accumulator.  Beside
 * fp32's roundings such a sum is off by up to GMM8_CUT of the sum of its products'
 * magnitudes; it shows where they cancel (of 2^16 - 2^16 + 4 in one eight nothing
 * is left).  Up to four rows are summed in fp32 from whole products.
 *
 * Conventions: as moebound.h (row-major contiguous device tensors, caller-
 * owned memory and workspace, no allocation or synchronisation, work enqueued
 * on `stream`, enum moe_status returns, host-side argument checks before
 * anything is enqueued).  Matrices are 16-byte aligned, scales and offsets
 * 4-byte aligned.  Outputs do not overlap inputs.
 *   offsets: int32 [E+1] on the device, ascending, in [0, R].  Rows outside
 *   [offsets[0], offsets[E]) are neither read nor written.  Offsets that break
 *   this give unspecified rows, but nothing outside the tensors is touched.
 *   A workspace serves one call at a time: calls that may overlap, on other
 *   streams or in graphs replayed side by side, each take their own.
 *   NaN or Inf in a row of X spoils that row of Y and its expert's dW; in W its
 *   expert's rows; nothing else.  A scale byte of 255 (E8M0's NaN) makes its
 *   block's numbers NaN.
 */
#ifndef GMM_H
#define GMM_H

#include <stddef.h>
#include <stdint.h>

#include "moebound.h"

#ifdef __cplusplus
extern "C" {
#endif

/* What the operands X and W are. */
enum gmm_operands {
    GMM_BF16 = 0, /* bfloat16: gmm_forward, gmm_backward_dx, gmm_backward_dw  */
    GMM_Q8 = 1    /* e4m3 with scales: gmm8_forward, gmm8_backward_dw         */
};

/* What seven of eight products lose at most, 2^-13 of the largest each (see above). */
#define GMM8_CUT (7.0 / 8192)

/* Filled by gmm_plan; passed unchanged to the other calls. */
typedef struct gmm_plan {
    uint32_t magic;    /* set by gmm_plan                                    */
    int32_t operands;  /* enum gmm_operands                                  */
    int64_t R;         /* rows                                               */
    int32_t K, N, E;
    int32_t row_pitch; /* bytes of a row of X: 2 K, or K to 128 in 8 bits    */
    int64_t fwd_workspace_bytes; /* forward and backward dX; may be 0        */
    int64_t bwd_workspace_bytes; /* backward dW; may be 0                    */
} gmm_plan_t;

/*
 * gmm_plan -- host only, pure.  R = 0 and E = 0 are valid (nothing to multiply;
 * backward dW still writes zeros).
 * Errors: MOE_EINVAL if out is NULL, R < 0, K < 1, N < 1, E < 0, operands
 *   unknown, N (and K in bfloat16) not a multiple of 8, or E = 0 with R > 0.
 *   MOE_EUNSUPPORTED if K or N > 65536, E > 1024, R >= 2^31 - 65536, 2 K N (the
 *   bytes of a matrix) >= 2^31, R max(K, N) >= 2^40, or a launch would have 2^32
 *   threads (within the limits before only near them: R past 2^31 - 2^19 over
 *   hundreds of experts).
 */
int gmm_plan(int64_t R, int32_t K, int32_t N, int32_t E, int32_t operands, gmm_plan_t* out);

/*
 * gmm_forward -- Y [R][N] = X [R][K] W[e].
 * offsets may be NULL where E = 1 (all rows).  workspace: at least
 *   plan->fwd_workspace_bytes bytes, 256-byte aligned; NULL where that is 0.
 * Errors: MOE_EINVAL (plan not from gmm_plan or of other operands, a pointer
 *   NULL with R > 0 or not aligned), MOE_EWORKSPACE, MOE_EHIP.
 */
int gmm_forward(const gmm_plan_t* plan, const void* X, const void* W, const int32_t* offsets,
                void* Y, void* workspace, size_t workspace_bytes, void* stream);

/* gmm_backward_dx -- dX [R][K] = dY [R][N] W[e]^T.  As gmm_forward. */
int gmm_backward_dx(const gmm_plan_t* plan, const void* dY, const void* W,
                    const int32_t* offsets, void* dX, void* workspace, size_t workspace_bytes,
                    void* stream);

/*
 * gmm_backward_dw -- dW [E][K][N] = X_e^T dY_e; with accumulate != 0 that is added
 * to what dW holds, one fp32 addition per element.
 * workspace: at least plan->bwd_workspace_bytes bytes, 256-byte aligned; NULL
 *   where that is 0.
 * Errors: as gmm_forward; X, dY may be NULL where R = 0.
 */
int gmm_backward_dw(const gmm_plan_t* plan, const void* X, const void* dY,
                    const int32_t* offsets, float* dW, int32_t accumulate, void* workspace,
                    size_t workspace_bytes, void* stream);

/*
 * gmm8_forward -- Y [R][N] = X Wt[e]^T in 8 bits; for R > 4 to GMM8_CUT (above).
 * Inputs (device): Xq [R][K to 128], Xs [R][ceil(K/128) to 4]; Wq [E][N][K to 128],
 *   Ws [E][ceil(N/128)][ceil(K/128) to 4].  The padding counts: zeros in q, and
 *   in s any byte but 255 past the last block.
 * Errors: as gmm_forward.
 */
int gmm8_forward(const gmm_plan_t* plan, const void* Xq, const void* Xs, const void* Wq,
                 const void* Ws, const int32_t* offsets, void* Y, void* workspace,
                 size_t workspace_bytes, void* stream);

/*
 * gmm8_backward_dw -- gmm_backward_dw with X in 8 bits; its values enter the
 * product as bfloat16, which holds them (scales of 2^-110 and more).
 */
int gmm8_backward_dw(const gmm_plan_t* plan, const void* Xq, const void* Xs, const void* dY,
                     const int32_t* offsets, float* dW, int32_t accumulate, void* workspace,
                     size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* GMM_H */
