/*
 * q8.h -- C ABI of rows in 8 bits, and of SwiGLU with activation checkpoints in
 * 8 bits (part of libmoebound.so), for AMD Instinct MI355X (gfx950).
 *
 * A matrix [N][H] in 8 bits is two arrays:
 *   q  e4m3 numbers (OCP: finite up to 448, NaN 0x7f / 0xff, no infinity), rows
 *      of row_pitch = H rounded up to a multiple of 128 bytes, zeros past H;
 *   s  scales, one byte b per row and 128 columns, standing for 2^(b - 127)
 *      (E8M0), rows of scale_pitch = ceil(H / 128) rounded up to a multiple of 4
 *      bytes, 127 past the last block.
 * The value is q 2^(b - 127).  A power of two costs an 8-bit floating-point
 * number nothing (its rounding is relative), the matrix instruction applies it
 * by itself, and every value whose scale is 2^-110 or more is a bfloat16 number.
 * The scale that the operators here write is the smallest power of two, from
 * 2^-110 up, under which the block's largest finite magnitude is at most 448;
 * quotients are rounded once, to the nearest, ties to even.  A value that is
 * NaN or infinite becomes NaN and has no part in the scale.  (A magnitude of
 * 1.9375 * 2^127 or more is nearest to 2^128: infinite when it is unpacked.)
 *
 * SwiGLU: h = silu(a) u = a u / (1 + e^-a).  Its backward pass needs a and u;
 * kept in 8 bits they take half the memory of bfloat16 and spare the products
 * that recomputing them would cost.  With a, u the values kept, g = 1 / (1 + e^-a):
 *   dU = dH a g,   dA = dH u g (1 + a (1 - g)).
 *
 * Conventions: as moebound.h (row-major contiguous device tensors, caller-
 * owned memory, no allocation or synchronisation, work enqueued on `stream`,
 * enum moe_status returns, host-side argument checks before anything is
 * enqueued).  q arrays are 16-byte aligned, s arrays 4-byte aligned; other
 * tensors have their element's alignment.  Outputs do not overlap inputs, but
 * for q8_swiglu_backward's dA, which may be dH.
 *   dtype MOE_BF16: unquantised tensors bfloat16; MOE_F32: fp32.
 */
#ifndef Q8_H
#define Q8_H

#include <stddef.h>
#include <stdint.h>

#include "moebound.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Filled by q8_plan; passed unchanged to the other calls. */
typedef struct q8_plan {
    uint32_t magic;      /* set by q8_plan                                 */
    int32_t dtype;       /* enum moe_dtype of the unquantised tensors      */
    int64_t N;           /* rows                                           */
    int32_t H;           /* row width                                      */
    int32_t row_pitch;   /* bytes of a row of q: H to a multiple of 128    */
    int32_t scale_pitch; /* bytes of a row of s: blocks to a multiple of 4 */
    int32_t reserved0;
} q8_plan_t;

/*
 * q8_plan -- host only, pure.  N = 0 is valid (every call is a no-op).
 * Errors: MOE_EINVAL if out is NULL, N < 0, H < 1, or dtype unknown.
 *   MOE_EUNSUPPORTED if H > 65536 or N >= 2^31.
 */
int q8_plan(int64_t N, int32_t H, int32_t dtype, q8_plan_t* out);

/*
 * q8_pack -- X [N][H] to q [N][row_pitch], s [N][scale_pitch], padding included.
 * Errors: MOE_EINVAL (plan not from q8_plan, a pointer NULL with N > 0 or not
 *   aligned), MOE_EHIP (enqueue failed).
 */
int q8_pack(const q8_plan_t* plan, const void* X, void* q, void* s, void* stream);

/*
 * q8_unpack -- the values of q, s to X [N][H] (bfloat16: rounded to the nearest
 * where a scale below 2^-110, which nothing here writes, leaves its range).  A
 * scale byte of 255 (E8M0's NaN) gives NaN.
 * Errors: as q8_pack.
 */
int q8_unpack(const q8_plan_t* plan, const void* q, const void* s, void* X, void* stream);

/*
 * q8_pack_weights -- E matrices W [E][K][N] in 8 bits with one scale per 128 x
 * 128 block (the same rule, over the block's elements), along either axis:
 *   q, s    [E][K][N to 128], [E][ceil(K / 128)][ceil(N / 128) to 4]:
 *           rows along N, for products that sum over N (dX = dY W^T);
 *   qt, st  [E][N][K to 128], [E][ceil(N / 128)][ceil(K / 128) to 4]:
 *           rows along K, for products that sum over K (Y = X W).
 * Either pair may be NULL (not wanted), not both.  Both pairs hold the same
 * numbers and scales.
 * Errors: MOE_EINVAL (E < 0, K < 1, N < 1, dtype unknown, W NULL or half a pair
 *   or both pairs NULL with E > 0, a pointer not aligned), MOE_EUNSUPPORTED
 *   (K or N > 65536, E > 65535), MOE_EHIP.  E = 0 is a no-op.
 */
int q8_pack_weights(int32_t E, int32_t K, int32_t N, int32_t dtype, const void* W, void* q,
                    void* s, void* qt, void* st, void* stream);

/*
 * q8_swiglu_forward -- h in 8 bits (the next product's operand), and the
 * checkpoint of a and u that q8_swiglu_backward reads.
 * Inputs (device): A, U [N][H].
 * Outputs (device, overwritten): Hq, Hs; Aq, As, Uq, Us, each pair [N][row_pitch],
 *   [N][scale_pitch].  The four of the checkpoint may be NULL together (no
 *   backward pass).  h is formed from A and U themselves, not from the checkpoint,
 *   and rounded to 8 bits as its 64-bit value is: in fp32, and again in 64 bits
 *   where that lies next to a border of e4m3 or of a scale.
 * Errors: as q8_pack; MOE_EINVAL also for a part of a checkpoint.
 */
int q8_swiglu_forward(const q8_plan_t* plan, const void* A, const void* U, void* Hq, void* Hs,
                      void* Aq, void* As, void* Uq, void* Us, void* stream);

/*
 * q8_swiglu_backward -- gradients of <h, dH> at the checkpoint's values.
 * Inputs (device): Aq, As, Uq, Us as q8_swiglu_forward wrote them; dH [N][H].
 * Outputs (device, overwritten): dA (may be dH itself), dU [N][H].
 * Errors: as q8_pack.
 */
int q8_swiglu_backward(const q8_plan_t* plan, const void* Aq, const void* As, const void* Uq,
                       const void* Us, const void* dH, void* dA, void* dU, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* Q8_H */
