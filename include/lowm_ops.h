/*
 * lowm_ops.h -- C ABI of the operators that stand next to the low-M GEMM of
 * lowm.h in a decode step, for AMD Instinct MI355X (gfx950).  Exported by
 * liblowm.so.
 *
 *   lowm_residual_norm   norm after a block, gate, residual add, norm before
 *                        the next block, to bf16 or to int8 with a row scale
 *   lowm_quantize_rows   rows to int8 with a scale per row
 *   lowm_gemm_i8         C = (A W^T) scaled per row and column, int8 operands
 *   lowm_moe             a mixture-of-experts layer for up to 64 tokens
 *   lowm_token_logprobs  log probability of a given token per row, entropy,
 *                        rank and the most likely alternatives
 *
 * Conventions are those of lowm.h: the caller owns every buffer, the library
 * allocates nothing and keeps no state between calls; a call validates its
 * arguments on the host before any HIP call, enqueues its kernels on `stream`
 * (a hipStream_t; NULL is the null stream) and returns.  Return values are
 * the LOWM_* codes of lowm.h; lowm_last_hip_error() gives the cause of
 * LOWM_ERR_LAUNCH.  Every struct below is read during the call only.  All
 * calls can be captured into a HIP graph.
 */
#ifndef LOWM_OPS_H
#define LOWM_OPS_H

#include <stddef.h>
#include <stdint.h>

#include "lowm.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Element types of the operands that may have more than one. */
#define LOWM_BF16 0
#define LOWM_F32 1
#define LOWM_I8 2

/*
 * Norms before and after a block, with the block's gate and the residual.
 * For each of M rows of D elements, in fp32:
 *
 *     p  = N(y) * w_post                (y itself without LOWM_NORM_POST)
 *     r' = residual_scale * r + branch_scale * gate * p
 *     x  = N(r') * w_pre                (skipped with LOWM_NORM_NO_PRE)
 *     N(v) = v / sqrt(mean(v^2) + eps)                     or, LOWM_NORM_CENTER,
 *     N(v) = (v - mean(v)) / sqrt(var(v) + eps)            (biased variance)
 *
 * r' is rounded once to the residual's type; x is computed from the unrounded
 * r' and rounded once to bf16, or stored as int8 with
 *     x_scale[row] = max|x| / 127,  q = rint(x / x_scale)  (ties to even);
 * an all-zero row has scale 0 and q 0; a row with an infinity or a NaN has
 * scale NaN and q 0.
 *
 * Rows start at ld_* elements from one another (>= D); elements of a row are
 * contiguous.  The gate's element (m, d) is gate[m * gate_row + d * gate_col]
 * (strides in elements, gate_col 0 or 1): (0, 1) is a gate per channel, (1, 0) one per row,
 * (D, 1) one per element.  NULL: w_post, w_pre, gate are ones.  r_out may be
 * r itself (same ld_r); otherwise no output may overlap an input or another
 * output.  y and x may not overlap.
 */
#define LOWM_NORM_POST 1
#define LOWM_NORM_NO_PRE 2
#define LOWM_NORM_CENTER 4
#define LOWM_NORM_MAX_D 16384
typedef struct lowm_residual_norm_args {
    const void* y;          /* [M, D] y_type: the block's output */
    const void* r;          /* [M, D] r_type: the residual stream */
    void* r_out;            /* [M, D] r_type */
    void* x;                /* [M, D] x_type (NULL with LOWM_NORM_NO_PRE) */
    float* x_scale;         /* [M], only for x_type LOWM_I8 */
    const void* w_post;     /* [D] w_type or NULL */
    const void* w_pre;      /* [D] w_type or NULL */
    const void* gate;       /* gate_type or NULL */
    int64_t ld_y, ld_r, ld_r_out, ld_x;
    int64_t gate_row, gate_col;
    int32_t M, D;
    int32_t y_type, r_type, w_type, gate_type;   /* LOWM_BF16 or LOWM_F32 */
    int32_t x_type;                              /* LOWM_BF16 or LOWM_I8 */
    int32_t flags;
    float residual_scale, branch_scale, eps;
} lowm_residual_norm_args;

/* Errors: NULL operand, M < 0, D < 1, ld < D, overlap, an unknown type or a
 * flag: LOWM_ERR_INVALID_ARG; D > LOWM_NORM_MAX_D, a pointer not aligned to
 * its element: LOWM_ERR_UNSUPPORTED.  M == 0 does nothing. */
int lowm_residual_norm(const lowm_residual_norm_args* args, void* stream);

/*
 * q[m][k] = rint(x[m][k] / scale[m]), scale[m] = max_k |x[m][k]| / 127, with
 * the zero and non-finite rows of lowm_residual_norm.  x bf16 or fp32 [M, K]
 * (rows ld_x apart), q int8 [M, K] dense, scale fp32 [M].  Any M; K <=
 * LOWM_QUANTIZE_MAX_K.  Errors as lowm_residual_norm.
 */
#define LOWM_QUANTIZE_MAX_K 32768
int lowm_quantize_rows(const void* x, int x_type, int64_t ld_x, int M, int K, void* q,
                       float* scale, void* stream);

#ifdef __cplusplus
}
#endif
#endif /* LOWM_OPS_H */
