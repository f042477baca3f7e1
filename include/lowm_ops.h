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
 * calls can be captured into a HIP graph.  The current device has to be that of
 * the buffers and of the stream.
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
 * output.  Column ranges of one buffer do not overlap if their ld are equal bytes.
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

/*
 * C[m][n] = (sum_k A[m][k] W[n][k]) * a_scale[m] * w_scale[n], the sum exact in
 * int32, scaled in fp32 and rounded once.  A [M, K] int8 with a_scale [M], or
 * bf16, which the call quantises per row as lowm_quantize_rows does (a row with
 * an infinity or a NaN gives a row of NaN); W [N, K] int8 with w_scale [N]; C
 * [M, N] bf16 or fp32; scales fp32.  All dense row-major; 1 <= M <= LOWM_MAX_M.
 *
 * The workspace (lowm_gemm_i8_workspace_bytes, 256-byte aligned) holds the
 * quantised rows of a bf16 A and the partial sums where K is split over
 * workgroups.  It is zeroed once before its first use; every call that completes
 * leaves what must be zero so, for any sizes.  The rest is not zero after a call:
 * a workspace serves this operator alone until it is zeroed again.  One workspace
 * per call in flight.  An int8 A may come without one (NULL): K is then not split.
 * lowm_workspace_status reads it, with N = LOWM_I8_STATUS_N.
 */
#define LOWM_I8_STATUS_N 8192
#define LOWM_I8_MAX_N 1073741568   /* 2^30 - 256 */
typedef struct lowm_gemm_i8_args {
    const void* A;
    const void* W;
    const float* a_scale;   /* only for an int8 A */
    const float* w_scale;
    void* C;
    void* workspace;
    size_t workspace_bytes;
    int32_t M, N, K;
    int32_t a_type;         /* LOWM_I8 or LOWM_BF16 */
    int32_t c_type;         /* LOWM_BF16 or LOWM_F32 */
} lowm_gemm_i8_args;

/* Bytes of workspace (0 for sizes the call would reject).  Host-only. */
size_t lowm_gemm_i8_workspace_bytes(int M, int N, int K);

/* Errors: NULL operand, a size < 1, an unknown type, an output or workspace
 * that overlaps another operand: LOWM_ERR_INVALID_ARG; M > LOWM_MAX_M, N >
 * LOWM_I8_MAX_N, K not a multiple of 16, K > 131056 (> LOWM_QUANTIZE_MAX_K for a
 * bf16 A), A or W not 16-byte, the workspace not 256-byte aligned, another pointer
 * not aligned to its element: LOWM_ERR_UNSUPPORTED; a workspace that is missing or too small:
 * LOWM_ERR_WORKSPACE. */
int lowm_gemm_i8(const lowm_gemm_i8_args* args, void* stream);

/*
 * A mixture-of-experts layer for T <= LOWM_MOE_MAX_T tokens:
 *
 *     l[t][e] = sum_d x[t][d] router[e][d]
 *     s       = softmax over e of l[t], or with LOWM_MOE_SIGMOID 1 / (1 + e^-l)
 *     the top_k experts of token t: the largest l, or with a bias the largest
 *         s + bias[e]; equal ones by e
 *     gate    = s of the chosen, divided by their sum unless LOWM_MOE_NO_RENORM,
 *         times routed_scale
 *     h       = silu(x[t] . w13[e][i]) * (x[t] . w13[e][I + i])    i < I
 *     out[t]  = sum over the chosen of gate * (h . w2[e][d])
 *
 * x, out [T, D], router [E, D], w13 [E, 2I, D] (gate rows, then up rows), w2
 * [E, D, I] bf16, all dense; bias fp32 [E] or NULL.  Sums are fp32; h is
 * rounded to bf16 between the two products (the matrix units' input type) and
 * out once.  ids (int32) and gates (fp32) [T, top_k], the chosen experts in
 * order, are written where not NULL.  The same inputs give the same bits.
 *
 * The workspace (lowm_moe_workspace_bytes, 256-byte aligned) is zeroed once
 * before its first use; every call that completes leaves what must be zero so,
 * for any sizes.  The rest is not zero after a call: a workspace serves this
 * operator alone until it is zeroed again.  One workspace per call in flight.
 * lowm_workspace_status of the GEMM reads it too, with N = D + 80.
 */
#define LOWM_MOE_MAX_T 64
#define LOWM_MOE_MAX_E 256
#define LOWM_MOE_MAX_K 16
#define LOWM_MOE_SIGMOID 1
#define LOWM_MOE_NO_RENORM 2
typedef struct lowm_moe_args {
    const void* x;
    const void* router;
    const float* bias;
    const void* w13;
    const void* w2;
    void* out;
    int32_t* ids;
    float* gates;
    void* workspace;
    size_t workspace_bytes;
    int32_t T, D, I, E, top_k;
    int32_t flags;
    float routed_scale;
} lowm_moe_args;

/* Bytes of workspace a call needs (0 for sizes it would reject).  Host-only. */
size_t lowm_moe_workspace_bytes(int T, int D, int I, int E, int top_k);

/* Errors: NULL operand, a size < 1, top_k > E, an unknown flag, overlap of an
 * output or the workspace with another operand: LOWM_ERR_INVALID_ARG; T, E or
 * top_k past its limit, D or I not a multiple of 8 or past 65536, an operand
 * not 16-byte (ids, gates, bias: 4-byte, workspace: 256-byte) aligned:
 * LOWM_ERR_UNSUPPORTED; a workspace that is missing or too small:
 * LOWM_ERR_WORKSPACE.  T == 0 does nothing. */
int lowm_moe(const lowm_moe_args* args, void* stream);

/*
 * Log probabilities of given tokens.  For each of M rows of V logits, with
 * m = max_v l[v], S = sum_v e^(l[v] - m) and log p[v] = l[v] - m - log S:
 *
 *     logprob = log p[token]
 *     entropy = -sum_v p[v] log p[v] = log S - (sum_v e^(l[v]-m) (l[v]-m)) / S
 *     rank    = how many logits are greater than the token's
 *     top_logprob, top_id [top_n]: the largest log p, in order; equal ones by id
 *
 * in fp32, from one pass over the logits.  A logit of -infinity is a masked
 * token: its probability is 0 and it is never an alternative.  Alternatives
 * past the last unmasked one have log p -infinity and id -1.  A row with
 * nothing unmasked has logprob -infinity, entropy 0, rank 0 and no alternatives.
 * A token outside 0 .. V-1 has logprob NaN and rank -1.  A row with a NaN or
 * a +infinity has no distribution: logprob, entropy and every top_logprob are
 * NaN and every top_id is -1.  The rank goes by comparison (a NaN is greater
 * than nothing, and nothing than it).
 *
 * logits bf16 or fp32, rows ld elements apart (>= V); tokens int64 or int32
 * [M]; logprob, entropy fp32 [M]; rank int32 [M]; top_logprob fp32 and top_id
 * int32 [M, top_n] (unused with top_n 0, at most LOWM_LOGPROBS_MAX_TOP).
 * logits must not overlap an output or the workspace.
 *
 * The workspace (256-byte aligned; it may be NULL where
 * lowm_token_logprobs_workspace_bytes is 0, as for many rows) joins the pieces
 * that few rows are cut into.  It is zeroed once before its first use; every
 * call that completes leaves it zero, for any sizes.  One workspace per call in
 * flight.  lowm_workspace_status reads it, with N = LOWM_LOGPROBS_STATUS_N.
 */
#define LOWM_LOGPROBS_STATUS_N 8192
#define LOWM_LOGPROBS_MAX_TOP 32
typedef struct lowm_token_logprobs_args {
    const void* logits;
    const void* tokens;
    float* logprob;
    float* entropy;
    int32_t* rank;
    float* top_logprob;
    int32_t* top_id;
    void* workspace;
    size_t workspace_bytes;
    int64_t ld;
    int32_t M, V, top_n;
    int32_t logits_type;    /* LOWM_BF16 or LOWM_F32 */
    int32_t tokens_bytes;   /* 8 (int64) or 4 (int32) */
} lowm_token_logprobs_args;

/* Bytes of workspace a call needs (0 for arguments it would reject).
 * Host-only. */
size_t lowm_token_logprobs_workspace_bytes(int M, int V, int top_n);

/* Errors: NULL operand, M < 0, V < 1, ld < V, top_n < 0, an unknown type,
 * overlap: LOWM_ERR_INVALID_ARG; top_n > LOWM_LOGPROBS_MAX_TOP, V > 2^30, a
 * pointer not aligned to its element (the workspace: to 256 bytes):
 * LOWM_ERR_UNSUPPORTED; a workspace that is missing or too small:
 * LOWM_ERR_WORKSPACE.  M == 0 does nothing. */
int lowm_token_logprobs(const lowm_token_logprobs_args* args, void* stream);

#ifdef __cplusplus
}
#endif
#endif /* LOWM_OPS_H */
