/*
 * lowm_cache.h -- C ABI of the attention part of a decode step and of the paged
 * 8-bit cache that it reads, for AMD Instinct MI355X (gfx950).  Exported by
 * liblowm.so.
 *
 *   lowm_rotary           rotary positions for queries and keys
 *   lowm_cache_append     new keys and values into the cache's pages
 *   lowm_cache_read       rows of the cache as bf16
 *   lowm_cache_attention  attention of each sequence's last rows over its cache
 *   lowm_fork_pages       sequences forked, reordered, freed; pages reserved
 *   lowm_compact_pages    pages moved to the lowest numbers
 *
 * Conventions are those of lowm_ops.h: the caller owns every buffer, the library
 * allocates nothing and keeps no state between calls; a call validates its
 * arguments on the host before any HIP call, enqueues its kernels on `stream` and
 * returns.  Every struct is read during the call only.  All calls can be captured
 * into a HIP graph: lengths, tables and positions are read on the device.  A
 * workspace serves one call at a time.
 *
 * The cache.  A page holds LOWM_PAGE = 64 tokens of every head of one layer, keys
 * and values apart, a byte an element, with one fp32 scale for each page and head:
 *
 *   k       [P][H][D / 16][64][16]    16 consecutive elements of a token together
 *   v       [P][H][4][D][16]          16 consecutive tokens of an element together
 *   k_scale, v_scale [P][H]
 *
 * so element d of token t of a page is byte [d / 16][t][d % 16] of its keys and
 * [t / 16][d][t % 16] of its values, and stands for that byte, as int8 or as e4m3
 * (1 sign, 4 exponent, 3 mantissa bits, bias 7, no infinity), times the scale, which
 * is not negative.  D is a multiple of 16 up to LOWM_CACHE_MAX_D.
 *
 * Sequences.  Row b of `table` [B][table_ld] (int32) lists the pages of sequence b
 * in order, and lens[b] (int32) counts its tokens, those of the call itself
 * included.  The call's rows lie one sequence after another: sequence b has rows
 * row_starts[b] .. row_starts[b + 1] - 1 of T (row_starts int32 [B + 1], not
 * falling), or T / B each where row_starts is NULL; row j of n stands at position
 * lens[b] - n + j, n and j by the bounds as they are given.  What cannot be is left
 * out, not followed, and moves nothing else: a position below 0 or past the table's
 * width, a page number outside 0 .. P - 1, rows outside 0 .. T - 1.
 */
#ifndef LOWM_CACHE_H
#define LOWM_CACHE_H

#include <stddef.h>
#include <stdint.h>

#include "lowm_ops.h"

#ifdef __cplusplus
extern "C" {
#endif

#define LOWM_E4M3 3

#define LOWM_PAGE 64
#define LOWM_CACHE_MAX_D 256
#define LOWM_CACHE_MAX_HEADS 1024
#define LOWM_CACHE_MAX_B 65536
#define LOWM_PAGES_MAX_R 4096
#define LOWM_PAGES_MAX_W 65536
#define LOWM_PAGES_MAX_P (1 << 24)

/* One layer of a cache (for lowm_fork_pages and lowm_compact_pages: `layers` of
 * them, one after another). */
typedef struct lowm_kv_cache {
    void* k;
    void* v;
    float* k_scale;
    float* v_scale;
    int32_t P, H, D;
    int32_t type;           /* LOWM_I8 or LOWM_E4M3 */
    int32_t layers;         /* 1 where one layer is meant */
} lowm_kv_cache;

typedef struct lowm_sequences {
    const int32_t* table;       /* [B][table_ld], W columns used */
    const int32_t* lens;        /* [B] */
    const int32_t* row_starts;  /* [B + 1] or NULL */
    int64_t table_ld;
    int32_t B, W, T;
} lowm_sequences;

/*
 * Rotary positions, for q [T, Hq, D] and, where it is not NULL, k [T, Hk, D].  Of
 * each head the R elements from `first` on are turned in pairs: elements i and
 * i + R/2 (LOWM_ROTARY_HALF) or 2i and 2i + 1 (LOWM_ROTARY_INTERLEAVED), i < R/2:
 *
 *     a = positions[t] * freqs[i]
 *     (x, y) -> scale * (x cos a - y sin a,  x sin a + y cos a)
 *
 * and the others are copied.  With LOWM_ROTARY_INVERSE the angle is -a (which is
 * also how a gradient goes back).  freqs fp64 [R/2], radians a position; the
 * product and its remainder by a turn are taken in fp64, so that far positions keep
 * their phase; the turn itself in fp32, rounded once to the type.
 *
 * q, k, and their outputs have one type, LOWM_BF16 or LOWM_F32; an element (t, h, d)
 * of x lies at t * x_row + h * x_head + d.  An output may be its own input (same
 * strides); no other overlap.  positions int32 or int64 [T].
 */
#define LOWM_ROTARY_HALF 0
#define LOWM_ROTARY_INTERLEAVED 1
#define LOWM_ROTARY_INVERSE 2
#define LOWM_ROTARY_MAX_D 1024
typedef struct lowm_rotary_args {
    const void* q;
    const void* k;
    void* q_out;
    void* k_out;
    const void* positions;
    const double* freqs;
    int64_t q_row, q_head, k_row, k_head, q_out_row, q_out_head, k_out_row, k_out_head;
    int32_t T, Hq, Hk, D, R, first;
    int32_t type;
    int32_t positions_bytes;    /* 8 or 4 */
    int32_t flags;
    float scale;
} lowm_rotary_args;

/* Errors: NULL operand, T < 0, a size < 1, R odd, first + R > D, a head or row
 * stride < 0 or rows that overlap, an unknown type or flag, overlap:
 * LOWM_ERR_INVALID_ARG; D past LOWM_ROTARY_MAX_D, heads past
 * LOWM_CACHE_MAX_HEADS, a pointer not aligned to its element: LOWM_ERR_UNSUPPORTED.
 * T == 0 does nothing. */
int lowm_rotary(const lowm_rotary_args* args, void* stream);

/*
 * New rows of keys and values into the cache, each page and head for itself:
 *
 *     s' = max |new| / top            top: 127 (int8) or 448 (e4m3)
 *     s' = max(s', s)                 where the page holds earlier tokens of the
 *                                     sequence (s: its scale before)
 *     new elements: round(x / s');    earlier ones, where s' > s: round(q * (s / s'))
 *
 * in fp32, round being to the nearest integer or e4m3 value, halves to even.  A page
 * of zeros has scale 0 and bytes 0.  A row with an infinity or a NaN makes the
 * page's scale NaN, until its first token is written again; its new bytes are 0 and
 * the earlier ones stay.  Bytes past the sequence's last token stay as they are.
 *
 * k, v [T, H, D] bf16 or fp32, both of one type, element (t, h, d) at
 * t * row + h * head + d.  A page that gets tokens must belong to one sequence
 * only (lowm_fork_pages sees to that).
 */
typedef struct lowm_cache_append_args {
    lowm_kv_cache cache;
    lowm_sequences seq;
    const void* k;
    const void* v;
    int64_t k_row, k_head, v_row, v_head;
    int32_t type;               /* LOWM_BF16 or LOWM_F32 */
} lowm_cache_append_args;

/* Errors, of this call and the next two: NULL operand, T or B or W < 0, a size < 1,
 * an unknown type, T no multiple of B where row_starts is NULL, a stride < 0 or rows of
 * k, v or q that overlap, an output that overlaps another operand:
 * LOWM_ERR_INVALID_ARG; D not a multiple of 16 or past LOWM_CACHE_MAX_D, B or heads
 * past their limits, k or v of the cache not 16-byte (another pointer: element)
 * aligned: LOWM_ERR_UNSUPPORTED.  T == 0 does nothing. */
int lowm_cache_append(const lowm_cache_append_args* args, void* stream);

/* The rows' keys and values as bf16 (byte times scale, rounded once), [T, H, D]
 * dense each; the inverse of an append.  Rows that are left out are not written. */
typedef struct lowm_cache_read_args {
    lowm_kv_cache cache;
    lowm_sequences seq;
    void* k_out;
    void* v_out;
} lowm_cache_read_args;
int lowm_cache_read(const lowm_cache_read_args* args, void* stream);

/*
 * Attention of the rows q [T, Hq, D] (bf16) over the cache of their sequences.  Head
 * h reads head h / (Hq / H) of the cache.  A row at position p sees tokens 0 .. p of
 * its sequence, or with window > 0 those from p - window + 1 on:
 *
 *     x_t = scale * q . k_t          lse = log sum_t e^x_t
 *     out = sum_t e^(x_t - lse) v_t
 *
 * out [T, Hq, D] bf16 dense, lse fp32 [T, Hq] where not NULL.  A row that sees
 * nothing has out 0 and lse -infinity; tokens on a page that the table does not
 * give (a number outside 0 .. P - 1) are not seen.  Rows of no sequence (behind the
 * last one) are not written.  What no row of a sequence sees may hold anything; but an
 * e4m3 NaN (lowm_cache_append writes none) among the values of a token that one of its
 * rows sees may reach that element of its other rows in the call too, and a page's scale
 * is every row's that sees a token of the page.
 *
 * Sums and softmax statistics are fp32, and a page's value scale may be any that is
 * finite, however far from another's.  The matrix products take fp16: a row of q scaled
 * by a power of two, the bytes as they are (both exact but for elements of q below 2^-28
 * of their row's largest), and each token's weight e^(x - lse) times its page's value
 * scale, rounded to 11 bits, or, below 2^-21 of the largest such product that the row
 * sees, to a multiple of 2^-31 of that, or of less.  So with w the weights, s the scales,
 * b the values' bytes and v = s b, an element of out is off by at most 2^-11 sum w |v| +
 * 2^-32 max (w s) sum |b| before it is rounded to bf16, beside fp32's own roundings: where
 * a page of much larger scale holds zeros in an element, little may be left of the others'.
 * The same inputs give the same bits.
 *
 * The workspace (lowm_cache_attention_workspace_bytes, 256-byte aligned) is zeroed once
 * before its first use; every call that completes leaves what must be zero so, for any
 * sizes.  The rest is not zero after a call: a workspace serves this operator alone
 * until it is zeroed again.
 */
typedef struct lowm_cache_attention_args {
    lowm_kv_cache cache;
    lowm_sequences seq;
    const void* q;
    void* out;
    float* lse;
    void* workspace;
    size_t workspace_bytes;
    int64_t q_row, q_head;      /* elements; rows of D are contiguous, 16-byte aligned */
    int32_t Hq;
    int32_t window;             /* 0: none */
    float scale;
} lowm_cache_attention_args;

/* Bytes of workspace a call needs (0 for sizes it would reject).  Host-only. */
size_t lowm_cache_attention_workspace_bytes(int T, int Hq, int H, int D);

/* Errors as lowm_cache_append; Hq no multiple of H, window < 0:
 * LOWM_ERR_INVALID_ARG; q, its strides or out not 16-byte, workspace not 256-byte
 * aligned, T Hq past 2^31 - 1, H (T Hq / (H R) + B + 1) (W + 72) past 2^30 - 1 with R =
 * 16, 32, 64 or 128 where T Hq is up to 16, 32 or 64 H B or more:
 * LOWM_ERR_UNSUPPORTED; a workspace that is missing or too small: LOWM_ERR_WORKSPACE. */
int lowm_cache_attention(const lowm_cache_attention_args* args, void* stream);

/*
 * The next step's sequences from this one's.  Row r goes on as its parent
 * parents[r] (itself, or any other; several rows may take one), or ends where that
 * is outside 0 .. R - 1.  With page counts n = ceil(len / 64):
 *
 *   - len' = len of the parent (0 for a row that ends; no more than the table's width
 *     holds), its first n pages shared with whoever has them;
 *   - a last page that is not full is the row's own to write on: of the rows whose
 *     unfinished last page it is, the lowest keeps it, if no other row has it as a
 *     whole page and `held` does not, and every other gets a copy, in all layers;
 *   - a row that goes on gets pages for `reserve` more tokens.
 *
 * New pages are the lowest that no row has and that are not held, first to the
 * lowest row, its copy before its reserve.  Pages past a row's n are given up:
 * freeing a sequence is a parent outside the rows.  Where pages run out, or the
 * table is too narrow, a row gets -1 there, a copy does not take place, and
 * missing counts them.  What is then appended there is lost, and is not seen later:
 * a row that goes on with an unfinished last page that the table does not give is
 * counted by every call, until that page is full (the next one is reserved as
 * usual) or the row ends.
 *
 * parents NULL: every row its own.  held (int32 [P], NULL: none): pages with a
 * value > 0 are in use by others and stay untouched.  refs' [P] counts the rows'
 * uses of each page, with held's.  Outputs may not overlap inputs.
 */
typedef struct lowm_fork_pages_args {
    lowm_kv_cache cache;
    const int32_t* table;       /* [R][W] dense */
    const int32_t* lens;        /* [R] */
    const int32_t* parents;     /* [R] or NULL */
    const int32_t* held;        /* [P] or NULL */
    int32_t* table_out;         /* [R][W] dense */
    int32_t* lens_out;          /* [R] */
    int32_t* refs_out;          /* [P] */
    int32_t* missing_out;       /* [1] */
    void* workspace;
    size_t workspace_bytes;
    int32_t R, W, reserve;
} lowm_fork_pages_args;

/* Bytes of workspace of this call and the next; it needs no clearing.  Host-only. */
size_t lowm_pages_workspace_bytes(int R, int W, int P);

/* Errors: NULL operand, a size < 1, reserve < 0, overlap: LOWM_ERR_INVALID_ARG; R
 * past LOWM_PAGES_MAX_R, W past LOWM_PAGES_MAX_W, P past LOWM_PAGES_MAX_P, reserve past
 * LOWM_PAGES_MAX_W pages, a wrong alignment: LOWM_ERR_UNSUPPORTED; LOWM_ERR_WORKSPACE
 * as above. */
int lowm_fork_pages(const lowm_fork_pages_args* args, void* stream);

/*
 * Compacting: the highest page that a row has moves to the lowest free one, the next
 * highest to the next lowest, and so on while that is lower; held pages stay.  The
 * bytes and scales of all layers move along, table' is the table with the new
 * numbers, refs' as above.  counts: [0] pages moved, [1] one more than the highest
 * page in use.  Every entry of the table counts (none is measured by a length).
 */
typedef struct lowm_compact_pages_args {
    lowm_kv_cache cache;
    const int32_t* table;
    const int32_t* held;
    int32_t* table_out;
    int32_t* refs_out;
    int32_t* counts_out;        /* [2] */
    void* workspace;
    size_t workspace_bytes;
    int32_t R, W;
} lowm_compact_pages_args;
int lowm_compact_pages(const lowm_compact_pages_args* args, void* stream);

#ifdef __cplusplus
}
#endif
#endif /* LOWM_CACHE_H */
