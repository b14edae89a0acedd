/*
 * puro_attention.h -- C ABI of the attention block's operators for AMD
 * Instinct MI355X (gfx950): what a Qwen3-shaped layer runs between the QKV
 * projection's output and the O projection's input, forward and backward.
 *
 *   rotary positions      puro_rope_table, puro_rope
 *   query/key norms with  puro_qk_norm_rope, puro_qk_norm_rope_append,
 *   the rotation          puro_qk_norm_rope_backward
 *   attention             puro_attention, puro_attention_backward
 *
 * The pages on Puro-2B keep attention and the norms in BF16/FP32 around the
 * FP8 linears (en.roboind.com article, section "FP8 takes advantage of the RTX
 * 5090's low precision efficiency") of a Qwen3-compatible model (ainews.surl.tw
 * article); they give no formulas, which this library fixes below.  Tensors are
 * bf16, statistics, sums and tables fp32.
 *
 * The conventions of puro.h hold for every call: device pointers, 16-byte
 * aligned; host validation first and nothing enqueued on an error; no device
 * allocation; work enqueued on `stream`; thread-safe; outputs must not overlap
 * inputs or other outputs.  In addition:
 *   - Head tensors are [tokens][heads][head_dim] with the heads of a token
 *     densely packed and a free distance between tokens, the `stride` that goes
 *     with each pointer: in elements, a multiple of 8, at least heads *
 *     head_dim and below 2^23.  Slices of a projection's output (its query, key and value
 *     columns) are passed as they lie.  Two slices of the same rows do not
 *     overlap when their strides are equal and their columns are apart.
 *   - head_dim is 64 or 128.
 *   - Integer tensors (positions, rows, sequence starts and lengths) are device
 *     memory, 4-byte aligned, and cannot be checked on the host.  A value out
 *     of its range never makes a kernel read or write out of bounds; what it
 *     gives is stated at each call.
 */
#ifndef PURO_ATTENTION_H
#define PURO_ATTENTION_H

#include "puro.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    PURO_ROPE_HALF = 0,        /* pairs (i, i + rot/2), i < rot/2 */
    PURO_ROPE_INTERLEAVED = 1  /* pairs (2i, 2i + 1) */
} puro_rope_layout;

typedef enum {
    PURO_ROPE_PLAIN = 0,   /* f_i = base^(-2i/rot) */
    PURO_ROPE_LINEAR = 1,  /* f_i / factor: positions pressed into the trained range */
    PURO_ROPE_NTK = 2,     /* base * factor^(rot/(rot-2)) in place of base */
    PURO_ROPE_YARN = 3     /* f_i ((1-g)/factor + g) with g = clamp((trained f_i / 2 pi - 1) / 31, 0, 1): pairs that
                              turn more than 32 times in the trained length keep their frequency, those under one
                              turn are stretched; table scaled by 0.1 ln(factor) + 1.  The ramp is the published one,
                              over turns; model code that ramps over pair numbers instead, between the (rounded)
                              numbers of the pairs that turn 32 times and once, has other frequencies in between: for
                              weights tuned with those the caller fills the table, in the same layout */
} puro_rope_scaling;

/*
 * puro_rope_table -- the rotation's cosines and sines, made once per model.
 *   table  [positions][2][rot/2] fp32 (output): of position p the rot/2 values
 *          m cos(p f_i), then the rot/2 values m sin(p f_i), evaluated in fp64
 *          and rounded once (m = 1 except for PURO_ROPE_YARN)
 *   rot    rotated dimensions of a head: a multiple of 16, at most 128
 *   base   > 1; factor >= 1 and trained (positions of the trained context) > 0
 *          are read by the scalings that name them
 * Positions are below 2^24.
 */
puro_status puro_rope_table(int64_t positions, int64_t rot, double base, puro_rope_scaling scaling, double factor,
                            int64_t trained, float *table, puro_stream_t stream);

/* The rotation of a call's tokens. */
typedef struct {
    const float *table;       /* as puro_rope_table writes it */
    int64_t positions;        /* its positions */
    int64_t rot;              /* its rotated dimensions, at most head_dim; the others pass through */
    puro_rope_layout layout;
    const int32_t *pos;       /* [tokens], or NULL: token t stands at position t.  The rotated dimensions of a token
                                 whose position is not in 0 .. positions-1 become NaN */
} puro_rotation;

/*
 * puro_rope -- rotary positions alone: for each pair (a, b) of a head,
 *   a' = a cos - b sin,  b' = b cos + a sin      (inverse == 0)
 *   a' = a cos + b sin,  b' = b cos - a sin      (inverse != 0: the transpose,
 *                                                 which is the call's gradient)
 * in fp32, rounded once to bf16.
 *   x  [tokens][heads][head_dim], x_stride (input)
 *   y  [tokens][heads][head_dim], y_stride (output)
 */
puro_status puro_rope(const puro_rotation *r, int inverse, const uint16_t *x, int64_t x_stride, int64_t tokens,
                      int64_t heads, int64_t head_dim, uint16_t *y, int64_t y_stride, puro_stream_t stream);

/*
 * puro_qk_norm_rope -- RMS norm of every query and key head, then the rotation,
 * in one pass over the QKV projection's output:
 *   n = x / sqrt(mean(x^2) + eps) * w,  y = rotate(n)      (fp32, one rounding)
 *   x   [tokens][q_heads + k_heads (+ any more)][head_dim], x_stride (input)
 *   wq, wk  [head_dim] bf16: the weights of the query and of the key norms
 *   q   [tokens][q_heads][head_dim], q_stride;  k  [tokens][k_heads][head_dim],
 *       k_stride (outputs)
 * eps > 0.  Either head count may be 0.  Inputs below 2^60 in magnitude.
 */
puro_status puro_qk_norm_rope(const puro_rotation *r, const uint16_t *x, int64_t x_stride, int64_t tokens,
                              int64_t q_heads, int64_t k_heads, int64_t head_dim, const uint16_t *wq,
                              const uint16_t *wk, float eps, uint16_t *q, int64_t q_stride, uint16_t *k,
                              int64_t k_stride, puro_stream_t stream);

/*
 * puro_qk_norm_rope_append -- the same for serving: the keys go into a cache,
 * and the value heads that follow the key heads in x are copied into theirs.
 *   x        [tokens][q_heads + 2 k_heads][head_dim]
 *   cache_k  [cache_rows][k_heads][head_dim], k_stride; cache_v likewise
 *   rows     [tokens]: the cache row of each token.  A row outside 0 ..
 *            cache_rows-1 leaves both caches alone (the token's q is still
 *            written).  Tokens of one call that name the same row leave an
 *            unspecified mixture of their keys and values in it, head by head.
 */
puro_status puro_qk_norm_rope_append(const puro_rotation *r, const uint16_t *x, int64_t x_stride, int64_t tokens,
                                     int64_t q_heads, int64_t k_heads, int64_t head_dim, const uint16_t *wq,
                                     const uint16_t *wk, float eps, uint16_t *q, int64_t q_stride, uint16_t *cache_k,
                                     int64_t k_stride, uint16_t *cache_v, int64_t v_stride, const int32_t *rows,
                                     int64_t cache_rows, puro_stream_t stream);

/* Device workspace of puro_qk_norm_rope_backward. */
size_t puro_qk_norm_rope_backward_workspace_bytes(int64_t tokens, int64_t head_dim);

/*
 * puro_qk_norm_rope_backward -- its gradient.  With g = rotate^T(dy), r = 1 /
 * sqrt(mean(x^2) + eps) and h = x r:
 *   dx = r (w g - h mean(w g h)),   dw = sum over tokens and heads of g h
 *   dq, dk  the gradients of q and k (inputs);  x, wq, wk as in the forward call
 *   dx      [tokens][q_heads + k_heads][head_dim], dx_stride (output): written
 *           into the first columns of the projection output's gradient
 *   dwq, dwk  [head_dim] fp32 (outputs), summed in a fixed order; zeros where
 *           there is nothing to sum
 */
puro_status puro_qk_norm_rope_backward(const puro_rotation *r, const uint16_t *dq, int64_t dq_stride,
                                       const uint16_t *dk, int64_t dk_stride, const uint16_t *x, int64_t x_stride,
                                       int64_t tokens, int64_t q_heads, int64_t k_heads, int64_t head_dim,
                                       const uint16_t *wq, const uint16_t *wk, float eps, uint16_t *dx,
                                       int64_t dx_stride, float *dwq, float *dwk, void *workspace,
                                       size_t workspace_bytes, puro_stream_t stream);

/*
 * The shape of an attention call.
 *
 * Sequences.  q_start [sequences + 1] and k_start [sequences + 1] give the
 * first row of each sequence in q (q_tokens rows) and in k, v (k_tokens rows);
 * NULL for both and sequences == 1: one sequence of all rows.  k_len
 * [sequences], where given, says how many of a sequence's rows hold keys (a
 * cache with room left); NULL: all of them.  The starts ascend from 0 to the
 * row count; a sequence may be empty.  Starts and lengths out of range are
 * clamped into it, and rows that belong to no sequence are left unwritten.
 *
 * Mask.  The queries of a sequence are its last positions: query i of ql
 * queries and kl keys stands at p = kl - ql + i and sees key j when
 *   j <= p  and  (window == 0  or  j > p - window  or  j < sinks).
 * Keys that no query sees, and queries that see no key, have no part in any other
 * row, whatever they and their gradients hold.  A NaN or an infinity in a key or
 * value that some query sees, or in such a query's gradient, spreads to all
 * rows that see it and, times a probability of 0, may reach rows of the same
 * sequence that do not.
 *
 * Heads.  k_heads divides q_heads; query head h reads key head h / (q_heads /
 * k_heads).
 *
 * Sizes.  At most 2^30 query and key rows, 2^24 sequences and 2^16 query heads;
 * (q_tokens + 512 sequences) q_heads below 2^31, in the backward call three
 * quarters of it, and (k_tokens + 512 sequences) k_heads likewise.
 */
typedef struct {
    int64_t q_tokens, k_tokens, sequences;
    int64_t q_heads, k_heads, head_dim;
    int64_t q_stride, k_stride, v_stride, o_stride;     /* o_stride: o, and do in the backward call */
    int64_t dq_stride, dk_stride, dv_stride;            /* backward call only */
    int64_t max_k;      /* keys of the longest sequence, for planning how far long ones are split: any value >= 0
                           gives right results; 0: taken as k_tokens / sequences */
    int64_t window;     /* >= 0; 0: no window */
    int64_t sinks;      /* >= 0: first keys that stay visible outside the window */
    float scale;        /* of q . k: finite, at least 1e-30 */
} puro_attention_shape;

/* Device workspace of puro_attention and of puro_attention_backward for a shape (0: none; a shape that the call
 * refuses gives 0). */
size_t puro_attention_workspace_bytes(const puro_attention_shape *a);
size_t puro_attention_backward_workspace_bytes(const puro_attention_shape *a);

/*
 * puro_attention -- with S = scale q.k over the visible keys,
 *   lse = log sum exp S,   o = sum exp(S - lse) v
 * A query that sees no key gives o = 0 and lse = -infinity.
 *   o    [q_tokens][q_heads][head_dim] bf16, o_stride (output)
 *   lse  [q_heads][q_tokens] fp32 (output), or NULL
 * Products are bf16 with fp32 sums; exp(S - running maximum) is rounded to bf16
 * (for few queries to two of them, 16 bits) for its product with v, its sum is
 * not.  Deterministic for a given shape.
 */
puro_status puro_attention(const puro_attention_shape *a, const uint16_t *q, const uint16_t *k, const uint16_t *v,
                           const int32_t *q_start, const int32_t *k_start, const int32_t *k_len, uint16_t *o,
                           float *lse, void *workspace, size_t workspace_bytes, puro_stream_t stream);

/*
 * puro_attention_backward -- gradients of puro_attention (without k_len).  With
 * P = exp(S - lse), D = sum(do o) per row, dS = P (do.v - D):
 *   dq = scale sum dS k,  dk = scale sum dS q,  dv = sum P do
 * dk and dv sum over the query heads of a key head.  Rows that see nothing, and
 * keys that nothing sees, get zeros.
 *   o, lse  as puro_attention wrote them;  d_o  the gradient of o, laid out as o
 * Products are bf16 with fp32 sums: P and dS are rounded to bf16 for theirs.  D
 * from the rounded o is put right by the sum of the row's dS (0 for the exact D):
 * always for dk, for dq where that sum reaches 2^-6 of the root of the squared dS;
 * below it, it adds scale (sum dS) (sum P k) to dq.
 * Deterministic for a given shape.
 */
puro_status puro_attention_backward(const puro_attention_shape *a, const uint16_t *d_o, const uint16_t *q,
                                    const uint16_t *k, const uint16_t *v, const uint16_t *o, const float *lse,
                                    const int32_t *q_start, const int32_t *k_start, uint16_t *dq, uint16_t *dk,
                                    uint16_t *dv, void *workspace, size_t workspace_bytes, puro_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* PURO_ATTENTION_H */
