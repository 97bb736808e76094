/*
 * seacells_token.h - C ABI of the token operators on MI355X (gfx950), in the
 * same library as seacells_fw.h (libseacells_fw.so).
 *
 * A fit gives cells (rows of K), archetypes and an assignment A. A model that
 * learns from them - cells or archetypes as tokens, K's neighbour lists as
 * training pairs, a cell's archetype as the class to predict - needs three
 * operators around its matrix products, each with its gradient:
 *
 *   embed        y[i] = scale * table[token[i]]
 *   embed_grad   d_table[t] = scale * sum of d_y[i] over token[i] = t
 *   layer_norm   y = (x - mean) * rstd * weight + bias, per row
 *   layer_norm_grad, with the sums of the weight's and the bias' gradient
 *   logprobs     log p of given classes, entropy, the top alternatives
 *   logprobs_grad
 *
 * Conventions (as in seacells_fw.h): the caller allocates every buffer; the
 * library never allocates or synchronises and enqueues all work on `stream`.
 * Return values are SEACELLS_OK or a negative SEACELLS_E_* code found on the
 * host before anything is enqueued; *status (device, where an entry point
 * takes one) is overwritten with the OR of SEACELLS_FLAG_* conditions the
 * kernels met. Results are deterministic (fixed summation orders, no
 * floating-point atomics); every call can be captured into a graph.
 *
 * Dense matrices are row-major with a row stride in elements (`*_ld`, at
 * least the row's length; anything the element type's alignment allows).
 * dtype arguments are SEACELLS_F32 / F16 / BF16. Sums, statistics and norms
 * are f32; each output element is rounded to its type once. n = 0 rows is
 * allowed and writes only what does not depend on rows. An output overlaps no
 * other operand, but where it is said that it may be one.
 */
#ifndef SEACELLS_TOKEN_H
#define SEACELLS_TOKEN_H

#include <stddef.h>
#include <stdint.h>

#include "seacells_fw.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Element types. */
#define SEACELLS_F32 0u
#define SEACELLS_F16 1u
#define SEACELLS_BF16 2u

/* An unknown or unsupported element type, or a pointer that is not aligned
 * to its element (return value). */
#define SEACELLS_E_TYPE (-6)

/* Longest row (elements of an embedding, a norm or a row of logits); row
 * counts and table rows may go to 2^31 - 1. SEACELLS_E_TOO_LARGE above. */
#define SEACELLS_MAX_WIDTH (1u << 23)

/* Most alternatives that seacells_logprobs returns per row. */
#define SEACELLS_TOP_MAX 64u

/*
 * Embedding lookup: out[i, :] = scale * table[tokens[i], :] for i < n.
 * table   device [v, d] of dtype, row stride table_ld; out [n, d] likewise.
 * tokens  device [n] int32. A negative token is padding: a row of zeros. A
 *         token >= v also gives zeros and sets SEACELLS_FLAG_BAD_INDEX.
 */
int seacells_embed(const void *table, uint32_t dtype, uint32_t v, uint32_t d, uint64_t table_ld,
                   const int32_t *tokens, uint32_t n, float scale, void *out, uint64_t out_ld,
                   uint32_t *status, seacells_stream_t stream);

/* Workspace bytes seacells_embed_grad needs. */
size_t seacells_embed_grad_workspace(uint32_t n, uint32_t v, uint32_t d);

/*
 * Gradient of the lookup's table: for every row t < v
 *   d_table[t, :] = add_to[t, :] + scale * sum of d_out[i, :] over the i with
 *   tokens[i] = t,
 * summed in f32 in a fixed order and rounded once. Rows without a token are
 * written too (add_to's row, or zeros). Negative tokens are skipped; tokens
 * >= v are skipped and set SEACELLS_FLAG_BAD_INDEX.
 * d_out    device [n, d] of d_out_type, row stride d_out_ld.
 * add_to   device [v, d] or NULL (nothing is added), of d_table's type and
 *          stride. add_to == d_table accumulates in place (rows without a
 *          token are then left alone); other overlaps are not allowed.
 * d_table  device [v, d] of d_table_type (d_out_type or SEACELLS_F32), row
 *          stride d_table_ld.
 * workspace: at least seacells_embed_grad_workspace(n, v, d) bytes, 256-byte
 * aligned.
 */
int seacells_embed_grad(const int32_t *tokens, uint32_t n, const void *d_out, uint32_t d_out_type,
                        uint64_t d_out_ld, uint32_t v, uint32_t d, float scale,
                        const void *add_to, void *d_table, uint32_t d_table_type,
                        uint64_t d_table_ld, void *workspace, size_t workspace_bytes,
                        uint32_t *status, seacells_stream_t stream);

/*
 * Layer norm of n rows of d elements: mean = sum x / d, rstd =
 * 1 / sqrt(sum (x - mean)^2 / d + eps), out = (x - mean) * rstd * weight + bias.
 * x, out        device [n, d] of dtype, row strides x_ld, out_ld. out may be x
 *               (same stride).
 * weight, bias  device [d] of weight_type (dtype or SEACELLS_F32); either may
 *               be NULL (1 and 0).
 * mean, rstd    device [n] f32 out, or NULL.
 * eps           finite, >= 0.
 * A row that holds NaN or an infinity gets NaN in out and rstd, and a mean that
 * is not finite.
 */
int seacells_layer_norm(const void *x, uint32_t dtype, uint32_t n, uint32_t d, uint64_t x_ld,
                        const void *weight, const void *bias, uint32_t weight_type, float eps,
                        void *out, uint64_t out_ld, float *mean, float *rstd,
                        seacells_stream_t stream);

/* Workspace bytes seacells_layer_norm_grad needs. */
size_t seacells_layer_norm_grad_workspace(uint32_t n, uint32_t d);

/*
 * Gradients of seacells_layer_norm, with h = (x - mean) * rstd, g = d_out * weight:
 *   d_x      = rstd * (g - mean_d(g) - h * mean_d(g * h))   per row
 *   d_weight = sum over rows of d_out * h
 *   d_bias   = sum over rows of d_out
 * d_out, x, d_x      device [n, d] of dtype with row strides; d_x may be
 *                    d_out or x (same stride), or NULL (not computed).
 * mean, rstd         device [n] f32 as the forward call wrote them.
 * weight             device [d] of weight_type, or NULL (1).
 * d_weight, d_bias   device [d] of weight_type, out; either may be NULL (not
 *                    computed). n = 0 gives zeros.
 * workspace: at least seacells_layer_norm_grad_workspace(n, d) bytes, 256-byte
 * aligned.
 */
int seacells_layer_norm_grad(const void *d_out, uint64_t d_out_ld, const void *x, uint32_t dtype,
                             uint32_t n, uint32_t d, uint64_t x_ld, const float *mean,
                             const float *rstd, const void *weight, uint32_t weight_type,
                             void *d_x, uint64_t d_x_ld, void *d_weight, void *d_bias,
                             void *workspace, size_t workspace_bytes, seacells_stream_t stream);

/* Workspace bytes seacells_logprobs needs. */
size_t seacells_logprobs_workspace(uint32_t n, uint32_t v, uint32_t top_k);

/*
 * Log probabilities of n rows of v logits. With m = max x and s =
 * log sum exp(x - m) over the row:
 *   stats[i]    = (m, s)                             device [n, 2] f32 out, or NULL
 *   logp[i]     = x[targets[i]] - m - s              device [n] f32 out, or NULL
 *   entropy[i]  = -sum p log p, p = exp(x - m - s)   device [n] f32 out, or NULL
 *   top_idx[i]  = columns of the top_k largest x in descending order, the
 *                 lowest column first among equals (-0 equals +0)
 *                                                    device [n, top_k] int32 out
 *   top_logp[i] = their log probabilities            device [n, top_k] f32 out
 * targets   device [n] int32, or NULL with logp NULL. A negative target is
 *           ignored (logp 0); a target >= v too, with SEACELLS_FLAG_BAD_INDEX.
 * top_k     0 (top_idx and top_logp unused) to SEACELLS_TOP_MAX.
 * Masks: a logit of -inf has p = 0 and is no alternative; where fewer than
 * top_k columns are left the rest is (-1, -inf). A row with nothing left has
 * stats (-inf, 0), logp -inf, entropy 0. A row that holds NaN or +inf has no
 * distribution: its f32 outputs are NaN (logp of an ignored target stays 0)
 * and its top_idx -1.
 * workspace: at least seacells_logprobs_workspace(n, v, top_k) bytes, 256-byte
 * aligned (may be NULL where that is 0).
 */
int seacells_logprobs(const void *logits, uint32_t dtype, uint32_t n, uint32_t v, uint64_t ld,
                      const int32_t *targets, uint32_t top_k, float *logp, float *entropy,
                      float *stats, int32_t *top_idx, float *top_logp, void *workspace,
                      size_t workspace_bytes, uint32_t *status, seacells_stream_t stream);

/*
 * Gradient of sum_i d_logp[i] logp[i] + d_entropy[i] entropy[i] to the logits:
 *   d_logits = d_logp (1[column = target] - p) - d_entropy p (log p + entropy)
 * logits, d_logits      device [n, v] of dtype, row strides ld, d_logits_ld.
 *                       d_logits may be logits (same stride).
 * targets               device [n] int32, or NULL (every row is ignored). An
 *                       ignored target (as above) takes no part of d_logp.
 * stats, entropy        as seacells_logprobs wrote them; entropy may be NULL
 *                       with d_entropy NULL.
 * d_logp, d_entropy     device [n] f32; either may be NULL (0).
 * Masked (-inf) logits and rows with nothing left get 0 (whatever d_logp and
 * d_entropy hold there); a row without a distribution (NaN stats) gets NaN.
 */
int seacells_logprobs_grad(const void *logits, uint32_t dtype, uint32_t n, uint32_t v,
                           uint64_t ld, const int32_t *targets, const float *stats,
                           const float *entropy, const float *d_logp, const float *d_entropy,
                           void *d_logits, uint64_t d_logits_ld, uint32_t *status,
                           seacells_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* SEACELLS_TOKEN_H */
