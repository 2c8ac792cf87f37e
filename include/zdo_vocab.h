/*
 * zdo_vocab.h — the two ends of a language model at the vocabulary matrix, on
 * the optimizer's own buffers, on AMD Instinct MI355X (gfx950): what reads
 * the parameter buffer that all_gather_params leaves, and what writes the
 * matrix's gradient into the contribution that the rank sends. The calls
 * stand beside those of zdo.h and share its plan, streams, error codes and
 * conventions (its first comment); every call only enqueues work, allocates
 * nothing and may be captured into a HIP graph.
 *
 * The matrix W is parameter `param_index` of the plan: rows of `dim` elements
 * one after the other from the parameter's first element, row v belonging to
 * token v. vocab * dim may be less than the parameter has elements: what lies
 * behind row vocab - 1 (rows that only pad the vocabulary) is never read. The
 * parameter may start at any element and dim may be any number, odd ones too;
 * the products run without a copy of W when W starts at a multiple of 8
 * elements and dim is a multiple of 64.
 *
 * Conventions beyond zdo.h's:
 *   - params: bf16, N elements (WORLD). grads: bf16, N elements (WORLD): a
 *     rank's contribution. Only the parameter's own elements are touched.
 *   - tokens, targets: n int64 in device memory. A number outside [0, vocab)
 *     names no row: such a token's output is zero, it takes part in no
 *     gradient, and its target makes a loss of zero. What its row of
 *     grad_out, hidden, lse or grad_loss holds (Inf and NaN too) reaches no
 *     other output.
 *   - Rows of activations (out, grad_out, hidden, grad_hidden) are `dim`
 *     consecutive elements, one row every `stride` elements (stride >= dim;
 *     with n <= 1 it is not used). They, and arrays with one element a token,
 *     need their type's own alignment only; 16 bytes and strides of a multiple
 *     of 8 are fastest.
 *   - Types of activations: ZDO_BF16 or ZDO_F32.
 *   - What a call writes must share no element with anything else of it. Rows may
 *     lie between the rows of another array if both strides have as many bytes
 *     (hidden and grad_hidden as two halves of one buffer's columns), and an array
 *     without gaps between two rows; with strides that differ, arrays whose extents
 *     meet are refused. What lies between rows is neither read nor written.
 *   - accumulate: 0 overwrites every element of the parameter in grads (those
 *     without a contribution become 0); otherwise the gradient is added to
 *     what is there, in fp32 and rounded once, and embedding_grad leaves rows
 *     that no token names as they were.
 *   - n is in [0, 2^30] (the loss: [0, 2^22]), vocab in [1, 2^30], dim in
 *     [1, 2^20], strides at most 2^30; with n = 0 the gradients are those of no
 *     tokens, and the token arrays may be NULL.
 *   - workspace: device memory, 16-byte aligned, as many bytes as the call's
 *     query says, this call's alone until it completes. Two graphs that may
 *     run at the same time need two.
 *   - Equal calls give equal bits: sums have a fixed order, which depends on the
 *     sizes and on where W starts and how long its rows are, and no result goes
 *     through an atomic addition.
 */
#ifndef ZDO_VOCAB_H
#define ZDO_VOCAB_H

#include <stdint.h>

#include "zdo.h"

#ifdef __cplusplus
extern "C" {
#endif

#define ZDO_BF16 0
#define ZDO_F32 1

/* out_i = scale * W[tokens_i] (one fp32 product, rounded once to out_type),
 * zero for a token that names no row. out must not overlap the inputs. */
int embedding_lookup(const zdo_plan *plan, int32_t param_index, int64_t vocab, int64_t dim, const uint16_t *params,
                     const int64_t *tokens, int64_t n, float scale, void *out, int32_t out_type, int64_t out_stride,
                     void *stream);

/* Workspace bytes embedding_grad needs; -1 for sizes out of range. */
int64_t zdo_embedding_grad_workspace_bytes(int64_t n, int64_t dim);

/* The lookup's gradient: for every row v, scale * (the sum of grad_out_i over
 * the tokens i that name v), added in fp32 in the tokens' order (in pieces, whose
 * sums are then added in order), multiplied by scale and rounded once to bf16,
 * into the parameter's elements of grads. The device orders the positions by
 * token, so that a row is summed without atomics however many tokens name it.
 * grads and workspace must not overlap the inputs or each other. */
int embedding_grad(const zdo_plan *plan, int32_t param_index, int64_t vocab, int64_t dim, const int64_t *tokens,
                   int64_t n, const void *grad_out, int32_t grad_type, int64_t grad_stride, float scale,
                   int32_t accumulate, uint16_t *grads, void *workspace, void *stream);

/* Workspace bytes linear_cross_entropy and linear_cross_entropy_grad need (the
 * same for both, so that one workspace serves a step); -1 for sizes out of
 * range (n here is at most 2^22, and so it is in both calls). It holds hidden in
 * bf16 and, for the gradient, its sum in fp32; a piece's d and its rows of W, at
 * most 256 MB each (or 512 bytes a token, and for each of dim); the sums of
 * splits, at most 128 MB for each gradient; for the loss, in the place of d and the
 * sums, 8 bytes for each token and 128 rows of W (64 for up to 32 tokens). */
int64_t zdo_linear_cross_entropy_workspace_bytes(int64_t n, int64_t vocab, int64_t dim);

/* Softmax cross entropy of the logits z_i = W hidden_i, which are never kept:
 *   lse_i  = log(sum over v < vocab of exp(z_i[v]))
 *   loss_i = lse_i - z_i[targets_i], 0 where the target names no row.
 * hidden: bf16. Products and sums in fp32, exponentials relative to a running
 * maximum m_i; the loss is (m_i - z_i[targets_i]) + log(sum over v of exp(z_i[v] -
 * m_i)), so that it is never negative and a small one keeps its digits however large
 * the logits are. loss and lse: fp32, n elements each; lse is written for every
 * token. Outputs and workspace must not overlap the inputs or each other. */
int linear_cross_entropy(const zdo_plan *plan, int32_t param_index, int64_t vocab, int64_t dim,
                         const uint16_t *params, const uint16_t *hidden, int64_t hidden_stride,
                         const int64_t *targets, int64_t n, float *loss, float *lse, void *workspace, void *stream);

/* The gradients of sum_i grad_loss_i * loss_i, from linear_cross_entropy's lse:
 *   d_i[v]      = (exp(z_i[v] - lse_i) - [v == targets_i]) * grad_loss_i
 *   grad_hidden_i = sum over v of d_i[v] * W[v]   (rounded to grad_hidden_type)
 *   W's gradient: row v = sum over i of d_i[v] * hidden_i   (into grads)
 * z is formed again, in pieces of the vocabulary. d is rounded to bf16 for the
 * two products, as their results are, and the products' sums are in fp32; what
 * the rounding leaves of d_i[targets_i], the largest term of most sums, is added
 * to grad_hidden in fp32, and for up to 128 tokens W's gradient takes d in two
 * bf16 parts. A token whose target names no row has a grad_hidden of zero.
 * grad_hidden or grads may be NULL (both only with n = 0): that gradient is not
 * computed.
 * hidden's rows of tokens whose target names no row are not used. An infinite
 * element of W leaves no finite number in its column of grad_hidden. Outputs
 * and workspace must not overlap the inputs or each other. */
int linear_cross_entropy_grad(const zdo_plan *plan, int32_t param_index, int64_t vocab, int64_t dim,
                              const uint16_t *params, const uint16_t *hidden, int64_t hidden_stride,
                              const int64_t *targets, int64_t n, const float *lse, const float *grad_loss,
                              void *grad_hidden, int32_t grad_hidden_type, int64_t grad_hidden_stride,
                              int32_t accumulate, uint16_t *grads, void *workspace, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* ZDO_VOCAB_H */
