/*
 * sv_logprobs.h -- C ABI of libsvlogprobs: log probabilities of given tokens
 * and distillation from a teacher's top logits, each with its gradient, on
 * one NVIDIA GB300 (sm_103a).
 *
 * spec_verify.h decides which tokens a round emits. What stands around that
 * decision reads the same rows of logits: the log probabilities that a server
 * returns with the emitted tokens and their alternatives, and the training of
 * the draft model on what the target thought of its drafts ("Speculative
 * decoding" (aihero.vn): the closer the draft's distribution q is to the
 * target's p, the more drafts are kept).
 *
 * Rows. With x the logits of a row, T the temperature and z = x / T,
 *   lse = log sum_v exp z_v,  log p_v = z_v - lse,  entropy = -sum_v p_v log p_v
 * (0 log 0 = 0). Order among a row's tokens is by logit, ties by lowest index.
 *
 * Data errors are found on the device, row by row; row_status, where given,
 * receives 0 or spec_verify.h's bits for every row:
 *   SV_SEQ_BAD_TOKEN  a token, or a teacher's token, below -1 or at or above
 *                     the vocabulary.
 *   SV_SEQ_NONFINITE  the row has a NaN or +inf, or nothing but -inf; or the
 *                     teacher's log probabilities have a NaN or +inf, or no
 *                     finite one where they are to be renormalised, or
 *                     probabilities that float32 cannot add up where they are
 *                     not (logarithms from some 88 up).
 * The row's floating outputs, gradients included, are then NaN, its whole
 * outputs -1. No input makes a kernel read or write outside the arrays.
 *
 * Sums and statistics are float32, gradients are rounded to the logits' type
 * once. Results do not depend on the order in which blocks run: the same
 * inputs give the same bits. Return codes are spec_verify.h's SV_OK and
 * SV_ERR_*. All calls are asynchronous on `stream`, allocate nothing and may be
 * captured into a CUDA graph.
 *
 * Workspace. Rows are cut into pieces whose blocks leave one another their sums.
 *   workspace  device, 256-byte aligned, at least sv_logprobs_workspace_bytes. Its
 *              first SV_LOGPROBS_COUNTER_BYTES must be 0 before it is used for the
 *              first time, with rows of whatever sizes; every call leaves them 0.
 *              Calls that share a workspace must be ordered (one stream, or events);
 *              a captured call's replays too.
 */
#ifndef SV_LOGPROBS_H
#define SV_LOGPROBS_H

#include <stddef.h>
#include <stdint.h>

#include "spec_verify.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Element type besides spec_verify.h's SV_F32 and SV_BF16 (sv_attention.h's). */
#ifndef SV_F16
#define SV_F16 2
#endif

/* Most top alternatives of a row, and most entries of a teacher's row. */
#define SV_MAX_TOP 128
/* Largest vocabulary whose top alternatives are given. */
#define SV_MAX_TOP_VOCAB (1 << 20)

/* The part of a workspace that has to be 0 before its first use. */
#define SV_LOGPROBS_COUNTER_BYTES 262144

/* Floats that the forward calls keep of a row for the backward ones. */
#define SV_ROW_STATS 8

/* What is made of the teacher's probability that its entries leave:
 * SV_TAIL_RENORMALISE  the entries are scaled to sum 1 (their log
 *                      probabilities may be off by a constant, as logits are).
 * SV_TAIL_BUCKET       all tokens without an entry are one outcome, of
 *                      probability max(0, 1 - the entries' sum). */
enum sv_tail { SV_TAIL_RENORMALISE = 0, SV_TAIL_BUCKET = 1 };

/*
 * Rows of logits: row o * inner + i, with 0 <= o < outer and 0 <= i < inner,
 * begins at logits + o * outer_stride + i * inner_stride (in elements) and has
 * vocab elements. Everything else that is said to be [rows] is contiguous, in
 * that order.
 *   logits   device, aligned to its elements. Rows that begin on 16-byte
 *            boundaries are read a little faster.
 *   outer, inner   >= 0, their product below 2^31. Strides are 0 .. 2^40 and
 *            not looked at where there is one of a kind.
 *   vocab    1 .. 2^31 - 1.
 *   dtype    SV_F32, SV_BF16 or SV_F16.
 *   temperature  > 0 and up to 2^117, with log2(e) / T and 1 / T finite in float32.
 */
typedef struct sv_logit_rows {
    const void* logits;
    int64_t outer, inner;
    int64_t outer_stride, inner_stride;
    int64_t vocab;
    int32_t dtype;
    float temperature;
} sv_logit_rows;

/*
 * Workspace for any of these calls on such rows, with up to top_k alternatives.
 * rows->logits and the strides are not looked at. Host only.
 */
int sv_logprobs_workspace_bytes(const sv_logit_rows* rows, int64_t top_k, size_t* bytes);

/*
 * Log probabilities, entropy and top alternatives of rows of logits, which are
 * read once.
 *   tokens        device int32 [rows], or NULL. -1: nothing is asked of the row,
 *                 which is not read; it gets log probability, entropy and lse 0,
 *                 rank and top tokens -1, top log probabilities -inf.
 *   top_k         0 .. min(SV_MAX_TOP, vocab); above 0 only for vocabularies up to
 *                 SV_MAX_TOP_VOCAB.
 *   logprobs      device float [rows]: log p of the token (needs tokens).
 *   rank          device int32 [rows]: tokens ahead of the token (needs tokens).
 *   entropy, lse  device float [rows].
 *   top_tokens, top_logprobs  device int32 and float [rows][top_k]: the first
 *                 top_k tokens in order, and their log p. Both or neither.
 *   row_stats     device float [rows][SV_ROW_STATS], 16-byte aligned: what the backward call
 *                 needs of this one.
 * Each output may be NULL. One launch.
 */
int sv_token_logprobs(const sv_logit_rows* rows, const int32_t* tokens, int64_t top_k,
                      float* logprobs, float* entropy, float* lse, int32_t* rank,
                      int32_t* top_tokens, float* top_logprobs, float* row_stats,
                      int32_t* row_status, void* workspace, size_t workspace_bytes, void* stream);

/*
 * The logits' gradient, from gradients a, b and c of log probability, entropy and
 * lse (device float [rows] each, NULL for zeros; grad_logprobs needs tokens):
 *   grad_v = (a ([v = token] - p_v) - b p_v (log p_v + entropy) + c p_v) / T.
 * The tokens may be others than the forward call's. Rows whose token is out of
 * range, here or there, get NaN; other rows of token -1, here or there, zeros.
 *   row_stats   what sv_token_logprobs wrote for these rows.
 *   grad        device, the logits' type, vocab elements a row; row o * inner + i
 *               begins at grad + o * grad_outer_stride + i * grad_inner_stride.
 *               Rows must not overlap. It may be the logits themselves, or must have no
 *               element in common with them (its rows may lie between theirs).
 * One launch.
 */
int sv_token_logprobs_backward(const sv_logit_rows* rows, const int32_t* tokens,
                               const float* row_stats, const float* grad_logprobs,
                               const float* grad_entropy, const float* grad_lse, void* grad,
                               int64_t grad_outer_stride, int64_t grad_inner_stride,
                               void* stream);

/*
 * Divergence of a teacher's entries from rows of logits, and its gradient.
 * A row's teacher is k pairs (token, log probability); pairs of token -1 are
 * none, and pairs of one token add their probabilities. With P the entries'
 * probabilities (renormalised or not), q = softmax(x / T), and with
 * SV_TAIL_BUCKET P_o what the entries leave and q_o the sum of q over the tokens
 * that have none (both left out where all tokens have one):
 *   loss = sum_v P_v (log P_v - log q_v)  [ + P_o (log P_o - log q_o) ]
 * over the tokens with entries (0 log 0 = 0; a P_o of up to 2^-20, the rounding of a
 * whole teacher's float32 logarithms, is 0 where q_o is below float32's range, as of
 * masked tokens), and with M the sum of all P, P_o too,
 *   dloss/dx_v = (M q_v - P_v) / T                  for tokens with entries
 *              = (M q_v - P_o q_v / q_o) / T        for the others.
 * Rows without entries are not read; they have loss 0 and gradient 0.
 *   teacher_tokens, teacher_logprobs  device int32 and float [rows][k],
 *               1 <= k <= SV_MAX_TOP.
 *   weights     device float [rows], or NULL for ones: factors of the rows'
 *               gradients (not of their losses).
 *   loss        device float [rows], or NULL.
 *   grad        as in sv_token_logprobs_backward, or NULL.
 *   row_stats   device float [rows][SV_ROW_STATS], 16-byte aligned, or NULL.
 * One launch; one more for the gradient of long rows, which are read again.
 */
int sv_distill(const sv_logit_rows* rows, const int32_t* teacher_tokens,
               const float* teacher_logprobs, int64_t k, int tail, const float* weights,
               float* loss, void* grad, int64_t grad_outer_stride, int64_t grad_inner_stride,
               float* row_stats, int32_t* row_status, void* workspace, size_t workspace_bytes,
               void* stream);

/*
 * The gradient alone, from row_stats of a sv_distill call on the same rows and
 * teacher: grad_loss[row] dloss/dx. One launch.
 */
int sv_distill_backward(const sv_logit_rows* rows, const int32_t* teacher_tokens,
                        const float* teacher_logprobs, int64_t k, int tail,
                        const float* row_stats, const float* grad_loss, void* grad,
                        int64_t grad_outer_stride, int64_t grad_inner_stride, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* SV_LOGPROBS_H */
