/*
 * engram_vocab.h -- C ABI of libengram.so, third part: the operators at the
 * vocabulary's end of the layer, on one AMD Instinct MI355X (gfx950):
 *   - distillation from a teacher's top logits: the loss, its gradient, or
 *     both in one call (with one entry a row, a label's cross entropy);
 *   - the selection of a beam search over beams and vocabulary;
 *   - the reordering of the decoding states after it: slots of rings
 *     (engram_ple_conv_step's, or any other state) and token histories.
 *
 * The conventions of engram.h hold: caller-owned device buffers; no
 * allocation, no state, no host synchronisation; arguments checked on the
 * host before anything is enqueued, with engram.h's status codes.  Rows of
 * logits and of gradients may lie apart (a stride in values, of at least the
 * row's length) and start at any address of their type; pools are 16-byte
 * aligned (EALIGN otherwise).  Buffers of one call do not overlap unless an
 * entry point says that they may.
 *
 * Types named by a call: ENGRAM_BF16 and ENGRAM_F32 (engram_layer.h).
 */
#ifndef ENGRAM_VOCAB_H
#define ENGRAM_VOCAB_H

#include "engram_layer.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Most entries of a teacher's row; most beams, and candidates, of a sequence;
 * most pools of one reordering. */
#define ENGRAM_DISTILL_MAX_TOP 1024
#define ENGRAM_BEAM_MAX 64
#define ENGRAM_FORK_MAX_POOLS 8

/*
 * engram_distill -- for each row t, with the student's logits z[v] (v in
 * [0, vocab)), q[v] = softmax(z / temperature), and the teacher's entries
 * (id_j, y_j), j in [0, top), of which those with an id in [0, vocab) are used:
 *   without d_teacher_lse: p_j = softmax over the used entries of
 *     y_j / temperature
 *   with d_teacher_lse (the log of the sum of exp(y / temperature) over the
 *     teacher's whole vocabulary): p_j = exp(y_j / temperature - teacher_lse)
 *   P[v] = sum of p_j over the entries with id_j = v (an id may repeat)
 *   m = sum of p_j;  r = 1 - m with `rest` (below 2^-20, the rounding of
 *     teacher_lse, it counts as 0), else 0
 *   s = sum of q[v] over the v that no used entry names
 *   loss = sum_v P[v] * log(P[v] / q[v]) + r * log(r / s)
 *   lse = log sum_v exp(z[v] / temperature),  lse_rest = lse + log s
 *   grad[v] = grad_loss / temperature
 *             * (q[v] * (m + r) - P[v] - (v unnamed ? r * q[v] / s : 0))
 * A term with P[v] = 0 (r = 0) is 0.  A row without a used entry, or whose used
 * entries all have y = -inf without d_teacher_lse, has no target: loss 0,
 * gradient 0.  A row with grad_loss = 0 has gradient 0, whatever its logits
 * hold.  A logit of -inf has q = 0 (a row of them: lse -inf, q 0); a target
 * with q = 0 gives a loss of +inf and a finite gradient.  NaN and +inf logits
 * make their own row's loss NaN, and its gradient where it is not 0.
 * Sums over the vocabulary: fp32 terms, summed in fp32 by each lane (128
 * chunks of 8 and a value at most) and in fp64 across lanes, in an order that
 * the sizes and the alignment of a row's address fix: a repeated call gives the
 * same bits.  The named logits' part, the teacher's and the logarithms are
 * fp64; a term of less than 2^-126 of the largest is lost.  The gradient is
 * rounded once to the logits' type.
 *   rows (up to 4,194,303, and rows * ceil(vocab / 16384) for a gradient up to
 *     16,500,000, / 8192 for fp32: a launch's threads), vocab (1 to 2^30), top
 *     (1 to ENGRAM_DISTILL_MAX_TOP).
 *   d_logits of logits_type, rows logits_stride values apart.
 *   d_ids int64 [rows, top]: -1 marks an unused entry; other ids outside
 *     [0, vocab) are treated the same and add one each to *d_err_count (when
 *     not NULL), once a call.
 *   d_teacher [rows, top] of teacher_type; d_teacher_lse fp32 [rows] or NULL.
 *   rest 0 or 1; 1 needs d_teacher_lse.
 *   temperature 2^-64 to 2^64.
 *   d_loss, d_lse, d_lse_rest (with rest only): fp32 [rows], written when not
 *     NULL.
 *   d_grad of logits_type, rows grad_stride values apart, written when not
 *     NULL; may be d_logits (with its stride).  Needs d_grad_loss fp32 [rows].
 *   The workspace (engram_distill_workspace bytes, 16-byte aligned) is needed
 *   where that is not 0.
 * engram_distill_backward -- the gradient alone, from the d_lse (and, with
 *   rest, d_lse_rest) that engram_distill wrote: q = exp(z / temperature - lse),
 *   q / s = exp(z / temperature - lse_rest).  A logarithm's rounding to fp32 is
 *   a relative error of these: 2^-19 below 64 and, used for bf16 logits only,
 *   2^-15 below 1024.  A row with a larger one (a low temperature, logits all
 *   at a mask's lowest value or far from 0; at a temperature below 1 an
 *   infinite one too) is summed again by one block, its gradient as exact as
 *   engram_distill's and two to six times as long.  No workspace; d_loss is
 *   NULL.
 * Errors: EINVAL, EWORKSPACE.  rows == 0 enqueues nothing.
 */
typedef struct engram_distill_args {
  int64_t rows, vocab, top;
  int64_t logits_stride, grad_stride;
  double temperature;
  int32_t logits_type, teacher_type, rest;
  int32_t reserved; /* 0 */
  const void *d_logits;
  const int64_t *d_ids;
  const void *d_teacher;
  const float *d_teacher_lse;
  const float *d_grad_loss;
  float *d_loss;
  float *d_lse;      /* engram_distill: written; backward: read */
  float *d_lse_rest; /* the same */
  void *d_grad;
  int64_t *d_err_count;
  void *d_workspace;
  size_t workspace_bytes;
  void *stream;
} engram_distill_args;

/* Bytes of workspace of engram_distill, grad 1 with d_grad and 0 without; (size_t)-1 for
 * sizes it refuses. */
size_t engram_distill_workspace(int64_t rows, int64_t vocab, int32_t grad);
int engram_distill(const engram_distill_args *args);
int engram_distill_backward(const engram_distill_args *args);

/*
 * engram_beam_select -- the best continuations of each sequence's beams.
 * With lse[b,w] = log sum_v exp(logits[b,w,v]), the candidate (w, v) of
 * sequence b has the value
 *     scores[b,w] + (logits[b,w,v] - lse[b,w])
 * in fp64 (lse: fp32 terms, summed in fp64 across lanes in an order that the
 * sizes fix, so that beams with equal logits have equal ones; its largest logit
 * is taken off first, so that a beam whose logits are all a mask's lowest value
 * keeps the logarithm of their number).  A finished beam has one candidate, (w,
 * eos_id) with the value scores[b,w]; its logits are not read.  The `count`
 * largest values are written in falling order, equal ones by the lower beam and
 * then the lower id.  A value that is -inf or NaN is never taken (a beam whose
 * score or lse is not finite has none): entries that nothing is left for have
 * score -inf, parent -1, token -1.
 *   batch, beams (1 to ENGRAM_BEAM_MAX), vocab (1 to 2^30), count (1 to
 *     ENGRAM_BEAM_MAX).
 *   d_logits [batch * beams] rows of `type`, logits_stride values apart.
 *   d_scores fp32 [batch, beams].
 *   d_finished uint8 [batch, beams] or NULL (none); with it eos_id is in
 *     [0, vocab).  eos_id -1: no id ends a beam.
 *   d_out_scores fp32, d_out_parents int64 (the beam's index in its
 *     sequence), d_out_tokens int64, d_out_finished uint8 (the parent was
 *     finished or the token is eos_id; may be NULL): [batch, count], written.
 *     With count == beams d_out_scores may be d_scores, and d_out_finished
 *     d_finished.
 *   The workspace holds engram_beam_select_workspace bytes, 16-byte aligned.
 * Errors: EINVAL, EWORKSPACE.  batch == 0 enqueues nothing.
 */
size_t engram_beam_select_workspace(int64_t batch, int64_t beams, int64_t vocab);
int engram_beam_select(const void *d_logits, int32_t type, int64_t logits_stride,
                       const float *d_scores, const uint8_t *d_finished, int64_t eos_id,
                       int64_t batch, int64_t beams, int64_t vocab, int64_t count,
                       float *d_out_scores, int64_t *d_out_parents, int64_t *d_out_tokens,
                       uint8_t *d_out_finished, void *d_workspace, size_t workspace_bytes,
                       void *stream);

/*
 * engram_beam_fork -- the states of the beams that a selection kept.  New beam
 * j of sequence b continues old beam parents[b,j].  Of the new beams with one
 * parent the first keeps the parent's slot; each other one, in rising order,
 * takes the next slot of an old beam without a child, and the parent's state
 * is copied there, in every pool.  So the new slots are the old ones in
 * another order, and only states that are needed twice are moved.
 *   d_parents int64 [batch, beams]; -1 marks an unused entry (it takes a slot
 *     without a child, nothing copied); other values outside [0, beams) are
 *     treated the same and add one to *d_err_count (when not NULL).
 *   d_slots int64 [batch, beams], distinct, or NULL (slot b * beams + j).  A
 *     slot outside [0, slot_count) is handed on like any other, but nothing is
 *     copied from or to it; one that is not -1 adds one to *d_err_count.
 *     Repeated slots race on their contents (in bounds).
 *   h_pools, h_slot_bytes: `pools` (0 to ENGRAM_FORK_MAX_POOLS) device
 *     buffers of slot_count slots of that many bytes (a multiple of 16).
 *   d_new_slots int64 [batch, beams], written; not d_slots or d_parents.
 *   d_history int64 [batch, beams, history_len] and d_new_history [batch,
 *     beams, new_len], 1 <= new_len <= history_len + 1, with d_tokens int64
 *     [batch, beams]: new row j is the last new_len values of the parent's
 *     row (an unused entry: its own) with tokens[b,j] after it.  All of the
 *     three or none (d_history may be NULL with history_len 0); d_new_history is not
 *     d_history.
 * Errors: EINVAL, EALIGN.  batch == 0 enqueues nothing.
 */
int engram_beam_fork(const int64_t *d_parents, const int64_t *d_slots, int64_t batch,
                     int64_t beams, void *const *h_pools, const int64_t *h_slot_bytes,
                     int32_t pools, int64_t slot_count, int64_t *d_new_slots,
                     const int64_t *d_tokens, const int64_t *d_history, int64_t history_len,
                     int64_t *d_new_history, int64_t new_len, int64_t *d_err_count,
                     void *stream);

#ifdef __cplusplus
}
#endif

#endif /* ENGRAM_VOCAB_H */
