/*
 * engram_layer.h -- C ABI of libengram.so, second part: the layer operators
 * around the hashed n-gram lookup, for training and for serving, on one AMD
 * Instinct MI355X (gfx950):
 *   - the residual norm: a block's output normed, gated, scaled and added to
 *     the residual stream, and the next block's norm of the sum;
 *   - 8-bit activation checkpoints, which the backward passes here read;
 *   - the gradients of the PLE causal dilated depthwise convolution
 *     (engram_ple_conv) and its form for single tokens;
 *   - the scaled token embedding and its gradient by sorted tokens.
 *
 * The conventions of engram.h hold: caller-owned device buffers, row-major
 * and contiguous; no allocation, no state, no host synchronisation; arguments
 * checked on the host before anything is enqueued, with engram.h's status
 * codes.  Data buffers (bf16, fp32 and int8 arrays of [..., channels]) are
 * 16-byte aligned (EALIGN otherwise); per-row and per-group statistics,
 * scales and ids have their type's own alignment.  Buffers of one call do not
 * overlap unless an entry point says that they may.
 *
 * Types named by a call: ENGRAM_BF16 and ENGRAM_F32.
 */
#ifndef ENGRAM_LAYER_H
#define ENGRAM_LAYER_H

#include "engram.h"

#ifdef __cplusplus
extern "C" {
#endif

#define ENGRAM_BF16 0
#define ENGRAM_F32 1

/* Channels that share one scale of an 8-bit checkpoint, and the widest norm
 * group. */
#define ENGRAM_ACT_BLOCK 128
#define ENGRAM_NORM_MAX_GROUP 16384

/*
 * engram_residual_norm -- with rows t, groups g of n = channels / groups
 * adjacent channels, and rms_g the root of a group's mean square:
 *     u[t,g]    = 1 / sqrt(mean_g(y[t]^2) + eps)
 *     a[t,c]    = 1 / (1 + exp(-gate)), or 1 without a gate
 *     out[t,c]  = residual_scale * residual[t,c]
 *                 + scale[c] * a[t,c] * w_post[c] * y[t,c] * u[t,g]
 *     v[t,g]    = 1 / sqrt(mean_g(out[t]^2) + eps)
 *     next[t,c] = out[t,c] * v[t,g] * w_next[c]
 * All of it in fp32.  out is rounded once to the residual's type, and v and
 * next are taken of the rounded value (what a separate norm would read), next
 * rounded once to bf16.  Non-finite values spread over their own group of
 * their own row only.
 *   rows, channels, groups: channels a multiple of 8 * groups; n at most
 *     ENGRAM_NORM_MAX_GROUP.
 *   d_residual  [rows, channels] of residual_type.
 *   d_y         bf16 [rows, channels], the block's output; NULL: no branch,
 *     next is the norm of the residual itself (the norm before a block), and
 *     d_out, d_gate, d_w_post, d_scale, d_rstd_post and d_y_codes are NULL and
 *     residual_scale is 1.
 *   d_gate      bf16 [rows, gate_width], gate_width = groups (one gate a
 *     group) or channels; NULL with gate_width 0: no gate.
 *   d_w_post, d_scale, d_w_next  bf16 [channels]; a NULL w_post or scale is 1.
 *     d_w_next NULL: no next norm (d_next, d_rstd_next, d_next_codes NULL).
 *   d_out       [rows, channels] of residual_type, written; may be d_residual.
 *   d_next      bf16 [rows, channels], written.
 *   d_rstd_post, d_rstd_next  fp32 [rows, groups], written when not NULL: u
 *     and v, which the backward reads.
 *   d_y_codes, d_y_scales, d_next_codes, d_next_scales  the 8-bit checkpoints
 *     of y and of next, written when not NULL (both of a pair), as
 *     engram_act_encode writes them for rows of n values: codes int8 [rows,
 *     channels], scales fp32 [rows, groups, ceil(n / ENGRAM_ACT_BLOCK)].
 *     Codes that are kept make keeping y itself needless.
 *   eps > 0 and finite.
 * Errors: EINVAL, EALIGN.  rows == 0 enqueues nothing.
 *
 * engram_residual_norm_backward -- its gradients.  With gx = grad_next *
 * w_next, xh = out * v, yh = y * u and mean_g over a group:
 *     dR        = grad_out + v * (gx - xh * mean_g(gx * xh))
 *     grad_residual = residual_scale * dR
 *     q         = dR * a * scale * w_post
 *     grad_y    = u * (q - yh * mean_g(q * yh))
 *     grad_gate = (1 - a) * q * yh (summed over the group for one gate a group)
 *     grad_w_next = sum_t grad_next * xh
 *     grad_w_post = scale * sum_t dR * a * yh,  grad_scale = w_post * (same sum)
 * in fp32; the sums over rows go in a fixed order (the same result run to
 * run), per block of rows in fp32 and over the blocks in fp64.
 *   d_out (as written by the forward; the residual without a branch),
 *   d_rstd_next, d_w_next: needed with a next norm.  d_rstd_post: needed with
 *   a branch, and exactly one of d_y and the pair d_y_codes / d_y_scales (the
 *   checkpoint is then what y stands for).
 *   d_grad_out [rows, channels] of residual_type, or NULL (zero);
 *   d_grad_next bf16 [rows, channels], given exactly with a next norm.  One
 *   of the two is given.
 *   d_grad_residual (residual_type; may be d_grad_out), d_grad_y (bf16),
 *   d_grad_gate (bf16, [rows, gate_width]), d_grad_w_post, d_grad_scale,
 *   d_grad_w_next (fp32 [channels]): written when not NULL; one of what the
 *   call has no input for is EINVAL.
 *   The workspace (engram_residual_norm_backward_workspace bytes, 16-byte
 *   aligned) is needed when a gradient over rows is asked for.
 * Errors: EINVAL, EALIGN, EWORKSPACE.  rows == 0 writes zeros into the
 * gradients over rows.
 */
typedef struct engram_norm_args {
  int64_t rows, channels, groups, gate_width;
  float eps, residual_scale;
  int32_t residual_type; /* ENGRAM_BF16 or ENGRAM_F32 */
  int32_t reserved;      /* 0 */
  const void *d_residual; /* forward */
  const void *d_y;
  const void *d_gate;
  const void *d_w_post;
  const void *d_scale;
  const void *d_w_next;
  void *d_out;            /* forward: written; backward: read */
  void *d_next;           /* forward */
  float *d_rstd_post;     /* forward: written; backward: read */
  float *d_rstd_next;
  int8_t *d_y_codes;      /* forward: written; backward: read */
  float *d_y_scales;
  int8_t *d_next_codes;   /* forward */
  float *d_next_scales;
  const void *d_grad_out; /* backward, as the rest */
  const void *d_grad_next;
  void *d_grad_residual;
  void *d_grad_y;
  void *d_grad_gate;
  float *d_grad_w_post;
  float *d_grad_scale;
  float *d_grad_w_next;
  void *d_workspace;
  size_t workspace_bytes;
  void *stream;
} engram_norm_args;

int engram_residual_norm(const engram_norm_args *args);

/* Bytes of workspace of the backward; (size_t)-1 for sizes it refuses. */
size_t engram_residual_norm_backward_workspace(int64_t rows, int64_t channels, int64_t groups);

int engram_residual_norm_backward(const engram_norm_args *args);

/*
 * engram_act_encode -- an activation's 8-bit checkpoint.  Each row's channels
 * are cut into blocks of ENGRAM_ACT_BLOCK (the last one may be shorter); with
 * m the largest magnitude in a block:
 *     scale = m / 127,  code = round(x * (127 / m))    (to nearest, ties to even)
 * in fp32, each quotient and product rounded once, so the codes are the same
 * wherever they are made.  A block with m < 2^-120 has scale 0 and codes 0; a
 * block that holds an infinity or a NaN has scale NaN and codes 0, so that it
 * is read back as NaN.
 *   d_x bf16 [rows, channels], channels a multiple of 8; d_codes int8 [rows,
 *   channels]; d_scales fp32 [rows, ceil(channels / ENGRAM_ACT_BLOCK)].
 * engram_act_decode -- the values: bf16(code * scale), into d_x bf16.
 * Errors: EINVAL, EALIGN.  rows == 0 enqueues nothing.
 */
int engram_act_encode(const void *d_x, int64_t rows, int64_t channels, int8_t *d_codes,
                      float *d_scales, void *stream);
int engram_act_decode(const int8_t *d_codes, const float *d_scales, int64_t rows,
                      int64_t channels, void *d_x, void *stream);

/*
 * engram_ple_conv_backward -- the gradients of engram_ple_conv.  For the
 * position p (the halo's included, as negative positions) and the tap j steps
 * of dilation back (k = K-1-j):
 *     grad_x[b,p,c]      = sum_j w[c,K-1-j] * grad_out[b, p + j*dilation, c]
 *     grad_weight[c,K-1-j] = sum_{b,p} grad_out[b, p + j*dilation, c] * x[b,p,c]
 *     grad_bias[c]       = sum_{b,p >= 0} grad_out[b,p,c]
 * where a term counts only if p + j*dilation lies in [0, seq) and no change
 * of the segment id lies between; a term that does not count is never
 * multiplied (a NaN there stays there).  fp32; grad_x and grad_halo rounded
 * once to bf16; the sums over positions in a fixed order (the same result run
 * to run), per slice of positions in fp32 and over the slices in fp64.
 *   d_grad_out bf16 [batch, seq, channels]; d_weight, halo_len, d_seq_ids,
 *   batch, seq, channels, kernel_size, dilation as for engram_ple_conv.
 *   x: d_x bf16 [batch, seq, channels], or its checkpoint d_x_codes int8
 *     [batch, seq, channels] with d_x_scales fp32 (rows of code_width
 *     channels: channels / code_width rows to a position; 0 = channels).
 *     Needed, one of the two, when d_grad_weight is asked for.
 *   d_halo bf16 [batch, halo_len, channels] (needed with halo_len > 0 and
 *     d_grad_weight).
 *   d_grad_x, d_grad_halo (bf16), d_grad_weight (fp32 [channels,
 *     kernel_size]), d_grad_bias (fp32 [channels]): written when not NULL.
 *   The workspace (engram_ple_conv_backward_workspace bytes, 16-byte aligned)
 *   is needed for d_grad_weight and d_grad_bias.
 * kernel_size 4 with dilation up to 8 runs the register-window kernel; other
 * shapes a plain one.  Errors: EINVAL, EALIGN, EWORKSPACE.  An empty batch or
 * sequence writes zeros into the weight's and bias's gradients and the halo's.
 */
size_t engram_ple_conv_backward_workspace(int64_t batch, int64_t seq, int64_t halo_len,
                                          int64_t channels, int32_t kernel_size,
                                          int32_t dilation);
int engram_ple_conv_backward(const void *d_grad_out, const void *d_x, const int8_t *d_x_codes,
                             const float *d_x_scales, int64_t code_width, const void *d_halo,
                             int64_t halo_len, const int64_t *d_seq_ids, const void *d_weight,
                             int64_t batch, int64_t seq, int64_t channels, int32_t kernel_size,
                             int32_t dilation, void *d_grad_x, void *d_grad_halo,
                             float *d_grad_weight, float *d_grad_bias, void *d_workspace,
                             size_t workspace_bytes, void *stream);

/*
 * engram_ple_conv_step -- engram_ple_conv for tokens that arrive one (or a
 * few) at a time, from a ring of each sequence's latest inputs.  Token i of
 * sequence b stands at the position p = positions[b] + i of its segment (0:
 * the segment's first token) and
 *     out[b,i,c] = bias[c] + sum_k w[c,k] * x at position p - (K-1-k)*dilation
 * with positions below 0 reading 0 (the ring is then not read); x[b,i] is
 * written to row p mod ring_rows of the sequence's ring.  The same sum, in
 * the same order, as engram_ple_conv: the outputs are bitwise the same.
 *   d_x, d_out bf16 [batch, tokens, channels]; d_out NULL: only the ring is
 *     written (a prompt's last ring_rows inputs, say).
 *   d_ring bf16 [ring_count, ring_rows, channels], updated in place.
 *     ring_rows >= (K-1)*dilation, and at least 1.  A ring with further rows
 *     can take `tokens` back: positions that have not been overwritten stay.
 *   d_positions int64 [batch]; a negative position, or one above INT64_MAX -
 *     tokens, is an invalid entry.
 *   d_ring_ids int64 [batch], the ring of each sequence, distinct, or NULL
 *     (ring b).  -1 marks an unused entry: its outputs are zero, no ring is
 *     touched.  Any other id outside [0, ring_count), and an invalid position,
 *     is treated the same and adds one to *d_err_count (when not NULL).
 *     Repeated ids race on the one ring's contents (in bounds).
 *   d_weight, d_bias, kernel_size, dilation as for engram_ple_conv.
 * Errors: EINVAL, EALIGN.  batch * tokens == 0 enqueues nothing.
 */
int engram_ple_conv_step(const void *d_x, void *d_ring, int64_t ring_count, int64_t ring_rows,
                         const int64_t *d_ring_ids, const int64_t *d_positions,
                         const void *d_weight, const void *d_bias, int64_t batch, int64_t tokens,
                         int64_t channels, int32_t kernel_size, int32_t dilation, void *d_out,
                         int64_t *d_err_count, void *stream);

/*
 * engram_embed -- out[t, :] = scale * table[tokens[t], :], the product in fp32
 * and rounded once to the output's type.
 *   d_tokens int64 [n]: -1 is padding (a zero row); other ids outside
 *   [0, table_rows) give zero rows and are counted in *d_err_count (when not
 *   NULL).  d_table bf16 [table_rows, channels]; d_out [n, channels] of
 *   out_type; channels a multiple of 8.
 * Errors: EINVAL, EALIGN.  n == 0 enqueues nothing.
 *
 * engram_embed_grad -- its gradient into the whole table, by sorted tokens:
 *     grad_table[r, :] = scale * sum over t with tokens[t] == r of grads[t, :]
 * for every row r (rows without a token get zeros); with accumulate, the
 * product is added to the row (one fp32 add) and rows without a token are
 * left alone.  The sum and the product are fp64, rounded once to fp32 (and
 * that to bf16 for a bf16 table): deterministic, and for gradients whose sums
 * fit fp64 the same in any order (engram_scatter_add has the limits, for bf16).
 *   d_tokens as above (padding and invalid ids are skipped, the latter
 *   counted); d_grads [n, channels] of grads_type; d_grad_table [table_rows,
 *   channels] of table_type (accumulate: fp32 only).  table_rows < 2^32 - 1, n < 2^32 - 1.
 *   The workspace holds engram_embed_grad_workspace bytes, 16-byte aligned.
 *   More than 65,536 tokens are sorted with engram.h's bounded waits: should
 *   one expire, ENGRAM_ERR_STALLED is added to *d_err_count (when not NULL), and
 *   every value of the table is NaN (accumulate: the table is left as it was,
 *   so only the counter tells).
 * Errors: EINVAL, EALIGN, EWORKSPACE.  n == 0 writes zeros (accumulate:
 * nothing).
 */
int engram_embed(const int64_t *d_tokens, int64_t n, const void *d_table, int64_t table_rows,
                 int64_t channels, float scale, int32_t out_type, void *d_out,
                 int64_t *d_err_count, void *stream);
size_t engram_embed_grad_workspace(int64_t n, int64_t channels, int64_t table_rows);
int engram_embed_grad(const int64_t *d_tokens, int64_t n, const void *d_grads,
                      int32_t grads_type, int64_t channels, float scale, int64_t table_rows,
                      int32_t table_type, int32_t accumulate, void *d_grad_table,
                      void *d_workspace, size_t workspace_bytes, int64_t *d_err_count,
                      void *stream);

#ifdef __cplusplus
}
#endif

#endif /* ENGRAM_LAYER_H */
