// engram_vocab_host.cpp -- the extern "C" entry points of include/
// engram_vocab.h: argument checks on the host, then the launchers of the HIP
// sources.  Plain C++ (no HIP headers), so that the checks also build for the
// CPU alone.  Every check runs before anything is enqueued.
#include "engram_vocab_host.h"

using namespace engram;

namespace {

bool type_ok(int32_t type) { return type == ENGRAM_BF16 || type == ENGRAM_F32; }

// Rows of logits: their count, length and stride.
bool rows_ok(int64_t rows, int64_t vocab, int64_t stride) {
  if (rows < 0 || vocab < 1 || vocab > kMaxVocab || stride < vocab) return false;
  return mul_fits(rows, stride, INT64_MAX / 16);
}

}  // namespace

// ------------------------------------------------------------ distillation --
extern "C" size_t engram_distill_workspace(int64_t rows, int64_t vocab, int32_t grad) {
  if (!rows_ok(rows, vocab, vocab) || grad < 0 || grad > 1) return (size_t)-1;
  return distill_workspace(rows, vocab, grad != 0);
}

namespace {

int check_distill(const engram_distill_args *a) {
  if (a == nullptr) return ENGRAM_EINVAL;
  if (!rows_ok(a->rows, a->vocab, a->logits_stride)) return ENGRAM_EINVAL;
  if (a->top < 1 || a->top > ENGRAM_DISTILL_MAX_TOP) return ENGRAM_EINVAL;
  if (!mul_fits(a->rows, a->top * 8, INT64_MAX / 16)) return ENGRAM_EINVAL;
  if (!type_ok(a->logits_type) || !type_ok(a->teacher_type)) return ENGRAM_EINVAL;
  if (a->rest != 0 && a->rest != 1) return ENGRAM_EINVAL;
  if (!(a->temperature >= 0x1p-64 && a->temperature <= 0x1p64)) return ENGRAM_EINVAL;
  if (a->reserved != 0) return ENGRAM_EINVAL;
  if (a->d_grad != nullptr && !rows_ok(a->rows, a->vocab, a->grad_stride)) return ENGRAM_EINVAL;
  if (a->d_grad != nullptr && a->d_grad == a->d_logits && a->grad_stride != a->logits_stride)
    return ENGRAM_EINVAL;
  if (a->rest == 0 && a->d_lse_rest != nullptr) return ENGRAM_EINVAL;
  if (a->rows == 0) return ENGRAM_OK;
  if (a->d_logits == nullptr || a->d_ids == nullptr || a->d_teacher == nullptr)
    return ENGRAM_EINVAL;
  if (a->rest == 1 && a->d_teacher_lse == nullptr) return ENGRAM_EINVAL;
  if ((a->d_grad != nullptr) != (a->d_grad_loss != nullptr)) return ENGRAM_EINVAL;
  return ENGRAM_OK;
}

}  // namespace

extern "C" int engram_distill(const engram_distill_args *a) {
  const int rc = check_distill(a);
  if (rc != ENGRAM_OK || a->rows == 0) return rc;
  if (a->d_loss == nullptr && a->d_lse == nullptr && a->d_lse_rest == nullptr &&
      a->d_grad == nullptr)
    return ENGRAM_EINVAL;
  // (a row's statistics are written while other blocks still read its inputs)
  const float *const outs[] = {a->d_loss, a->d_lse, a->d_lse_rest};
  for (int i = 0; i < 3; ++i)
    if (outs[i] != nullptr && (outs[i] == a->d_grad_loss || outs[i] == a->d_teacher_lse ||
                               outs[i] == outs[(i + 1) % 3]))
      return ENGRAM_EINVAL;
  const size_t need = distill_workspace(a->rows, a->vocab, a->d_grad != nullptr);
  if (need > 0 && (a->d_workspace == nullptr || !aligned16(a->d_workspace) ||
                   a->workspace_bytes < need))
    return ENGRAM_EWORKSPACE;
  return launch_distill(*a);
}

extern "C" int engram_distill_backward(const engram_distill_args *a) {
  const int rc = check_distill(a);
  if (rc != ENGRAM_OK || a->rows == 0) return rc;
  if (a->d_grad == nullptr || a->d_loss != nullptr || a->d_lse == nullptr ||
      (a->rest == 1 && a->d_lse_rest == nullptr))
    return ENGRAM_EINVAL;
  return launch_distill_backward(*a);
}

// --------------------------------------------------------------- selection --
namespace {

bool beams_ok(int64_t batch, int64_t beams) {
  return batch >= 0 && beams >= 1 && beams <= ENGRAM_BEAM_MAX &&
         mul_fits(batch, beams, INT64_MAX / 64);
}

}  // namespace

extern "C" size_t engram_beam_select_workspace(int64_t batch, int64_t beams, int64_t vocab) {
  if (!beams_ok(batch, beams) || !rows_ok(batch * beams, vocab, vocab)) return (size_t)-1;
  const int64_t rows = batch * beams;
  if (rows == 0) return 0;
  return beam_parts_bytes(rows, vocab) + (size_t)rows * (size_t)beam_groups(vocab) * 4;
}

extern "C" int engram_beam_select(const void *d_logits, int32_t type, int64_t logits_stride,
                                  const float *d_scores, const uint8_t *d_finished,
                                  int64_t eos_id, int64_t batch, int64_t beams, int64_t vocab,
                                  int64_t count, float *d_out_scores, int64_t *d_out_parents,
                                  int64_t *d_out_tokens, uint8_t *d_out_finished,
                                  void *d_workspace, size_t workspace_bytes, void *stream) {
  if (!beams_ok(batch, beams) || !rows_ok(batch * beams, vocab, logits_stride) || !type_ok(type))
    return ENGRAM_EINVAL;
  if (count < 1 || count > ENGRAM_BEAM_MAX) return ENGRAM_EINVAL;
  if (eos_id < -1 || eos_id >= vocab || (d_finished != nullptr && eos_id < 0))
    return ENGRAM_EINVAL;
  if (batch == 0) return ENGRAM_OK;
  if (d_logits == nullptr || d_scores == nullptr || d_out_scores == nullptr ||
      d_out_parents == nullptr || d_out_tokens == nullptr)
    return ENGRAM_EINVAL;
  if (count != beams &&
      (d_out_scores == d_scores || (d_finished != nullptr && d_out_finished == d_finished)))
    return ENGRAM_EINVAL;
  if (d_workspace == nullptr || !aligned16(d_workspace) ||
      workspace_bytes < engram_beam_select_workspace(batch, beams, vocab))
    return ENGRAM_EWORKSPACE;
  char *ws = static_cast<char *>(d_workspace);
  const BeamCall c = {d_logits, type, logits_stride, d_scores, d_finished, eos_id, batch, beams,
                      vocab, count, d_out_scores, d_out_parents, d_out_tokens, d_out_finished,
                      reinterpret_cast<ScanPart *>(ws),
                      reinterpret_cast<float *>(ws + beam_parts_bytes(batch * beams, vocab))};
  return launch_beam_select(c, stream);
}

extern "C" int engram_beam_fork(const int64_t *d_parents, const int64_t *d_slots, int64_t batch,
                                int64_t beams, void *const *h_pools, const int64_t *h_slot_bytes,
                                int32_t pools, int64_t slot_count, int64_t *d_new_slots,
                                const int64_t *d_tokens, const int64_t *d_history,
                                int64_t history_len, int64_t *d_new_history, int64_t new_len,
                                int64_t *d_err_count, void *stream) {
  if (!beams_ok(batch, beams) || slot_count < 0) return ENGRAM_EINVAL;
  if (pools < 0 || pools > ENGRAM_FORK_MAX_POOLS ||
      (pools > 0 && (h_pools == nullptr || h_slot_bytes == nullptr)))
    return ENGRAM_EINVAL;
  ForkCall c = {};
  bool misaligned = false;
  for (int32_t i = 0; i < pools; ++i) {
    if (h_slot_bytes[i] < 16 || h_slot_bytes[i] % 16 != 0 ||
        !mul_fits(slot_count, h_slot_bytes[i], INT64_MAX / 16))
      return ENGRAM_EINVAL;
    if (h_pools[i] == nullptr && slot_count > 0 && batch > 0) return ENGRAM_EINVAL;
    for (int32_t k = 0; k < i; ++k)
      if (h_pools[i] == h_pools[k] && h_pools[i] != nullptr) return ENGRAM_EINVAL;
    misaligned |= !aligned16(h_pools[i]);
    c.pools[i] = h_pools[i];
    c.slot_bytes[i] = h_slot_bytes[i];
  }
  if (d_new_history != nullptr || d_history != nullptr || d_tokens != nullptr) {
    if (history_len < 0 || history_len > kMaxDim || new_len < 1 || new_len > history_len + 1)
      return ENGRAM_EINVAL;
    if (!mul_fits(batch * beams, history_len + 1, INT64_MAX / 64)) return ENGRAM_EINVAL;
    if (batch > 0 && (d_new_history == nullptr || d_tokens == nullptr ||
                      (d_history == nullptr && history_len > 0) || d_new_history == d_history))
      return ENGRAM_EINVAL;
  }
  // (without explicit slots every beam has one of its own)
  if (pools > 0 && d_slots == nullptr && slot_count < batch * beams) return ENGRAM_EINVAL;
  if (batch == 0) return ENGRAM_OK;
  if (d_parents == nullptr || d_new_slots == nullptr || d_new_slots == d_slots ||
      d_new_slots == d_parents)
    return ENGRAM_EINVAL;
  if (misaligned) return ENGRAM_EALIGN;
  c.parents = d_parents;
  c.slots = d_slots;
  c.batch = batch;
  c.beams = beams;
  c.pool_count = pools;
  c.slot_count = slot_count;
  c.new_slots = d_new_slots;
  c.tokens = d_tokens;
  c.history = d_history;
  c.history_len = history_len;
  c.new_history = d_new_history;
  c.new_len = new_len;
  c.err = d_err_count;
  return launch_beam_fork(c, stream);
}
