// vocab_launch_stub.cpp -- stand-ins for the HIP launchers of the vocabulary
// operators, beside host_launch_stub.cpp: with them csrc/engram_vocab_host.cpp
// builds and runs on a CPU alone, under host sanitizers.  Each only checks that
// the entry point handed it a consistent call.
#include <cstdlib>

#include "engram_vocab_host.h"

namespace engram {

namespace {
void require(bool ok) {
  if (!ok) std::abort();
}
}  // namespace

int launch_distill(const engram_distill_args &a) {
  require(a.rows > 0 && a.vocab > 0 && a.d_logits && a.d_ids && a.d_teacher);
  require((a.d_grad != nullptr) == (a.d_grad_loss != nullptr));
  const size_t need = distill_workspace(a.rows, a.vocab, a.d_grad != nullptr);
  require(need == 0 || (a.d_workspace && a.workspace_bytes >= need));
  const ScanShape s = distill_shape(a.rows, a.vocab);
  require(s.segs * s.seg_len >= a.vocab && (s.segs - 1) * s.seg_len < a.vocab);
  return ENGRAM_OK;
}

int launch_distill_backward(const engram_distill_args &a) {
  require(a.rows > 0 && a.d_grad && a.d_lse && (!a.rest || a.d_lse_rest));
  return ENGRAM_OK;
}

int launch_beam_select(const BeamCall &c, void *) {
  require(c.batch > 0 && c.beams > 0 && c.count > 0 && c.logits && c.parts && c.maxima);
  const ScanShape s = beam_shape(c.batch * c.beams, c.vocab);
  require(s.segs * s.seg_len >= c.vocab && (s.segs - 1) * s.seg_len < c.vocab);
  return ENGRAM_OK;
}

int launch_beam_fork(const ForkCall &c, void *) {
  require(c.batch > 0 && c.parents && c.new_slots && c.pool_count >= 0);
  for (int p = 0; p < c.pool_count; ++p) require(c.slot_bytes[p] % 16 == 0);
  return ENGRAM_OK;
}

}  // namespace engram
