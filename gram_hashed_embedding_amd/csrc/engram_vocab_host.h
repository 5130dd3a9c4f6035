// engram_vocab_host.h -- the host side of the operators at the vocabulary's
// end (include/engram_vocab.h) in plain C++: how rows of logits are cut, the
// workspaces, and the launchers of the HIP sources.
#pragma once

#include "engram_layer_host.h"
#include "engram_vocab.h"

namespace engram {

// A row of logits is read in chunks of 8 values, a lane to a chunk, by blocks
// of kScanThreads lanes; a block's step takes kScanSteps chunks a lane.
constexpr int kScanThreads = 256;
constexpr int64_t kScanTile = 8 * kScanThreads;  // values
constexpr int64_t kMaxVocab = int64_t(1) << 30;

// Rows are cut into `segs` segments of seg_len values (a multiple of
// kScanTile), a block to each.
struct ScanShape {
  int64_t segs, seg_len;
};
// At least `blocks` blocks where the rows are long enough, and segments of at
// most `most` values.
inline ScanShape scan_shape(int64_t rows, int64_t vocab, int64_t blocks, int64_t most) {
  const int64_t tiles = ceil_div(vocab, kScanTile);
  int64_t want = ceil_div(blocks, rows > 0 ? rows : 1);
  if (want > tiles) want = tiles;
  int64_t per = ceil_div(tiles, want);
  if (per * kScanTile > most) per = most / kScanTile;
  return {ceil_div(tiles, per), per * kScanTile};
}

// The sum of exp((z - max) / temperature) over a segment, beside its max.
struct ScanPart {
  double sum;
  float max;
  uint32_t pad;
};

// ------------------------------------------------------------ distillation --
// Chunks of 8 values that a lane holds of a row, for values of `size` bytes (of the 128
// registers that a lane has in blocks of 1024, or four blocks of 256, on a CU), and of a
// segment in the backward pass.
constexpr int distill_held(size_t size) { return size == 2 ? 20 : 10; }
constexpr int distill_held_backward(size_t size) { return size == 2 ? 8 : 4; }
// Rows are cut where a gradient is asked for and there are few of them, and where a row's
// bits (one a value: whether a teacher's row names it) would take more than 32 KB of LDS.
constexpr int64_t kDistillMaxSeg = int64_t(1) << 18;
constexpr int64_t kDistillBlocks = 1024;
constexpr int64_t kDistillFewRows = 128, kDistillFewVocab = 65536;
inline ScanShape distill_shape(int64_t rows, int64_t vocab) {
  return scan_shape(rows, vocab, kDistillBlocks, kDistillMaxSeg);
}
// The threads of a block that holds a whole row for its gradient; 0 where none does.
inline int distill_threads(int64_t rows, int64_t vocab, size_t size) {
  if (vocab < 8 || (rows <= kDistillFewRows && vocab >= kDistillFewVocab)) return 0;
  for (int threads = 256; threads <= 1024; threads *= 2)
    if (vocab <= (threads - 64) * 8 * distill_held(size)) return threads;  // (one wavefront less)
  return 0;
}
// What a segment of a row leaves: its sums (of the values that the teacher does not name,
// and of those it does) beside their maxima, and its part of the loss.
struct DistillPart {
  double rest_sum, named_sum, loss;
  float rest_max, named_max;
};
// The parts of every segment; nothing where a block takes a row.
inline size_t distill_workspace(int64_t rows, int64_t vocab, int32_t type, bool grad) {
  const bool cut = grad ? distill_threads(rows, vocab, type == ENGRAM_BF16 ? 2 : 4) == 0
                        : vocab > kDistillMaxSeg;
  if (rows == 0 || !cut) return 0;
  return (size_t)rows * (size_t)distill_shape(rows, vocab).segs * sizeof(DistillPart);
}

// --------------------------------------------------------------- selection --
// The scan leaves the largest logit of every kBeamGroup values.
constexpr int64_t kBeamGroup = 128;
constexpr int64_t kBeamBlocks = 1024;
constexpr int64_t kBeamMaxSeg = int64_t(1) << 18;
inline ScanShape beam_shape(int64_t rows, int64_t vocab) {
  return scan_shape(rows, vocab, kBeamBlocks, kBeamMaxSeg);
}
struct BeamCall {
  const void *logits;
  int32_t type;
  int64_t stride;
  const float *scores;
  const uint8_t *finished;
  int64_t eos, batch, beams, vocab, count;
  float *out_scores;
  int64_t *out_parents, *out_tokens;
  uint8_t *out_finished;
  ScanPart *parts;  // [batch * beams][segs]
  float *maxima;    // [batch * beams][groups]
};
inline size_t beam_parts_bytes(int64_t rows, int64_t vocab) {
  return (size_t)rows * (size_t)beam_shape(rows, vocab).segs * sizeof(ScanPart);
}

struct ForkCall {
  const int64_t *parents, *slots;
  int64_t batch, beams;
  void *pools[ENGRAM_FORK_MAX_POOLS];
  int64_t slot_bytes[ENGRAM_FORK_MAX_POOLS];
  int32_t pool_count;
  int64_t slot_count;
  int64_t *new_slots;
  const int64_t *tokens, *history;
  int64_t history_len;
  int64_t *new_history;
  int64_t new_len;
  int64_t *err;
};

// -------------------------------------------------------------- launchers --
int launch_distill(const engram_distill_args &a);
int launch_distill_backward(const engram_distill_args &a);
int launch_beam_select(const BeamCall &c, void *stream);
int launch_beam_fork(const ForkCall &c, void *stream);

}  // namespace engram
