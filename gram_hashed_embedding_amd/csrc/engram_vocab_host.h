// engram_vocab_host.h -- the host side of the operators at the vocabulary's
// end (include/engram_vocab.h) in plain C++: how rows of logits are cut, the
// workspaces, and the launchers of the HIP sources.
#pragma once

#include "engram_layer_host.h"
#include "engram_vocab.h"

namespace engram {

// A row of logits is read in chunks of 8 values, a lane to a chunk, by blocks
// of kScanThreads lanes.
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
// Chunks of 8 values that a lane of the backward pass holds, 32 registers of them: 2049 x
// 32,000 in fp32 takes 105.4 us, with half as many 106.4 (the teacher's row is read by twice
// the blocks), with twice as many 109.2 (fewer wavefronts fit a CU).
constexpr int distill_held_backward(size_t size) { return size == 2 ? 8 : 4; }
// A block takes a whole row, but for a few long rows with a gradient, which would leave CUs
// idle, and where a row's bits (one a value: whether a teacher's row names it) would take
// more than 32 KB of LDS: those are cut.  Loss and gradient of rows of 151,936 bf16 values,
// cut / not: 16 rows 19.7 / 29.6 us, 64 rows 20.9 / 30.1, 128 rows 28.7 / 35.4, 192 rows
// 42.8 / 38.1 (fp32: 64 rows 28.8 / 43.8, 128 rows 51.3 / 61.6, 192 rows 70.6 / 77.7).  Of
// 65,536 fp32 values, 64 rows 19.6 / 20.4, 128 rows 24.5 / 22.4; bf16 rows of that length lose 2
// to 3 us by it.  The loss alone gains nothing: its one pass is short beside what a second
// launch costs.
constexpr int64_t kDistillMaxSeg = int64_t(1) << 18;
constexpr int64_t kDistillBlocks = 1024;
constexpr int64_t kDistillFewRows = 128, kDistillFewVocab = 65536;
inline ScanShape distill_shape(int64_t rows, int64_t vocab) {
  return scan_shape(rows, vocab, kDistillBlocks, kDistillMaxSeg);
}
inline bool distill_cut(int64_t rows, int64_t vocab, bool grad) {
  return vocab > kDistillMaxSeg || (grad && rows <= kDistillFewRows && vocab >= kDistillFewVocab);
}
// What a segment of a row leaves: its sums (of the values that the teacher does not name,
// and of those it does) beside their maxima, its part of the loss, and the probability
// that this part is over.
struct DistillPart {
  double rest_sum, named_sum, loss, mass;
  float rest_max, named_max;
};
// The parts of every segment; nothing where a block takes a row.
inline size_t distill_workspace(int64_t rows, int64_t vocab, bool grad) {
  if (rows == 0 || !distill_cut(rows, vocab, grad)) return 0;
  return (size_t)rows * (size_t)distill_shape(rows, vocab).segs * sizeof(DistillPart);
}

// --------------------------------------------------------------- selection --
// The scan leaves the largest logit of every kBeamGroup values (16 lanes' chunks): the
// choice reads 1/64 of a bf16 row's bytes for them, and at most 96 groups of it again.  A
// selection among 512 rows of 151,936 bf16 values takes 44.2 us with 1024 blocks (two to a
// row), 46.7 with 2048 and 47.3 with 4096: a block's join is paid more often.
constexpr int64_t kBeamGroup = 128;
constexpr int64_t kBeamBlocks = 1024;
constexpr int64_t kBeamMaxSeg = int64_t(1) << 18;
inline ScanShape beam_shape(int64_t rows, int64_t vocab) {
  return scan_shape(rows, vocab, kBeamBlocks, kBeamMaxSeg);
}
inline int64_t beam_groups(int64_t vocab) { return ceil_div(vocab, kBeamGroup); }
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
