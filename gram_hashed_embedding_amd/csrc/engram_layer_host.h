// engram_layer_host.h -- the host side of the layer operators (include/
// engram_layer.h) in plain C++: the calls' checked arguments, the sizes of
// their workspaces, and the launchers of the HIP sources.  As engram_host.h:
// the entry points (engram_layer_host.cpp) check, then call one launcher.
#pragma once

#include "engram_host.h"
#include "engram_layer.h"

namespace engram {

constexpr int64_t kActBlock = ENGRAM_ACT_BLOCK;
inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// ----------------------------------------------------------- residual norm --
// How a norm kernel covers [rows, groups] groups of n = 8 * chunks channels.
// A group belongs to `lanes` threads, each holding `items` chunks of 8
// channels; a block of `threads` threads holds threads / lanes groups at a
// time: `gcols` adjacent groups of each of `trows` rows.  The grid is
// `colblocks` column blocks times `rowblocks` row blocks, which take the rows
// `trows` at a time in turn: the blocks that run together then work on one
// stretch of memory that moves on.
struct NormShape {
  int64_t rows, channels, groups, chunks;
  int lanes, items, threads, gcols, trows;
  int64_t colblocks, rowblocks;
};

// The shape for a kernel that holds at most max_items chunks a lane, with
// about `blocks` blocks when there is work for them; sums: each row block also
// leaves sums over its rows.
NormShape norm_shape(int64_t rows, int64_t channels, int64_t groups, int max_items,
                     int64_t blocks, bool sums);

constexpr int kNormForwardItems = 4;
constexpr int kNormBackwardItems = 2;
// The forward: a block takes a few rows and ends, so that the blocks that run
// together stay together in memory (65,536 x 6144: 32,768 blocks 943 us, 4096
// 1040, one for each row 960).  The backward: as many blocks of 256 threads as
// stay on the GPU together where a lane holds one chunk (3 wavefronts a SIMD),
// since each leaves sums (65,536 x 6144 in 24 groups: 768 blocks 1236 us, 1536
// 1274, 3072 1291).  That shape is where the count was measured.  Kernels of two
// chunks a lane keep 2 wavefronts a SIMD, so 768 of their blocks run in one and a
// half rounds; blocks of 1024 threads are scaled to 192, fewer than the 256 CUs
// ([16384, 4096] as one group takes 192 us against a floor of 124, [8192, 6144]
// 213 against 140).
constexpr int64_t kNormForwardBlocks = 32768;
constexpr int64_t kNormBackwardBlocks = 768;
// Most rows a lane sums in fp32 before the sums go on in fp64.
constexpr int64_t kNormMaxSteps = 256;

inline NormShape norm_forward_shape(int64_t rows, int64_t channels, int64_t groups) {
  return norm_shape(rows, channels, groups, kNormForwardItems, kNormForwardBlocks, false);
}
inline NormShape norm_backward_shape(int64_t rows, int64_t channels, int64_t groups) {
  return norm_shape(rows, channels, groups, kNormBackwardItems, kNormBackwardBlocks, true);
}
// The backward's sums over rows: each row block leaves two fp32 rows.
inline int64_t norm_partial_floats(const NormShape &s) { return s.rowblocks * 2 * s.channels; }

// ------------------------------------------------------------- convolution --
// The backward's work: waves of 64 lanes, each owning 4 channels a lane
// (256 channels) and `slice` consecutive positions of a row's halo (the first
// halo_slices slices) or of its sequence.  Each leaves kernel_size + 1 fp32
// sums a channel.
constexpr int64_t kConvMaxSlice = 1024;
// The shapes of the register-window kernel.
inline bool conv_windowed(int32_t K, int32_t dilation) { return K == 4 && dilation <= 8; }
struct ConvBackwardShape {
  int64_t quads, groups, slice, halo_slices, slices;  // slices: a row's, the halo's included
};
ConvBackwardShape conv_backward_shape(int64_t batch, int64_t seq, int64_t halo_len,
                                      int64_t channels, int32_t K, int32_t dilation);

struct ConvBackwardCall {
  const void *grad_out, *x;
  const int8_t *codes;
  const float *scales;
  int64_t code_width;
  const void *halo;
  int64_t halo_len;
  const int64_t *seg;
  const void *weight;
  int64_t batch, seq, channels;
  int32_t K, dilation;
  void *grad_x, *grad_halo;
  float *grad_weight, *grad_bias;
  float *partials;  // [batch * slices][K + 1][channels]
};

struct ConvStepCall {
  const void *x;
  void *ring;
  int64_t ring_count, ring_rows;
  const int64_t *ring_ids, *positions;
  const void *weight, *bias;
  int64_t batch, tokens, channels;
  int32_t K, dilation;
  void *out;
  int64_t *err;
};

// --------------------------------------------------------------- embedding --
// The gradient's sorted tokens are cut into chunks of a power of two of
// positions, one to a walker of row_lanes threads.  A chunk leaves up to two
// fp64 rows: the part of the run that enters it, and of the one that leaves it.
inline int embed_row_lanes(int64_t channels) {
  int l = 1;
  while (l < channels / 8 && l < 256) l *= 2;
  return l;
}
inline int64_t embed_chunk(int64_t n, int64_t channels) {
  // about 512 blocks of walkers, so that a frequent token's run is spread over
  // the GPU while its parts stay few
  const int64_t walkers = 512 * (256 / embed_row_lanes(channels));
  int64_t chunk = 16;
  while (chunk < 128 && chunk * walkers < n) chunk *= 2;
  return chunk;
}

constexpr int64_t kEmbedMarkRows = 4096;

struct EmbedGradCall {
  const int64_t *tokens;
  int64_t n;
  const void *grads;
  int32_t grads_type;
  int64_t channels;
  float scale;
  int64_t table_rows;
  int32_t type, accumulate;
  void *grad_table;
  double *partials;  // [chunks][2][channels]
  uint8_t *present;  // [table_rows, rounded up to whole kEmbedMarkRows]
  int64_t *err;
};

// -------------------------------------------------------------- launchers --
int launch_residual_norm(const engram_norm_args &a);
int launch_residual_norm_backward(const engram_norm_args &a);
int launch_act_encode(const void *d_x, int64_t rows, int64_t channels, int8_t *d_codes,
                      float *d_scales, void *stream);
int launch_act_decode(const int8_t *d_codes, const float *d_scales, int64_t rows,
                      int64_t channels, void *d_x, void *stream);
int launch_conv_backward(const ConvBackwardCall &c, void *stream);
int launch_conv_step(const ConvStepCall &c, void *stream);
int launch_embed(const int64_t *d_tokens, int64_t n, const void *d_table, int64_t table_rows,
                 int64_t channels, float scale, int32_t out_type, void *d_out,
                 int64_t *d_err_count, void *stream);
// launch_plan's sort for ids that crowd together (a vocabulary's frequent
// tokens have neighbouring ids): every digit in a pass of its own, none left to
// buckets of the top digit, which one block would sort nearly whole.  It leaves
// the sorted keys and positions and the stall flag; no slots, no stamp.
int launch_sort_crowded(const int64_t *d_row_ids, int64_t n, int64_t table_rows, const Plan &p,
                        void *d_workspace, int64_t *d_err_count, void *stream);
int launch_embed_grad(const EmbedGradCall &c, const Plan &p, void *d_workspace, void *stream);

}  // namespace engram
