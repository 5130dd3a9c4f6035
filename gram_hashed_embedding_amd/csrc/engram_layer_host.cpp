// engram_layer_host.cpp -- the extern "C" entry points of include/
// engram_layer.h: argument checks on the host, then the launchers of the HIP
// sources.  Plain C++ (no HIP headers), so that the checks also build for the
// CPU alone.  Every check runs before anything is enqueued.
#include "engram_layer_host.h"

#include <cmath>
#include <initializer_list>

namespace engram {

NormShape norm_shape(int64_t rows, int64_t channels, int64_t groups, int max_items,
                     int64_t blocks, bool sums) {
  NormShape s = {};
  s.rows = rows;
  s.channels = channels;
  s.groups = groups;
  s.chunks = channels / groups / 8;
  // A group of up to 64 chunks: one chunk a lane, within a wavefront.  Longer
  // groups: a wavefront with up to max_items chunks a lane while there are
  // groups enough to fill the GPU so, else whole blocks (the fewer chunks a
  // lane holds, the shorter its row takes).
  s.threads = 256;
  if (s.chunks <= 64) {
    s.items = 1;
    s.lanes = 4;
    while (s.lanes < s.chunks) s.lanes *= 2;
  } else if (s.chunks <= 64 * (int64_t)max_items && rows * groups >= 4096) {
    s.lanes = 64;
    s.items = (int)ceil_div(s.chunks, 64);
  } else {
    s.lanes = s.chunks <= 256 * (int64_t)max_items && (s.chunks <= 256 || rows * groups >= 1024)
                  ? 256
                  : 1024;
    s.threads = s.lanes;
    s.items = (int)ceil_div(s.chunks, s.lanes);
  }
  const int slots = s.threads / s.lanes;
  s.gcols = 1;
  while (s.gcols < groups && s.gcols < slots) s.gcols *= 2;
  s.trows = slots / s.gcols;
  s.colblocks = ceil_div(groups, s.gcols);
  const int64_t steps = rows > 0 ? ceil_div(rows, s.trows) : 1;  // of trows rows each
  int64_t want = blocks * 256 / s.threads / s.colblocks;
  if (want < 1) want = 1;
  if (sums) {
    // Few rows: four steps a block while that leaves 512 blocks (the sums' rows
    // that the blocks leave cost as much as their idle threads: [4099, 1024] with
    // 16 groups took 26.3 us so, 32 us with a block to a step or two).
    const int64_t least = ceil_div(512, s.colblocks), four = steps / 4;
    if (want > four && want > least) want = four > least ? four : least;
    if (want * kNormMaxSteps < steps) want = ceil_div(steps, kNormMaxSteps);
  }
  s.rowblocks = steps < want ? steps : want;
  return s;
}

ConvBackwardShape conv_backward_shape(int64_t batch, int64_t seq, int64_t halo_len,
                                      int64_t channels, int32_t K, int32_t dilation) {
  ConvBackwardShape s = {};
  s.quads = channels / 4;
  s.groups = ceil_div(s.quads, 64);
  // about 2048 waves, as many as stay on 256 CUs at a time (8 each; 4 each where the
  // window's registers leave one wave a SIMD, from dilation 5 or 6 on: those run in two
  // rounds); a slice not so short that the rows it reads past its end (the register
  // window's) outweigh its own, nor so long that its fp32 sums lose bits
  const int64_t want = ceil_div(2048, (batch > 0 ? batch : 1) * s.groups);
  const int64_t ahead = conv_windowed(K, dilation) ? (int64_t)(K - 1) * dilation : 0;
  const int64_t least = 2 * ahead > 32 ? 2 * ahead : 32;
  s.slice = ceil_div(seq > 0 ? seq : 1, want);
  if (s.slice < least) s.slice = least;
  if (s.slice > kConvMaxSlice) s.slice = kConvMaxSlice;
  s.halo_slices = ceil_div(halo_len, s.slice);
  s.slices = s.halo_slices + ceil_div(seq, s.slice);
  return s;
}

}  // namespace engram

using namespace engram;

namespace {

bool any_misaligned(std::initializer_list<const void *> ptrs) {
  for (const void *p : ptrs)
    if (!aligned16(p)) return true;
  return false;
}

// The sizes of a residual norm.
bool norm_sizes_ok(int64_t rows, int64_t channels, int64_t groups) {
  if (rows < 0 || channels <= 0 || groups <= 0 || channels > kMaxDim || groups > channels / 8)
    return false;
  if (channels % (8 * groups) != 0 || channels / groups > ENGRAM_NORM_MAX_GROUP) return false;
  return mul_fits(rows, channels * 4, INT64_MAX / 4);
}

// The arguments the norm and its backward share.
int check_norm(const engram_norm_args *a) {
  if (a == nullptr) return ENGRAM_EINVAL;
  if (!norm_sizes_ok(a->rows, a->channels, a->groups) || a->reserved != 0) return ENGRAM_EINVAL;
  if (a->residual_type != ENGRAM_BF16 && a->residual_type != ENGRAM_F32) return ENGRAM_EINVAL;
  if (!std::isfinite(a->residual_scale)) return ENGRAM_EINVAL;
  if (a->gate_width != 0 && a->gate_width != a->groups && a->gate_width != a->channels)
    return ENGRAM_EINVAL;
  if (a->rows > 0 && (a->gate_width != 0) != (a->d_gate != nullptr)) return ENGRAM_EINVAL;
  if ((a->d_y_codes != nullptr) != (a->d_y_scales != nullptr)) return ENGRAM_EINVAL;
  if ((a->d_next_codes != nullptr) != (a->d_next_scales != nullptr)) return ENGRAM_EINVAL;
  return ENGRAM_OK;
}

}  // namespace

// ----------------------------------------------------------- residual norm --
extern "C" int engram_residual_norm(const engram_norm_args *a) {
  const int rc = check_norm(a);
  if (rc != ENGRAM_OK) return rc;
  if (!(a->eps > 0.0f) || !std::isfinite(a->eps)) return ENGRAM_EINVAL;
  const bool next = a->d_w_next != nullptr;
  if (!next && (a->d_next != nullptr || a->d_rstd_next != nullptr || a->d_next_codes != nullptr))
    return ENGRAM_EINVAL;
  if (a->rows == 0) return ENGRAM_OK;
  if (a->d_residual == nullptr) return ENGRAM_EINVAL;
  if (a->d_y == nullptr) {
    if (a->d_out != nullptr || a->d_gate != nullptr || a->d_w_post != nullptr ||
        a->d_scale != nullptr || a->d_rstd_post != nullptr || a->d_y_codes != nullptr ||
        a->residual_scale != 1.0f || !next)
      return ENGRAM_EINVAL;
  } else if (a->d_out == nullptr) {
    return ENGRAM_EINVAL;
  }
  if (next && a->d_next == nullptr) return ENGRAM_EINVAL;
  if (any_misaligned({a->d_residual, a->d_y, a->d_w_post, a->d_scale, a->d_w_next, a->d_out,
                      a->d_next, a->d_y_codes, a->d_next_codes}) ||
      (a->gate_width == a->channels && !aligned16(a->d_gate)))
    return ENGRAM_EALIGN;
  return launch_residual_norm(*a);
}

extern "C" size_t engram_residual_norm_backward_workspace(int64_t rows, int64_t channels,
                                                          int64_t groups) {
  if (!norm_sizes_ok(rows, channels, groups)) return (size_t)-1;
  if (rows == 0) return 0;
  return (size_t)norm_partial_floats(norm_backward_shape(rows, channels, groups)) * 4;
}

extern "C" int engram_residual_norm_backward(const engram_norm_args *a) {
  const int rc = check_norm(a);
  if (rc != ENGRAM_OK) return rc;
  const bool next = a->d_w_next != nullptr;
  const bool sums = a->d_grad_w_post != nullptr || a->d_grad_scale != nullptr ||
                    a->d_grad_w_next != nullptr;
  if (!next && a->d_grad_w_next != nullptr) return ENGRAM_EINVAL;
  if (a->rows > 0) {
    if (next != (a->d_grad_next != nullptr)) return ENGRAM_EINVAL;
    if (a->d_grad_out == nullptr && a->d_grad_next == nullptr) return ENGRAM_EINVAL;
    if (next && (a->d_out == nullptr || a->d_rstd_next == nullptr)) return ENGRAM_EINVAL;
    if (a->d_y != nullptr && a->d_y_codes != nullptr) return ENGRAM_EINVAL;
    const bool branch = a->d_y != nullptr || a->d_y_codes != nullptr;
    if (branch && a->d_rstd_post == nullptr) return ENGRAM_EINVAL;
    if (!branch && (a->d_grad_y != nullptr || a->d_gate != nullptr || a->d_w_post != nullptr ||
                    a->d_scale != nullptr || a->residual_scale != 1.0f))
      return ENGRAM_EINVAL;
    if (a->d_gate == nullptr && a->d_grad_gate != nullptr) return ENGRAM_EINVAL;
  }
  if (a->d_w_post == nullptr && a->d_grad_w_post != nullptr) return ENGRAM_EINVAL;
  if (a->d_scale == nullptr && a->d_grad_scale != nullptr) return ENGRAM_EINVAL;
  if (any_misaligned({a->d_y, a->d_y_codes, a->d_w_post, a->d_scale, a->d_w_next, a->d_out,
                      a->d_grad_out, a->d_grad_next, a->d_grad_residual, a->d_grad_y,
                      a->d_grad_w_post, a->d_grad_scale, a->d_grad_w_next}) ||
      (a->gate_width == a->channels && any_misaligned({a->d_gate, a->d_grad_gate})))
    return ENGRAM_EALIGN;
  if (sums && a->rows > 0) {
    const size_t need =
        engram_residual_norm_backward_workspace(a->rows, a->channels, a->groups);
    if (a->d_workspace == nullptr || !aligned16(a->d_workspace) || a->workspace_bytes < need)
      return ENGRAM_EWORKSPACE;
  }
  if (!sums && (a->rows == 0 || (a->d_grad_residual == nullptr && a->d_grad_y == nullptr &&
                                 a->d_grad_gate == nullptr)))
    return ENGRAM_OK;
  return launch_residual_norm_backward(*a);
}

// ------------------------------------------------------- 8-bit checkpoints --
namespace {

int check_act(const void *x, const void *codes, const float *scales, int64_t rows,
              int64_t channels) {
  if (rows < 0 || channels <= 0 || channels % 8 != 0 || channels > kMaxDim) return ENGRAM_EINVAL;
  if (!mul_fits(rows, channels * 2, INT64_MAX / 16)) return ENGRAM_EINVAL;
  if (rows == 0) return ENGRAM_OK;
  if (x == nullptr || codes == nullptr || scales == nullptr) return ENGRAM_EINVAL;
  if (any_misaligned({x, codes})) return ENGRAM_EALIGN;
  return ENGRAM_OK;
}

}  // namespace

extern "C" int engram_act_encode(const void *d_x, int64_t rows, int64_t channels,
                                 int8_t *d_codes, float *d_scales, void *stream) {
  const int rc = check_act(d_x, d_codes, d_scales, rows, channels);
  if (rc != ENGRAM_OK || rows == 0) return rc;
  return launch_act_encode(d_x, rows, channels, d_codes, d_scales, stream);
}

extern "C" int engram_act_decode(const int8_t *d_codes, const float *d_scales, int64_t rows,
                                 int64_t channels, void *d_x, void *stream) {
  const int rc = check_act(d_x, d_codes, d_scales, rows, channels);
  if (rc != ENGRAM_OK || rows == 0) return rc;
  return launch_act_decode(d_codes, d_scales, rows, channels, d_x, stream);
}

// ------------------------------------------------------------- convolution --
namespace {

bool conv_sizes_ok(int64_t batch, int64_t seq, int64_t halo_len, int64_t channels,
                   int32_t kernel_size, int32_t dilation) {
  if (batch < 0 || seq < 0 || channels <= 0 || channels % 8 != 0 || channels > kMaxDim ||
      halo_len < 0)
    return false;
  if (kernel_size < 1 || kernel_size > kConvMaxKernel || dilation < 1) return false;
  if (seq > INT64_MAX / 4 - halo_len || !mul_fits(batch, seq + halo_len, INT64_MAX / 64))
    return false;
  return mul_fits(batch * (seq + halo_len), channels * 4, INT64_MAX / 16);
}

}  // namespace

extern "C" size_t engram_ple_conv_backward_workspace(int64_t batch, int64_t seq,
                                                     int64_t halo_len, int64_t channels,
                                                     int32_t kernel_size, int32_t dilation) {
  if (!conv_sizes_ok(batch, seq, halo_len, channels, kernel_size, dilation)) return (size_t)-1;
  const ConvBackwardShape s =
      conv_backward_shape(batch, seq, halo_len, channels, kernel_size, dilation);
  return (size_t)(batch * s.slices) * (size_t)(kernel_size + 1) * (size_t)channels * 4;
}

extern "C" int engram_ple_conv_backward(
    const void *d_grad_out, const void *d_x, const int8_t *d_x_codes, const float *d_x_scales,
    int64_t code_width, const void *d_halo, int64_t halo_len, const int64_t *d_seq_ids,
    const void *d_weight, int64_t batch, int64_t seq, int64_t channels, int32_t kernel_size,
    int32_t dilation, void *d_grad_x, void *d_grad_halo, float *d_grad_weight,
    float *d_grad_bias, void *d_workspace, size_t workspace_bytes, void *stream) {
  if (!conv_sizes_ok(batch, seq, halo_len, channels, kernel_size, dilation))
    return ENGRAM_EINVAL;
  if (code_width < 0 || code_width % 8 != 0 || (code_width > 0 && channels % code_width != 0))
    return ENGRAM_EINVAL;
  if ((d_x_codes != nullptr) != (d_x_scales != nullptr) ||
      (d_x_codes != nullptr && d_x != nullptr))
    return ENGRAM_EINVAL;
  if (halo_len == 0 && (d_halo != nullptr || d_grad_halo != nullptr)) return ENGRAM_EINVAL;
  if (batch > 0 && seq > 0) {
    if (d_grad_out == nullptr || d_weight == nullptr) return ENGRAM_EINVAL;
    if (d_grad_weight != nullptr && d_x == nullptr && d_x_codes == nullptr) return ENGRAM_EINVAL;
    if (d_grad_weight != nullptr && halo_len > 0 && d_halo == nullptr) return ENGRAM_EINVAL;
  }
  if (any_misaligned({d_grad_out, d_x, d_x_codes, d_halo, d_weight, d_grad_x, d_grad_halo,
                      d_grad_weight, d_grad_bias}))
    return ENGRAM_EALIGN;
  if (d_grad_weight != nullptr || d_grad_bias != nullptr) {
    const size_t need = engram_ple_conv_backward_workspace(batch, seq, halo_len, channels,
                                                           kernel_size, dilation);
    if (need > 0 && (d_workspace == nullptr || !aligned16(d_workspace) || workspace_bytes < need))
      return ENGRAM_EWORKSPACE;
  }
  if (d_grad_x == nullptr && d_grad_halo == nullptr && d_grad_weight == nullptr &&
      d_grad_bias == nullptr)
    return ENGRAM_OK;
  const ConvBackwardCall c = {d_grad_out, d_x,      d_x_codes, d_x_scales,
                              code_width > 0 ? code_width : channels,
                              d_halo,     halo_len, d_seq_ids, d_weight,
                              batch,      seq,      channels,  kernel_size,
                              dilation,   d_grad_x, d_grad_halo, d_grad_weight,
                              d_grad_bias, static_cast<float *>(d_workspace)};
  return launch_conv_backward(c, stream);
}

extern "C" int engram_ple_conv_step(const void *d_x, void *d_ring, int64_t ring_count,
                                    int64_t ring_rows, const int64_t *d_ring_ids,
                                    const int64_t *d_positions, const void *d_weight,
                                    const void *d_bias, int64_t batch, int64_t tokens,
                                    int64_t channels, int32_t kernel_size, int32_t dilation,
                                    void *d_out, int64_t *d_err_count, void *stream) {
  if (!conv_sizes_ok(batch, tokens, 0, channels, kernel_size, dilation)) return ENGRAM_EINVAL;
  if (ring_count < 0 || ring_rows < 1 || ring_rows < (int64_t)(kernel_size - 1) * dilation)
    return ENGRAM_EINVAL;
  if (!mul_fits(ring_count, ring_rows, INT64_MAX / 64) ||
      !mul_fits(ring_count * ring_rows, channels * 2, INT64_MAX / 16))
    return ENGRAM_EINVAL;
  if (d_ring_ids == nullptr && ring_count < batch) return ENGRAM_EINVAL;
  if (batch == 0 || tokens == 0) return ENGRAM_OK;
  if (d_x == nullptr || d_positions == nullptr || d_weight == nullptr ||
      (d_ring == nullptr && ring_count > 0))
    return ENGRAM_EINVAL;
  if (any_misaligned({d_x, d_ring, d_weight, d_bias, d_out})) return ENGRAM_EALIGN;
  const ConvStepCall c = {d_x, d_ring, ring_count, ring_rows, d_ring_ids, d_positions,
                          d_weight, d_bias, batch, tokens, channels, kernel_size, dilation,
                          d_out, d_err_count};
  return launch_conv_step(c, stream);
}

// --------------------------------------------------------------- embedding --
namespace {

bool embed_sizes_ok(int64_t n, int64_t channels, int64_t table_rows, int32_t type) {
  if (n < 0 || channels <= 0 || channels % 8 != 0 || channels > kMaxDim || table_rows < 0)
    return false;
  if (type != ENGRAM_BF16 && type != ENGRAM_F32) return false;
  return mul_fits(n, channels * 8, INT64_MAX / 16) &&
         mul_fits(table_rows, channels * 4, INT64_MAX / 16);
}

// The plan of the tokens as row ids (its own partial rows, 8 values wide, are
// not used: the gradient has its own after it).
bool embed_plan(int64_t n, int64_t table_rows, Plan *p) {
  return sorted_limits_ok(n, table_rows) && make_plan(n, table_rows, 8, p) &&
         grid_fits(apply_blocks(*p, 8), kWalkThreads);
}

size_t embed_partials(int64_t n, int64_t channels) {
  return (size_t)ceil_div(n, embed_chunk(n, channels)) * 2 * (size_t)channels * 8;
}

size_t embed_marks(int64_t table_rows) {
  return (size_t)(ceil_div(table_rows, kEmbedMarkRows) * kEmbedMarkRows);
}

}  // namespace

extern "C" int engram_embed(const int64_t *d_tokens, int64_t n, const void *d_table,
                            int64_t table_rows, int64_t channels, float scale, int32_t out_type,
                            void *d_out, int64_t *d_err_count, void *stream) {
  if (!embed_sizes_ok(n, channels, table_rows, out_type)) return ENGRAM_EINVAL;
  if (n == 0) return ENGRAM_OK;
  if (d_tokens == nullptr || d_out == nullptr || (d_table == nullptr && table_rows > 0))
    return ENGRAM_EINVAL;
  if (any_misaligned({d_table, d_out})) return ENGRAM_EALIGN;
  return launch_embed(d_tokens, n, d_table, table_rows, channels, scale, out_type, d_out,
                      d_err_count, stream);
}

extern "C" size_t engram_embed_grad_workspace(int64_t n, int64_t channels, int64_t table_rows) {
  Plan p;
  if (!embed_sizes_ok(n, channels, table_rows, ENGRAM_F32) || !embed_plan(n, table_rows, &p))
    return (size_t)-1;
  return p.total + embed_partials(n, channels) + embed_marks(table_rows);
}

extern "C" int engram_embed_grad(const int64_t *d_tokens, int64_t n, const void *d_grads,
                                 int32_t grads_type, int64_t channels, float scale,
                                 int64_t table_rows, int32_t table_type, int32_t accumulate,
                                 void *d_grad_table, void *d_workspace, size_t workspace_bytes,
                                 int64_t *d_err_count, void *stream) {
  Plan p;
  if (!embed_sizes_ok(n, channels, table_rows, table_type) || !embed_plan(n, table_rows, &p))
    return ENGRAM_EINVAL;
  if (grads_type != ENGRAM_BF16 && grads_type != ENGRAM_F32) return ENGRAM_EINVAL;
  if (accumulate != 0 && (accumulate != 1 || table_type != ENGRAM_F32)) return ENGRAM_EINVAL;
  if (table_rows > 0 && d_grad_table == nullptr && !(n == 0 && accumulate)) return ENGRAM_EINVAL;
  if (n > 0 && (d_tokens == nullptr || d_grads == nullptr)) return ENGRAM_EINVAL;
  if (any_misaligned({d_grads, d_grad_table})) return ENGRAM_EALIGN;
  if (n > 0 && (d_workspace == nullptr || !aligned16(d_workspace) ||
                workspace_bytes < engram_embed_grad_workspace(n, channels, table_rows)))
    return ENGRAM_EWORKSPACE;
  if (n == 0 && (accumulate || table_rows == 0)) return ENGRAM_OK;
  double *partials =
      n > 0 ? reinterpret_cast<double *>(static_cast<char *>(d_workspace) + p.total) : nullptr;
  uint8_t *present =
      n > 0 ? reinterpret_cast<uint8_t *>(partials) + embed_partials(n, channels) : nullptr;
  const EmbedGradCall c = {d_tokens,   n,          d_grads,    grads_type,   channels, scale,
                           table_rows, table_type, accumulate, d_grad_table, partials, present,
                           d_err_count};
  return launch_embed_grad(c, p, d_workspace, stream);
}
