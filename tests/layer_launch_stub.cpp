// layer_launch_stub.cpp -- stand-ins for the HIP launchers of the layer
// operators, beside host_launch_stub.cpp: with them csrc/engram_layer_host.cpp
// builds and runs on a CPU alone, under host sanitizers.  Each only checks that
// the entry point handed it a consistent call.
#include <cstdlib>

#include "engram_layer_host.h"

namespace engram {

namespace {
void require(bool ok) {
  if (!ok) std::abort();
}
}  // namespace

int launch_residual_norm(const engram_norm_args &a) {
  require(a.rows > 0 && a.d_residual != nullptr && a.channels % (8 * a.groups) == 0);
  require(a.d_y == nullptr ? a.d_out == nullptr && a.d_next != nullptr : a.d_out != nullptr);
  require((a.d_w_next != nullptr) == (a.d_next != nullptr));
  const NormShape s = norm_forward_shape(a.rows, a.channels, a.groups);
  require((int64_t)s.lanes * s.items >= s.chunks && s.rowblocks >= 1);
  return ENGRAM_OK;
}

int launch_residual_norm_backward(const engram_norm_args &a) {
  const bool sums = a.d_grad_w_post || a.d_grad_scale || a.d_grad_w_next;
  require(a.rows > 0 || sums);
  const NormShape s = norm_backward_shape(a.rows, a.channels, a.groups);
  require((int64_t)s.lanes * s.items >= s.chunks && s.items <= kNormBackwardItems);
  require(!sums || a.rows == 0 ||
          a.workspace_bytes >= (size_t)norm_partial_floats(s) * sizeof(float));
  return ENGRAM_OK;
}

int launch_act_encode(const void *d_x, int64_t rows, int64_t channels, int8_t *d_codes,
                      float *d_scales, void *) {
  require(d_x && d_codes && d_scales && rows > 0 && channels % 8 == 0);
  return ENGRAM_OK;
}

int launch_act_decode(const int8_t *d_codes, const float *d_scales, int64_t rows,
                      int64_t channels, void *d_x, void *) {
  require(d_x && d_codes && d_scales && rows > 0 && channels % 8 == 0);
  return ENGRAM_OK;
}

int launch_conv_backward(const ConvBackwardCall &c, void *) {
  require(c.grad_x || c.grad_halo || c.grad_weight || c.grad_bias);
  require(c.code_width > 0 && c.channels % c.code_width == 0);
  if (c.batch > 0 && c.seq > 0) {
    require(c.grad_out && c.weight);
    require(!c.grad_weight || c.x || c.codes);
    require(!(c.grad_weight || c.grad_bias) || c.partials);
    const ConvBackwardShape s =
        conv_backward_shape(c.batch, c.seq, c.halo_len, c.channels, c.K, c.dilation);
    require(s.halo_slices * s.slice >= c.halo_len &&
            (s.slices - s.halo_slices) * s.slice >= c.seq);
  }
  return ENGRAM_OK;
}

int launch_conv_step(const ConvStepCall &c, void *) {
  require(c.batch > 0 && c.tokens > 0 && c.x && c.positions && c.weight);
  require(c.ring_rows >= (int64_t)(c.K - 1) * c.dilation && (c.ring || c.ring_count == 0));
  return ENGRAM_OK;
}

int launch_embed(const int64_t *d_tokens, int64_t n, const void *d_table, int64_t table_rows,
                 int64_t, float, int32_t, void *d_out, int64_t *, void *) {
  require(n > 0 && d_tokens && d_out && (d_table || table_rows == 0));
  return ENGRAM_OK;
}

int launch_embed_grad(const EmbedGradCall &c, const Plan &p, void *d_workspace, void *) {
  require(c.n >= 0 && (c.grad_table || c.table_rows == 0));
  require(c.n == 0 || (c.tokens && c.grads && d_workspace && c.partials && p.total > 0));
  return ENGRAM_OK;
}

}  // namespace engram
