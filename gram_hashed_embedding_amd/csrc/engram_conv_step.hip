// engram_conv_step.hip -- the PLE convolution for tokens that arrive one at a
// time, from a ring of each sequence's latest inputs, for gfx950.
//
// What is computed is stated with engram_ple_conv_step in include/
// engram_layer.h; it is engram_ple_conv (the NeMo AutoModel v0.7 API page
// "qwen3_8_flash_next.engram", _causal_short_conv) with the history kept
// between calls, the taps summed in the same order.
//
// Bound by latency: a serving batch moves a few megabytes at most (6 rows of
// a sequence: x, three taps, the ring's new row, out).  So one launch, a lane
// to 8 channels of a sequence (16-byte accesses), and the taps' loads go out
// together: 2.9 us for 4 sequences of 1024 channels, 6.1 us for 256 of 8192
// (25 MB, 4.1 TB/s) on MI355X.  A lane reads and writes only its own channels of the ring, so
// the oldest row may be the one that this call overwrites.
#include "engram_layer_dev.h"

namespace engram {
namespace {

constexpr int kStepThreads = 256;

struct StepArgs {
  const u32x4 *x;
  u32x4 *ring;
  int64_t ring_count, ring_rows;
  const int64_t *ring_ids, *positions;
  const uint16_t *w;
  const u32x4 *bias;
  int64_t batch, tokens, chunks;
  int K, dil;
  u32x4 *out;
  int64_t *err;
};

template <int K>  // 0: any
__global__ __launch_bounds__(kStepThreads) void conv_step_kernel(const StepArgs a) {
  const int taps = K > 0 ? K : a.K;
  const int64_t i = (int64_t)blockIdx.x * kStepThreads + threadIdx.x;
  if (i >= a.batch * a.chunks) return;
  const int64_t b = i / a.chunks, ch = i - b * a.chunks;
  const int64_t id = a.ring_ids != nullptr ? a.ring_ids[b] : b, pos = a.positions[b];
  // (a position whose tokens would pass the largest number is as invalid)
  const bool ok =
      id >= 0 && id < a.ring_count && pos >= 0 && pos <= INT64_MAX - a.tokens;
  if (!ok) {
    if (ch == 0 && id != -1) count_errors(1, a.err);
    if (a.out != nullptr)
      for (int64_t n = 0; n < a.tokens; ++n)
        a.out[(b * a.tokens + n) * a.chunks + ch] = u32x4{0u, 0u, 0u, 0u};
    return;
  }
  u32x4 *ring = a.ring + id * a.ring_rows * a.chunks + ch;
  float bias[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
  if (a.bias != nullptr) unpack_bf16x8(a.bias[ch], bias);
  const uint16_t *w = a.w + ch * 8 * taps;
  for (int64_t n = 0; n < a.tokens; ++n) {
    const int64_t p = pos + n;
    const int64_t slot = p % a.ring_rows;
    const u32x4 x = a.x[(b * a.tokens + n) * a.chunks + ch];
    if (a.out != nullptr) {
      float acc[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) acc[e] = bias[e];
      if (K > 0) {
        u32x4 v[K > 0 ? K : 1];
#pragma unroll
        for (int k = 0; k < K; ++k) {
          const int64_t back = (int64_t)(K - 1 - k) * a.dil;
          int64_t s = slot - back;  // back <= ring_rows, so one wrap
          if (s < 0) s += a.ring_rows;
          v[k] = u32x4{0u, 0u, 0u, 0u};
          if (back == 0)
            v[k] = x;
          else if (p >= back)
            v[k] = ring[s * a.chunks];
        }
#pragma unroll
        for (int k = 0; k < K; ++k) {
          float f[8];
          unpack_bf16x8(v[k], f);
#pragma unroll
          for (int e = 0; e < 8; ++e) acc[e] += bf16_lo(w[e * K + k]) * f[e];
        }
      } else {
        for (int k = 0; k < taps; ++k) {
          const int64_t back = (int64_t)(taps - 1 - k) * a.dil;
          int64_t s = slot - back;
          if (s < 0) s += a.ring_rows;
          u32x4 v = {0u, 0u, 0u, 0u};
          if (back == 0)
            v = x;
          else if (p >= back)
            v = ring[s * a.chunks];
          float f[8];
          unpack_bf16x8(v, f);
          for (int e = 0; e < 8; ++e) acc[e] += bf16_lo(w[e * taps + k]) * f[e];
        }
      }
      a.out[(b * a.tokens + n) * a.chunks + ch] = pack_bf16x8(acc);
    }
    ring[slot * a.chunks] = x;
  }
}

}  // namespace
}  // namespace engram

int engram::launch_conv_step(const ConvStepCall &c, void *stream) {
  StepArgs a = {};
  a.x = static_cast<const u32x4 *>(c.x);
  a.ring = static_cast<u32x4 *>(c.ring);
  a.ring_count = c.ring_count;
  a.ring_rows = c.ring_rows;
  a.ring_ids = c.ring_ids;
  a.positions = c.positions;
  a.w = static_cast<const uint16_t *>(c.weight);
  a.bias = static_cast<const u32x4 *>(c.bias);
  a.batch = c.batch;
  a.tokens = c.tokens;
  a.chunks = c.channels / 8;
  a.K = c.K;
  a.dil = c.dilation;
  a.out = static_cast<u32x4 *>(c.out);
  a.err = c.err;
  const int64_t blocks = ceil_div(a.batch * a.chunks, kStepThreads);
  if (!grid_fits(blocks, kStepThreads)) return ENGRAM_EINVAL;
  const dim3 grid((unsigned)blocks), block(kStepThreads);
  if (c.K == 4)
    hipLaunchKernelGGL(conv_step_kernel<4>, grid, block, 0, as_stream(stream), a);
  else
    hipLaunchKernelGGL(conv_step_kernel<0>, grid, block, 0, as_stream(stream), a);
  return launch_status();
}
