// engram_act8.hip -- 8-bit activation checkpoints, for gfx950.
//
// The format is stated with engram_act_encode in include/engram_layer.h: int8
// codes with one fp32 scale per 128 channels, round(x * (127 / m)) with m the
// block's largest magnitude.  A code is off by at most half a step, m / 254.
// Blocks of 128 keep the scales at 3% of the codes and a block inside 16
// lanes of 8 channels, so its maximum is four DPP steps.
//
// Bound by HBM: the encoder reads 2 bytes and writes 1 a value, the decoder
// the reverse, with about 10 operations between.  A lane moves one chunk of 8
// channels of each of kActUnroll blocks, all loads before the first use.
// Measured on MI355X: 537M values encoded in 281 us (5.8 TB/s), 33.7M decoded in
// 17.5 us (5.8 TB/s).  1, 2 and 8 blocks a lane were no faster (331, 291 and 288
// us); non-temporal code stores gained 1% there but cost a decode that follows
// soon 20%.
#include "engram_layer_dev.h"

namespace engram {
namespace {

constexpr int kActThreads = 256;
constexpr int kActUnroll = 4;

// Slots of 16 lanes walk the 8-bit blocks of [rows, blocks per row] in order,
// kActUnroll of them a thread, a grid's width apart.
struct ActArgs {
  const u32x4 *x;
  u32x4 *out;
  u32x2 *codes;
  float *scales;
  int64_t blocks;      // all rows' 8-bit blocks
  uint32_t per_row;    // 8-bit blocks of a row
  int64_t row_chunks;  // chunks of 8 channels of a row
};

struct ActPlace {
  int64_t block, chunk;
  bool ok;
};

__device__ __forceinline__ ActPlace act_place(const ActArgs &a, int64_t block) {
  ActPlace p;
  const bool in = block < a.blocks;
  p.block = in ? block : 0;
  const int64_t row = a.blocks <= 0xffffffffll ? (uint32_t)p.block / a.per_row
                                               : p.block / (int64_t)a.per_row;
  const int64_t j = (p.block - row * a.per_row) * 16 + (threadIdx.x & 15);
  p.ok = in && j < a.row_chunks;
  p.chunk = row * a.row_chunks + (p.ok ? j : 0);
  return p;
}

constexpr int kSlots = kActThreads / 16;

__global__ __launch_bounds__(kActThreads) void act_encode_kernel(const ActArgs a) {
  const int64_t first = (int64_t)blockIdx.x * (kSlots * kActUnroll) + threadIdx.x / 16;
  ActPlace p[kActUnroll];
  u32x4 v[kActUnroll];
#pragma unroll
  for (int k = 0; k < kActUnroll; ++k) {
    p[k] = act_place(a, first + k * kSlots);
    v[k] = a.x[p[k].chunk];
  }
#pragma unroll
  for (int k = 0; k < kActUnroll; ++k) {
    float f[8];
    unpack_bf16x8(v[k], f);
    const CodeScale cs = code_scale(lanes_max<16>(p[k].ok ? max_magnitude(f) : 0u));
    if (!p[k].ok) continue;
    a.codes[p[k].chunk] = code_bytes8(f, cs.inv);
    if ((threadIdx.x & 15) == 0) a.scales[p[k].block] = cs.scale;
  }
}

__global__ __launch_bounds__(kActThreads) void act_decode_kernel(const ActArgs a) {
  const int64_t first = (int64_t)blockIdx.x * (kSlots * kActUnroll) + threadIdx.x / 16;
  ActPlace p[kActUnroll];
  u32x2 v[kActUnroll];
  float s[kActUnroll];
#pragma unroll
  for (int k = 0; k < kActUnroll; ++k) {
    p[k] = act_place(a, first + k * kSlots);
    v[k] = a.codes[p[k].chunk];
    s[k] = a.scales[p[k].block];
  }
#pragma unroll
  for (int k = 0; k < kActUnroll; ++k) {
    if (!p[k].ok) continue;
    float f[8];
    code_values(v[k].x, s[k], f);
    code_values(v[k].y, s[k], f + 4);
    a.out[p[k].chunk] = pack_bf16x8(f);
  }
}

ActArgs act_args(int64_t rows, int64_t channels) {
  ActArgs a = {};
  a.row_chunks = channels / 8;
  a.per_row = (uint32_t)ceil_div(channels, kActBlock);
  a.blocks = rows * a.per_row;
  return a;
}

}  // namespace
}  // namespace engram

int engram::launch_act_encode(const void *d_x, int64_t rows, int64_t channels, int8_t *d_codes,
                              float *d_scales, void *stream) {
  ActArgs a = act_args(rows, channels);
  a.x = static_cast<const u32x4 *>(d_x);
  a.codes = reinterpret_cast<u32x2 *>(d_codes);
  a.scales = d_scales;
  const int64_t blocks = ceil_div(a.blocks, kSlots * kActUnroll);
  if (!grid_fits(blocks, kActThreads)) return ENGRAM_EINVAL;
  hipLaunchKernelGGL(act_encode_kernel, dim3((unsigned)blocks), dim3(kActThreads), 0,
                     as_stream(stream), a);
  return launch_status();
}

int engram::launch_act_decode(const int8_t *d_codes, const float *d_scales, int64_t rows,
                              int64_t channels, void *d_x, void *stream) {
  ActArgs a = act_args(rows, channels);
  a.out = static_cast<u32x4 *>(d_x);
  a.codes = reinterpret_cast<u32x2 *>(const_cast<int8_t *>(d_codes));
  a.scales = const_cast<float *>(d_scales);
  const int64_t blocks = ceil_div(a.blocks, kSlots * kActUnroll);
  if (!grid_fits(blocks, kActThreads)) return ENGRAM_EINVAL;
  hipLaunchKernelGGL(act_decode_kernel, dim3((unsigned)blocks), dim3(kActThreads), 0,
                     as_stream(stream), a);
  return launch_status();
}
