// engram_layer_dev.h -- device helpers of the layer operators: bf16 packing,
// sums and maxima over aligned groups of lanes, and the 8-bit codes.
#pragma once

#include "engram_internal.h"
#include "engram_layer_host.h"

namespace engram {

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));

// Two fp32 values as bf16 bits (to nearest, ties to even): one instruction.
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const bf16x2 p = __builtin_convertvector(f32x2{lo, hi}, bf16x2);
  return __builtin_bit_cast(uint32_t, p);
}

__device__ __forceinline__ u32x4 pack_bf16x8(const float (&f)[8]) {
  return u32x4{pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]), pack_bf16(f[4], f[5]),
               pack_bf16(f[6], f[7])};
}

// ------------------------------------------------- reductions over lanes --
// Sum and maximum over aligned groups of LANES lanes, left in each of them.
// Up to 16 lanes a step is one DPP move (lanes i^1, i^2, then the mirror
// images within 8 and within 16, which hold the other half's total by then);
// 32 and 64 swap half-rows and halves of the wavefront.  Every lane of the
// wavefront takes part.
template <int CTRL>
__device__ __forceinline__ uint32_t dpp_move(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xf, 0xf, true);
}
constexpr int kDppXor1 = 0xB1, kDppXor2 = 0x4E, kDppHalfMirror = 0x141, kDppMirror = 0x140;

template <class OP>
__device__ __forceinline__ uint32_t combine_rows16(uint32_t v, OP op) {
  const auto r = __builtin_amdgcn_permlane16_swap(v, v, false, false);
  return op(r[0], r[1]);
}
template <class OP>
__device__ __forceinline__ uint32_t combine_halves(uint32_t v, OP op) {
  const auto r = __builtin_amdgcn_permlane32_swap(v, v, false, false);
  return op(r[0], r[1]);
}

template <int LANES, class OP>
__device__ __forceinline__ uint32_t lanes_reduce(uint32_t v, OP op) {
  if (LANES >= 2) v = op(v, dpp_move<kDppXor1>(v));
  if (LANES >= 4) v = op(v, dpp_move<kDppXor2>(v));
  if (LANES >= 8) v = op(v, dpp_move<kDppHalfMirror>(v));
  if (LANES >= 16) v = op(v, dpp_move<kDppMirror>(v));
  if (LANES >= 32) v = combine_rows16(v, op);
  if (LANES >= 64) v = combine_halves(v, op);
  return v;
}

template <int LANES>
__device__ __forceinline__ float lanes_sum(float v) {
  return __uint_as_float(lanes_reduce<LANES>(__float_as_uint(v), [](uint32_t a, uint32_t b) {
    return __float_as_uint(__uint_as_float(a) + __uint_as_float(b));
  }));
}
template <int LANES>
__device__ __forceinline__ uint32_t lanes_max(uint32_t v) {
  return lanes_reduce<LANES>(v, [](uint32_t a, uint32_t b) { return a > b ? a : b; });
}

// ------------------------------------------------------------ 8-bit codes --
// A block's scale and the factor its values are multiplied by, from the bits
// of its largest magnitude (bits order as magnitudes do, infinity and NaN
// above all).  Both quotients are rounded once, so codes made by any kernel
// are the same.
struct CodeScale {
  float scale, inv;
};
__device__ __forceinline__ CodeScale code_scale(uint32_t max_bits) {
  const float m = __uint_as_float(max_bits);
  if (max_bits >= 0x7f800000u) return {__uint_as_float(0x7fc00000u), 0.0f};
  if (m < 0x1p-120f) return {0.0f, 0.0f};
  return {__fdiv_rn(m, 127.0f), __fdiv_rn(127.0f, m)};
}

// Four codes as bytes.  A product with inv = 0 is masked to zero by the
// caller's inv (0 times an infinity would be NaN, which converts to 0).
__device__ __forceinline__ uint32_t code_bytes(const float *x, float inv) {
  uint32_t w = 0;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float q = inv == 0.0f ? 0.0f : __builtin_rintf(__fmul_rn(x[e], inv));
    w |= ((uint32_t)(int)q & 0xffu) << (8 * e);
  }
  return w;
}
__device__ __forceinline__ u32x2 code_bytes8(const float (&x)[8], float inv) {
  return u32x2{code_bytes(x, inv), code_bytes(x + 4, inv)};
}

// The largest magnitude (as bits) among eight values.
__device__ __forceinline__ uint32_t max_magnitude(const float (&x)[8]) {
  uint32_t m = 0;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const uint32_t b = __float_as_uint(x[e]) & 0x7fffffffu;
    m = b > m ? b : m;
  }
  return m;
}

// Four codes' values.  A byte with its top bit flipped is the code plus 128, which
// one instruction turns into a float.  (128 is taken off before the product: 128
// scales of the largest blocks are past fp32.)
__device__ __forceinline__ void code_values(uint32_t word, float scale, float *f) {
  const uint32_t biased = word ^ 0x80808080u;
#pragma unroll
  for (int e = 0; e < 4; ++e)
    f[e] = ((float)((biased >> (8 * e)) & 0xffu) - 128.0f) * scale;
}

// ------------------------------------------------- sums of rows of partials --
// The sum over rows of the fp32 column that `column` starts, in fp64 and in a
// fixed order: a block of kJoinThreads takes COLUMNS adjacent columns, each of
// its other threads of a column every so many rows.  The sum is left in the
// first thread of each column.
constexpr int kJoinThreads = 1024;
template <int COLUMNS>
__device__ __forceinline__ double join_column(const float *column, int64_t rows, int64_t stride,
                                              bool on) {
  constexpr int kSlots = kJoinThreads / COLUMNS;
  __shared__ double part[kSlots][COLUMNS];
  const int slot = threadIdx.x / COLUMNS, c = threadIdx.x % COLUMNS;
  double s = 0.0;
  if (on) {
#pragma unroll 8
    for (int64_t r = slot; r < rows; r += kSlots) s += column[r * stride];
  }
  part[slot][c] = s;
  __syncthreads();
  s = 0.0;
  if (slot == 0)
#pragma unroll
    for (int q = 0; q < kSlots; ++q) s += part[q][c];
  __syncthreads();
  return s;
}
// Few rows leave 16 threads a column enough to do; many take 64.
constexpr int64_t kJoinFewRows = 256;
inline int join_columns(int64_t rows) { return rows <= kJoinFewRows ? 64 : 16; }

}  // namespace engram
