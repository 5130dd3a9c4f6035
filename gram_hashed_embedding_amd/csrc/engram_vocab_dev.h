// engram_vocab_dev.h -- device helpers for rows of logits: chunks of eight
// values at any alignment, the running maximum and sum of a softmax, and its
// joins over lanes, segments and rows.
//
// A lane keeps the largest logit it has seen and the sum of
//     2^(z c - M),  c = log2(e) / temperature,  M = round(max c)
// (one fma and one v_exp_f32 a value); a new maximum scales the sum by
// 2^(M_old - M_new).  Sums leave the lane in fp64.  The logarithm is taken in
// fp64 at the end: lse = max / temperature + ln(sum) + (M - max c) ln 2, so
// that M's rounding is no error.
#pragma once

#include "engram_layer_dev.h"
#include "engram_vocab_host.h"

namespace engram {

constexpr float kNegInf = -__builtin_inff();

__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }

// max(a, b, c) in one instruction (fmaxf quiets its operands first).
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("v_max3_f32 %0, %1, %2, %3" : "=v"(r) : "v"(a), "v"(b), "v"(c));
  return r;
}

// Eight values from any address of their type: the loads are 16 bytes wide
// (global memory takes them at any alignment).
template <class T>
struct Chunk;
template <>
struct Chunk<uint16_t> {
  u32x4 r;
  __device__ __forceinline__ void load(const uint16_t *p) { __builtin_memcpy(&r, p, 16); }
  __device__ __forceinline__ void values(float (&z)[8]) const { unpack_bf16x8(r, z); }
  __device__ static __forceinline__ float one(uint16_t v) { return bf16_lo(v); }
};
template <>
struct Chunk<float> {
  f32x4 a, b;
  __device__ __forceinline__ void load(const float *p) {
    __builtin_memcpy(&a, p, 16);
    __builtin_memcpy(&b, p + 4, 16);
  }
  __device__ __forceinline__ void values(float (&z)[8]) const {
    z[0] = a.x; z[1] = a.y; z[2] = a.z; z[3] = a.w;
    z[4] = b.x; z[5] = b.y; z[6] = b.z; z[7] = b.w;
  }
  __device__ static __forceinline__ float one(float v) { return v; }
};

__device__ __forceinline__ float max8(float m, const float (&z)[8]) {
  return max3(max3(max3(m, z[0], z[1]), z[2], z[3]), max3(z[4], z[5], z[6]), z[7]);
}

// ---------------------------------------------------- running softmax sum --
// The exponent's reference of a maximum: 0 while there is none, so that no
// difference of infinities arises.
__device__ __forceinline__ float ref_of(float max, float c) {
  return max == kNegInf ? 0.0f : __fmul_rn(max, c);
}

struct Running {
  float max = kNegInf, sum = 0.0f;
  // raises the maximum to at least m, and gives the exponent's reference
  __device__ __forceinline__ float raise(float m, float c) {
    const float ref = ref_of(m, c);
    sum *= exp2_fast(__fmul_rn(max, c) - ref);  // (2^-inf while there was none)
    max = m;
    return ref;
  }
  __device__ __forceinline__ void add(const float (&z)[8], float c, float ref) {
    float e[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) e[i] = exp2_fast(__builtin_fmaf(z[i], c, -ref));
    sum += ((e[0] + e[1]) + (e[2] + e[3])) + ((e[4] + e[5]) + (e[6] + e[7]));
  }
};

// A sum with its maximum, of a lane, a segment or a row.
struct RowSum {
  float max;
  double sum;
};
__device__ __forceinline__ RowSum join_sums(const RowSum &a, const RowSum &b, float c) {
  // (a NaN maximum is one of a NaN sum)
  const float m = a.max > b.max ? a.max : b.max;
  const float ref = ref_of(m, c);
  // the terms of an empty side are 0, whatever its reference
  const double sa = a.max == kNegInf ? a.sum : a.sum * (double)exp2_fast(ref_of(a.max, c) - ref);
  const double sb = b.max == kNegInf ? b.sum : b.sum * (double)exp2_fast(ref_of(b.max, c) - ref);
  return {m, sa + sb};
}

// Joined over a wavefront, left in every lane: the order is the same for every row.
__device__ __forceinline__ RowSum wave_join(RowSum v, float c) {
#pragma unroll
  for (int d = 1; d < kWave; d *= 2) {
    const RowSum o = {__shfl_xor(v.max, d), __shfl_xor(v.sum, d)};
    // the lower lane's side first in both
    v = (threadIdx.x & d) ? join_sums(o, v, c) : join_sums(v, o, c);
  }
  return v;
}

// Joined over a block; `part` holds a slot a wavefront.  Left in every lane.
template <int THREADS>
__device__ __forceinline__ RowSum block_join(RowSum v, float c, RowSum *part) {
  v = wave_join(v, c);
  if (threadIdx.x % kWave == 0) part[threadIdx.x / kWave] = v;
  __syncthreads();
  v = part[0];
#pragma unroll
  for (int w = 1; w < THREADS / kWave; ++w) v = join_sums(v, part[w], c);
  __syncthreads();
  return v;
}

// log of the sum of exp(z / temperature).
__device__ __forceinline__ double log_sum(const RowSum &v, double temperature, float c) {
  if (v.max == kNegInf && v.sum == 0.0) return -__builtin_inf();
  const double m = v.max;
  return m / temperature + log(v.sum) +
         ((double)ref_of(v.max, c) - m * (double)c) * 0.693147180559945309417;
}

template <int THREADS>
__device__ __forceinline__ double block_sum(double v, double *part) {
#pragma unroll
  for (int d = 1; d < kWave; d *= 2) v += __shfl_xor(v, d);
  if (threadIdx.x % kWave == 0) part[threadIdx.x / kWave] = v;
  __syncthreads();
  v = part[0];
#pragma unroll
  for (int w = 1; w < THREADS / kWave; ++w) v += part[w];
  __syncthreads();
  return v;
}
template <int THREADS>
__device__ __forceinline__ double block_max(double v, double *part) {
#pragma unroll
  for (int d = 1; d < kWave; d *= 2) v = fmax(v, __shfl_xor(v, d));
  if (threadIdx.x % kWave == 0) part[threadIdx.x / kWave] = v;
  __syncthreads();
  v = part[0];
#pragma unroll
  for (int w = 1; w < THREADS / kWave; ++w) v = fmax(v, part[w]);
  __syncthreads();
  return v;
}

// -------------------------------------------------------- reading a segment --
// A lane's chunks of the values [lo, hi) of a row (lo a multiple of kScanTile),
// U at a time: use(chunks' first index / 8, z) is called by every lane of the
// block, for chunks that lie before hi; values past hi are -inf.
template <class T, int U, class USE>
__device__ __forceinline__ void each_chunks(const T *row, int64_t lo, int64_t hi, USE use) {
  const int t = threadIdx.x;
  int64_t at = lo;
  for (; at + U * kScanTile <= hi; at += U * kScanTile) {
    Chunk<T> r[U];
#pragma unroll
    for (int u = 0; u < U; ++u) r[u].load(row + at + u * kScanTile + 8 * t);
    float z[U][8];
#pragma unroll
    for (int u = 0; u < U; ++u) r[u].values(z[u]);
    use(at, z);
  }
  if (at < hi) {
    float z[U][8];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t i = at + u * kScanTile + 8 * t;
      if (i + 8 <= hi) {
        Chunk<T> r;
        r.load(row + i);
        r.values(z[u]);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) z[u][e] = i + e < hi ? Chunk<T>::one(row[i + e]) : kNegInf;
      }
    }
    use(at, z);
  }
}

}  // namespace engram
