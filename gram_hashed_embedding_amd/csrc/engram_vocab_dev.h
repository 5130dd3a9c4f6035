// engram_vocab_dev.h -- device helpers for rows of logits: chunks of eight
// values at any alignment, the running maximum and sum of a softmax, and its
// joins over lanes, segments and rows.
//
// A lane keeps the largest logit it has seen and the sum of
//     exp((z - max) / temperature) = 2^((z - max) c),  c = log2(e) / temperature
// (a subtraction, a product and a v_exp_f32 a value).  One fma, z c - (max c), would
// do, but max c overflows for a row whose logits are all a mask's lowest value;
// the difference is exact there.  Sums leave the lane in fp64, where the
// logarithm is taken too.
#pragma once

#include <math.h>

#include "engram_layer_dev.h"
#include "engram_vocab_host.h"

namespace engram {

constexpr float kNegInf = -__builtin_inff();

__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }

// max(a, b, c) in one instruction, v_maximum3_f32; NaN if any is one.  (fmaxf quiets its
// operands first.  The compiler has to know the instruction: it puts wait states between a
// vector instruction and one that moves its result across lanes.)
__device__ __forceinline__ float max3(float a, float b, float c) {
  return __builtin_elementwise_maximum(__builtin_elementwise_maximum(a, b), c);
}

// Eight values at any address of their type: the loads and stores are 16 bytes wide
// (global memory takes them at any alignment).  ONCE: not read again, or not soon, so that
// the caches keep what is.
typedef uint32_t u32x4_any __attribute__((ext_vector_type(4), aligned(2)));
typedef float f32x4_any __attribute__((ext_vector_type(4), aligned(4)));
template <class T>
struct Chunk;
template <>
struct Chunk<uint16_t> {
  u32x4 r;
  template <bool ONCE = false>
  __device__ __forceinline__ void load(const uint16_t *p) {
    const u32x4_any *q = reinterpret_cast<const u32x4_any *>(p);
    r = ONCE ? __builtin_nontemporal_load(q) : *q;
  }
  __device__ __forceinline__ void values(float (&z)[8]) const { unpack_bf16x8(r, z); }
  __device__ static __forceinline__ float one(uint16_t v) { return bf16_lo(v); }
  __device__ static __forceinline__ void store_one(uint16_t *p, float v) {
    *p = (uint16_t)pack_bf16(v, 0.0f);
  }
  __device__ static __forceinline__ void store_once(uint16_t *p, const float (&v)[8]) {
    const u32x4 w = pack_bf16x8(v);
    __builtin_nontemporal_store(w, reinterpret_cast<u32x4_any *>(p));
  }
};
template <>
struct Chunk<float> {
  f32x4 a, b;
  template <bool ONCE = false>
  __device__ __forceinline__ void load(const float *p) {
    const f32x4_any *q = reinterpret_cast<const f32x4_any *>(p);
    a = ONCE ? __builtin_nontemporal_load(q) : *q;
    b = ONCE ? __builtin_nontemporal_load(q + 1) : q[1];
  }
  __device__ __forceinline__ void values(float (&z)[8]) const {
    z[0] = a.x; z[1] = a.y; z[2] = a.z; z[3] = a.w;
    z[4] = b.x; z[5] = b.y; z[6] = b.z; z[7] = b.w;
  }
  __device__ static __forceinline__ float one(float v) { return v; }
  __device__ static __forceinline__ void store_one(float *p, float v) { *p = v; }
  __device__ static __forceinline__ void store_once(float *p, const float (&v)[8]) {
    f32x4_any *q = reinterpret_cast<f32x4_any *>(p);
    __builtin_nontemporal_store(f32x4{v[0], v[1], v[2], v[3]}, q);
    __builtin_nontemporal_store(f32x4{v[4], v[5], v[6], v[7]}, q + 1);
  }
};

// Values before the first at a whole cache line, of `n` that start at p: a block's chunks
// start behind them.  (At odd multiples of 2 bytes a 16-byte access takes about a fifth more
// time, at other places than whole lines about a twentieth.)
constexpr int kLine = 128;
template <class T>
__device__ __forceinline__ int lead_of(const T *p, int64_t n) {
  const int lead = (int)(-reinterpret_cast<uintptr_t>(p) % kLine / sizeof(T));
  return lead < n ? lead : (int)n;
}

__device__ __forceinline__ float max8(float m, const float (&z)[8]) {
  return max3(max3(max3(m, z[0], z[1]), z[2], z[3]), max3(z[4], z[5], z[6]), z[7]);
}

// ---------------------------------------------------- running softmax sum --
// The point that exponents are taken from: the maximum, or 0 while there is none,
// so that no difference of infinities arises.
__device__ __forceinline__ float ref_of(float max) { return max == kNegInf ? 0.0f : max; }

// log2(e) / temperature, in two parts: rounded to one, it would be off by up to 2^-25 of
// it, which in the exponent of a term far below the maximum is more than fp32's rounding.
// The second part is above 0, so that -inf times it is -inf as well.
struct Scale {
  float hi, lo;
};
inline Scale scale_of(double temperature) {
  const double c = 1.4426950408889634 / temperature;
  float hi = (float)c;
  while ((double)hi >= c) hi = nextafterf(hi, 0.0f);
  return {hi, (float)(c - (double)hi)};
}
__device__ __forceinline__ float exp_scaled(float d, Scale c) {
  return exp2_fast(__builtin_fmaf(d, c.lo, d * c.hi));
}

struct Running {
  float max = kNegInf, sum = 0.0f;
  // raises the maximum to at least m, and gives the point that exponents are taken from
  __device__ __forceinline__ float raise(float m, Scale c) {
    const float ref = ref_of(m);
    sum *= exp_scaled(max - ref, c);  // (2^-inf while there was none)
    max = m;
    return ref;
  }
  __device__ __forceinline__ void add(const float (&z)[8], float ref, Scale c) {
    float e[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) e[i] = exp_scaled(z[i] - ref, c);
    sum += ((e[0] + e[1]) + (e[2] + e[3])) + ((e[4] + e[5]) + (e[6] + e[7]));
  }
};

// exp in fp64 by its series around 0 (|r| <= ln(2) / 2: the 11th power's term is
// 2e-13), in few registers.
__device__ __forceinline__ double exp64(double x) {
  x = x < -800.0 ? -800.0 : x > 800.0 ? 800.0 : x;  // (0 and +inf; a NaN stays one)
  const double n = rint(x * 1.44269504088896340736);
  const double r = fma(-n, 0.693147180559945309417, x);
  double p = 1.0 / 3628800.0;
  p = fma(p, r, 1.0 / 362880.0);
  p = fma(p, r, 1.0 / 40320.0);
  p = fma(p, r, 1.0 / 5040.0);
  p = fma(p, r, 1.0 / 720.0);
  p = fma(p, r, 1.0 / 120.0);
  p = fma(p, r, 1.0 / 24.0);
  p = fma(p, r, 1.0 / 6.0);
  p = fma(p, r, 0.5);
  p = fma(p, r, 1.0);
  p = fma(p, r, 1.0);
  return ldexp(p, (int)n);
}

// log in fp64: of x = 2^e m, m in [1/2, 1), from y = log(m) in fp32 (an error of about 1e-7)
// and one step of Newton's method, log(m) = y + log(1 + d), d = m exp(-y) - 1, of which d^3 is
// beyond fp64.
__device__ __forceinline__ double log64(double x) {
  if (!(x > 0.0) || __builtin_isinf(x))
    return x == 0.0 ? -__builtin_inf() : x > 0.0 ? x : __builtin_nan("");
  int e;
  const double m = frexp(x, &e);
  const double y = (double)(__builtin_amdgcn_logf((float)m) * 0.693147182464599609375f);
  const double d = fma(m, exp64(-y), -1.0);
  return fma((double)e, 0.693147180559945309417, y + (d - 0.5 * d * d));
}

// ----------------------------------------------- reductions over wavefronts --
template <int LANES>
__device__ __forceinline__ float lanes_max_of(float v) {
  return __uint_as_float(lanes_reduce<LANES>(__float_as_uint(v), [](uint32_t a, uint32_t b) {
    return __float_as_uint(__builtin_fmaxf(__uint_as_float(a), __uint_as_float(b)));
  }));
}
__device__ __forceinline__ float wave_max(float v) { return lanes_max_of<kWave>(v); }
__device__ __forceinline__ double double_of(uint32_t lo, uint32_t hi) {
  return __longlong_as_double((long long)((uint64_t)hi << 32 | lo));
}
__device__ __forceinline__ uint32_t low_of(double v) {
  return (uint32_t)__double_as_longlong(v);
}
__device__ __forceinline__ uint32_t high_of(double v) {
  return (uint32_t)((uint64_t)__double_as_longlong(v) >> 32);
}
template <int CTRL>
__device__ __forceinline__ double dpp_move(double v) {
  return double_of(dpp_move<CTRL>(low_of(v)), dpp_move<CTRL>(high_of(v)));
}
// A commutative op over aligned groups of LANES lanes, left in each of them.
template <int LANES, class OP>
__device__ __forceinline__ double lanes_reduce(double v, OP op) {
  if (LANES >= 2) v = op(v, dpp_move<kDppXor1>(v));
  if (LANES >= 4) v = op(v, dpp_move<kDppXor2>(v));
  if (LANES >= 8) v = op(v, dpp_move<kDppHalfMirror>(v));
  if (LANES >= 16) v = op(v, dpp_move<kDppMirror>(v));
  if (LANES >= 32) {
    const uint32_t l = low_of(v), h = high_of(v);
    const auto x = __builtin_amdgcn_permlane16_swap(l, l, false, false);
    const auto y = __builtin_amdgcn_permlane16_swap(h, h, false, false);
    v = op(double_of(x[0], y[0]), double_of(x[1], y[1]));
  }
  if (LANES >= 64) {
    const uint32_t l = low_of(v), h = high_of(v);
    const auto x = __builtin_amdgcn_permlane32_swap(l, l, false, false);
    const auto y = __builtin_amdgcn_permlane32_swap(h, h, false, false);
    v = op(double_of(x[0], y[0]), double_of(x[1], y[1]));
  }
  return v;
}
__device__ __forceinline__ double wave_sum(double v) {
  return lanes_reduce<kWave>(v, [](double a, double b) { return a + b; });
}
__device__ __forceinline__ double wave_max(double v) {
  return lanes_reduce<kWave>(v, [](double a, double b) { return fmax(a, b); });
}

// A value that every lane has alike, in scalar registers.
__device__ __forceinline__ uint32_t uniform(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_readfirstlane((int)v);
}
__device__ __forceinline__ float uniform(float v) {
  return __uint_as_float(uniform(__float_as_uint(v)));
}
__device__ __forceinline__ double uniform(double v) {
  return double_of(uniform(low_of(v)), uniform(high_of(v)));
}

// Every lane's stores to LDS before, for the other lanes of its wavefront after.
__device__ __forceinline__ void wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

// A sum of exponentials with its maximum: of exp((z - max) / temperature).
struct RowSum {
  float max;
  double sum;
};
// s, taken from max, as taken from ref.
__device__ __forceinline__ double moved(double s, float max, float ref, Scale c) {
  return max == kNegInf ? s : s * (double)exp_scaled(max - ref, c);
}
// The lanes' running sums over a block of WAVES wavefronts, in a fixed order: one barrier, after
// which every wavefront joins the others' for itself.
template <int WAVES>
struct JoinLds {
  float max[WAVES];
  double sum[WAVES];
};
// (RUN: a Running, or a RowSum of several.)
template <int WAVES, class RUN>
__device__ __forceinline__ RowSum block_join(const RUN &run, Scale c, JoinLds<WAVES> &l) {
  const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
  const float own = wave_max(run.max);
  const double part = wave_sum(moved(run.sum, run.max, ref_of(own), c));
  if (lane == 0) {
    l.max[wave] = own;
    l.sum[wave] = part;
  }
  __syncthreads();
  const float other = l.max[lane % WAVES];
  const float m = uniform(lanes_max_of<WAVES>(other));
  const double s = moved(l.sum[lane % WAVES], other, ref_of(m), c);
  return {m, uniform(lanes_reduce<WAVES>(s, [](double a, double b) { return a + b; }))};
}
// The sums of a row's segments, joined by a wavefront.
__device__ __forceinline__ RowSum wave_join(const ScanPart *parts, int64_t n, Scale c) {
  float m = kNegInf;
  for (int64_t i = threadIdx.x % kWave; i < n; i += kWave) m = max3(m, parts[i].max, kNegInf);
  m = wave_max(m);
  double s = 0.0;
  for (int64_t i = threadIdx.x % kWave; i < n; i += kWave)
    s += moved(parts[i].sum, parts[i].max, ref_of(m), c);
  return {m, wave_sum(s)};
}

// -------------------------------------------------------- reading a segment --
// The values [lo, hi) of a row by a block, U chunks a lane at a time: use(at, z) is
// called by every lane with the chunks that start at at + 8 * (u * THREADS + lane);
// values past hi are -inf.  The next chunks' loads are on their way meanwhile; first() is
// called once, behind the first ones.
template <class T, int THREADS, int U, bool ONCE, class FIRST, class USE>
__device__ __forceinline__ void each_chunks(const T *row, int64_t lo, int64_t hi, FIRST first,
                                            USE use) {
  constexpr int kTile = 8 * THREADS, kStep = U * kTile;
  const int t = threadIdx.x;
  const int64_t last = lo + (hi - lo) / kStep * kStep - kStep;  // the last whole step
  int64_t at = lo;
  if (at <= last) {
    Chunk<T> r[U];
#pragma unroll
    for (int u = 0; u < U; ++u) r[u].template load<ONCE>(row + at + u * kTile + 8 * t);
    first();
    for (; at < last; at += kStep) {
      float z[U][8];
      Chunk<T> n[U];
#pragma unroll
      for (int u = 0; u < U; ++u) n[u].template load<ONCE>(row + at + kStep + u * kTile + 8 * t);
#pragma unroll
      for (int u = 0; u < U; ++u) r[u].values(z[u]);
      use(at, z);
#pragma unroll
      for (int u = 0; u < U; ++u) r[u] = n[u];
    }
    float z[U][8];
#pragma unroll
    for (int u = 0; u < U; ++u) r[u].values(z[u]);
    use(at, z);
    at += kStep;
  } else {
    first();
  }
  if (at < hi) {
    float z[U][8];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t i = at + u * kTile + 8 * t;
      if (i + 8 <= hi) {
        Chunk<T> r;
        r.template load<ONCE>(row + i);
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
