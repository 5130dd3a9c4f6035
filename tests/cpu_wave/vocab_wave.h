// vocab_wave.h -- what the vocabulary operators' kernels use beyond hip_runtime.h's
// stand-ins, in the same manner: every lane of a wavefront calls a cross-lane operation.
#pragma once

#include <hip/hip_runtime.h>

inline long long __double_as_longlong(double v) { return __builtin_bit_cast(long long, v); }
inline double __longlong_as_double(long long v) { return __builtin_bit_cast(double, v); }
inline uint32_t __umulhi(uint32_t a, uint32_t b) { return (uint32_t)((uint64_t)a * b >> 32); }
inline int __ffsll(unsigned long long v) { return __builtin_ffsll((long long)v); }
inline float __double2float_rd(double v) {
  const float f = (float)v;
  return (double)f > v ? nextafterf(f, -HUGE_VALF) : f;
}
inline int atomicAdd(int *p, int v) {
  const int old = *p;
  *p = old + v;
  return old;
}
inline uint32_t atomicOr(uint32_t *p, uint32_t v) {
  const uint32_t old = *p;
  *p = old | v;
  return old;
}

// Any value's words, from the lane that `from` gives for this one.
template <class T, class FROM>
inline T cpu_wave_get(T v, FROM from) {
  static_assert(sizeof(T) % 4 == 0, "words");
  uint32_t words[sizeof(T) / 4];
  memcpy(words, &v, sizeof(T));
  for (uint32_t &w : words) w = cpu_wave::share(w)[from(cpu_wave::lane())];
  memcpy(&v, words, sizeof(T));
  return v;
}
template <class T>
inline T __shfl(T v, int lane) {
  return cpu_wave_get(v, [&](unsigned) { return (unsigned)lane % 64u; });
}
template <class T>
inline T __shfl_xor(T v, int mask) {
  return cpu_wave_get(v, [&](unsigned l) { return l ^ (unsigned)mask; });
}

#define __builtin_amdgcn_readfirstlane(v) ((int)cpu_wave::share((uint32_t)(v))[0])
#define __builtin_amdgcn_exp2f(x) exp2f(x)
#define __builtin_amdgcn_logf(x) log2f(x)
#define __builtin_amdgcn_fence(order, scope) ((void)0)
#define __builtin_amdgcn_wave_barrier() ((void)cpu_wave::share(0u))
