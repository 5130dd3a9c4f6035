// hip_runtime.h -- a stand-in for HIP's header with which a kernel source of
// this library builds as ordinary C++ and runs on a CPU, a block at a time, for
// the tests that need an order of the wavefronts which a GPU gives only now and
// then (and for results that a GPU is not made to produce on purpose).
//
// Every thread is a fiber.  A wavefront's cross-lane operations wait for its 64
// lanes, a barrier for the block's threads.  The wavefronts take turns in a fixed
// order, each running as far as it can: the one that completes a barrier runs on
// to the next before any other has left the first.  That is the worst order for
// LDS that is written again too early.
#pragma once

#include <math.h>
#include <stdint.h>
#include <stdio.h>
#include <stdlib.h>
#include <string.h>
#include <ucontext.h>

#include <functional>
#include <memory>
#include <vector>

#define __global__
#define __device__
#define __forceinline__ inline
#define __launch_bounds__(...)
#define __shared__ static

struct dim3 {
  unsigned x, y, z;
  dim3(unsigned x_ = 1, unsigned y_ = 1, unsigned z_ = 1) : x(x_), y(y_), z(z_) {}
};
struct uint2 {
  uint32_t x, y;
};
typedef void *hipStream_t;
typedef int hipError_t;
constexpr hipError_t hipSuccess = 0;
inline hipError_t hipGetLastError() { return hipSuccess; }

namespace cpu_wave {

constexpr int kLanes = 64;
constexpr size_t kStack = 64 << 10;

struct Wave {
  uint64_t arrived = 0;
  uint32_t value[2][kLanes];
};
struct Fiber {
  ucontext_t context;
  std::unique_ptr<char[]> stack;
  dim3 thread;
  Wave *wave;
  uint64_t wave_round = 0, block_round = 0;
  const uint64_t *waits_for = nullptr;  // runs again once *waits_for >= target
  uint64_t target = 0;
  bool done = false;
};

inline ucontext_t scheduler;
inline Fiber *self = nullptr;
inline dim3 block_index, block_size;
inline uint64_t block_arrived;
inline const std::function<void()> *body;
inline bool descending = false;  // the order in which the wavefronts take turns

inline void wait_until(const uint64_t *counter, uint64_t target) {
  self->waits_for = counter;
  self->target = target;
  swapcontext(&self->context, &scheduler);
}
inline void run_body() {
  (*body)();
  self->done = true;
  swapcontext(&self->context, &scheduler);
}
// Every lane's value; all 64 lanes of the wavefront call it.
inline const uint32_t *share(uint32_t v) {
  Wave &w = *self->wave;
  uint32_t *values = w.value[self->wave_round++ & 1];
  values[self->thread.x % kLanes] = v;
  ++w.arrived;
  wait_until(&w.arrived, self->wave_round * kLanes);
  return values;
}
inline unsigned lane() { return self->thread.x % kLanes; }
inline void barrier() {
  ++self->block_round;
  ++block_arrived;
  wait_until(&block_arrived, self->block_round * block_size.x);
}

inline void run_block(std::vector<Fiber> &fibers, std::vector<Wave> &waves) {
  block_arrived = 0;
  for (Wave &w : waves) w = Wave();
  for (unsigned t = 0; t < fibers.size(); ++t) {
    Fiber &f = fibers[t];
    std::unique_ptr<char[]> stack = std::move(f.stack);
    f = Fiber();
    f.stack = stack ? std::move(stack) : std::unique_ptr<char[]>(new char[kStack]);
    f.thread = dim3(t, 0, 0);
    f.wave = &waves[t / kLanes];
    getcontext(&f.context);
    f.context.uc_stack.ss_sp = f.stack.get();
    f.context.uc_stack.ss_size = kStack;
    f.context.uc_link = nullptr;
    makecontext(&f.context, run_body, 0);
  }
  size_t left = fibers.size();
  while (left > 0) {
    bool any = false;
    for (size_t i = 0; i < waves.size(); ++i) {
      const size_t w = descending ? waves.size() - 1 - i : i;
      for (bool progress = true; progress;) {
        progress = false;
        for (size_t t = w * kLanes; t < (w + 1) * kLanes && t < fibers.size(); ++t) {
          Fiber &f = fibers[t];
          if (f.done || (f.waits_for != nullptr && *f.waits_for < f.target)) continue;
          self = &f;
          swapcontext(&scheduler, &f.context);
          left -= f.done;
          progress = any = true;
        }
      }
    }
    if (!any) {
      fprintf(stderr, "cpu_wave: every thread waits\n");
      abort();
    }
  }
}

inline void launch(dim3 grid, dim3 block, const std::function<void()> &kernel) {
  block_size = block;
  body = &kernel;
  std::vector<Fiber> fibers(block.x);
  std::vector<Wave> waves((block.x + kLanes - 1) / kLanes);
  for (unsigned b = 0; b < grid.x; ++b) {
    block_index = dim3(b, 0, 0);
    run_block(fibers, waves);
  }
}

}  // namespace cpu_wave

#define threadIdx (::cpu_wave::self->thread)
#define blockIdx (::cpu_wave::block_index)
#define hipLaunchKernelGGL(kernel, grid, block, lds, stream, ...) \
  ((void)(stream), ::cpu_wave::launch(grid, block, [&]() { (kernel)(__VA_ARGS__); }))

inline void __syncthreads() { cpu_wave::barrier(); }
inline uint64_t __ballot(bool v) {
  const uint32_t *values = cpu_wave::share(v);
  uint64_t mask = 0;
  for (int l = 0; l < cpu_wave::kLanes; ++l) mask |= (uint64_t)(values[l] != 0) << l;
  return mask;
}
inline int __popcll(uint64_t v) { return __builtin_popcountll(v); }

// The cross-lane moves that the kernels use: a permutation of each four lanes
// (control values up to 0xff), the mirror images within 16 and within 8 lanes.
inline int cpu_wave_dpp(int, int v, int control, int, int, bool) {
  const uint32_t *values = cpu_wave::share((uint32_t)v);
  const unsigned l = cpu_wave::lane();
  if (control <= 0xff) return (int)values[(l & ~3u) | ((control >> (2 * (l & 3))) & 3)];
  if (control == 0x140) return (int)values[l ^ 15];
  if (control == 0x141) return (int)values[l ^ 7];
  abort();
}
struct cpu_wave_pair {
  uint32_t v[2];
  uint32_t operator[](int i) const { return v[i]; }
};
// Rows (halves) exchanged between two copies of one register: what each lane then
// holds is its pair of rows' (the two halves') values.
inline cpu_wave_pair cpu_wave_swap(uint32_t v, unsigned width) {
  const uint32_t *values = cpu_wave::share(v);
  const unsigned l = cpu_wave::lane();
  return cpu_wave_pair{{values[l & ~width], values[l | width]}};
}
#define __builtin_amdgcn_update_dpp(...) cpu_wave_dpp(__VA_ARGS__)
#define __builtin_amdgcn_permlane16_swap(a, b, x, y) cpu_wave_swap(a, 16)
#define __builtin_amdgcn_permlane32_swap(a, b, x, y) cpu_wave_swap(a, 32)

inline uint32_t __float_as_uint(float f) { return __builtin_bit_cast(uint32_t, f); }
inline float __uint_as_float(uint32_t u) { return __builtin_bit_cast(float, u); }
inline float __expf(float x) { return expf(x); }
inline float __fmul_rn(float a, float b) { return a * b; }
inline float __fdiv_rn(float a, float b) { return a / b; }
inline unsigned long long atomicAdd(unsigned long long *p, unsigned long long v) {
  const unsigned long long old = *p;
  *p = old + v;
  return old;
}
template <class T>
inline T min(T a, T b) {
  return b < a ? b : a;
}
template <class T>
inline T max(T a, T b) {
  return a < b ? b : a;
}

// float to bf16 (to nearest, ties to even), which the compiler calls for.
extern "C" inline __attribute__((used)) __bf16 __truncsfbf2(float f) {
  uint32_t u = __builtin_bit_cast(uint32_t, f);
  u = f != f ? (u >> 16) | 0x40u : (u + 0x7fffu + ((u >> 16) & 1u)) >> 16;
  return __builtin_bit_cast(__bf16, (uint16_t)u);
}
