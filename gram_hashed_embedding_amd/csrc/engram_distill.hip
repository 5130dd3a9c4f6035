// engram_distill.hip -- distillation from a teacher's top logits: the loss of
// every row, its gradient, or both, for gfx950.  What is computed is stated
// with engram_distill in include/engram_vocab.h.
//
// The vocabulary's part is one pass over a row's logits for the sum of their
// exponentials, and one that writes the gradient.  With r (the teacher's mass
// on the ids it does not name) the first pass leaves the named ids out: s and
// the sum of all are then sums of positive terms, and s - r, which the
// gradient of the others is made of, keeps its digits when s is near r.  The
// second pass treats every id as unnamed; the few named ones are written
// after it.
#include "engram_vocab_dev.h"

namespace engram {
namespace {

struct DistillArgs {
  int64_t vocab, top, stride, grad_stride, segs, seg_len;
  float temperature, c;  // c = log2(e) / temperature
  int rest;
  const void *logits;
  const int64_t *ids;
  const void *teacher;
  const float *teacher_lse, *grad_loss;
  float *loss, *lse, *lse_rest;
  void *grad;
  int64_t *err;
  ScanPart *parts;
};

// What a block keeps of the teacher's row in LDS, `top` values each.
struct Entries {
  double *p;     // the entry's probability; after merge(), its id's
  int32_t *ids;  // -1: unused; after merge(), also where an earlier entry has the id
  float *z;      // the student's logit
  __device__ Entries(char *lds, int64_t top)
      : p(reinterpret_cast<double *>(lds)), ids(reinterpret_cast<int32_t *>(p + top)),
        z(reinterpret_cast<float *>(ids + top)) {}
};
constexpr size_t kEntryBytes = 16;

template <class T>
__device__ __forceinline__ float teacher_value(const void *p, int64_t i) {
  return Chunk<T>::one(static_cast<const T *>(p)[i]);
}

// The teacher's row: m, r, and whether it has a target at all.
struct Target {
  double m, r;
  bool none;
};

template <class Y>
__device__ Target read_target(const DistillArgs &a, int64_t row, Entries e, double *part,
                              int64_t *err) {
  const double T = a.temperature;
  double most = -__builtin_inf();
  int used = 0, bad = 0;
  for (int64_t j = threadIdx.x; j < a.top; j += kScanThreads) {
    const int64_t id = a.ids[row * a.top + j];
    const bool ok = id >= 0 && id < a.vocab;
    bad += !ok && id != -1;
    used |= ok;
    const double y = ok ? teacher_value<Y>(a.teacher, row * a.top + j) / T : -__builtin_inf();
    e.ids[j] = ok ? (int32_t)id : -1;
    e.p[j] = y;
    most = fmax(most, y);
  }
  count_errors(bad, err);
  double ref;
  if (a.teacher_lse != nullptr) {
    ref = a.teacher_lse[row];
  } else {
    ref = block_max<kScanThreads>(most, part);
    if (ref == -__builtin_inf()) ref = 0.0;
  }
  double sum = 0.0;
  for (int64_t j = threadIdx.x; j < a.top; j += kScanThreads) {
    const double p = e.ids[j] >= 0 ? exp(e.p[j] - ref) : 0.0;
    e.p[j] = p;
    sum += p;
  }
  sum = block_sum<kScanThreads>(sum, part);
  Target t = {sum, 0.0, __syncthreads_or(used) == 0};
  if (a.teacher_lse == nullptr) {
    t.none |= sum == 0.0;
    for (int64_t j = threadIdx.x; j < a.top; j += kScanThreads)
      if (sum != 0.0) e.p[j] /= sum;
    t.m = sum == 0.0 ? 0.0 : sum / sum;
  } else if (a.rest) {
    // (a smaller difference from 1 is what rounding teacher_lse to fp32 leaves)
    const double r = 1.0 - sum;
    t.r = !t.none && r >= 0x1p-20 ? r : 0.0;
  }
  __syncthreads();
  return t;
}

// Entries of one id become one: the first has their sum, in their order.
__device__ void merge(int64_t top, Entries e) {
  constexpr int kMost = ENGRAM_DISTILL_MAX_TOP / kScanThreads;
  double p[kMost];
  bool first[kMost];
#pragma unroll
  for (int k = 0; k < kMost; ++k) {
    const int64_t j = threadIdx.x + k * kScanThreads;
    p[k] = 0.0;
    first[k] = true;
    if (j >= top) continue;
    const int32_t id = e.ids[j];
    if (id < 0) continue;
    for (int64_t i = 0; i < top; ++i)
      if (e.ids[i] == id) {
        p[k] += e.p[i];
        first[k] &= i >= j;
      }
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < kMost; ++k) {
    const int64_t j = threadIdx.x + k * kScanThreads;
    if (j >= top) continue;
    e.p[j] = p[k];
    if (!first[k]) e.ids[j] = -1;
  }
  __syncthreads();
}

// One bit a value of the segment [lo, hi) that the teacher names.
__device__ void mark_named(uint32_t *bits, int64_t words, const int64_t *ids, int64_t top,
                           int64_t lo, int64_t hi) {
  for (int64_t i = threadIdx.x; i < words; i += kScanThreads) bits[i] = 0u;
  __syncthreads();
  for (int64_t j = threadIdx.x; j < top; j += kScanThreads) {
    const int64_t id = ids[j] - lo;
    if (id >= 0 && id < hi - lo) atomicOr(&bits[id >> 5], 1u << (id & 31));
  }
  __syncthreads();
}

// The sum over a segment, the named values left out with REST.
template <class T, bool REST>
__device__ __forceinline__ RowSum scan_segment(const T *row, int64_t lo, int64_t hi, float c,
                                               const uint8_t *bits, RowSum *part) {
  constexpr int U = sizeof(T) == 2 ? 4 : 2;
  Running run;
  each_chunks<T, U>(row, lo, hi, [&](int64_t at, float (&z)[U][8]) {
    if (REST) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int64_t i = at + u * kScanTile + 8 * threadIdx.x;
        const uint32_t named = i < hi ? bits[(i - lo) >> 3] : 0u;
        if (named != 0u)
#pragma unroll
          for (int k = 0; k < 8; ++k)
            if (named >> k & 1u) z[u][k] = kNegInf;
      }
    }
    float m = run.max;
#pragma unroll
    for (int u = 0; u < U; ++u) m = max8(m, z[u]);
    const float ref = run.raise(m, c);
#pragma unroll
    for (int u = 0; u < U; ++u) run.add(z[u], c, ref);
  });
  return block_join<kScanThreads>(RowSum{run.max, (double)run.sum}, c, part);
}

struct RowStats {
  double lse, lse_rest;
};

// log(q) of a value, log(s): with no finite logit at all every q is 0.
__device__ __forceinline__ double log_share(double x, double lse) {
  return lse == -__builtin_inf() ? lse : x - lse;
}

// The row's statistics from its sum (of the unnamed values with REST) and its loss.
template <class T, bool REST>
__device__ RowStats finish_row(const DistillArgs &a, int64_t row, const RowSum &sum, Entries e,
                               const Target &t, double *part) {
  const double T_ = a.temperature;
  const T *z = static_cast<const T *>(a.logits) + row * a.stride;
  for (int64_t j = threadIdx.x; j < a.top; j += kScanThreads)
    e.z[j] = e.ids[j] >= 0 ? Chunk<T>::one(z[e.ids[j]]) : kNegInf;
  RowStats s;
  s.lse = s.lse_rest = log_sum(sum, T_, a.c);
  if (REST) {
    double most = -__builtin_inf(), named = 0.0;
    for (int64_t j = threadIdx.x; j < a.top; j += kScanThreads)
      most = fmax(most, e.z[j] / T_);
    most = block_max<kScanThreads>(most, part);
    const double ref = most == -__builtin_inf() ? 0.0 : most;
    for (int64_t j = threadIdx.x; j < a.top; j += kScanThreads)
      if (e.ids[j] >= 0) named += exp(e.z[j] / T_ - ref);
    named = block_sum<kScanThreads>(named, part);
    // log(exp(lse_rest) + named * exp(ref)), from the larger of the two
    const double ln = ref + log(named);
    if (named == 0.0)
      s.lse = s.lse_rest;
    else if (s.lse_rest > ln)
      s.lse = s.lse_rest + log1p(exp(ln - s.lse_rest));
    else
      s.lse = ln + log1p(exp(s.lse_rest - ln));
  }
  if (a.loss != nullptr) {
    double loss = 0.0;
    for (int64_t j = threadIdx.x; j < a.top; j += kScanThreads)
      if (e.ids[j] >= 0 && e.p[j] != 0.0)
        loss += e.p[j] * (log(e.p[j]) - log_share(e.z[j] / T_, s.lse));
    loss = block_sum<kScanThreads>(loss, part);
    if (REST && t.r != 0.0) loss += t.r * (log(t.r) - log_share(s.lse_rest, s.lse));
    if (threadIdx.x == 0) a.loss[row] = t.none ? 0.0f : (float)loss;
  }
  if (threadIdx.x == 0) {
    if (a.lse != nullptr) a.lse[row] = (float)s.lse;
    if (REST && a.lse_rest != nullptr) a.lse_rest[row] = (float)s.lse_rest;
  }
  return s;
}

// Stores of eight values, or of the last ones before hi.
__device__ __forceinline__ void store8(uint16_t *p, const float (&v)[8], int64_t left) {
  const u32x4 w = pack_bf16x8(v);
  if (left >= 8) {
    __builtin_memcpy(p, &w, 16);
  } else {
    const uint32_t h[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (e < left) p[e] = (uint16_t)(h[e / 2] >> (16 * (e % 2)));
  }
}
__device__ __forceinline__ void store8(float *p, const float (&v)[8], int64_t left) {
  if (left >= 8) {
    __builtin_memcpy(p, v, 32);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (e < left) p[e] = v[e];
  }
}
__device__ __forceinline__ void store1(uint16_t *p, float v) { *p = (uint16_t)pack_bf16(v, 0.0f); }
__device__ __forceinline__ void store1(float *p, float v) { *p = v; }

// The gradient of the values [lo, hi) of a row.  Every value is first written as
// an unnamed one,
//     factor * exp(z / temperature - base),
// base the log of the sum of all (of the unnamed with REST, whose share s makes
// factor = g / temperature * ((m + r) s - r)): one subtraction, product, v_exp_f32
// and product.  The named ones follow.
template <class T, bool REST>
__device__ void write_gradient(const DistillArgs &a, int64_t row, int64_t lo, int64_t hi,
                               const RowStats &s, Entries e, const Target &t) {
  const double T_ = a.temperature;
  const T *zrow = static_cast<const T *>(a.logits) + row * a.stride;
  T *grow = static_cast<T *>(a.grad) + row * a.grad_stride;
  const float g = a.grad_loss[row];
  constexpr int U = sizeof(T) == 2 ? 4 : 2;
  if (g == 0.0f || t.none) {
    const float zero[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
    for (int64_t i = lo + 8 * threadIdx.x; i < hi; i += kScanTile) store8(grow + i, zero, hi - i);
    return;
  }
  const double gt = g / T_, base = REST ? s.lse_rest : s.lse;
  const bool empty = base == -__builtin_inf();
  const float r0 = empty || base != base ? 0.0f : (float)(base * T_);
  double f = gt * t.m;
  if (REST) f = gt * ((t.m + t.r) * (empty ? 0.0 : exp(s.lse_rest - s.lse)) - t.r);
  const float factor = empty ? 0.0f : (float)(f * exp(r0 / T_ - base));
  each_chunks<T, U>(zrow, lo, hi, [&](int64_t at, float (&z)[U][8]) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t i = at + u * kScanTile + 8 * threadIdx.x;
#pragma unroll
      for (int k = 0; k < 8; ++k) z[u][k] = factor * exp2_fast((z[u][k] - r0) * a.c);
      if (i < hi) store8(grow + i, z[u], hi - i);
    }
  });
  __syncthreads();
  for (int64_t j = threadIdx.x; j < a.top; j += kScanThreads) {
    const int32_t id = e.ids[j];
    if (id < lo || id >= hi) continue;
    const double q = s.lse == -__builtin_inf() ? 0.0 : exp(e.z[j] / T_ - s.lse);
    store1(grow + id, (float)(gt * ((t.m + t.r) * q - e.p[j])));
  }
}

extern __shared__ __align__(16) char lds[];

// A block to a row: the loss and, with GRAD, the gradient.
template <class T, class Y, bool REST, bool GRAD>
__global__ __launch_bounds__(kScanThreads) void distill_row_kernel(const DistillArgs a) {
  __shared__ RowSum sums[kScanThreads / kWave];
  __shared__ double part[kScanThreads / kWave];
  const int64_t row = blockIdx.x;
  Entries e(lds, a.top);
  uint32_t *bits = reinterpret_cast<uint32_t *>(lds + a.top * kEntryBytes);
  const Target t = read_target<Y>(a, row, e, part, a.err);
  if (REST)
    mark_named(bits, a.seg_len / 32, a.ids + row * a.top, a.top, 0, a.vocab);
  merge(a.top, e);
  const T *z = static_cast<const T *>(a.logits) + row * a.stride;
  const RowSum sum = scan_segment<T, REST>(z, 0, a.vocab, a.c,
                                           reinterpret_cast<const uint8_t *>(bits), sums);
  const RowStats s = finish_row<T, REST>(a, row, sum, e, t, part);
  if (GRAD) {
    __syncthreads();  // (the logits of the named ids are read before any is overwritten)
    write_gradient<T, REST>(a, row, 0, a.vocab, s, e, t);
  }
}

// A block to a segment of a row: its sum.
template <class T, bool REST>
__global__ __launch_bounds__(kScanThreads) void distill_scan_kernel(const DistillArgs a) {
  __shared__ RowSum sums[kScanThreads / kWave];
  const int64_t row = blockIdx.x / a.segs, seg = blockIdx.x - row * a.segs;
  const int64_t lo = seg * a.seg_len, hi = lo + a.seg_len < a.vocab ? lo + a.seg_len : a.vocab;
  uint32_t *bits = reinterpret_cast<uint32_t *>(lds);
  if (REST) mark_named(bits, a.seg_len / 32, a.ids + row * a.top, a.top, lo, hi);
  const T *z = static_cast<const T *>(a.logits) + row * a.stride;
  const RowSum s = scan_segment<T, REST>(z, lo, hi, a.c,
                                         reinterpret_cast<const uint8_t *>(bits), sums);
  if (threadIdx.x == 0) a.parts[row * a.segs + seg] = {s.sum, s.max, 0u};
}

// A block to a row: the segments' sums joined, the row's statistics and loss.
template <class T, class Y, bool REST>
__global__ __launch_bounds__(kScanThreads) void distill_finish_kernel(const DistillArgs a) {
  __shared__ RowSum sums[kScanThreads / kWave];
  __shared__ double part[kScanThreads / kWave];
  const int64_t row = blockIdx.x;
  Entries e(lds, a.top);
  const Target t = read_target<Y>(a, row, e, part, a.err);
  merge(a.top, e);
  RowSum v = {kNegInf, 0.0};
  for (int64_t i = threadIdx.x; i < a.segs; i += kScanThreads) {
    const ScanPart p = a.parts[row * a.segs + i];
    v = join_sums(v, RowSum{p.max, p.sum}, a.c);
  }
  v = block_join<kScanThreads>(v, a.c, sums);
  finish_row<T, REST>(a, row, v, e, t, part);
}

// A block to a segment of a row: its gradient, from the statistics that were kept.
template <class T, class Y, bool REST>
__global__ __launch_bounds__(kScanThreads) void distill_backward_kernel(const DistillArgs a) {
  __shared__ double part[kScanThreads / kWave];
  const int64_t row = blockIdx.x / a.segs, seg = blockIdx.x - row * a.segs;
  const int64_t lo = seg * a.seg_len, hi = lo + a.seg_len < a.vocab ? lo + a.seg_len : a.vocab;
  Entries e(lds, a.top);
  const Target t = read_target<Y>(a, row, e, part, seg == 0 ? a.err : nullptr);
  merge(a.top, e);
  const T *z = static_cast<const T *>(a.logits) + row * a.stride;
  // (other segments may be overwritten already)
  for (int64_t j = threadIdx.x; j < a.top; j += kScanThreads) {
    const int32_t id = e.ids[j];
    e.z[j] = id >= lo && id < hi ? Chunk<T>::one(z[id]) : kNegInf;
  }
  __syncthreads();
  const RowStats s = {a.lse[row], REST ? a.lse_rest[row] : 0.0};
  write_gradient<T, REST>(a, row, lo, hi, s, e, t);
}

DistillArgs device_args(const engram_distill_args &h, const ScanShape &shape) {
  DistillArgs a = {};
  a.vocab = h.vocab;
  a.top = h.top;
  a.stride = h.logits_stride;
  a.grad_stride = h.grad_stride;
  a.segs = shape.segs;
  a.seg_len = shape.seg_len;
  a.temperature = h.temperature;
  a.c = (float)(1.4426950408889634 / (double)h.temperature);
  a.rest = h.rest;
  a.logits = h.d_logits;
  a.ids = h.d_ids;
  a.teacher = h.d_teacher;
  a.teacher_lse = h.d_teacher_lse;
  a.grad_loss = h.d_grad_loss;
  a.loss = h.d_loss;
  a.lse = h.d_lse;
  a.lse_rest = h.d_lse_rest;
  a.grad = h.d_grad;
  a.err = h.d_err_count;
  return a;
}

// Calls f with the types and the switch as template arguments.
template <class F>
void with_types(const engram_distill_args &h, F f) {
  const auto rest = [&](auto t, auto y) {
    if (h.rest)
      f(t, y, std::true_type{});
    else
      f(t, y, std::false_type{});
  };
  const auto teacher = [&](auto t) {
    if (h.teacher_type == ENGRAM_BF16)
      rest(t, uint16_t{});
    else
      rest(t, float{});
  };
  if (h.logits_type == ENGRAM_BF16)
    teacher(uint16_t{});
  else
    teacher(float{});
}

void enqueue_backward(const engram_distill_args &h, const DistillArgs &a, hipStream_t stream) {
  const dim3 grid((unsigned)(h.rows * a.segs)), block(kScanThreads);
  const size_t entries = (size_t)h.top * kEntryBytes;
  with_types(h, [&](auto t, auto y, auto rest) {
    hipLaunchKernelGGL((distill_backward_kernel<decltype(t), decltype(y), rest.value>), grid,
                       block, entries, stream, a);
  });
}

}  // namespace
}  // namespace engram

int engram::launch_distill(const engram_distill_args &h) {
  const ScanShape shape = distill_shape(h.rows, h.vocab);
  if (!grid_fits(h.rows * shape.segs, kScanThreads)) return ENGRAM_EINVAL;
  DistillArgs a = device_args(h, shape);
  const hipStream_t stream = as_stream(h.stream);
  const size_t entries = (size_t)h.top * kEntryBytes, bits = h.rest ? shape.seg_len / 8 : 0;
  const dim3 rows((unsigned)h.rows), block(kScanThreads);
  if (shape.segs == 1) {
    with_types(h, [&](auto t, auto y, auto rest) {
      using T = decltype(t);
      using Y = decltype(y);
      if (h.d_grad != nullptr)
        hipLaunchKernelGGL((distill_row_kernel<T, Y, rest.value, true>), rows, block,
                           entries + bits, stream, a);
      else
        hipLaunchKernelGGL((distill_row_kernel<T, Y, rest.value, false>), rows, block,
                           entries + bits, stream, a);
    });
    return launch_status();
  }
  a.parts = static_cast<ScanPart *>(h.d_workspace);
  float *kept = reinterpret_cast<float *>(a.parts + h.rows * shape.segs);
  if (h.d_grad != nullptr) {
    if (a.lse == nullptr) a.lse = kept;
    if (a.lse_rest == nullptr) a.lse_rest = kept + h.rows;
  }
  with_types(h, [&](auto t, auto y, auto rest) {
    using T = decltype(t);
    using Y = decltype(y);
    hipLaunchKernelGGL((distill_scan_kernel<T, rest.value>),
                       dim3((unsigned)(h.rows * shape.segs)), block, bits, stream, a);
    hipLaunchKernelGGL((distill_finish_kernel<T, Y, rest.value>), rows, block, entries, stream,
                       a);
  });
  if (h.d_grad != nullptr) {
    a.err = nullptr;  // counted already
    enqueue_backward(h, a, stream);
  }
  return launch_status();
}

int engram::launch_distill_backward(const engram_distill_args &h) {
  const ScanShape shape = distill_shape(h.rows, h.vocab);
  if (!grid_fits(h.rows * shape.segs, kScanThreads)) return ENGRAM_EINVAL;
  enqueue_backward(h, device_args(h, shape), as_stream(h.stream));
  return launch_status();
}
