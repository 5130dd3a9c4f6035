// engram_distill.hip -- distillation from a teacher's top logits: the loss of
// every row, its gradient, or both, for gfx950.  What is computed is stated
// with engram_distill in include/engram_vocab.h.
//
// With N the ids that a row's teacher names and R the others, the sums
//     S_R = sum over R of exp(z / T),  S_N the same over N
// are kept apart: S_R is the pass over the vocabulary, in fp32 terms, S_N a few
// terms in fp64.  The named ids are where a row's large terms lie, so lse =
// log(S_R + S_N) keeps its digits, and so do s = S_R / (S_R + S_N) and s - r,
// which the gradient of the unnamed ids is made of.  The gradient is written
// for every id as if it were unnamed; the few named ones are written after it.
//
// For loss and gradient together a block holds its whole row in registers between
// the two passes, so a row is read once (distill_hold_kernel); rows that no block
// can hold, and a few long rows, which would leave CUs idle, are cut into segments
// and read again for the gradient (distill_scan_kernel, distill_backward_kernel).
#include "engram_vocab_dev.h"

namespace engram {
namespace {

struct DistillArgs {
  int64_t rows, vocab, top, stride, grad_stride, segs, seg_len;
  double temperature;
  Scale c;  // log2(e) / temperature
  int teacher_type, rest;
  const void *logits;
  const int64_t *ids;
  const void *teacher;
  const float *teacher_lse, *grad_loss;
  float *loss, *lse, *lse_rest;
  void *grad;
  int64_t *err;
  DistillPart *parts;
};

// What a block keeps of the teacher's row in LDS, `top` values each, and behind
// them one bit a value of its part of the vocabulary: whether it is named.
struct Entries {
  double *p;      // the probability of the entry, then of its id; where there is one
  int32_t *ids;   // -1: unused, or an earlier entry has the id
  float *z;       // the student's logit
  uint32_t *bits;
  __device__ Entries(char *lds, int64_t top) : Entries(lds, lds, top) {}
  // (the bits behind another row's entries)
  __device__ Entries(char *lds, char *before, int64_t top)
      : p(reinterpret_cast<double *>(lds)), ids(reinterpret_cast<int32_t *>(p + top)),
        z(reinterpret_cast<float *>(ids + top)),
        bits(reinterpret_cast<uint32_t *>(before + top * 16)) {}
};
constexpr size_t kEntryBytes = 16;

// An entry as it is loaded; a lane has up to kMost of them.
template <int THREADS>
struct RawEntries {
  static constexpr int kMost = ENGRAM_DISTILL_MAX_TOP / THREADS;
  int64_t id[kMost];
  float y[kMost], lse, weight;
  __device__ __forceinline__ void load(const DistillArgs &a, int64_t row, int thread) {
    lse = a.teacher_lse != nullptr ? a.teacher_lse[row] : 0.0f;
    weight = a.grad_loss != nullptr ? a.grad_loss[row] : 0.0f;
#pragma unroll
    for (int k = 0; k < kMost; ++k) {
      const int j = thread + k * THREADS;
      id[k] = -1;
      y[k] = kNegInf;
      if (j < a.top) {
        id[k] = a.ids[row * a.top + j];
        y[k] = a.teacher_type == ENGRAM_BF16
                   ? bf16_lo(static_cast<const uint16_t *>(a.teacher)[row * a.top + j])
                   : static_cast<const float *>(a.teacher)[row * a.top + j];
      }
    }
  }
};

// The teacher's row: m, r, and whether it has a target at all.
struct Target {
  double m, r;
  bool none;
};

// Fills e.ids and e.p; with `words` of bits, marks the ids that lie in [lo, hi).
// Entries of one id become one, the first, with their sum in their order.
template <int THREADS>
__device__ __forceinline__ Target read_target(const DistillArgs &a, int64_t row, const RawEntries<THREADS> &raw,
                              int64_t lo, int64_t hi, int words, Entries e, double *part,
                              int64_t *err, const int thread = threadIdx.x) {
  constexpr int kMost = RawEntries<THREADS>::kMost;
  __shared__ int flags;  // 1: an entry is used, 2: an id may repeat
  const double T = a.temperature;
  const int top = (int)a.top;
  if (thread == 0) flags = 0;
  for (int i = thread; i < words; i += THREADS) e.bits[i] = 0u;
  double most = -__builtin_inf();
  int bad = 0, seen = 0;
#pragma unroll
  for (int k = 0; k < kMost; ++k) {
    const int j = thread + k * THREADS;
    if (j < top) {
      const int64_t id = raw.id[k];
      const bool ok = id >= 0 && id < a.vocab;
      bad += !ok && id != -1;
      seen |= ok;
      const double y = ok ? raw.y[k] / T : -__builtin_inf();
      e.ids[j] = ok ? (int32_t)id : -1;
      e.p[j] = y;
      most = fmax(most, y);
    }
  }
  count_errors(bad, err);
  double ref;
  if (a.teacher_lse != nullptr) {
    ref = raw.lse;
    __syncthreads();
  } else {
    ref = block_max<THREADS>(most, part, thread);
    if (ref == -__builtin_inf()) ref = 0.0;
  }
  double sum = 0.0;
  for (int j = thread; j < top; j += THREADS) {
    const int32_t id = e.ids[j];
    const double p = id >= 0 ? exp64(e.p[j] - ref) : 0.0;
    e.p[j] = p;
    sum += p;
    if (words > 0 && id >= lo && id < hi) {
      const uint32_t bit = 1u << ((id - lo) & 31);
      if (atomicOr(&e.bits[(id - lo) >> 5], bit) & bit) seen |= 2;
    }
  }
  if (seen != 0) atomicOr(&flags, seen);
  sum = block_sum<THREADS>(sum, part, thread);
  const uint32_t flag = uniform((uint32_t)flags);
  Target t = {sum, 0.0, (flag & 1) == 0};
  if (a.teacher_lse == nullptr) {
    t.none |= sum == 0.0;
    if (sum != 0.0)
      for (int j = thread; j < top; j += THREADS) e.p[j] /= sum;
    t.m = uniform(sum == 0.0 ? 0.0 : sum / sum);
  } else if (a.rest) {
    // (a smaller difference from 1 is what rounding teacher_lse to fp32 leaves)
    const double r = 1.0 - sum;
    t.r = uniform(!t.none && r >= 0x1p-20 ? r : 0.0);
  }
  if (words == 0 || (flag & 2) != 0) {
    __syncthreads();
    double p[kMost];
    bool first[kMost];
#pragma unroll
    for (int k = 0; k < kMost; ++k) {
      const int j = thread + k * THREADS;
      const int32_t id = j < top ? e.ids[j] : -1;
      double total = 0.0;
      bool least = true;
      if (id >= 0)
        for (int i = 0; i < top; ++i)
          if (e.ids[i] == id) {
            total += e.p[i];
            least &= i >= j;
          }
      p[k] = total;
      first[k] = least;
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kMost; ++k) {
      const int j = thread + k * THREADS;
      if (j < top) {
        e.p[j] = p[k];
        if (!first[k]) e.ids[j] = -1;
      }
    }
  }
  __syncthreads();
  return t;
}

// -inf in the place of a chunk's named values.
__device__ __forceinline__ void leave_out(float (&z)[8], uint32_t named) {
  if (named != 0u)
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (named >> k & 1u) z[k] = kNegInf;
}

// The sum over both sides, taken from the larger maximum, and the unnamed side's share in
// it (none in an empty sum).
struct Whole {
  RowSum all;
  double s;
};
__device__ __forceinline__ Whole both(const RowSum &rest, const RowSum &named, double T) {
  const bool up = rest.max >= named.max;
  const double d = up ? (double)named.max - (double)rest.max
                      : (double)rest.max - (double)named.max;
  const double w = rest.max == named.max ? 1.0 : exp64(d / T);  // (two empty sides are level)
  const double a = up ? rest.sum : rest.sum * w, b = up ? named.sum * w : named.sum;
  const double sum = uniform(a + b);
  return {{uniform(up ? rest.max : named.max), sum}, uniform(sum == 0.0 ? 0.0 : a / sum)};
}

// The named logits' sum, in fp64, over the block; e.z is read by its own lanes.
template <int THREADS>
__device__ __forceinline__ RowSum sum_named(const DistillArgs &a, Entries e, double *part,
                                            const int thread = threadIdx.x) {
  const int top = (int)a.top;
  float m = kNegInf;
  for (int j = thread; j < top; j += THREADS) m = max3(m, e.z[j], kNegInf);
  m = block_max<THREADS>(m, reinterpret_cast<float *>(part), thread);
  double sum = 0.0;
  for (int j = thread; j < top; j += THREADS)
    if (e.ids[j] >= 0) sum += exp64(((double)e.z[j] - (double)ref_of(m)) / a.temperature);
  return {m, block_sum<THREADS>(sum, part, thread)};
}

// Loss and statistics of a row, written.
template <int THREADS>
__device__ __forceinline__ void write_row(const DistillArgs &a, int64_t row, const RowSum &rest,
                          const RowSum &all, Entries e, const Target &t, double *part,
                          const int thread = threadIdx.x) {
  const double T = a.temperature;
  const double none = -__builtin_inf();
  const int top = (int)a.top;
  double loss = 0.0, lse = 0.0;
  if (thread < (unsigned)top) {  // (the first lane is one of them)
    lse = log_sum(all, T);
    if (a.loss != nullptr)
      for (int j = thread; j < top; j += THREADS) {
        const double p = e.p[j];
        if (e.ids[j] >= 0 && p != 0.0)
          // (where no logit is finite every q is 0)
          loss += p * (log64(p) - (lse == none ? none : e.z[j] / T - lse));
      }
  }
  if (a.loss != nullptr) loss = block_sum<THREADS>(loss, part, thread);
  if (thread != 0) return;
  if (a.lse != nullptr) a.lse[row] = (float)lse;
  const double lse_rest = a.rest ? log_sum(rest, T) : 0.0;
  if (a.rest && a.lse_rest != nullptr) a.lse_rest[row] = (float)lse_rest;
  if (a.loss != nullptr) {
    if (t.r != 0.0) loss += t.r * (log64(t.r) - (lse_rest == none ? none : lse_rest - lse));
    a.loss[row] = t.none ? 0.0f : (float)loss;
  }
}

// ------------------------------------------------------------ held rows --
__device__ __forceinline__ void store8(uint16_t *p, const float (&v)[8]) {
  const u32x4 w = pack_bf16x8(v);
  __builtin_memcpy(p, &w, 16);
}
__device__ __forceinline__ void store8(float *p, const float (&v)[8]) {
  __builtin_memcpy(p, v, 32);
}
__device__ __forceinline__ void store1(uint16_t *p, float v) { *p = (uint16_t)pack_bf16(v, 0.0f); }
__device__ __forceinline__ void store1(float *p, float v) { *p = v; }

// The n >= 8 values of a row that start at `row`, in the registers of a block: chunk k
// of a lane starts at 8 * (k * THREADS + lane).  A chunk that would pass the end is the
// last eight values instead, of which those before its start are not its own, so
// every load is made, in a row, at an address inside.
template <class T, int THREADS, int N>
struct Held {
  Chunk<T> r[N];
  // whether any lane has values in chunk k; whether all have eight (uniform)
  __device__ static __forceinline__ bool any(int n, int k) { return 8 * k * THREADS < n; }
  __device__ static __forceinline__ bool full(int n, int k) { return 8 * (k + 1) * THREADS <= n; }
  // the address of a value: a uniform base and 32 bits of a lane's own
  __device__ static __forceinline__ const T *value(const T *row, uint32_t at) {
    return reinterpret_cast<const T *>(reinterpret_cast<const char *>(row) +
                                       (uint32_t)(at * sizeof(T)));
  }
  // where the eight values of a lane's chunk lie; its own start `first` (at most 8) later
  __device__ static __forceinline__ uint32_t place(int n, int k, int lane) {
    const int at = 8 * (k * THREADS + lane);
    return (uint32_t)(at + 8 <= n ? at : n - 8);
  }
  __device__ static __forceinline__ int first(int n, int k, int lane) {
    const int over = 8 * (k * THREADS + lane) + 8 - n;
    return over <= 0 ? 0 : over < 8 ? over : 8;
  }
  __device__ __forceinline__ void load(const T *row, int n) {
#pragma unroll
    for (int k = 0; k < N; ++k) r[k].load(value(row, place(n, k, threadIdx.x)));
  }
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int k = 0; k < N; ++k) r[k].clear();
  }

  // The running sum of the unnamed values.
  __device__ __forceinline__ void sum(int n, Scale c, const uint32_t *bits, Running &run) const {
    const uint8_t *bytes = reinterpret_cast<const uint8_t *>(bits);
    constexpr int G = sizeof(T) == 2 ? 2 : 1;
    const int lane = hidden_thread();
#pragma unroll
    for (int g = 0; g < N; g += G) {
      if (g + G <= N && full(n, g + G - 1)) {
        float z[G][8], m = run.max;
#pragma unroll
        for (int u = 0; u < G; ++u) {
          r[g + u].values(z[u]);
          leave_out(z[u], bytes[(g + u) * THREADS + lane]);
          m = max8(m, z[u]);
        }
        const float ref = run.raise(m, c);
#pragma unroll
        for (int u = 0; u < G; ++u) run.add(z[u], ref, c);
      } else {
#pragma unroll
      for (int u = 0; u < G; ++u)
        if (g + u < N && any(n, g + u)) {
          float z[8];
          r[g + u].values(z);
          const int from = first(n, g + u, lane);
          const uint32_t at = place(n, g + u, lane);
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if (i < from || (bits[(at + i) >> 5] >> ((at + i) & 31) & 1u)) z[i] = kNegInf;
          run.add(z, run.raise(max8(run.max, z), c), c);
        }
      }
    }
  }

  // factor * exp((z - ref) / T) in the place of every value.  (The values are unpacked
  // and placed anew: kept from the sum they would take twice the registers.)  With RELOAD
  // a chunk that is done is loaded from the row `next`, or, without one, from one place.
  template <bool RELOAD>
  __device__ __forceinline__ void write(T *row, int n, float factor, float ref, Scale c,
                                        const T *next, bool more) {
    const int lane = hidden_thread();
    const uint32_t all = more ? ~0u : 0u;
#pragma unroll
    for (int k = 0; k < N; ++k) {
      if (any(n, k)) {
        r[k].renew();
        float z[8];
        r[k].values(z);
#pragma unroll
        for (int i = 0; i < 8; ++i)
          // (rounded to bf16 the second part of c is lost)
          z[i] = factor * (sizeof(T) == 2 ? exp2_fast((z[i] - ref) * c.hi)
                                          : exp_scaled(z[i] - ref, c));
        T *to = const_cast<T *>(value(row, place(n, k, lane)));
        const int from = full(n, k) ? 0 : first(n, k, lane);
        if (from == 0) {
          store8(to, z);
        } else {
#pragma unroll
          for (int i = 1; i < 8; ++i)
            if (i >= from) store1(to + i, z[i]);
        }
      }
      if (RELOAD) r[k].load(value(next, place(n, k, lane) & all));
    }
  }
};

template <class T>
__device__ __forceinline__ void write_zeros(T *row, int64_t lo, int64_t hi, int threads) {
  const float zero[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
  for (int64_t i = lo + 8 * threadIdx.x; i < hi; i += 8 * threads) {
    if (i + 8 <= hi)
      store8(row + i, zero);
    else
      for (int64_t j = i; j < hi; ++j) store1(row + j, 0.0f);
  }
}

// The gradient of the named values in [lo, hi): q by q_of(z).
template <class T, int THREADS, class Q>
__device__ __forceinline__ void write_named(const DistillArgs &a, T *row, int64_t lo, int64_t hi,
                                            double gt, Entries e, const Target &t, Q q_of,
                                            const int thread = threadIdx.x) {
  for (int j = thread; j < (int)a.top; j += THREADS) {
    const int32_t id = e.ids[j];
    if (id >= lo && id < hi)
      store1(row + id, (float)(gt * ((t.m + t.r) * q_of(e.z[j]) - e.p[j])));
  }
}

constexpr int64_t kComputeUnits = 256;
constexpr int64_t kDistillWideRows = 512;

extern __shared__ __align__(16) char lds[];

// Loss and gradient of rows that a block's registers hold.  As many blocks as stay on the
// GPU together take the rows in turn.  All wavefronts but one hold the row: they sum it
// (while its last chunks arrive), write its gradient chunk by chunk, and load the next
// row's chunks into the registers that this leaves, so that loads, stores and arithmetic
// go on side by side.  The last wavefront does what is not the vocabulary's: it reads the
// next row's target while a gradient is written, and writes the named values and the loss
// of the row before while one is summed.  Two barriers a row.
//
// One row of the CU's registers at a time, its 2 x 304 KB (151,936 bf16 values) against the
// arithmetic of two exponentials a value: without the wavefront of its own, each row's
// target, sums' joins and loss were waited for in turn (4096 rows: 610 us).
struct RowInfo {
  double m, r, named_sum;
  float named_max, weight;
  int none;
};

// Every lane's stores to LDS before, for the other lanes of its wavefront after.
__device__ __forceinline__ void wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

// A wavefront's read_target() and sum_named() for a whole row.
template <class T>
__device__ __forceinline__ void prepare_row(const DistillArgs &a, int64_t row, Entries e,
                                            RowInfo *info, int lane) {
  const double T_ = a.temperature;
  const int top = (int)a.top;
  const int words = (int)((a.vocab + 31) / 32);
  double most = -__builtin_inf();
  int bad = 0;
  bool used = false;
  for (int j = lane; j < top; j += kWave) {
    const int64_t id = a.ids[row * a.top + j];
    const float y = a.teacher_type == ENGRAM_BF16
                        ? bf16_lo(static_cast<const uint16_t *>(a.teacher)[row * a.top + j])
                        : static_cast<const float *>(a.teacher)[row * a.top + j];
    const bool ok = id >= 0 && id < a.vocab;
    bad += !ok && id != -1;
    used |= ok;
    const double v = ok ? y / T_ : -__builtin_inf();
    e.ids[j] = ok ? (int32_t)id : -1;
    e.p[j] = v;
    most = fmax(most, v);
  }
  for (int i = lane; i < words; i += kWave) e.bits[i] = 0u;
  count_errors(bad, a.err);
  wave_sync();
  double ref;
  if (a.teacher_lse != nullptr) {
    ref = a.teacher_lse[row];
  } else {
    ref = uniform(wave_max(most));
    if (ref == -__builtin_inf()) ref = 0.0;
  }
  const T *z = static_cast<const T *>(a.logits) + row * a.stride;
  double sum = 0.0;
  float max = kNegInf;
  bool again = false;
  for (int j = lane; j < top; j += kWave) {
    const int32_t id = e.ids[j];
    const float x = id >= 0 ? Chunk<T>::one(z[id]) : kNegInf;
    const double p = id >= 0 ? exp64(e.p[j] - ref) : 0.0;
    if (id >= 0) {
      const uint32_t bit = 1u << (id & 31);
      again |= (atomicOr(&e.bits[id >> 5], bit) & bit) != 0;
    }
    e.p[j] = p;
    e.z[j] = x;
    sum += p;
    max = __builtin_fmaxf(max, x);
  }
  sum = uniform(wave_sum(sum));
  double m = sum, r = 0.0;
  bool none = __ballot(used) == 0;
  if (a.teacher_lse == nullptr) {
    none |= sum == 0.0;
    if (sum != 0.0)
      for (int j = lane; j < top; j += kWave) e.p[j] /= sum;
    m = sum == 0.0 ? 0.0 : sum / sum;
  } else if (a.rest) {
    r = 1.0 - sum;
    r = !none && r >= 0x1p-20 ? r : 0.0;
  }
  wave_sync();
  if (__ballot(again) != 0) {
    // (64 entries at a time: those before them are done, and the first of an id keeps it)
    for (int c = 0; c < top; c += kWave) {
      const int j = c + lane;
      const int32_t id = j < top ? e.ids[j] : -1;
      double total = 0.0;
      bool first = true;
      if (id >= 0)
        for (int i = 0; i < top; ++i)
          if (e.ids[i] == id) {
            total += e.p[i];
            first &= i >= j;
          }
      wave_sync();
      if (id >= 0) {
        if (first)
          e.p[j] = total;
        else
          e.ids[j] = -1;
      }
      wave_sync();
    }
  }
  max = uniform(wave_max(max));
  double named = 0.0;
  for (int j = lane; j < top; j += kWave)
    if (e.ids[j] >= 0) named += exp64(((double)e.z[j] - (double)ref_of(max)) / T_);
  named = wave_sum(named);
  if (lane == 0)
    *info = {m, r, named, max, a.grad_loss[row], none};
}

// A wavefront's write_named() and write_row().
template <class T>
__device__ __forceinline__ void finish_row(const DistillArgs &a, int64_t row, Entries e,
                                           const RowInfo &info, const RowSum &rest,
                                           const RowSum &all, int lane) {
  const double T_ = a.temperature, none = -__builtin_inf();
  const int top = (int)a.top;
  const double lse = log_sum(all, T_);
  T *grad = static_cast<T *>(a.grad) + row * a.grad_stride;
  const bool counts = info.weight != 0.0f && info.none == 0;
  const double gt = info.weight / T_;
  double loss = 0.0;
  for (int j = lane; j < top; j += kWave) {
    const int32_t id = e.ids[j];
    if (id < 0) continue;
    const double p = e.p[j], z = e.z[j];
    if (p != 0.0)  // (where no logit is finite every q is 0)
      loss += p * (log64(p) - (lse == none ? none : z / T_ - lse));
    if (counts) {
      const double q =
          all.sum == 0.0 ? 0.0 : exp64((z - (double)ref_of(all.max)) / T_) / all.sum;
      store1(grad + id, (float)(gt * ((info.m + info.r) * q - p)));
    }
  }
  loss = wave_sum(loss);
  if (lane != 0) return;
  const double lse_rest = a.rest ? log_sum(rest, T_) : 0.0;
  if (a.lse != nullptr) a.lse[row] = (float)lse;
  if (a.rest && a.lse_rest != nullptr) a.lse_rest[row] = (float)lse_rest;
  if (a.loss != nullptr) {
    if (info.r != 0.0)
      loss += info.r * (log64(info.r) - (lse_rest == none ? none : lse_rest - lse));
    a.loss[row] = info.none != 0 ? 0.0f : (float)loss;
  }
}

template <class T, int THREADS>
__global__ __launch_bounds__(THREADS, 4) void distill_hold_kernel(const DistillArgs a) {
  constexpr int kLast = THREADS / kWave - 1;
  constexpr int N = distill_held(sizeof(T));
  __shared__ RowInfo infos[2];
  __shared__ double wave_sums[THREADS / kWave];
  __shared__ float wave_maxima[THREADS / kWave];
  const int n = (int)a.vocab;
  const double T_ = a.temperature;
  // two rows' entries, and the bits of one behind them
  char *other = lds + a.top * kEntryBytes;
  const bool holds = uniform(threadIdx.x / kWave) != kLast;
  Held<T, THREADS - kWave, N> held;
  int64_t row = blockIdx.x, before = -1;
  if (holds)
    held.load(static_cast<const T *>(a.logits) + row * a.stride, n);
  else
    prepare_row<T>(a, row, Entries(lds, other, a.top), &infos[0], threadIdx.x % kWave);
  if (threadIdx.x % kWave == 0 && !holds) {
    wave_sums[kLast] = 0.0;
    wave_maxima[kLast] = kNegInf;
  }
  __syncthreads();
  RowSum rest = {kNegInf, 0.0}, all = rest;
  for (int odd = 0;; odd ^= 1) {
    const int thread = hidden_thread(), lane = thread % kWave;
    const Entries e(odd ? other : lds, other, a.top), was(odd ? lds : other, other, a.top);
    if (holds) {
      Running run;
      held.sum(hidden(n), a.c, e.bits, run);
      const float m = wave_max(run.max);
      const double s = wave_sum(moved(run.sum, run.max, ref_of(m), a.c));
      if (lane == 0) {
        wave_maxima[thread / kWave] = m;
        wave_sums[thread / kWave] = s;
      }
    } else if (before >= 0) {
      finish_row<T>(a, before, was, infos[odd ^ 1], rest, all, lane);
    }
    __syncthreads();
    const RowInfo &info = infos[odd];
    {
      constexpr int kWaves = THREADS / kWave;
      const float m1 = wave_maxima[lane % kWaves];
      const float m = uniform(lanes_max_of<kWaves>(m1));
      const double s = moved(wave_sums[lane % kWaves], m1, ref_of(m), a.c);
      rest = {m, uniform(lanes_reduce<kWaves>(s, [](double x, double y) { return x + y; }))};
    }
    const Whole whole = both(rest, RowSum{info.named_max, info.named_sum}, T_);
    all = whole.all;
    const bool more = row + gridDim.x < a.rows;
    const int64_t next = more ? row + gridDim.x : row;
    if (holds) {
      // (a row that does not count: zeros, whatever it holds)
      const bool counts = info.weight != 0.0f && info.none == 0;
      if (!counts) held.clear();
      const float factor =
          uniform(!counts || rest.sum == 0.0
                      ? 0.0f
                      : (float)(info.weight / T_ * ((info.m + info.r) * whole.s - info.r) /
                                rest.sum));
      held.template write<true>(static_cast<T *>(a.grad) + row * a.grad_stride, hidden(n),
                                factor, counts ? ref_of(rest.max) : 0.0f, a.c,
                                static_cast<const T *>(a.logits) + next * a.stride, more);
    } else if (more) {
      prepare_row<T>(a, next, was, &infos[odd ^ 1], lane);
    }
    __syncthreads();
    before = row;
    row = next;
    if (!more) {
      if (!holds) finish_row<T>(a, before, e, info, rest, all, lane);
      return;
    }
  }
}

// The unnamed values of [lo, hi) of a row, summed while the teacher's entries are read and
// their logits (of those that lie in it) loaded.
template <class T, int THREADS>
__device__ __forceinline__ RowSum scan_row(const DistillArgs &a, int64_t row, int64_t lo,
                                           int64_t hi, Entries e, Target &t, double *part,
                                           int64_t *err) {
  constexpr int U = sizeof(T) == 2 ? 2 : 1;
  const T *z = static_cast<const T *>(a.logits) + row * a.stride;
  const uint8_t *bytes = reinterpret_cast<const uint8_t *>(e.bits);
  RawEntries<THREADS> raw;
  raw.load(a, row, threadIdx.x);
  Running run;
  each_chunks<T, THREADS, U>(
      z, lo, hi,
      [&] {
        t = read_target<THREADS>(a, row, raw, lo, hi, (int)(hi - lo + 31) / 32, e, part, err);
        for (int j = threadIdx.x; j < (int)a.top; j += THREADS) {
          const int32_t id = e.ids[j];
          e.z[j] = id >= lo && id < hi ? Chunk<T>::one(z[id]) : kNegInf;
        }
      },
      [&](int64_t at, float (&v)[U][8]) {
        float m = run.max;
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int64_t i = at + (u * THREADS + (int)threadIdx.x) * 8;
          leave_out(v[u], i < hi ? bytes[(i - lo) >> 3] : 0u);
          m = max8(m, v[u]);
        }
        const float ref = run.raise(m, a.c);
#pragma unroll
        for (int u = 0; u < U; ++u) run.add(v[u], ref, a.c);
      });
  return block_join<THREADS>(run, a.c, part);
}

// A block to a row: its statistics and loss.
template <class T, int THREADS>
__global__ __launch_bounds__(THREADS, 8) void distill_row_kernel(const DistillArgs a) {
  __shared__ double part[THREADS / kWave];
  Entries e(lds, a.top);
  Target t;
  const int64_t row = blockIdx.x;
  const RowSum rest = scan_row<T, THREADS>(a, row, 0, a.vocab, e, t, part, a.err);
  const RowSum named = sum_named<THREADS>(a, e, part);
  write_row<THREADS>(a, row, rest, both(rest, named, a.temperature).all, e, t, part);
}

// A block to a segment of a row: its part of the sums and of the loss.
template <class T>
__global__ __launch_bounds__(kScanThreads, 8) void distill_scan_kernel(const DistillArgs a) {
  __shared__ double part[kScanThreads / kWave];
  Entries e(lds, a.top);
  Target t;
  const int64_t row = blockIdx.x / a.segs, seg = blockIdx.x - row * a.segs;
  const int64_t lo = seg * a.seg_len, hi = lo + a.seg_len < a.vocab ? lo + a.seg_len : a.vocab;
  const RowSum rest =
      scan_row<T, kScanThreads>(a, row, lo, hi, e, t, part, seg == 0 ? a.err : nullptr);
  const RowSum named = sum_named<kScanThreads>(a, e, part);
  double loss = 0.0;  // but for the part of lse
  for (int j = threadIdx.x; j < (int)a.top; j += kScanThreads) {
    const int32_t id = e.ids[j];
    const double p = e.p[j];
    if (id >= lo && id < hi && p != 0.0) loss += p * (log64(p) - e.z[j] / a.temperature);
  }
  loss = block_sum<kScanThreads>(loss, part);
  if (threadIdx.x == 0)
    a.parts[row * a.segs + seg] = {rest.sum, named.sum, loss, rest.max, named.max};
}

// A row's parts, joined by every wavefront for itself.
struct Joined {
  RowSum rest, named;
  double loss;
};
__device__ __forceinline__ Joined join_parts(const DistillArgs &a, int64_t row) {
  const DistillPart *parts = a.parts + row * a.segs;
  const int lane = threadIdx.x % kWave;
  float mr = kNegInf, mn = kNegInf;
  for (int64_t i = lane; i < a.segs; i += kWave) {
    mr = max3(mr, parts[i].rest_max, kNegInf);
    mn = max3(mn, parts[i].named_max, kNegInf);
  }
  mr = wave_max(mr);
  mn = wave_max(mn);
  double sr = 0.0, sn = 0.0, loss = 0.0;
  for (int64_t i = lane; i < a.segs; i += kWave) {
    const DistillPart p = parts[i];
    sr += moved(p.rest_sum, p.rest_max, ref_of(mr), a.c);
    // (fp64 terms: the step is too)
    sn += p.named_max == kNegInf
              ? p.named_sum
              : p.named_sum * exp64(((double)p.named_max - (double)ref_of(mn)) / a.temperature);
    loss += p.loss;
  }
  return {{mr, wave_sum(sr)}, {mn, wave_sum(sn)}, wave_sum(loss)};
}

// Loss and statistics of a row from its parts, written by one lane.
__device__ __forceinline__ void write_joined(const DistillArgs &a, int64_t row, const Joined &v,
                                             const Whole &whole, const Target &t) {
  const double T_ = a.temperature, none = -__builtin_inf();
  const double lse = log_sum(whole.all, T_), lse_rest = a.rest ? log_sum(v.rest, T_) : 0.0;
  if (a.lse != nullptr) a.lse[row] = (float)lse;
  if (a.rest && a.lse_rest != nullptr) a.lse_rest[row] = (float)lse_rest;
  if (a.loss == nullptr) return;
  // (where no logit is finite the parts hold the infinite loss of their targets)
  double loss = lse == none || t.m == 0.0 ? v.loss : v.loss + t.m * lse;
  if (t.r != 0.0) loss += t.r * (log64(t.r) - (lse_rest == none ? none : lse_rest - lse));
  a.loss[row] = t.none ? 0.0f : (float)loss;
}

// A wavefront to a row: its parts joined.
__global__ __launch_bounds__(kScanThreads) void distill_finish_kernel(const DistillArgs a) {
  __shared__ double part[kScanThreads / kWave];
  const int64_t row = blockIdx.x;
  RawEntries<kScanThreads> raw;
  raw.load(a, row, threadIdx.x);
  Entries e(lds, a.top);
  const Target t = read_target<kScanThreads>(a, row, raw, 0, 0, 0, e, part, nullptr);
  if (threadIdx.x >= kWave) return;
  const Joined v = join_parts(a, row);
  const Whole whole = both(v.rest, v.named, a.temperature);
  if (threadIdx.x == 0) write_joined(a, row, v, whole, t);
}

// A block to a segment of a row: its gradient, from the statistics that were kept or, with
// PARTS, from the parts that distill_scan_kernel left (the first segment's block then also
// writes the row's loss and statistics).  SHORT: a vocabulary of less than eight values.
template <class T, bool SHORT, bool PARTS>
__global__ __launch_bounds__(kScanThreads) void distill_backward_kernel(const DistillArgs a,
                                                                        const int64_t segs) {
  constexpr int N = distill_held_backward(sizeof(T));
  __shared__ double part[kScanThreads / kWave];
  const int64_t row = blockIdx.x / segs, seg = blockIdx.x - row * segs;
  // (whole chunks are shared out, so that every segment has eight values or more)
  const int64_t chunks = a.vocab / 8, lo = chunks * seg / segs * 8;
  const int64_t hi = seg + 1 == segs ? a.vocab : chunks * (seg + 1) / segs * 8;
  const T *z = static_cast<const T *>(a.logits) + row * a.stride;
  T *grad = static_cast<T *>(a.grad) + row * a.grad_stride;
  const double T_ = a.temperature;
  RawEntries<kScanThreads> raw;
  raw.load(a, row, threadIdx.x);
  Held<T, kScanThreads, N> held;
  if (!SHORT) held.load(z + lo, (int)(hi - lo));
  Entries e(lds, a.top);
  const Target t = read_target<kScanThreads>(a, row, raw, lo, hi, (int)(hi - lo + 31) / 32, e,
                                             part, !PARTS && seg == 0 ? a.err : nullptr);
  // the unnamed: factor * exp((z - ref) / T); the named: q = exp(z / T - below) * scale
  double below, scale = 1.0, f;
  const double gt = raw.weight / T_;
  float ref;
  if (PARTS) {
    const Joined v = join_parts(a, row);
    const Whole whole = both(v.rest, v.named, T_);
    if (seg == 0 && threadIdx.x == 0) write_joined(a, row, v, whole, t);
    ref = ref_of(v.rest.max);
    f = v.rest.sum == 0.0 ? 0.0 : gt * ((t.m + t.r) * whole.s - t.r) / v.rest.sum;
    below = ref_of(whole.all.max) / T_;
    scale = whole.all.sum == 0.0 ? 0.0 : 1.0 / whole.all.sum;
  } else {
    // base: the log of the unnamed values' own sum, or of the whole one without a class for
    // the rest
    const double lse = a.lse[row], base = a.rest ? a.lse_rest[row] : lse;
    const bool empty = base == -__builtin_inf();
    ref = empty || base != base ? 0.0f : (float)(base * T_);
    f = gt * t.m;
    if (a.rest) f = gt * ((t.m + t.r) * (empty ? 0.0 : exp64(base - lse)) - t.r);
    f = empty ? 0.0 : f * exp64(ref / T_ - base);
    below = lse == -__builtin_inf() ? 0.0 : lse;
    scale = lse == -__builtin_inf() ? 0.0 : 1.0;
  }
  if (raw.weight == 0.0f || t.none) {
    write_zeros(grad, lo, hi, kScanThreads);
    return;
  }
  // (other segments' logits may be overwritten already)
  for (int j = threadIdx.x; j < (int)a.top; j += kScanThreads) {
    const int32_t id = e.ids[j];
    e.z[j] = id >= lo && id < hi ? Chunk<T>::one(z[id]) : kNegInf;
  }
  const float factor = (float)f;
  float one = kNegInf;
  if (SHORT && threadIdx.x < a.vocab) one = Chunk<T>::one(z[threadIdx.x]);
  __syncthreads();
  if (!SHORT)
    held.template write<false>(grad + lo, (int)(hi - lo), factor, ref, a.c, nullptr, false);
  else if (threadIdx.x < a.vocab)
    store1(grad + threadIdx.x, factor * exp_scaled(one - ref, a.c));
  __syncthreads();
  write_named<T, kScanThreads>(a, grad, lo, hi, gt, e, t, [&](float x) {
    return scale == 0.0 ? 0.0 : exp64(x / T_ - below) * scale;
  });
}

DistillArgs device_args(const engram_distill_args &h, const ScanShape &shape) {
  DistillArgs a = {};
  a.rows = h.rows;
  a.vocab = h.vocab;
  a.top = h.top;
  a.stride = h.logits_stride;
  a.grad_stride = h.grad_stride;
  a.segs = shape.segs;
  a.seg_len = shape.seg_len;
  a.temperature = h.temperature;
  a.c = scale_of(h.temperature);
  a.teacher_type = h.teacher_type;
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

size_t lds_bytes(int64_t top, int64_t values) {
  return (size_t)top * kEntryBytes + (size_t)ceil_div(values, 32) * 4;
}

template <class T, int THREADS>
void enqueue_hold(const DistillArgs &a, hipStream_t stream) {
  // as many blocks as stay on the GPU together
  const int64_t most = kComputeUnits * (1024 / THREADS);
  hipLaunchKernelGGL((distill_hold_kernel<T, THREADS>),
                     dim3((unsigned)(a.rows < most ? a.rows : most)), dim3(THREADS),
                     lds_bytes(2 * a.top, a.vocab), stream, a);
}

template <class T, bool PARTS>
int enqueue_backward(const DistillArgs &a, hipStream_t stream) {
  const int64_t most = kScanThreads * distill_held_backward(sizeof(T));
  // (a segment of a row's chunks, and what is left of the last)
  const int64_t segs = a.vocab < 8 ? 1 : ceil_div(a.vocab / 8, most - 1);
  if (!grid_fits(a.rows * segs, kScanThreads)) return ENGRAM_EINVAL;
  const dim3 grid((unsigned)(a.rows * segs)), block(kScanThreads);
  const size_t bytes = lds_bytes(a.top, most * 8);
  if (a.vocab < 8)
    hipLaunchKernelGGL((distill_backward_kernel<T, true, PARTS>), grid, block, bytes, stream, a,
                       segs);
  else
    hipLaunchKernelGGL((distill_backward_kernel<T, false, PARTS>), grid, block, bytes, stream, a,
                       segs);
  return launch_status();
}

template <class T>
int enqueue(const engram_distill_args &h) {
  const ScanShape shape = distill_shape(h.rows, h.vocab);
  DistillArgs a = device_args(h, shape);
  const hipStream_t stream = as_stream(h.stream);
  const bool grad = h.d_grad != nullptr;
  const int threads = grad ? distill_threads(h.rows, h.vocab, sizeof(T)) : 0;
  if (!grid_fits(h.rows, 1024) || !grid_fits(h.rows * shape.segs, kScanThreads))
    return ENGRAM_EINVAL;
  if (threads == 256) {
    enqueue_hold<T, 256>(a, stream);
  } else if (threads == 512) {
    enqueue_hold<T, 512>(a, stream);
  } else if (threads == 1024) {
    enqueue_hold<T, 1024>(a, stream);
  } else if (!grad && h.vocab <= kDistillMaxSeg) {
    const dim3 rows((unsigned)h.rows);
    const size_t bytes = lds_bytes(h.top, h.vocab);
    if (h.rows <= kDistillWideRows)
      hipLaunchKernelGGL((distill_row_kernel<T, 1024>), rows, dim3(1024), bytes, stream, a);
    else
      hipLaunchKernelGGL((distill_row_kernel<T, 256>), rows, dim3(256), bytes, stream, a);
  } else {
    a.parts = static_cast<DistillPart *>(h.d_workspace);
    hipLaunchKernelGGL(distill_scan_kernel<T>, dim3((unsigned)(h.rows * shape.segs)),
                       dim3(kScanThreads), lds_bytes(h.top, shape.seg_len), stream, a);
    if (grad) return enqueue_backward<T, true>(a, stream);
    hipLaunchKernelGGL(distill_finish_kernel, dim3((unsigned)h.rows), dim3(kScanThreads),
                       lds_bytes(h.top, 0), stream, a);
  }
  return launch_status();
}

}  // namespace
}  // namespace engram

int engram::launch_distill(const engram_distill_args &h) {
  return h.logits_type == ENGRAM_BF16 ? enqueue<uint16_t>(h) : enqueue<float>(h);
}

int engram::launch_distill_backward(const engram_distill_args &h) {
  const DistillArgs a = device_args(h, ScanShape{});
  const hipStream_t stream = as_stream(h.stream);
  return h.logits_type == ENGRAM_BF16 ? enqueue_backward<uint16_t, false>(a, stream)
                                      : enqueue_backward<float, false>(a, stream);
}
