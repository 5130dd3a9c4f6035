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
// What is not the vocabulary's, the teacher's entries and the loss, is one
// wavefront's work in every kernel, with the block's other wavefronts waiting at
// three barriers a row at most.
//
// For loss and gradient together a block reads its row twice, the second time
// from the Infinity Cache (256 MB) as long as the rows in flight fit it, and the
// gradient is stored past it (distill_row_kernel, distill_threads).
//
// What bounds it is memory: a value costs 2 or 4 bytes and a subtraction, a
// product, a v_exp_f32 and an addition, so the floor is each logit read once and
// each gradient written once.  At each kernel below stands what it reaches of
// the 6.6 TB/s that a large streaming copy does here.
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
  float *z;       // the student's logit; -inf outside the block's part
  uint32_t *bits;
  __device__ Entries(char *lds, int64_t top)
      : p(reinterpret_cast<double *>(lds)), ids(reinterpret_cast<int32_t *>(p + top)),
        z(reinterpret_cast<float *>(ids + top)), bits(reinterpret_cast<uint32_t *>(z + top)) {}
};
constexpr size_t kEntryBytes = 16;
constexpr int kLead = kWave;  // bits before the first chunk's
static_assert(kLead * 2 >= kLine, "a wavefront reads a lead");

// What the teacher's row gives beside them.
struct RowInfo {
  double m, r;
  RowSum named;  // of the logits in the block's part
  float weight;  // the loss' gradient; 0 where only the loss is asked for
  int none;      // no target
};

// The sum over the named logits in the block's part, by one wavefront; max: each lane's largest.
__device__ __forceinline__ RowSum named_sum(const DistillArgs &a, Entries e, float max) {
  double sum = 0.0;
  max = wave_max(max);
  for (int j = threadIdx.x; j < (int)a.top; j += kWave)
    if (e.ids[j] >= 0) sum += exp64(((double)e.z[j] - (double)ref_of(max)) / a.temperature);
  return {max, wave_sum(sum)};
}

// An id's entries, found by those that met its bit (`again`, one for each of the lane's entries),
// become its first one, with their sum.  (Only rows that repeat ids pay for it: 64 x 151,936 with
// 300 entries a row takes 30 us, 35 where 1 in 4 rows repeats one.)
__device__ __forceinline__ void merge_repeated(int top, Entries e, uint32_t again) {
  const int lane = threadIdx.x;
  for (int c = 0; c < top; c += kWave)
    for (uint64_t met = __ballot(again >> (c / kWave) & 1u); met != 0; met &= met - 1) {
      const int32_t id = e.ids[c + __ffsll((unsigned long long)met) - 1];
      if (id < 0) continue;
      double total = 0.0;
      int first = -1, count = 0;
      for (int b = 0; b < top; b += kWave) {
        const int i = b + lane;
        const bool same = i < top && e.ids[i] == id;
        const uint64_t all = __ballot(same);
        if (first < 0 && all != 0) first = b + __ffsll((unsigned long long)all) - 1;
        count += __popcll(all);
        if (same) total += e.p[i];
        if (same && i != first) e.ids[i] = -1;
      }
      if (count > 1) {
        total = wave_sum(total);
        if (lane == 0) e.p[first] = total;
      }
      wave_sync();
    }
}

// Reads the teacher's row, by one wavefront: e and *info, for the values [lo, hi) of the
// vocabulary, of which first_bit (kLead before lo at most) has the first bit.  Entries of one id
// become one, the first, with their sum.  WHOLE: the statistics' sum over the named logits too.
template <class T, bool WHOLE>
__device__ __forceinline__ void read_target(const DistillArgs &a, int64_t row, int64_t lo,
                                            int64_t hi, int64_t first_bit, Entries e,
                                            RowInfo *info, int64_t *err) {
  const double T_ = a.temperature;
  const int top = (int)a.top, lane = threadIdx.x;
  const T *z = static_cast<const T *>(a.logits) + row * a.stride;
  // (loaded here, their latency is beside that of the ids)
  const float whole = a.teacher_lse != nullptr ? a.teacher_lse[row] : 0.0f;
  const float weight = a.grad_loss != nullptr ? a.grad_loss[row] : 0.0f;
  double most = -__builtin_inf();
  float max = kNegInf;
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
  count_errors(bad, err);
  for (int i = lane; i < (int)((hi - first_bit + 31) / 32); i += kWave) e.bits[i] = 0u;
  wave_sync();
  double ref;
  if (a.teacher_lse != nullptr) {
    ref = whole;
  } else {
    ref = wave_max(most);
    if (ref == -__builtin_inf()) ref = 0.0;
  }
  double sum = 0.0;
  uint32_t again = 0;  // a bit for each of the lane's entries
  for (int j = lane; j < top; j += kWave) {
    const int32_t id = e.ids[j];
    const bool here = id >= lo && id < hi;
    const float x = here ? Chunk<T>::one(z[id]) : kNegInf;
    const double p = id >= 0 ? exp64(e.p[j] - ref) : 0.0;
    if (here) {
      const uint32_t at = (uint32_t)(id - first_bit), bit = 1u << (at & 31);
      if ((atomicOr(&e.bits[at >> 5], bit) & bit) != 0) again |= 1u << (j / kWave);
    }
    e.p[j] = p;
    e.z[j] = x;
    sum += p;
    max = __builtin_fmaxf(max, x);
  }
  sum = wave_sum(sum);
  double m = sum, r = 0.0;
  bool none = __ballot(used) == 0;
  if (a.teacher_lse == nullptr) {
    none |= sum == 0.0;
    if (sum != 0.0)
      for (int j = lane; j < top; j += kWave) e.p[j] /= sum;
    m = sum == 0.0 ? 0.0 : sum / sum;
  } else if (a.rest) {
    // (a smaller difference from 1 is what rounding teacher_lse to fp32 leaves)
    r = 1.0 - sum;
    r = !none && r >= 0x1p-20 ? r : 0.0;
  }
  wave_sync();
  merge_repeated(top, e, again);
  RowSum named = {kNegInf, 0.0};
  if (WHOLE) named = named_sum(a, e, max);
  if (lane == 0) *info = {m, r, named, weight, none};
  wave_sync();
}

// -inf in the place of a chunk's named values.
__device__ __forceinline__ void leave_out(float (&z)[8], uint32_t named) {
  if (named != 0u)
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (named >> k & 1u) z[k] = kNegInf;
}

// The unnamed values of [lo, hi) of a row, summed by a block; the first wavefront reads the
// teacher's row while the first values are on their way.  (Were the named ids not left out
// here but subtracted afterwards, losses would be off by 1e-6 to 3e-6: the sum's rounding
// against what is left of it.  Left out they are within 5e-8.)
template <class T, int THREADS>
__device__ __forceinline__ RowSum scan_row(const DistillArgs &a, int64_t row, int64_t lo,
                                           int64_t hi, Entries e, RowInfo *info,
                                           JoinLds<THREADS / kWave> &join, int64_t *err) {
  constexpr int U = sizeof(T) == 2 ? 2 : 1;
  const T *z = static_cast<const T *>(a.logits) + row * a.stride;
  const uint8_t *bytes = reinterpret_cast<const uint8_t *>(e.bits);
  const int lead = lead_of(z + lo, hi - lo), lane = threadIdx.x;
  const int64_t body = lo + lead;
  float one = lane < lead ? Chunk<T>::one(z[lo + lane]) : kNegInf;
  Running run;
  each_chunks<T, THREADS, U, false>(
      z, body, hi,
      [&] {
        if (lane < kWave) {
          read_target<T, true>(a, row, lo, hi, body - kLead, e, info, err);
          const int bit = kLead - lead + lane;
          if (lane < lead && (e.bits[bit >> 5] >> (bit & 31) & 1u) == 0u) {
            const float ref = run.raise(one, a.c);
            run.sum += exp_scaled(one - ref, a.c);
          }
        }
        __syncthreads();
      },
      [&](int64_t at, float (&v)[U][8]) {
        float m = run.max;
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int64_t i = at + (u * THREADS + (int)threadIdx.x) * 8;
          leave_out(v[u], i < hi ? bytes[kLead / 8 + ((i - body) >> 3)] : 0u);
          m = max8(m, v[u]);
        }
        const float ref = run.raise(m, a.c);
#pragma unroll
        for (int u = 0; u < U; ++u) run.add(v[u], ref, a.c);
      });
  return block_join(run, a.c, join);
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
  const double sum = a + b;
  return {{up ? rest.max : named.max, sum}, sum == 0.0 ? 0.0 : a / sum};
}

// How a row's gradient is written: an unnamed value as
//     factor * exp((z - ref) / T),  factor = g / T * ((m + r) s - r) / S_R
// (a subtraction, a product, a v_exp_f32 and a product), a named one from its share.
struct Gradient {
  float factor, ref;
  bool zero;  // the row does not count
};
__device__ __forceinline__ Gradient gradient_of(const RowInfo &info, const RowSum &rest, double s,
                                                double T) {
  const double f =
      rest.sum == 0.0 ? 0.0 : info.weight / T * ((info.m + info.r) * s - info.r) / rest.sum;
  return {uniform((float)f), ref_of(rest.max), info.weight == 0.0f || info.none != 0};
}

template <class T>
__device__ __forceinline__ float gradient_value(float z, const Gradient &g, Scale c) {
  // (rounded to bf16 the second part of c is lost)
  return g.factor * (sizeof(T) == 2 ? exp2_fast((z - g.ref) * c.hi) : exp_scaled(z - g.ref, c));
}
template <class T>
__device__ __forceinline__ void gradient_values(float (&z)[8], const Gradient &g, Scale c) {
#pragma unroll
  for (int i = 0; i < 8; ++i) z[i] = gradient_value<T>(z[i], g, c);
}

template <class T>
__device__ void write_zeros(T *row, int64_t lo, int64_t hi, int threads) {
  const float zero[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
  for (int64_t i = lo + 8 * (int)threadIdx.x; i < hi; i += 8 * threads) {
    if (i + 8 <= hi)
      Chunk<T>::store_once(row + i, zero);
    else
      for (int64_t j = i; j < hi; ++j) Chunk<T>::store_one(row + j, 0.0f);
  }
}

// The gradient of the named values in [lo, hi), by one wavefront: q is exp(z / T - below)
// times scale.
template <class T>
__device__ __forceinline__ void write_named(const DistillArgs &a, T *row, int64_t lo, int64_t hi,
                                            Entries e, const RowInfo &info, double below,
                                            double scale) {
  const double gt = info.weight / a.temperature, whole = info.m + info.r;
  for (int j = threadIdx.x; j < (int)a.top; j += kWave) {
    const int32_t id = e.ids[j];
    if (id < lo || id >= hi) continue;
    const double q = scale == 0.0 ? 0.0 : exp64(e.z[j] / a.temperature - below) * scale;
    Chunk<T>::store_one(row + id, (float)(gt * (whole * q - e.p[j])));
  }
}

// sum of p (log(p) - (z - ref) / T) over the named values of the block's part, by one
// wavefront, and the sum of p.  (Logits are taken from a point near them: beside a mask's
// lowest value nothing else would be left.)
struct NamedLoss {
  double loss, mass;
};
__device__ __forceinline__ NamedLoss named_loss(const DistillArgs &a, Entries e, int64_t lo,
                                                int64_t hi, float ref) {
  double loss = 0.0, mass = 0.0;
  for (int j = threadIdx.x; j < (int)a.top; j += kWave) {
    const int32_t id = e.ids[j];
    const double p = e.p[j];
    if (id < lo || id >= hi || p == 0.0) continue;
    loss += p * (log64(p) - ((double)e.z[j] - (double)ref) / a.temperature);
    mass += p;
  }
  return {wave_sum(loss), wave_sum(mass)};
}

// Loss and statistics of a row, written by one lane; loss: over the named values, taken from
// the largest logit.
__device__ __forceinline__ void write_row(const DistillArgs &a, int64_t row, const RowSum &rest,
                                          const RowSum &all, double loss, const RowInfo &info) {
  const double T_ = a.temperature, log_all = log64(all.sum), log_rest = log64(rest.sum);
  const double all_at = ref_of(all.max) / T_, rest_at = ref_of(rest.max) / T_;
  if (a.lse != nullptr) a.lse[row] = (float)(all_at + log_all);
  if (a.rest && a.lse_rest != nullptr) a.lse_rest[row] = (float)(rest_at + log_rest);
  if (a.loss == nullptr) return;
  // (where no logit is finite every q is 0, and a target's loss infinite already)
  if (all.sum != 0.0 && info.m != 0.0) loss += info.m * log_all;
  if (info.r != 0.0)
    loss += info.r * (log64(info.r) -
                      (rest.sum == 0.0 ? log_rest : (rest_at - all_at) + (log_rest - log_all)));
  a.loss[row] = info.none != 0 ? 0.0f : (float)loss;
}

extern __shared__ __align__(16) char lds[];

// A block to a row: its loss and statistics and, with GRAD, its gradient, for which the row
// is read again.  8 wavefronts a SIMD in blocks of each size.
//
// Without GRAD it is one pass: 4096 x 151,936 bf16 228 us (5.5 TB/s), 4096 x 50,257 84 us
// (4.9), 1031 x 50,257 27 us (3.9: four blocks a CU and no second round of them, so that the
// teacher's row before it and the joins behind it are not hidden), 16,384 x 1000 29 us (a
// wavefront to a row, each waiting for its teacher's entries and their logits in turn).  With
// GRAD 4096 x 151,936 bf16 takes 527 us, 4.7 TB/s of the floor's bytes, its blocks reading and
// writing in turn.  Tried instead for these 2.5 GB: the row held in registers from one pass to
// the other, so that nothing is read twice, 566 us (304 KB leave a CU one block, whose joins
// then stall it), the same with persistent blocks 610; all rows scanned, then written, 128 to
// 1024 rows at a time 721 to 1114; ordinary stores 618 against 534 in turn (the gradient
// pushes rows out of the Infinity Cache); the second pass backwards, or 1 or 4 chunks a lane
// and step, no change.
//
// Chunks start at whole cache lines of the logits, which the gradient usually shares: with
// the row's first value at the first chunk 4096 x 50,257 bf16 took 226 us with its gradient
// and 92 without (now 194 and 83), 50,256 192 and 82 (184, 82).
template <class T, int THREADS, bool GRAD>
__global__ __launch_bounds__(THREADS, 8) void distill_row_kernel(const DistillArgs a) {
  __shared__ JoinLds<THREADS / kWave> join;
  __shared__ RowInfo info;
  Entries e(lds, a.top);
  const int64_t row = blockIdx.x;
  const RowSum rest = scan_row<T, THREADS>(a, row, 0, a.vocab, e, &info, join, a.err);
  const Whole whole = both(rest, info.named, a.temperature);
  if (GRAD) {
    T *grad = static_cast<T *>(a.grad) + row * a.grad_stride;
    const Gradient g = gradient_of(info, rest, whole.s, a.temperature);
    if (g.zero) {
      write_zeros(grad, 0, a.vocab, THREADS);
    } else {
      constexpr int U = sizeof(T) == 2 ? 2 : 1;
      const T *z = static_cast<const T *>(a.logits) + row * a.stride;
      const int lead = lead_of(z, a.vocab), thread = threadIdx.x;
      each_chunks<T, THREADS, U, true>(
          z, lead, a.vocab,
          [&] {
            if (thread >= lead) return;
            const float one = gradient_value<T>(Chunk<T>::one(z[thread]), g, a.c);
            Chunk<T>::store_one(grad + thread, one);
          },
          [&](int64_t at, float (&v)[U][8]) {
#pragma unroll
            for (int u = 0; u < U; ++u) {
              const int64_t i = at + (u * THREADS + (int)threadIdx.x) * 8;
              gradient_values<T>(v[u], g, a.c);
              if (i + 8 <= a.vocab) {
                Chunk<T>::store_once(grad + i, v[u]);
              } else {
#pragma unroll
                for (int k = 0; k < 8; ++k)
                  if (i + k < a.vocab) Chunk<T>::store_one(grad + i + k, v[u][k]);
              }
            }
          });
      __syncthreads();
      if (threadIdx.x < kWave)
        write_named<T>(a, grad, 0, a.vocab, e, info, ref_of(whole.all.max) / a.temperature,
                       whole.all.sum == 0.0 ? 0.0 : 1.0 / whole.all.sum);
    }
  }
  if (threadIdx.x >= kWave) return;
  const double loss =
      a.loss != nullptr ? named_loss(a, e, 0, a.vocab, ref_of(whole.all.max)).loss : 0.0;
  if (threadIdx.x == 0) write_row(a, row, rest, whole.all, loss, info);
}

// A block to a segment of a row: its part of the sums and of the loss.  64 x 151,936 bf16,
// 16 blocks to a row: 11.3 us, of which the bytes are 3; the rest is the launch and the
// latency of one block's chain (ids, their logits, their sum, the joins).
template <class T>
__global__ __launch_bounds__(kScanThreads, 8) void distill_scan_kernel(const DistillArgs a) {
  __shared__ JoinLds<kScanThreads / kWave> join;
  __shared__ RowInfo info;
  Entries e(lds, a.top);
  const int64_t row = blockIdx.x / a.segs, seg = blockIdx.x - row * a.segs;
  const int64_t lo = seg * a.seg_len, hi = lo + a.seg_len < a.vocab ? lo + a.seg_len : a.vocab;
  const RowSum rest = scan_row<T, kScanThreads>(a, row, lo, hi, e, &info, join,
                                                seg == 0 ? a.err : nullptr);
  if (threadIdx.x >= kWave) return;
  const NamedLoss own = named_loss(a, e, lo, hi, ref_of(info.named.max));
  if (threadIdx.x == 0)
    a.parts[row * a.segs + seg] = {rest.sum,  info.named.sum, own.loss,
                                   own.mass, rest.max,       info.named.max};
}

// A row's parts, joined by a wavefront; the loss taken from the largest logit.
struct Joined {
  RowSum rest, named;
  double loss;
};
__device__ __forceinline__ Joined join_parts(const DistillArgs &a, int64_t row) {
  const DistillPart *parts = a.parts + row * a.segs;
  const int lane = threadIdx.x % kWave;
  float mr = kNegInf, mn = kNegInf;
  for (int64_t i = lane; i < a.segs; i += kWave) {
    mr = __builtin_fmaxf(mr, parts[i].rest_max);
    mn = __builtin_fmaxf(mn, parts[i].named_max);
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
    if (p.mass != 0.0)
      loss += p.mass * (((double)ref_of(mr > mn ? mr : mn) - (double)ref_of(p.named_max)) /
                        a.temperature);
  }
  return {{mr, wave_sum(sr)}, {mn, wave_sum(sn)}, wave_sum(loss)};
}

// A wavefront to a row: its parts joined.  Few bytes: it is the latency of a launch and of
// the teacher's row, read again.
template <class T>
__global__ __launch_bounds__(kWave) void distill_finish_kernel(const DistillArgs a) {
  __shared__ RowInfo info;
  const int64_t row = blockIdx.x;
  read_target<T, false>(a, row, 0, 0, 0, Entries(lds, a.top), &info, nullptr);
  const Joined v = join_parts(a, row);
  const Whole whole = both(v.rest, v.named, a.temperature);
  if (threadIdx.x == 0) write_row(a, row, v.rest, whole.all, v.loss, info);
}

// Whether a row's kept logarithms are too coarse to take its gradient from.  Half a step of fp32
// is a relative error of every exponential: 2^-19 below 64, and 2^-15 below 1024, which is 1/64 of
// the rounding of a bf16 gradient.  Beside a mask's lowest value nothing is left of the sum's own
// logarithm, and the quotient by a temperature below 1 may be past fp32.  (-inf is exact
// otherwise: an empty sum.)
template <class T>
__device__ __forceinline__ bool coarse(float lse, double temperature) {
  return __builtin_fabsf(lse) >= (sizeof(T) == 2 ? 1024.0f : 64.0f) &&
         !(lse == kNegInf && temperature >= 1.0);
}
template <class T>
__device__ __forceinline__ bool coarse_row(const DistillArgs &a, int64_t row) {
  return coarse<T>(a.lse[row], a.temperature) ||
         (a.rest && coarse<T>(a.lse_rest[row], a.temperature));
}

// The gradient of a whole row by one block, from sums of its own that it takes first, `part`
// values at a time (as many as e has bits for).  One block, because the gradient may take the
// logits' place.  With every row coarse (temperature 0.001) 4096 x 151,936 bf16 take 937 us (415
// with none), 4096 x 50,257 348 (142), 2049 x 32,000 fp32 188 (102), 16,384 x 1000 bf16 132 (30).
template <class T, int THREADS>
__device__ __forceinline__ void write_row_anew(const DistillArgs &a, int64_t row, int64_t part,
                                               Entries e, RowInfo *info,
                                               JoinLds<THREADS / kWave> &join) {
  const T *z = static_cast<const T *>(a.logits) + row * a.stride;
  T *grad = static_cast<T *>(a.grad) + row * a.grad_stride;
  const uint8_t *bytes = reinterpret_cast<const uint8_t *>(e.bits);
  const int thread = threadIdx.x, top = (int)a.top;
  if (thread < kWave) read_target<T, false>(a, row, 0, 0, 0, e, info, nullptr);
  RowSum own = {kNegInf, 0.0};
  for (int64_t lo = 0; lo < a.vocab; lo += part) {
    const int64_t hi = lo + part < a.vocab ? lo + part : a.vocab;
    __syncthreads();  // (the bits of the part before were read)
    if (thread < kWave) {
      for (int i = thread; i < (int)((hi - lo + 31) / 32); i += kWave) e.bits[i] = 0u;
      wave_sync();
      uint32_t again = 0;
      for (int j = thread; j < top; j += kWave) {
        const int32_t id = e.ids[j];
        if (id < lo || id >= hi) continue;
        const uint32_t at = (uint32_t)(id - lo), bit = 1u << (at & 31);
        if ((atomicOr(&e.bits[at >> 5], bit) & bit) != 0) again |= 1u << (j / kWave);
        e.z[j] = Chunk<T>::one(z[id]);
      }
      wave_sync();
      merge_repeated(top, e, again);
    }
    __syncthreads();
    Running run;
    const int n = (int)(hi - lo);
    for (int i = 8 * thread; i + 8 <= n; i += 8 * THREADS) {
      float v[8];
      Chunk<T> r;
      r.load(z + lo + i);
      r.values(v);
      leave_out(v, bytes[i >> 3]);
      const float ref = run.raise(max8(run.max, v), a.c);
      run.add(v, ref, a.c);
    }
    const int tail = n / 8 * 8 + thread;
    if (tail < n && (bytes[tail >> 3] >> (tail & 7) & 1) == 0) {
      const float one = Chunk<T>::one(z[lo + tail]);
      const float ref = run.raise(max3(run.max, one, kNegInf), a.c);
      run.sum += exp_scaled(one - ref, a.c);
    }
    const float m = max3(own.max, run.max, kNegInf);
    own = {m, moved(own.sum, own.max, ref_of(m), a.c) +
                  moved(run.sum, run.max, ref_of(m), a.c)};
  }
  const RowSum rest = block_join(own, a.c, join);
  if (thread < kWave) {
    float most = kNegInf;
    for (int j = thread; j < top; j += kWave)
      if (e.ids[j] >= 0) most = __builtin_fmaxf(most, e.z[j]);
    const RowSum named = named_sum(a, e, most);
    if (thread == 0) info->named = named;
  }
  __syncthreads();
  const Whole whole = both(rest, info->named, a.temperature);
  const Gradient g = gradient_of(*info, rest, whole.s, a.temperature);
  if (g.zero) {
    write_zeros(grad, 0, a.vocab, THREADS);
    return;
  }
  for (int64_t i = 8 * thread; i + 8 <= a.vocab; i += 8 * THREADS) {
    float v[8];
    Chunk<T> r;
    r.load(z + i);
    r.values(v);
    gradient_values<T>(v, g, a.c);
    Chunk<T>::store_once(grad + i, v);
  }
  const int64_t tail = a.vocab / 8 * 8 + thread;
  if (tail < a.vocab)
    Chunk<T>::store_one(grad + tail, gradient_value<T>(Chunk<T>::one(z[tail]), g, a.c));
  __syncthreads();
  if (thread < kWave)
    write_named<T>(a, grad, 0, a.vocab, e, *info, ref_of(whole.all.max) / a.temperature,
                   whole.all.sum == 0.0 ? 0.0 : 1.0 / whole.all.sum);
}

// The coarse rows among `index`, index + blocks, ... (64 of them) by a block, one after another.
// (They are shared out without a word between blocks; every wavefront finds the same ones.)
template <class T, int THREADS>
__device__ __forceinline__ void write_coarse_rows(const DistillArgs &a, uint32_t index,
                                                  uint32_t blocks, int64_t part, Entries e,
                                                  RowInfo *info,
                                                  JoinLds<THREADS / kWave> &join) {
  const int64_t mine = index + (int64_t)(threadIdx.x % kWave) * blocks;
  uint64_t left = __ballot(mine < a.rows && coarse_row<T>(a, mine) && a.grad_loss[mine] != 0.0f);
  for (; left != 0; left &= left - 1) {
    const uint32_t nth = __ffsll((unsigned long long)left) - 1;
    write_row_anew<T, THREADS>(a, index + nth * blocks, part, e, info, join);
    __syncthreads();  // (before e and *info are written again)
  }
}

// A block to a segment of a row: its gradient, from the statistics that were kept or, with
// PARTS, from the parts that distill_scan_kernel left (the first segment's block then also
// writes the row's loss and statistics).  The segment's values are in registers while the
// teacher's row is read.
//
// 2049 x 32,000 fp32: 102 us (5.1 TB/s of reads and writes; loads that stay in the caches
// 124 against 110 timed alike), 16,384 x 32,000 bf16 363 (5.8), 4096 x 151,936 bf16 415
// (6.0), 4096 x 50,257 bf16 142 (5.8; 179 and 149 without and with the alignment to cache lines,
// timed alike).  Its 80 registers leave 6 wavefronts to a SIMD; of 5, 1031 x 50,257 bf16 took 41.6
// us instead of 39.4.  With PARTS, 64 x 151,936 bf16: 9.9 us, latency as in the scan (11.8 with the
// parts joined by every wavefront behind the teacher's row, timed when it was 10.2).
template <class T, int THREADS, bool PARTS>
__global__ __launch_bounds__(THREADS) void distill_backward_kernel(const DistillArgs a,
                                                                   const uint32_t segs,
                                                                   const uint32_t blocks) {
  constexpr int N = distill_held_backward(sizeof(T));
  static_assert(!PARTS || THREADS >= 2 * kWave, "the second wavefront joins the parts");
  __shared__ RowInfo info;
  __shared__ Joined joined;
  __shared__ JoinLds<THREADS / kWave> join;
  Entries e(lds, a.top);
  if (!PARTS && blockIdx.x >= blocks) {
    write_coarse_rows<T, THREADS>(a, blockIdx.x - blocks, gridDim.x - blocks, 8 * THREADS * N, e,
                                  &info, join);
    return;
  }
  const int64_t row = blockIdx.x / segs;
  const uint32_t seg = blockIdx.x - (uint32_t)row * segs;
  const double T_ = a.temperature;
  constexpr int kLineValues = kLine / sizeof(T);
  const T *z = static_cast<const T *>(a.logits) + row * a.stride;
  T *grad = static_cast<T *>(a.grad) + row * a.grad_stride;
  // whole cache lines are shared out; the first segment has the values before them too, the
  // last those behind: one of each to a lane of the block's last wavefront
  const int lead = lead_of(z, a.vocab);
  const uint32_t lines = (uint32_t)(a.vocab - lead) / kLineValues;
  const uint32_t each = lines / segs, more = lines - each * segs;  // (the first `more` one more)
  const int64_t body = lead + (int64_t)(each * seg + (seg < more ? seg : more)) * kLineValues;
  const int n = (int)(each + (seg < more)) * kLineValues, thread = threadIdx.x;
  const int64_t end = body + n;
  const int64_t lo = seg == 0 ? 0 : body, hi = seg + 1 == segs ? a.vocab : end;
  Chunk<T> r[N];
#pragma unroll
  for (int k = 0; k < N; ++k) {
    const int i = 8 * (k * THREADS + thread);
    if (i < n) r[k].template load<true>(z + body + i);
  }
  if (thread < kWave) {
    read_target<T, false>(a, row, lo, hi, lo, e, &info, !PARTS && seg == 0 ? a.err : nullptr);
  } else if (PARTS && thread < 2 * kWave) {
    const Joined v = join_parts(a, row);
    if (thread == kWave) joined = v;
  }
  __syncthreads();
  Gradient g;
  Whole whole;
  double below, scale;
  if (PARTS) {
    whole = both(joined.rest, joined.named, T_);
    g = gradient_of(info, joined.rest, whole.s, T_);
    below = ref_of(whole.all.max) / T_;
    scale = whole.all.sum == 0.0 ? 0.0 : 1.0 / whole.all.sum;
  } else {
    // the unnamed: exp(z / T - base), base the log of their own sum, or of the whole one
    // without a class for the rest
    const double lse = a.lse[row], base = a.rest ? a.lse_rest[row] : lse;
    const bool empty = base == -__builtin_inf();
    g.ref = empty || base != base ? 0.0f : (float)(base * T_);
    double f = info.weight / T_ * info.m;
    if (a.rest)
      f = info.weight / T_ *
          ((info.m + info.r) * (empty ? 0.0 : exp64(base - lse)) - info.r);
    g.factor = uniform(empty ? 0.0f : (float)(f * exp64(g.ref / T_ - base)));
    g.zero = info.weight == 0.0f || info.none != 0;
    below = lse;
    scale = lse == -__builtin_inf() ? 0.0 : 1.0;
    if (!g.zero && coarse_row<T>(a, row)) return;  // (one of the last blocks has it)
  }
  if (PARTS && seg == 0 && thread == THREADS - 1)
    write_row(a, row, joined.rest, whole.all, joined.loss, info);
  if (g.zero) {
    write_zeros(grad, lo, hi, THREADS);
    return;
  }
  const int lane = thread - (THREADS - kWave);
  const bool before = lane >= 0 && lo + lane < body, behind = lane >= 0 && end + lane < hi;
  const float first = before ? Chunk<T>::one(z[lo + lane]) : kNegInf;
  const float last = behind ? Chunk<T>::one(z[end + lane]) : kNegInf;
#pragma unroll
  for (int k = 0; k < N; ++k) {
    const int i = 8 * (k * THREADS + thread);
    if (i < n) {
      float v[8];
      r[k].values(v);
      gradient_values<T>(v, g, a.c);
      Chunk<T>::store_once(grad + body + i, v);
    }
  }
  if (before) Chunk<T>::store_one(grad + lo + lane, gradient_value<T>(first, g, a.c));
  if (behind) Chunk<T>::store_one(grad + end + lane, gradient_value<T>(last, g, a.c));
  __syncthreads();
  if (thread < kWave) write_named<T>(a, grad, lo, hi, e, info, below, scale);
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
  return (size_t)top * kEntryBytes + (size_t)ceil_div(values + kLead, 32) * 4;
}

template <class T, int THREADS>
void enqueue_rows(const DistillArgs &a, hipStream_t stream) {
  const dim3 grid((unsigned)a.rows), block(THREADS);
  const size_t bytes = lds_bytes(a.top, a.vocab);
  if (a.grad != nullptr)
    hipLaunchKernelGGL((distill_row_kernel<T, THREADS, true>), grid, block, bytes, stream, a);
  else
    hipLaunchKernelGGL((distill_row_kernel<T, THREADS, false>), grid, block, bytes, stream, a);
}

// Blocks for the rows whose statistics are coarse: four to a CU, each of at most 64 rows.  They
// are the last ones of the launch and as a rule find nothing to do (2049 x 32,000 fp32 101.8 us,
// 103.1 without them; 4096 x 50,257 bf16 142.4 and 139.4).  Tried instead: the look at a row's
// statistics before each block's first chunks 107.9 and 143.5, a launch of its own 106.8 and 140.7
// and 2.5 us more for any call.
inline int64_t coarse_blocks(int64_t rows) {
  const int64_t least = ceil_div(rows, kWave), want = least < 1024 ? 1024 : least;
  return want < rows ? want : rows;
}
// (PARTS: none, the statistics are the call's own.)
template <class T, int THREADS, bool PARTS>
int enqueue_backward(const DistillArgs &a, hipStream_t stream) {
  const int64_t most = 8 * THREADS * distill_held_backward(sizeof(T));  // values
  const int64_t segs = ceil_div(a.vocab, most), blocks = a.rows * segs;
  const int64_t all = blocks + (PARTS ? 0 : coarse_blocks(a.rows));
  if (!grid_fits(all, kScanThreads)) return ENGRAM_EINVAL;
  hipLaunchKernelGGL((distill_backward_kernel<T, THREADS, PARTS>), dim3((unsigned)all),
                     dim3(THREADS), lds_bytes(a.top, most + 2 * kLead), stream, a, (uint32_t)segs,
                     (uint32_t)blocks);
  return launch_status();
}
// A row that a wavefront holds (8192 bytes) goes by one: 16,384 rows of 2000 bytes in bf16 29 us,
// by 256 threads 62, 8000 bytes 62 and 79 (fp32 28 and 58, 72 and 79); the teacher's row is each
// block's first work.  Longer ones take as long either way, and more for more entries in
// narrower blocks, each of which reads them: fp32 rows of 128,000 bytes 884 by 64 threads and
// 819 by 256.
template <class T>
int enqueue_kept(const DistillArgs &a, hipStream_t stream) {
  if (a.vocab <= 8 * kWave * distill_held_backward(sizeof(T)))
    return enqueue_backward<T, kWave, false>(a, stream);
  return enqueue_backward<T, kScanThreads, false>(a, stream);
}

// Threads of a row's block.  Few rows have a CU each and gain by every thread; of many, narrow
// blocks are quicker at what is not the vocabulary's, and more of them overlap.  us with / without
// a gradient, calls of a graph, bf16 (fp32 likewise by its bytes), 64 / 128 / 256 / 512 / 1024:
//   256 rows of 8000 bytes    11.6  10.0   9.1   9.6  11.2      8.6   7.7   7.3   7.5   8.0
//              24,000         19.6  14.5  12.2  11.7  11.7     13.0  10.2   8.9   8.4   8.5
//              64,000         36.4  24.1  17.2  14.9  15.0     21.9  15.6  11.8  10.6  10.6
//   1500 rows of 2000         11.3  12.3  14.9  21.4  35.6      8.4   9.1  10.4  14.2  22.9
//                8000         16.5  15.9  15.9  23.1  37.4     11.6  11.2  11.2  16.0  24.7
//              32,000         34.1  29.9  28.6  32.1  40.8     20.7  19.5  18.2  20.8  27.7
//   16,384 rows of 2000       41    59    90    178   334      29    41    61    123   217
//                8000         75    84    113   204   358      45    55    73    141   240
//              16,000         137   126   144   222   390      66    74    90    147   252
//              32,000         263   242   225   291   437      110   109   121   171   281
//              64,000         552   487   454   430   554      203   194   185   218   321
// With a gradient long rows are also kept from crowding each other out of the Infinity Cache
// before they are read again: 2048 of them are in flight by 256 threads, 1024 by 512 and 512 by
// 1024, up to 112 MB for rows of up to 110,000 bytes.  Longer ones have 512 in flight whatever
// their length: 156 MB at 303,872 bytes, all of the cache at 500,000, more than it holds above.
// 4096 rows, us by 256 / 512 / 1024 threads: 80,000 bytes 158 / 145 / 160, 120,000 253 / 230 / 218,
// 196,000 421 / 382 / 364, 303,872 646 / 548 / 538; by 1024, TB/s of the floor's bytes: 303,872
// 4.7, 496,640 4.7, 607,744 (2048 rows) 3.7, 993,280 3.7.
constexpr int64_t kDistillManyRows = 2048;
int distill_threads(int64_t rows, int64_t bytes, bool grad) {
  if (rows <= 256) return bytes <= 12000 ? 256 : bytes <= 48000 ? 512 : 1024;
  const bool many = rows > kDistillManyRows;
  if (bytes <= (!many ? 4000 : grad ? 9000 : 20000)) return 64;
  if (many && bytes <= (grad ? 20000 : 40000)) return 128;
  if (!grad || bytes <= 55000) return 256;
  return bytes <= 110000 ? 512 : 1024;
}

template <class T>
int enqueue(const engram_distill_args &h) {
  const ScanShape shape = distill_shape(h.rows, h.vocab);
  const DistillArgs plain = device_args(h, shape);
  const hipStream_t stream = as_stream(h.stream);
  const bool grad = h.d_grad != nullptr;
  if (!grid_fits(h.rows, 1024) || !grid_fits(h.rows * shape.segs, kScanThreads))
    return ENGRAM_EINVAL;
  if (!distill_cut(h.rows, h.vocab, grad)) {
    switch (distill_threads(h.rows, h.vocab * (int64_t)sizeof(T), grad)) {
      case 64: enqueue_rows<T, 64>(plain, stream); break;
      case 128: enqueue_rows<T, 128>(plain, stream); break;
      case 256: enqueue_rows<T, 256>(plain, stream); break;
      case 512: enqueue_rows<T, 512>(plain, stream); break;
      default: enqueue_rows<T, 1024>(plain, stream);
    }
    return launch_status();
  }
  DistillArgs a = plain;
  a.parts = static_cast<DistillPart *>(h.d_workspace);
  hipLaunchKernelGGL(distill_scan_kernel<T>, dim3((unsigned)(h.rows * shape.segs)),
                     dim3(kScanThreads), lds_bytes(h.top, shape.seg_len), stream, a);
  if (grad) return enqueue_backward<T, kScanThreads, true>(a, stream);
  hipLaunchKernelGGL(distill_finish_kernel<T>, dim3((unsigned)h.rows), dim3(kWave),
                     lds_bytes(h.top, 0), stream, a);
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
  return h.logits_type == ENGRAM_BF16 ? enqueue_kept<uint16_t>(a, stream)
                                      : enqueue_kept<float>(a, stream);
}
