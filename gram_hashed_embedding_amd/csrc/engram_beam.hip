// engram_beam.hip -- beam search: the selection over beams and vocabulary, and
// the reordering of the decoding states after it, for gfx950.  What is computed
// is stated with engram_beam_select and engram_beam_fork in include/
// engram_vocab.h.
//
// Selection.  One pass over the logits (beam_scan_kernel) leaves each segment's
// sum of exponentials and the largest logit of every kBeamGroup adjacent
// values.  The `count` best candidates lie in the `count` best groups (by their
// largest value, equal ones by place: the candidate before which `count` others
// come cannot be one of the first `count`), so beam_choose_kernel, a block to a
// sequence, finds those among 1/128 of the values, reads them again and takes
// the best of `count` times 128 candidates.  Both choices are exact in fp64.
//
// Reordering.  A new beam that is the first child of its parent keeps the
// parent's slot; only the others' states are copied, into slots of beams that
// ended.  Every block works the order out for itself from one wavefront's
// ballots, so one launch does all of it and nothing is read that is written.
#include "engram_vocab_dev.h"

namespace engram {
namespace {

// ------------------------------------------------------------------- scan --
struct ScanArgs {
  const void *logits;
  int64_t vocab, stride, segs, seg_len, groups;
  Scale c;
  const float *scores;
  const uint8_t *finished;
  ScanPart *parts;
  float *maxima;
};

// Whether a beam's logits are needed.
__device__ __forceinline__ bool beam_live(const float *scores, const uint8_t *finished,
                                          int64_t row) {
  return __builtin_isfinite(scores[row]) && (finished == nullptr || finished[row] == 0);
}

// A block to a segment of a beam's logits.  Memory bounds it: 512 beams of 151,936 bf16 values
// are read in 29 to 32 us (5.4 to 4.9 TB/s); 4 chunks a lane and step instead of 2 are no faster.
// The groups' maxima wait in LDS and are written 4 bytes a lane next to each other at the end, not
// by every 16th lane in between.  Chunks start with the row, wherever it lies, so that beams with
// equal logits have equal sums to the last bit and tie as they should; from whole cache lines on
// a selection among 4096 beams of 50,257 bf16 values takes 95 us instead of 106, of 50,256 94
// instead of 98, 512 beams of 151,935 43.5 instead of 47.7.  One beam or a few: 4 to 6 us, a
// block's own latency.
template <class T>
__global__ __launch_bounds__(kScanThreads) void beam_scan_kernel(const ScanArgs a) {
  __shared__ JoinLds<kScanThreads / kWave> join;
  __shared__ float most_of[kBeamMaxSeg / kBeamGroup];
  const int64_t row = blockIdx.x / a.segs, seg = blockIdx.x - row * a.segs;
  if (!beam_live(a.scores, a.finished, row)) return;
  const T *z = static_cast<const T *>(a.logits) + row * a.stride;
  const int64_t lo = seg * a.seg_len, hi = lo + a.seg_len < a.vocab ? lo + a.seg_len : a.vocab;
  float *maxima = a.maxima + row * a.groups;
  constexpr int U = sizeof(T) == 2 ? 2 : 1;
  Running run;
  each_chunks<T, kScanThreads, U, true>(z, lo, hi, [] {}, [&](int64_t at, float (&z)[U][8]) {
    float m = run.max;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const float own = max8(kNegInf, z[u]);
      m = max3(m, own, kNegInf);
      const float most = lanes_max_of<16>(own);
      const int64_t i = at + u * kScanTile + 8 * threadIdx.x;
      if (threadIdx.x % 16 == 0 && i < hi) most_of[(i - lo) / kBeamGroup] = most;
    }
    const float ref = run.raise(m, a.c);
#pragma unroll
    for (int u = 0; u < U; ++u) run.add(z[u], ref, a.c);
  });
  const RowSum s = block_join(run, a.c, join);  // (with a barrier)
  const int n = (int)((hi - lo + kBeamGroup - 1) / kBeamGroup);
  for (int i = threadIdx.x; i < n; i += kScanThreads) maxima[lo / kBeamGroup + i] = most_of[i];
  if (threadIdx.x == 0) a.parts[row * a.segs + seg] = {s.sum, s.max, 0u};
}

// ----------------------------------------------------------------- choice --
constexpr int kChooseThreads = 1024;
constexpr int kChooseList = 2048;
constexpr int kChooseGroups = 96;  // (at least ENGRAM_BEAM_MAX; kKeep values a thread)

// A candidate: its value, and its place among all of them.
struct Candidate {
  double value;
  int64_t at;
};
__device__ __forceinline__ bool before(const Candidate &x, const Candidate &y) {
  return x.value > y.value || (x.value == y.value && x.at < y.at);
}
constexpr double kNone = -__builtin_inf();

struct ChooseLds {
  Candidate list[kChooseList];
  Candidate best[ENGRAM_BEAM_MAX];  // the answer, in order
  Candidate wave_best[kChooseThreads / kWave];
  uint32_t row_best[kChooseThreads / 16];
  int listed;
};

// Bits that order as the values do (rounded down to fp32), and a value that has at least
// these bits.
__device__ __forceinline__ uint32_t order_bits(double v) {
  const uint32_t u = __float_as_uint(__double2float_rd(v));
  return u ^ ((u >> 31) != 0 ? 0xffffffffu : 0x80000000u);
}
constexpr uint32_t kNoneBits = 0x007fffffu;  // of kNone
__device__ __forceinline__ double value_of_bits(uint32_t k) {
  if (k <= kNoneBits) return kNone;
  return __uint_as_float(k ^ ((k >> 31) != 0 ? 0x80000000u : 0xffffffffu));
}

// Lists the candidates 0 .. n-1 of which the first `count` are some, in l.list in no order;
// gives their number.  logit(i) loads what value(i, logit) is made of (kNone where there is
// no candidate); place(i) is what equal values are ordered by; meanwhile() is done while
// the first loads are on their way and ends in a barrier.
//
// A threshold first: of the largest values of 64 rows of 16 threads, the count-th
// largest has at least `count` values at or above it (its leading 20 bits are enough,
// found bit by bit from ballots).  What reaches it is listed.  Where that is more than
// the list holds (long runs of equal values), the first `count` are listed one at a
// time instead, each the first after the one before: where a mask of a large finite value
// leaves fewer ids than are asked for, 16 of 4 beams of 151,936 take 0.9 ms instead of 17 us,
// 64 of 64 beams 2.5 ms instead of 96 us (a mask of -inf has no such candidates).  A thread
// keeps its first kKeep values; their loads go out together.
constexpr int kKeep = 12;
template <class LOGIT, class VALUE, class PLACE, class MEANWHILE>
__device__ __forceinline__ int list_best(ChooseLds &l, int n, int count, LOGIT logit, VALUE value,
                                         PLACE place, MEANWHILE meanwhile) {
  const int t = threadIdx.x;
  float raw[kKeep];
#pragma unroll
  for (int k = 0; k < kKeep; ++k) {
    const int i = t + k * kChooseThreads;
    if (k * kChooseThreads < n) raw[k] = logit(i < n ? i : n - 1);
  }
  if (t == 0) l.listed = 0;
  meanwhile();
  double kept[kKeep], mine = kNone;
#pragma unroll
  for (int k = 0; k < kKeep; ++k) {
    const int i = t + k * kChooseThreads;
    kept[k] = kNone;
    if (k * kChooseThreads < n && i < n) kept[k] = value(i, raw[k]);
    mine = fmax(mine, kept[k]);
  }
  for (int i = t + kKeep * kChooseThreads; i < n; i += kChooseThreads)
    mine = fmax(mine, value(i, logit(i)));
  const uint32_t row = lanes_max<16>(order_bits(mine));
  if (t % 16 == 0) l.row_best[t / 16] = row;
  __syncthreads();
  const uint32_t of_row = l.row_best[t % kWave];
  uint32_t bits = 0;
#pragma unroll
  for (int b = 31; b >= 12; --b) {
    const uint32_t test = bits | 1u << b;
    if (__popcll(__ballot(of_row >= test)) >= count) bits = test;
  }
  const double least = value_of_bits(bits);
  const auto list = [&](int i, double v) {
    if (v > kNone && v >= least) {
      const int k = atomicAdd(&l.listed, 1);
      if (k < kChooseList) l.list[k] = {v, place(i)};
    }
  };
  if (mine > kNone && mine >= least) {
#pragma unroll
    for (int k = 0; k < kKeep; ++k) list(t + k * kChooseThreads, kept[k]);
    for (int i = t + kKeep * kChooseThreads; i < n; i += kChooseThreads)
      list(i, value(i, logit(i)));
  }
  __syncthreads();
  const int listed = l.listed;
  if (listed <= kChooseList) return listed;
  // (at least `count` candidates there)
  Candidate last = {__builtin_inf(), -1};
  for (int r = 0; r < count; ++r) {
    Candidate m = {kNone, INT64_MAX};
    for (int i = t; i < n; i += kChooseThreads) {
      const double v = value(i, logit(i));
      if (v > kNone && v <= last.value && v >= m.value) {
        const Candidate c = {v, place(i)};
        if (before(last, c) && before(c, m)) m = c;
      }
    }
#pragma unroll
    for (int d = 1; d < kWave; d *= 2) {
      const Candidate o = {__shfl_xor(m.value, d), __shfl_xor(m.at, d)};
      if (before(o, m)) m = o;
    }
    if (t % kWave == 0) l.wave_best[t / kWave] = m;
    __syncthreads();
    last = l.wave_best[0];
    for (int w = 1; w < kChooseThreads / kWave; ++w)
      if (before(l.wave_best[w], last)) last = l.wave_best[w];
    if (t == 0) l.list[r] = last;
    __syncthreads();
  }
  return count;
}

// The first `count` of the listed candidates, in order, in l.best: each one's rank is the
// number of those before it, counted by a wavefront.
__device__ __forceinline__ void rank_listed(ChooseLds &l, int listed, int count) {
  const int lane = threadIdx.x % kWave;
  for (int k = threadIdx.x / kWave; k < listed; k += kChooseThreads / kWave) {
    const Candidate c = l.list[k];
    int ahead = 0;
    for (int o = lane; o - lane < listed; o += kWave)
      ahead += __popcll(__ballot(o < listed && before(l.list[o], c)));
    if (lane == 0 && ahead < count) l.best[ahead] = c;
  }
  __syncthreads();
}

struct ChooseArgs {
  BeamCall c;
  int64_t segs, groups;
  uint32_t per_group;  // (2^32 - 1) / groups, rounded down
  Scale log2e;
};

// A block to a sequence.  Its bytes are few (8 beams of 151,936 values: 38 KB of maxima and 24
// KB of groups read again): it is a chain of loads, barriers and ballots, 10.1 us for 4 beams
// and 14.2 for 64 sequences of 8, so it runs once whatever the batch.  What shortened it: the
// loads of a pass all sent before the first is used and behind the beams' sums, no division
// of 64 bits, and the first choice's groups left unordered (21 to 23 us -> 14).  Of 512
// threads, tried before that, a whole selection took 56 us where it took 50 of 1024.
template <class T>
__global__ __launch_bounds__(kChooseThreads) void beam_choose_kernel(const ChooseArgs a) {
  __shared__ ChooseLds l;
  // lse, in two parts: beside a mask's lowest value nothing would be left of the sum's logarithm
  __shared__ double top[ENGRAM_BEAM_MAX];    // the largest logit
  __shared__ double lse[ENGRAM_BEAM_MAX];    // from there; NaN: no candidate but a finished beam's
  __shared__ double score[ENGRAM_BEAM_MAX];
  __shared__ bool done[ENGRAM_BEAM_MAX];     // (out_scores and out_finished may be the inputs)
  __shared__ int64_t group_at[kChooseGroups];  // of each chosen group: its first value
  __shared__ int64_t group_end[kChooseGroups];  // what it ends before
  __shared__ int group_beam[kChooseGroups];
  const BeamCall &c = a.c;
  const int64_t b = blockIdx.x, first_row = b * c.beams;
  const int t = threadIdx.x, beams = (int)c.beams, count = (int)c.count;
  const int groups = (int)a.groups;
  const auto value_of = [&](int w, float z) {
    const double v = score[w] + (((double)z - top[w]) - lse[w]);
    return v == v ? v : kNone;
  };
  // i / groups by the whole part of (2^32 - 1) / groups, which is at most one too small
  const auto beam_of = [&](uint32_t i) {
    const uint32_t w = __umulhi(i, a.per_group);
    return (int)(i - w * groups >= (uint32_t)groups ? w + 1 : w);
  };
  // the best groups; a finished beam's candidate is a group of its own (its first)
  int chosen = list_best(
      l, beams * groups, count,
      // (of beams that were not scanned whatever the memory holds)
      [&](int i) { return c.maxima[first_row * groups + i]; },
      [&](int i, float z) {
        const int w = beam_of(i);
        if (lse[w] == lse[w]) return value_of(w, z);
        return i == w * groups && done[w] ? score[w] : kNone;
      },
      [&](int i) { return (int64_t)i; },
      [&] {
        // each beam's lse, a wavefront to a beam
        for (int w = t / kWave; w < beams; w += kChooseThreads / kWave) {
          const int64_t row = first_row + w;
          double m = 0.0, v = __builtin_nan("");
          if (beam_live(c.scores, c.finished, row)) {
            const RowSum sum = wave_join(c.parts + row * a.segs, a.segs, a.log2e);
            m = sum.max;
            v = log64(sum.sum);
            if (!__builtin_isfinite(m) || !__builtin_isfinite(v)) v = __builtin_nan("");
          }
          if (t % kWave == 0) {
            top[w] = m;
            lse[w] = v;
            score[w] = c.scores[row];
            done[w] = c.finished != nullptr && c.finished[row] != 0 &&
                      __builtin_isfinite(c.scores[row]);
          }
        }
        __syncthreads();
      });
  // more than a few are cut to the first `count`
  const bool ranked = chosen > kChooseGroups;
  if (ranked) {
    rank_listed(l, chosen, count);
    chosen = chosen < count ? chosen : count;
  }
  if (t < chosen) {
    const int at = (int)(ranked ? l.best[t].at : l.list[t].at), w = beam_of(at);
    const int g = at - w * groups;
    group_beam[t] = w;
    group_at[t] = (int64_t)g * kBeamGroup;
    // (of a finished beam nothing is read)
    group_end[t] = lse[w] != lse[w] ? 0 : c.vocab;
  }
  __syncthreads();
  const int listed = list_best(
      l, chosen * (int)kBeamGroup, count,
      [&](int i) {
        const int w = group_beam[i / kBeamGroup];
        const int64_t v = group_at[i / kBeamGroup] + i % kBeamGroup;
        const T *z = static_cast<const T *>(c.logits) + (first_row + w) * c.stride;
        return v < group_end[i / kBeamGroup] ? Chunk<T>::one(z[v]) : kNegInf;
      },
      [&](int i, float z) {
        const int w = group_beam[i / kBeamGroup];
        if (lse[w] == lse[w]) return value_of(w, z);
        return i % kBeamGroup == 0 ? score[w] : kNone;
      },
      [&](int i) {
        const int w = group_beam[i / kBeamGroup];
        return w * c.vocab + (lse[w] != lse[w] ? c.eos : group_at[i / kBeamGroup] + i % kBeamGroup);
      },
      [] { __syncthreads(); });
  rank_listed(l, listed, count);
  if (t < count) {
    const bool there = t < listed;
    const Candidate best = l.best[there ? t : 0];
    const int64_t w = there ? best.at / c.vocab : -1, v = there ? best.at - w * c.vocab : -1;
    const int64_t o = b * count + t;
    c.out_scores[o] = there ? (float)best.value : kNegInf;
    c.out_parents[o] = w;
    c.out_tokens[o] = v;
    if (c.out_finished != nullptr)
      c.out_finished[o] = there && (v == c.eos || done[w]);
  }
}

// ------------------------------------------------------------- reordering --
constexpr int kForkThreads = 256;
constexpr int kForkSteps = 4;
constexpr int64_t kForkChunk = (int64_t)kForkThreads * kForkSteps * 16;  // bytes a block copies

// Blocks: `chunks` of every new beam (the pools' slots one after another); the first
// of them also writes the beam's slot and history.  A block copies 16 KB, 4 loads of 16
// bytes in flight a lane.  64 x 8 beams with slots of 192 KB, of which about a third are
// copied: 13.5 us, 5.2 TB/s (70 MB in all, too few for more); a few beams 3.9 us, a launch's
// latency.
__global__ __launch_bounds__(kForkThreads) void beam_fork_kernel(const ForkCall c,
                                                                 const int64_t chunks) {
  const int64_t entry = blockIdx.x / chunks;
  int64_t chunk = blockIdx.x - entry * chunks;
  const int64_t b = entry / c.beams;
  const int j = (int)(entry - b * c.beams), lane = threadIdx.x % kWave;
  const int beams = (int)c.beams;
  int64_t raw = -1, slot = -1;  // a lane to a beam
  if (lane < beams) {
    raw = c.parents[b * beams + lane];
    slot = c.slots != nullptr ? c.slots[b * beams + lane] : b * beams + lane;
  }
  const bool valid = raw >= 0 && raw < beams;
  const int parent = valid ? (int)raw : -1;
  uint64_t keeps = 0, bare = 0;  // first children; old beams without a child
  for (int w = 0; w < beams; ++w) {
    const uint64_t children = __ballot(parent == w);
    if (children != 0)
      keeps |= children & -children;
    else
      bare |= uint64_t(1) << w;
  }
  const int from = __shfl(parent, j);
  const int64_t source = from >= 0 ? __shfl(slot, from) : -1;
  int to = from;
  if (!(keeps >> j & 1)) {
    // as many new beams before j keep nothing as bare beams come before its own
    int skip = __popcll(~keeps & ((uint64_t(1) << j) - 1));
    uint64_t left = bare;
    while (skip-- > 0) left &= left - 1;
    to = __ffsll((unsigned long long)left) - 1;
  }
  const int64_t target = __shfl(slot, to);
  if (chunk == 0) {
    if (threadIdx.x == 0) c.new_slots[entry] = target;
    if (threadIdx.x < kWave && lane == j) {
      const int bad = (!valid && raw != -1) + (c.pool_count > 0 && slot != -1 &&
                                               (slot < 0 || slot >= c.slot_count));
      count_errors(bad, c.err);
    }
    if (c.new_history != nullptr) {
      const int64_t row = b * beams + (from >= 0 ? from : j);
      const int64_t drop = c.history_len + 1 - c.new_len;
      for (int64_t i = threadIdx.x; i < c.new_len; i += kForkThreads)
        c.new_history[entry * c.new_len + i] =
            i + 1 == c.new_len ? c.tokens[entry] : c.history[row * c.history_len + drop + i];
    }
  }
  if (source < 0 || source >= c.slot_count || target < 0 || target >= c.slot_count ||
      source == target)
    return;
  for (int p = 0; p < c.pool_count; ++p) {
    const int64_t bytes = c.slot_bytes[p], mine = (bytes + kForkChunk - 1) / kForkChunk;
    if (chunk >= mine) {
      chunk -= mine;
      continue;
    }
    const u32x4 *in = reinterpret_cast<const u32x4 *>(static_cast<char *>(c.pools[p]) +
                                                      source * bytes);
    u32x4 *out = reinterpret_cast<u32x4 *>(static_cast<char *>(c.pools[p]) + target * bytes);
    const int64_t n = bytes / 16, at = chunk * (kForkChunk / 16) + threadIdx.x;
    u32x4 v[kForkSteps];
#pragma unroll
    for (int k = 0; k < kForkSteps; ++k)
      if (at + k * kForkThreads < n) v[k] = in[at + k * kForkThreads];
#pragma unroll
    for (int k = 0; k < kForkSteps; ++k)
      if (at + k * kForkThreads < n) out[at + k * kForkThreads] = v[k];
    return;
  }
}

}  // namespace
}  // namespace engram

int engram::launch_beam_select(const BeamCall &c, void *stream) {
  const int64_t rows = c.batch * c.beams;
  const ScanShape shape = beam_shape(rows, c.vocab);
  if (!grid_fits(rows * shape.segs, kScanThreads) || !grid_fits(c.batch, kChooseThreads))
    return ENGRAM_EINVAL;
  const Scale log2e = scale_of(1.0);
  const int64_t groups = beam_groups(c.vocab);
  const ScanArgs s = {c.logits, c.vocab, c.stride, shape.segs, shape.seg_len, groups, log2e,
                      c.scores, c.finished, c.parts, c.maxima};
  const ChooseArgs a = {c, shape.segs, groups,
                        (uint32_t)(0xffffffffu / groups), log2e};
  const dim3 grid((unsigned)(rows * shape.segs)), block(kScanThreads);
  const dim3 sequences((unsigned)c.batch), wide(kChooseThreads);
  if (c.type == ENGRAM_BF16) {
    hipLaunchKernelGGL(beam_scan_kernel<uint16_t>, grid, block, 0, as_stream(stream), s);
    hipLaunchKernelGGL(beam_choose_kernel<uint16_t>, sequences, wide, 0, as_stream(stream), a);
  } else {
    hipLaunchKernelGGL(beam_scan_kernel<float>, grid, block, 0, as_stream(stream), s);
    hipLaunchKernelGGL(beam_choose_kernel<float>, sequences, wide, 0, as_stream(stream), a);
  }
  return launch_status();
}

int engram::launch_beam_fork(const ForkCall &c, void *stream) {
  int64_t chunks = 0;
  for (int p = 0; p < c.pool_count; ++p) chunks += ceil_div(c.slot_bytes[p], kForkChunk);
  if (chunks < 1) chunks = 1;
  const int64_t entries = c.batch * c.beams;
  if (!mul_fits(entries, chunks, kMaxGridItems) || !grid_fits(entries * chunks, kForkThreads))
    return ENGRAM_EINVAL;
  hipLaunchKernelGGL(beam_fork_kernel, dim3((unsigned)(entries * chunks)), dim3(kForkThreads), 0,
                     as_stream(stream), c, chunks);
  return launch_status();
}
