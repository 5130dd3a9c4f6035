// engram_embed.hip -- the scaled token embedding and its gradient by sorted
// tokens, for gfx950.
//
// What is computed is stated with engram_embed in include/engram_layer.h: the
// ordinary token table beside the hashed one, its rows scaled on the way out,
// and the gradient of the whole table.
//
// Bound by HBM.  The forward reads a row and writes one; the gradient's
// floor is one write of the whole table beside one read of the tokens'
// gradients, and most rows of a vocabulary have no token in a batch.
//
// The gradient.  The tokens are sorted as the hashed rows are (the plan of
// engram_sort.hip), so a row's terms are one run of the sorted order and no
// atomic is needed: the result does not depend on timing, and each row is
// written once.  Walkers take equal chunks of the sorted positions, however
// the tokens crowd: a run inside a chunk is summed and written by its walker;
// a run that crosses chunks leaves a part in each, which the walker of the
// chunk it begins in adds up in a second, short kernel.  Beside the walkers,
// in the same launch, the other blocks write the zeros of the rows without a
// token (most of a vocabulary), found by a 64-way search of the sorted tokens
// a block.  Sums are fp64, as the hashed table's.
#include "engram_layer_dev.h"
#include "engram_scatter_dev.h"

namespace engram {
namespace {

constexpr int kEmbedThreads = 256;
constexpr int kEmbedRows = 4;  // rows of a lane in flight

template <class OUT>
__device__ __forceinline__ void store8(OUT *row, int64_t chunk, const float (&f)[8]);
template <>
__device__ __forceinline__ void store8<uint16_t>(uint16_t *row, int64_t chunk,
                                                 const float (&f)[8]) {
  __builtin_nontemporal_store(pack_bf16x8(f), reinterpret_cast<u32x4 *>(row) + chunk);
}
template <>
__device__ __forceinline__ void store8<float>(float *row, int64_t chunk, const float (&f)[8]) {
  f32x4 *q = reinterpret_cast<f32x4 *>(row) + 2 * chunk;
  q[0] = f32x4{f[0], f[1], f[2], f[3]};
  q[1] = f32x4{f[4], f[5], f[6], f[7]};
}

template <class OUT>
__global__ __launch_bounds__(kEmbedThreads) void embed_kernel(
    const int64_t *__restrict__ tokens, int64_t n, const u32x4 *__restrict__ table,
    int64_t table_rows, int64_t chunks, int lanes, float scale, OUT *__restrict__ out,
    int64_t *err) {
  const int slots = kEmbedThreads / lanes;
  const int slot = threadIdx.x / lanes, lane = threadIdx.x % lanes;
  const int64_t first = (int64_t)blockIdx.x * slots * kEmbedRows + slot;
  int64_t row[kEmbedRows];
  int bad = 0;
#pragma unroll
  for (int k = 0; k < kEmbedRows; ++k) {
    const int64_t t = first + k * slots;
    row[k] = t < n ? tokens[t] : -1;
    if (row[k] < 0 || row[k] >= table_rows) {
      bad += lane == 0 && row[k] != -1 ? 1 : 0;
      row[k] = -1;
    }
  }
  count_errors(bad, err);
  for (int64_t c = lane; c < chunks; c += lanes) {
    u32x4 v[kEmbedRows];
#pragma unroll
    for (int k = 0; k < kEmbedRows; ++k)
      v[k] = row[k] >= 0 ? table[row[k] * chunks + c] : u32x4{0u, 0u, 0u, 0u};
#pragma unroll
    for (int k = 0; k < kEmbedRows; ++k) {
      const int64_t t = first + k * slots;
      if (t >= n) continue;
      float f[8];
      unpack_bf16x8(v[k], f);
#pragma unroll
      for (int e = 0; e < 8; ++e) f[e] = row[k] >= 0 ? f[e] * scale : 0.0f;
      store8<OUT>(out + t * chunks * 8, c, f);
    }
  }
}

// ---------------------------------------------------------------- gradient --
// A row of `chunks` chunks of 8 channels is covered by `lanes` threads (a
// power of two, at most a block).
struct EmbedGradArgs {
  const uint32_t *keys, *vals;  // sorted tokens and their positions
  const PlanScalars *plan;      // of the sort, or null (sorted without one)
  const void *grads;
  double *partials;  // [walks][2][channels]: of the run that enters, that leaves
  int64_t n, chunks, table_rows;
  int64_t walks, walk_len, walk_blocks;
  int lanes, rows_per_block;
  float scale;
  void *out;
};

// Whether the order is valid (a wait of the sort that expired has marked the
// error counter; nothing is read by such an order, and nothing written).
__device__ __forceinline__ bool order_holds(const EmbedGradArgs &g) {
  return g.plan == nullptr || g.plan->stalled == 0;
}

// A few thousand tokens are sorted by counting, in one launch: a token's place
// is the number of smaller ones, and of equal ones before it.  A block places
// kRankBlock tokens; its threads are kRankBlock tokens wide and share out the
// tokens to compare with, four at a time from LDS.  n^2 comparisons over the
// whole GPU beat the sort's passes, which wait on one another, up to
// kRankTokens.
constexpr int kRankThreads = 1024, kRankBlock = 16, kRankParts = kRankThreads / kRankBlock;
constexpr int64_t kRankTokens = 8192;

__global__ __launch_bounds__(kRankThreads) void embed_rank_kernel(
    const int64_t *__restrict__ tokens, int n, uint32_t table_rows, uint32_t *keys,
    uint32_t *vals, int64_t *err) {
  __shared__ u32x4 s_key4[kRankTokens / 4];
  __shared__ uint32_t s_count[kRankParts][kRankBlock];
  uint32_t *s_key = reinterpret_cast<uint32_t *>(s_key4);
  const int i0 = blockIdx.x * kRankBlock;
  int bad = 0;
  for (int j = threadIdx.x; j < ((n + 3) & ~3); j += kRankThreads) {
    uint32_t k = 0xffffffffu;  // past the end: above every key
    if (j < n) {
      const int64_t t = tokens[j];
      const bool ok = t >= 0 && t < (int64_t)table_rows;
      k = ok ? (uint32_t)t : table_rows;
      bad += !ok && t != -1 && j >= i0 && j < i0 + kRankBlock ? 1 : 0;
    }
    s_key[j] = k;
  }
  count_errors(bad, err);
  __syncthreads();
  const int lane = threadIdx.x % kRankBlock, part = threadIdx.x / kRankBlock;
  const int i = i0 + lane;
  const uint32_t key = i < n ? s_key[i] : 0u;
  const int quads = (n + 3) / 4;
  uint32_t count = 0;
  // the block's own tokens lie in quads [i0 / 4, i0 / 4 + kRankBlock / 4)
  for (int q = part; q < quads; q += kRankParts) {
    const u32x4 k = s_key4[q];
    if (q < i0 / 4) {
      count += (k.x <= key) + (k.y <= key) + (k.z <= key) + (k.w <= key);
    } else if (q >= i0 / 4 + kRankBlock / 4) {
      count += (k.x < key) + (k.y < key) + (k.z < key) + (k.w < key);
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint32_t other = e == 0 ? k.x : e == 1 ? k.y : e == 2 ? k.z : k.w;
        count += other < key || (other == key && q * 4 + e < i) ? 1u : 0u;
      }
    }
  }
  s_count[part][lane] = count;
  __syncthreads();
  if (threadIdx.x >= kRankBlock || i >= n) return;
  uint32_t place = 0;
#pragma unroll
  for (int p = 0; p < kRankParts; ++p) place += s_count[p][lane];
  keys[place] = key;
  vals[place] = (uint32_t)i;
}

template <class OUT, bool ACCUMULATE>
__device__ __forceinline__ void write_row(const EmbedGradArgs &g, int64_t row, int64_t c,
                                          const double (&sum)[8]) {
  OUT *dst = static_cast<OUT *>(g.out) + row * g.chunks * 8;
  float f[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) f[e] = (float)(sum[e] * (double)g.scale);
  if (ACCUMULATE) {
    const float *old = reinterpret_cast<const float *>(dst) + c * 8;
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] = old[e] + f[e];
  }
  store8<OUT>(dst, c, f);
}

__device__ __forceinline__ void write_part(const EmbedGradArgs &g, int64_t walk, int which,
                                           int64_t c, const double (&sum)[8]) {
  f64x2 *dst = reinterpret_cast<f64x2 *>(g.partials + ((walk * 2 + which) * g.chunks + c) * 8);
#pragma unroll
  for (int e = 0; e < 4; ++e) dst[e] = f64x2{sum[2 * e], sum[2 * e + 1]};
}

// A walker's chunk [a, b) of the sorted positions: its runs' sums.
// Eight values of a gradient row, bf16 (uint16_t) or float.
template <class G>
struct GradRow;
template <>
struct GradRow<uint16_t> {
  static constexpr int kAhead = 8;  // rows in flight
  typedef u32x4 Raw;
  static __device__ __forceinline__ Raw load(const void *p, int64_t chunk) {
    return static_cast<const u32x4 *>(p)[chunk];
  }
  static __device__ __forceinline__ void unpack(const Raw &r, float (&f)[8]) {
    unpack_bf16x8(r, f);
  }
};
template <>
struct GradRow<float> {
  static constexpr int kAhead = 4;
  struct Raw {
    f32x4 a, b;
  };
  static __device__ __forceinline__ Raw load(const void *p, int64_t chunk) {
    const f32x4 *q = static_cast<const f32x4 *>(p) + 2 * chunk;
    return Raw{q[0], q[1]};
  }
  static __device__ __forceinline__ void unpack(const Raw &r, float (&f)[8]) {
    f[0] = r.a.x; f[1] = r.a.y; f[2] = r.a.z; f[3] = r.a.w;
    f[4] = r.b.x; f[5] = r.b.y; f[6] = r.b.z; f[7] = r.b.w;
  }
};

template <class G, class OUT, bool ACCUMULATE>
__device__ void walk_chunk(const EmbedGradArgs &g, int64_t walk, int lane) {
  const int64_t a = walk * g.walk_len, b = min(a + g.walk_len, g.n);
  const uint32_t before = a > 0 ? g.keys[a - 1] : 0xffffffffu;  // no key (they are smaller)
  const uint32_t after = b < g.n ? g.keys[b] : 0xffffffffu;
  for (int64_t c = lane; c < g.chunks; c += g.lanes) {
    double sum[8] = {0.0, 0.0, 0.0, 0.0, 0.0, 0.0, 0.0, 0.0};
    uint32_t run = g.keys[a];
    bool entered = run == before;
    constexpr int kAhead = GradRow<G>::kAhead;
    for (int64_t i = a; i < b; i += kAhead) {
      uint32_t key[kAhead];
      typename GradRow<G>::Raw v[kAhead];
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        const int64_t at = min(i + k, b - 1);
        key[k] = g.keys[at];
        v[k] = GradRow<G>::load(g.grads, (int64_t)g.vals[at] * g.chunks + c);
      }
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        if (i + k >= b) break;
        if (key[k] != run) {  // a run has ended in this chunk
          if (run < g.table_rows) {
            if (entered)
              write_part(g, walk, 0, c, sum);
            else
              write_row<OUT, ACCUMULATE>(g, run, c, sum);
          }
          run = key[k];
          entered = false;
#pragma unroll
          for (int e = 0; e < 8; ++e) sum[e] = 0.0;
        }
        float f[8];
        GradRow<G>::unpack(v[k], f);
#pragma unroll
        for (int e = 0; e < 8; ++e) sum[e] += f[e];
      }
    }
    if (run >= g.table_rows) continue;  // padding and invalid ids sort last
    if (entered)
      write_part(g, walk, 0, c, sum);
    else if (run == after)
      write_part(g, walk, 1, c, sum);
    else
      write_row<OUT, ACCUMULATE>(g, run, c, sum);
  }
}

// The first sorted position in [lo, n) whose key is at least `key` (a
// wavefront together: 64 probes a step).
__device__ __forceinline__ int64_t lower_bound(const EmbedGradArgs &g, int64_t lo, int64_t key) {
  int64_t hi = g.n;
  while (lo < hi) {
    const int64_t step = (hi - lo + 63) / 64;
    const int64_t at = lo + ((int64_t)(threadIdx.x & 63) + 1) * step - 1;
    const bool below = at < hi && (int64_t)g.keys[at] < key;
    const int64_t passed = __popcll(__ballot(below));  // probes below are the first ones
    lo = min(lo + passed * step, hi);
    // the answer is in [lo, lo + step - 1], or the short last part
    hi = min(lo + step - 1, hi);
  }
  return lo;
}

constexpr int kMaxRowsPerBlock = 256;

// Blocks below walk_blocks walk the sorted tokens; the others write the zeros
// of the rows without one.
template <class G, class OUT, bool ACCUMULATE>
__global__ __launch_bounds__(kEmbedThreads) void embed_grad_kernel(const EmbedGradArgs g) {
  __shared__ int64_t bound[2];
  __shared__ uint32_t present[kMaxRowsPerBlock];
  if (!order_holds(g)) return;
  const int slots = kEmbedThreads / g.lanes;
  const int slot = threadIdx.x / g.lanes, lane = threadIdx.x % g.lanes;
  if (blockIdx.x < g.walk_blocks) {
    const int64_t walk = (int64_t)blockIdx.x * slots + slot;
    if (walk < g.walks) walk_chunk<G, OUT, ACCUMULATE>(g, walk, lane);
    return;
  }
  const int64_t r0 = ((int64_t)blockIdx.x - g.walk_blocks) * g.rows_per_block;
  const int64_t rows = min((int64_t)g.rows_per_block, g.table_rows - r0);
  int64_t lo = 0, hi = 0;
  if (g.n > 0) {
    const int wave = threadIdx.x / kWave;
    if (wave < 2) {
      const int64_t at = lower_bound(g, 0, r0 + (wave == 0 ? 0 : rows));
      if ((threadIdx.x & 63) == 0) bound[wave] = at;
    }
    __syncthreads();
    lo = bound[0];
    hi = bound[1];
  }
  if (threadIdx.x < rows) present[threadIdx.x] = 0u;
  __syncthreads();
  for (int64_t i = lo + threadIdx.x; i < hi; i += kEmbedThreads) present[g.keys[i] - r0] = 1u;
  __syncthreads();
  // 16 bytes a lane, side by side
  const int64_t words = g.chunks * (int64_t)(sizeof(OUT) / 2);
  for (int64_t r = slot; r < rows; r += slots) {
    if (present[r] != 0u) continue;
    u32x4 *row = reinterpret_cast<u32x4 *>(static_cast<OUT *>(g.out) + (r0 + r) * g.chunks * 8);
    for (int64_t c = lane; c < words; c += g.lanes)
      __builtin_nontemporal_store(u32x4{0u, 0u, 0u, 0u}, row + c);
  }
}

// The runs that cross chunks: a block of the chunk that one begins in adds its
// parts.  It takes up to 64 chunks of 8 channels; its other threads share the
// parts out, so a frequent token's hundreds of them are on their way together,
// and their sums are added in order.
template <class OUT, bool ACCUMULATE>
__global__ __launch_bounds__(kEmbedThreads) void embed_join_kernel(const EmbedGradArgs g,
                                                                   int64_t col_blocks) {
  __shared__ double sums[kEmbedThreads][9];  // (9: rows in other banks)
  const int64_t walk = blockIdx.x / col_blocks;
  if (walk + 1 >= g.walks || !order_holds(g)) return;
  const int64_t a = walk * g.walk_len, b = a + g.walk_len;
  const uint32_t run = g.keys[b - 1];
  if (run >= g.table_rows || g.keys[b] != run) return;           // does not leave
  if (g.keys[a] == run && a > 0 && g.keys[a - 1] == run) return;  // entered: another's
  // the last chunk it reaches: those after begin with its key, 64 tested at once
  int64_t last = walk;
  for (int more = 64; more == 64; last += more) {
    const int64_t q = last + 1 + (threadIdx.x & 63);
    more = __popcll(__ballot(q < g.walks && g.keys[q * g.walk_len] == run));
  }
  const int cols = g.lanes < 64 ? g.lanes : 64, parts = kEmbedThreads / cols;
  const int col = threadIdx.x % cols, part = threadIdx.x / cols;
  const int64_t c = (blockIdx.x % col_blocks) * cols + col;
  const bool on = c < g.chunks;
  double sum[8] = {0.0, 0.0, 0.0, 0.0, 0.0, 0.0, 0.0, 0.0};
  // part 0 begins with the run's first piece, the one that leaves `walk`
  for (int64_t q = walk + part; on && q <= last; q += parts) {
    const f64x2 *src = reinterpret_cast<const f64x2 *>(g.partials) +
                       ((q * 2 + (q == walk ? 1 : 0)) * g.chunks + c) * 4;
    f64x2 v[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = src[e];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      sum[2 * e] += v[e].x;
      sum[2 * e + 1] += v[e].y;
    }
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) sums[threadIdx.x][e] = sum[e];
  __syncthreads();
  if (part != 0 || !on) return;
  for (int q = 1; q < parts; ++q)
#pragma unroll
    for (int e = 0; e < 8; ++e) sum[e] += sums[q * cols + col][e];
  write_row<OUT, ACCUMULATE>(g, run, c, sum);
}

template <class OUT, bool ACCUMULATE>
void launch_grad(const EmbedGradArgs &g, bool float_grads, unsigned blocks, hipStream_t s) {
  const dim3 block(kEmbedThreads);
  if (float_grads)
    hipLaunchKernelGGL((embed_grad_kernel<float, OUT, ACCUMULATE>), dim3(blocks), block, 0, s, g);
  else
    hipLaunchKernelGGL((embed_grad_kernel<uint16_t, OUT, ACCUMULATE>), dim3(blocks), block, 0, s,
                       g);
  if (g.walks > 1) {
    const int64_t col_blocks = ceil_div(g.chunks, 64);
    hipLaunchKernelGGL((embed_join_kernel<OUT, ACCUMULATE>), dim3((unsigned)(g.walks * col_blocks)),
                       block, 0, s, g, col_blocks);
  }
}

}  // namespace
}  // namespace engram

int engram::launch_embed(const int64_t *d_tokens, int64_t n, const void *d_table,
                         int64_t table_rows, int64_t channels, float scale, int32_t out_type,
                         void *d_out, int64_t *d_err_count, void *stream) {
  const int64_t chunks = channels / 8;
  const int lanes = embed_row_lanes(channels);
  const int64_t blocks = ceil_div(n, (int64_t)(kEmbedThreads / lanes) * kEmbedRows);
  if (!grid_fits(blocks, kEmbedThreads)) return ENGRAM_EINVAL;
  const dim3 grid((unsigned)blocks), block(kEmbedThreads);
  const u32x4 *table = static_cast<const u32x4 *>(d_table);
  if (out_type == ENGRAM_F32)
    hipLaunchKernelGGL(embed_kernel<float>, grid, block, 0, as_stream(stream), d_tokens, n,
                       table, table_rows, chunks, lanes, scale, static_cast<float *>(d_out),
                       d_err_count);
  else
    hipLaunchKernelGGL(embed_kernel<uint16_t>, grid, block, 0, as_stream(stream), d_tokens, n,
                       table, table_rows, chunks, lanes, scale, static_cast<uint16_t *>(d_out),
                       d_err_count);
  return launch_status();
}

int engram::launch_embed_grad(const EmbedGradCall &c, const Plan &p, void *d_workspace,
                              void *stream) {
  hipStream_t st = as_stream(stream);
  EmbedGradArgs g = {};
  g.grads = c.grads;
  g.partials = c.partials;
  g.n = c.n;
  g.chunks = c.channels / 8;
  g.table_rows = c.table_rows;
  g.lanes = embed_row_lanes(c.channels);
  g.scale = c.scale;
  g.out = c.grad_table;
  // about 128 KB of rows a block of zeros
  const int64_t row_bytes = c.channels * (c.type == ENGRAM_F32 ? 4 : 2);
  g.rows_per_block = 8;
  while (g.rows_per_block < kMaxRowsPerBlock && g.rows_per_block * row_bytes < (128 << 10))
    g.rows_per_block *= 2;
  g.walk_len = embed_chunk(c.n, c.channels);
  g.walks = ceil_div(c.n, g.walk_len);
  g.walk_blocks = ceil_div(g.walks, kEmbedThreads / g.lanes);
  const int64_t zero_blocks = c.accumulate ? 0 : ceil_div(c.table_rows, g.rows_per_block);
  const int64_t blocks = g.walk_blocks + zero_blocks;
  if (!grid_fits(blocks, kEmbedThreads) ||
      !grid_fits(g.walks * ceil_div(g.chunks, 64), kEmbedThreads))
    return ENGRAM_EINVAL;
  if (c.n > 0) {
    const Views v = views_of(p, d_workspace);
    g.keys = v.sorted_keys;
    g.vals = v.sorted_vals;
    if (c.n <= kRankTokens) {
      hipLaunchKernelGGL(embed_rank_kernel, dim3((unsigned)ceil_div(c.n, kRankBlock)),
                         dim3(kRankThreads), 0, st, c.tokens, (int)c.n, (uint32_t)c.table_rows,
                         const_cast<uint32_t *>(g.keys), const_cast<uint32_t *>(g.vals), c.err);
    } else {
      g.plan = v.scalars;
      const int rc =
          launch_sort_crowded(c.tokens, c.n, c.table_rows, p, d_workspace, c.err, stream);
      if (rc != ENGRAM_OK) return rc;
    }
    if (c.table_rows == 0) return launch_status();
  }
  const bool wide = c.grads_type == ENGRAM_F32;
  if (c.accumulate)
    launch_grad<float, true>(g, wide, (unsigned)blocks, st);
  else if (c.type == ENGRAM_F32)
    launch_grad<float, false>(g, wide, (unsigned)blocks, st);
  else
    launch_grad<uint16_t, false>(g, wide, (unsigned)blocks, st);
  return launch_status();
}
