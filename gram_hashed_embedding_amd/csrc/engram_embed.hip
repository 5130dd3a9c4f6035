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
// written once.  A block owns a range of adjacent table rows, finds its part
// of the sorted tokens by a 64-way search and writes its rows from zero or
// from their runs.  A frequent token's run is too long for one block: every
// 64 sorted positions that are all of one token are summed beforehand into an
// fp64 row, and the row's owner adds those.  Sums are fp64, as the hashed
// table's, so runs may be cut anywhere.
#include "engram_layer_dev.h"
#include "engram_scatter_dev.h"

namespace engram {
namespace {

constexpr int kEmbedThreads = 256;
constexpr int kEmbedRows = 4;  // rows of a lane in flight

// A row of `chunks` chunks of 8 channels is covered by `lanes` threads (a
// power of two, at most a block); a block takes 256 / lanes rows at a time.
inline int row_lanes(int64_t chunks) {
  int l = 1;
  while (l < chunks && l < kEmbedThreads) l *= 2;
  return l;
}

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
  __builtin_nontemporal_store(f32x4{f[0], f[1], f[2], f[3]}, q);
  __builtin_nontemporal_store(f32x4{f[4], f[5], f[6], f[7]}, q + 1);
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
struct EmbedGradArgs {
  const uint32_t *keys, *vals;  // sorted tokens and their positions
  const PlanScalars *plan;
  const u32x4 *grads;
  double *partials;
  int64_t n, chunks, table_rows;
  int lanes, rows_per_block;
  float scale;
  void *out;
};

// Whether the plan holds a valid order (a wait of it that expired has marked
// the error counter; nothing is read by such an order, and nothing written).
__device__ __forceinline__ bool plan_holds(const EmbedGradArgs &g) {
  return g.plan->stalled == 0 && g.plan->n == (uint64_t)g.n;
}

// Adds the gradient rows of the sorted positions [a, b), chunk c.
__device__ __forceinline__ void add_rows(const EmbedGradArgs &g, int64_t a, int64_t b, int64_t c,
                                         double (&sum)[8]) {
  constexpr int kAhead = 8;
  for (int64_t i = a; i < b; i += kAhead) {
    u32x4 v[kAhead];
#pragma unroll
    for (int k = 0; k < kAhead; ++k)
      v[k] = i + k < b ? g.grads[(int64_t)g.vals[i + k] * g.chunks + c] : u32x4{0u, 0u, 0u, 0u};
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      float f[8];
      unpack_bf16x8(v[k], f);
#pragma unroll
      for (int e = 0; e < 8; ++e) sum[e] += f[e];
    }
  }
}

// Sums of the kEmbedChunk-position chunks that are all of one token.
__global__ __launch_bounds__(kEmbedThreads) void embed_chunk_kernel(const EmbedGradArgs g) {
  const int64_t chunk = blockIdx.x;
  const int64_t a = chunk * kEmbedChunk, b = a + kEmbedChunk;
  if (!plan_holds(g)) return;
  const uint32_t key = g.keys[a];
  if (key >= g.table_rows || key != g.keys[b - 1]) return;
  for (int64_t c = threadIdx.x; c < g.chunks; c += kEmbedThreads) {
    double sum[8] = {0.0, 0.0, 0.0, 0.0, 0.0, 0.0, 0.0, 0.0};
    add_rows(g, a, b, c, sum);
    double *dst = g.partials + (chunk * g.chunks + c) * 8;
#pragma unroll
    for (int e = 0; e < 8; ++e) dst[e] = sum[e];
  }
}

// The first sorted position whose key is at least `key` (a wavefront
// together: 64 probes a step).
__device__ __forceinline__ int64_t lower_bound(const EmbedGradArgs &g, int64_t key) {
  int64_t lo = 0, hi = g.n;
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

template <class OUT, bool ACCUMULATE>
__global__ __launch_bounds__(kEmbedThreads) void embed_rows_kernel(const EmbedGradArgs g) {
  __shared__ int64_t bound[2];
  __shared__ uint32_t begin[kMaxRowsPerBlock], end[kMaxRowsPerBlock];
  const int64_t r0 = (int64_t)blockIdx.x * g.rows_per_block;
  const int64_t rows = min((int64_t)g.rows_per_block, g.table_rows - r0);
  int64_t lo = 0, hi = 0;
  if (g.n > 0) {
    if (!plan_holds(g)) return;
    const int wave = threadIdx.x / kWave;
    if (wave < 2) {
      const int64_t at = lower_bound(g, r0 + (wave == 0 ? 0 : rows));
      if ((threadIdx.x & 63) == 0) bound[wave] = at;
    }
    __syncthreads();
    lo = bound[0];
    hi = bound[1];
  }
  for (int i = threadIdx.x; i < rows; i += kEmbedThreads) begin[i] = end[i] = 0u;
  __syncthreads();
  for (int64_t i = lo + threadIdx.x; i < hi; i += kEmbedThreads) {
    const uint32_t k = g.keys[i];
    if (i == lo || g.keys[i - 1] != k) begin[k - r0] = (uint32_t)i;
    if (i == hi - 1 || g.keys[i + 1] != k) end[k - r0] = (uint32_t)(i + 1);
  }
  __syncthreads();
  const int slots = kEmbedThreads / g.lanes;
  const int lane = threadIdx.x % g.lanes;
  for (int64_t r = threadIdx.x / g.lanes; r < rows; r += slots) {
    const int64_t a = begin[r], b = end[r];
    OUT *row = static_cast<OUT *>(g.out) + (r0 + r) * g.chunks * 8;
    if (a == b) {
      if (ACCUMULATE) continue;
      const float zero[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
      for (int64_t c = lane; c < g.chunks; c += g.lanes) store8<OUT>(row, c, zero);
      continue;
    }
    const int64_t c0 = (a + kEmbedChunk - 1) / kEmbedChunk, c1 = b / kEmbedChunk;
    for (int64_t c = lane; c < g.chunks; c += g.lanes) {
      double sum[8] = {0.0, 0.0, 0.0, 0.0, 0.0, 0.0, 0.0, 0.0};
      if (c0 < c1) {
        add_rows(g, a, c0 * kEmbedChunk, c, sum);
#pragma unroll 4
        for (int64_t q = c0; q < c1; ++q) {
          const double *src = g.partials + (q * g.chunks + c) * 8;
#pragma unroll
          for (int e = 0; e < 8; ++e) sum[e] += src[e];
        }
        add_rows(g, c1 * kEmbedChunk, b, c, sum);
      } else {
        add_rows(g, a, b, c, sum);
      }
      float f[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) f[e] = (float)(sum[e] * (double)g.scale);
      if (ACCUMULATE) {
        const float *old = reinterpret_cast<const float *>(row) + c * 8;
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] = old[e] + f[e];
      }
      store8<OUT>(row, c, f);
    }
  }
}

}  // namespace
}  // namespace engram

int engram::launch_embed(const int64_t *d_tokens, int64_t n, const void *d_table,
                         int64_t table_rows, int64_t channels, float scale, int32_t out_type,
                         void *d_out, int64_t *d_err_count, void *stream) {
  const int64_t chunks = channels / 8;
  const int lanes = row_lanes(chunks);
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
  g.grads = static_cast<const u32x4 *>(c.grads);
  g.partials = c.partials;
  g.n = c.n;
  g.chunks = c.channels / 8;
  g.table_rows = c.table_rows;
  g.lanes = row_lanes(g.chunks);
  g.scale = c.scale;
  g.out = c.grad_table;
  // about 128 KB of fp32 rows a block
  g.rows_per_block = 8;
  while (g.rows_per_block < kMaxRowsPerBlock && g.rows_per_block * c.channels < 32768)
    g.rows_per_block *= 2;
  const int64_t blocks = ceil_div(c.table_rows, g.rows_per_block);
  const int64_t full_chunks = c.n / kEmbedChunk;
  if (!grid_fits(blocks, kEmbedThreads) || !grid_fits(full_chunks, kEmbedThreads))
    return ENGRAM_EINVAL;
  if (c.n > 0) {
    const Views v = views_of(p, d_workspace);
    g.keys = v.sorted_keys;
    g.vals = v.sorted_vals;
    g.plan = v.scalars;
    const int rc = launch_plan(c.tokens, nullptr, c.n, c.table_rows, p, d_workspace, c.err,
                               stream);
    if (rc != ENGRAM_OK || c.table_rows == 0) return rc;
    if (full_chunks > 0)
      hipLaunchKernelGGL(embed_chunk_kernel, dim3((unsigned)full_chunks), dim3(kEmbedThreads), 0,
                         st, g);
  }
  const dim3 grid((unsigned)blocks), block(kEmbedThreads);
  if (c.accumulate)
    hipLaunchKernelGGL((embed_rows_kernel<float, true>), grid, block, 0, st, g);
  else if (c.type == ENGRAM_F32)
    hipLaunchKernelGGL((embed_rows_kernel<float, false>), grid, block, 0, st, g);
  else
    hipLaunchKernelGGL((embed_rows_kernel<uint16_t, false>), grid, block, 0, st, g);
  return launch_status();
}
