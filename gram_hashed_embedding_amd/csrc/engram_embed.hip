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
// The gradient.  The tokens are sorted (by counting, many of them by the passes
// of engram_sort.hip), so a row's terms are one run of the sorted order and no
// atomic is needed: the result does not depend on timing, and each row is
// written once.  Walkers take equal chunks of the sorted positions, however
// the tokens crowd: a run inside a chunk is summed and written by its walker;
// a run that crosses chunks leaves a part in each, which a block of the chunk
// it begins in adds up in a second, short kernel.  Beside the walkers, in the
// same launch, small blocks write the zeros of the rows without a token (most
// of a vocabulary), which a mark a row tells apart.  Sums are fp64, as the
// hashed table's.
//
// Measured on MI355X, 151,936 rows, tokens of Zipf exponent 1.1: 65,536 x 2048
// looked up in 53.7 us (6.0 TB/s; into floats 92 us, 6.4 TB/s); the gradient of
// as many into floats 290 us, of which sorting takes 35, marks 7, the walkers and
// zeros 228 (7.0 TB/s) and the join 8; of 4099 x 1024 into bf16 59 us (counting
// and marks 6, walkers and zeros 49, join 5).  From float gradients the 65,536 x 2048
// take 391 us (4.5 TB/s: four rows of a lane in flight, not eight); accumulated into
// the rows with tokens alone 215 us from bf16 and 252 from floats, where no zeros hide
// the sort and the walkers' waits.  More and shorter chunks were slower (at most 64
// positions: 362 us, 32: 388, against 306 then at 128).
#include "engram_layer_dev.h"
#include "engram_scatter_dev.h"

namespace engram {
namespace {

constexpr int kEmbedThreads = 256;
constexpr int kEmbedRows = 4;  // rows of a lane in flight

// A thread's eight columns: two runs of four, at the quads a and b of the row.
// Adjacent when what is read and written is bf16 (16 bytes a lane); else a row's
// lanes apart, so that a wavefront's 16-byte accesses of floats lie side by side
// (two stores of 16 bytes, 32 apart, write every line twice).  G: the rows read;
// OUT: those written.
struct Cols {
  int64_t a, b;
  bool on_b;
};
template <class G, class OUT>
constexpr bool kSplitCols = sizeof(G) == 4 || sizeof(OUT) == 4;
template <class G, class OUT>
__device__ __forceinline__ Cols cols_of(int64_t base, int lane, int lanes, int64_t quads) {
  if (!kSplitCols<G, OUT>) return Cols{base + 2 * lane, base + 2 * lane + 1, true};
  return Cols{base + lane, base + lane + lanes, base + lane + lanes < quads};
}

__device__ __forceinline__ void store4(uint16_t *row, int64_t quad, const float *f) {
  __builtin_nontemporal_store(u32x2{pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3])},
                              reinterpret_cast<u32x2 *>(row) + quad);
}
__device__ __forceinline__ void store4(float *row, int64_t quad, const float *f) {
  __builtin_nontemporal_store(f32x4{f[0], f[1], f[2], f[3]},
                              reinterpret_cast<f32x4 *>(row) + quad);
}

// Eight values of a row that is read, bf16 (uint16_t) or float; row: its first quad.
template <class G, bool SPLIT>
struct RowIn;
template <bool SPLIT>
struct RowIn<uint16_t, SPLIT> {
  static constexpr int kAhead = 8;  // rows in flight
  typedef u32x4 Raw;
  static __device__ __forceinline__ Raw load(const void *p, int64_t row, const Cols &c) {
    if (!SPLIT) return static_cast<const u32x4 *>(p)[(row + c.a) / 2];
    const u32x2 *q = static_cast<const u32x2 *>(p) + row;
    const u32x2 x = q[c.a], y = q[c.on_b ? c.b : c.a];
    return u32x4{x.x, x.y, y.x, y.y};
  }
  static __device__ __forceinline__ void unpack(const Raw &r, float (&f)[8]) {
    unpack_bf16x8(r, f);
  }
};
template <bool SPLIT>
struct RowIn<float, SPLIT> {
  static constexpr int kAhead = 4;
  struct Raw {
    f32x4 a, b;
  };
  static __device__ __forceinline__ Raw load(const void *p, int64_t row, const Cols &c) {
    const f32x4 *q = static_cast<const f32x4 *>(p) + row;
    return Raw{q[c.a], q[c.on_b ? c.b : c.a]};
  }
  static __device__ __forceinline__ void unpack(const Raw &r, float (&f)[8]) {
    f[0] = r.a.x; f[1] = r.a.y; f[2] = r.a.z; f[3] = r.a.w;
    f[4] = r.b.x; f[5] = r.b.y; f[6] = r.b.z; f[7] = r.b.w;
  }
};

// Writes a thread's eight values.
template <class G, class OUT>
__device__ __forceinline__ void store_cols(OUT *row, const Cols &c, const float (&f)[8]) {
  if constexpr (!kSplitCols<G, OUT>) {
    __builtin_nontemporal_store(pack_bf16x8(f), reinterpret_cast<u32x4 *>(row) + c.a / 2);
  } else {
    store4(row, c.a, f);
    if (c.on_b) store4(row, c.b, f + 4);
  }
}

template <class OUT>
__global__ __launch_bounds__(kEmbedThreads) void embed_kernel(
    const int64_t *__restrict__ tokens, int64_t n, const void *__restrict__ table,
    int64_t table_rows, int64_t chunks, int lanes, float scale, OUT *__restrict__ out,
    int64_t *err) {
  typedef RowIn<uint16_t, kSplitCols<uint16_t, OUT>> Row;
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
  const int64_t quads = chunks * 2;
  for (int64_t base = 0; base < quads; base += 2 * lanes) {
    const Cols c = cols_of<uint16_t, OUT>(base, lane, lanes, quads);
    if (c.a >= quads) break;
    u32x4 v[kEmbedRows];
#pragma unroll
    for (int k = 0; k < kEmbedRows; ++k) {
      v[k] = u32x4{0u, 0u, 0u, 0u};
      if (row[k] >= 0) v[k] = Row::load(table, row[k] * quads, c);
    }
#pragma unroll
    for (int k = 0; k < kEmbedRows; ++k) {
      const int64_t t = first + k * slots;
      if (t >= n) continue;
      float f[8];
      unpack_bf16x8(v[k], f);
#pragma unroll
      for (int e = 0; e < 8; ++e) f[e] = row[k] >= 0 ? f[e] * scale : 0.0f;
      store_cols<uint16_t, OUT>(out + t * chunks * 8, c, f);
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
  const uint8_t *present;  // [table_rows]: rows with a token (n > 0)
  int lanes, rows_per_block;
  float scale;
  void *out;
};

// Whether the order is valid (a wait of the sort that expired has marked the
// error counter; no sum is read or written by such an order).
__device__ __forceinline__ bool order_holds(const EmbedGradArgs &g) {
  return g.plan == nullptr || g.plan->stalled == 0;
}

// Which rows have a token, from the sorted tokens: a thread searches for its row
// (the threads of a wavefront take nearly the same steps).  Without a valid order
// it fills its row with NaN, so that a caller who counts no errors cannot take what
// the table held for a gradient (here and not beside the walkers, whose kernel of
// 65,536 x 2048 took 1% longer with the fill in it).
template <class OUT>
__global__ __launch_bounds__(kEmbedThreads) void embed_mark_kernel(const EmbedGradArgs g,
                                                                   uint8_t *present) {
  const int64_t row = (int64_t)blockIdx.x * kEmbedThreads + threadIdx.x;
  if (row >= g.table_rows) return;
  if (!order_holds(g)) {
    const uint32_t nan = sizeof(OUT) == 4 ? 0x7fc00000u : 0x7fc07fc0u;
    const int64_t words = g.chunks * (int64_t)(sizeof(OUT) / 2);
    u32x4 *dst = static_cast<u32x4 *>(g.out) + row * words;
    for (int64_t c = 0; c < words; ++c) dst[c] = u32x4{nan, nan, nan, nan};
    return;
  }
  int64_t lo = 0, hi = g.n;  // the first key not below the row lies in [lo, hi]
  while (lo < hi) {
    const int64_t mid = lo + (hi - lo) / 2;
    if ((int64_t)g.keys[mid] < row)
      lo = mid + 1;
    else
      hi = mid;
  }
  present[row] = lo < g.n && (int64_t)g.keys[lo] == row ? 1 : 0;
}

// The same from a few tokens in any order: a block takes kMarkRows rows and
// looks at every token.
constexpr int kMarkThreads = 1024, kMarkRows = 4096;
__device__ __forceinline__ void mark_rows(const int64_t *tokens, int64_t n, int64_t first,
                                          uint32_t *flags, uint8_t *present) {
  for (int i = threadIdx.x; i < kMarkRows / 4; i += kMarkThreads) flags[i] = 0u;
  __syncthreads();
  for (int64_t j = threadIdx.x; j < n; j += kMarkThreads) {
    const uint64_t r = (uint64_t)tokens[j] - (uint64_t)first;
    if (r < (uint64_t)kMarkRows) reinterpret_cast<uint8_t *>(flags)[r] = 1;
  }
  __syncthreads();
  // (the array is padded to whole blocks' rows)
  for (int i = threadIdx.x; i < kMarkRows / 4; i += kMarkThreads)
    reinterpret_cast<uint32_t *>(present + first)[i] = flags[i];
}

// Tokens are sorted by counting, a piece of at most kRankTokens at a time: a
// token's place in its piece is the number of smaller ones, and of equal ones
// before it.  A block places BLOCK tokens; its threads are BLOCK tokens wide and
// share out the piece's tokens to compare with, four at a time from LDS.  A few
// thousand tokens are one piece: one launch, in which the blocks after
// rank_blocks mark the rows that have a token.  More are pieces of kPieceTokens,
// merged by embed_merge_kernel: up to kMergeTokens the comparisons and searches,
// spread over the whole GPU, beat the sort's passes, which wait on one another
// (the whole gradient at 256 channels: 9000 tokens 44 us against 60 with the
// passes, 20,000 52 and 67, 65,536 81 and 89, 90,000 107 and 86; where the two
// cross between the last two was not looked for).
constexpr int kRankThreads = kMarkThreads;
constexpr int64_t kRankTokens = 8192, kPieceTokens = 2048, kMergeTokens = 65536;
constexpr int kRankBlock = 16, kPieceBlock = 64;

template <int BLOCK>
__global__ __launch_bounds__(kRankThreads) void embed_rank_kernel(
    const int64_t *__restrict__ tokens, int64_t n, int piece, uint32_t table_rows,
    uint32_t rank_blocks, uint32_t *keys, uint32_t *vals, uint8_t *present, int64_t *err) {
  constexpr int kParts = kRankThreads / BLOCK;
  __shared__ u32x4 s_key4[kRankTokens / 4];
  __shared__ uint32_t s_count[kParts][BLOCK];
  uint32_t *s_key = reinterpret_cast<uint32_t *>(s_key4);
  if (blockIdx.x >= rank_blocks) {
    mark_rows(tokens, n, (int64_t)(blockIdx.x - rank_blocks) * kMarkRows, s_key, present);
    return;
  }
  // this block's piece of the tokens (a whole number of blocks long), and the
  // first token of the piece that it places
  const int64_t start = (int64_t)blockIdx.x * BLOCK / piece * piece;
  const int i0 = (int)((int64_t)blockIdx.x * BLOCK - start);
  const int len = (int)min((int64_t)piece, n - start);
  int bad = 0;
  for (int j = threadIdx.x; j < ((len + 3) & ~3); j += kRankThreads) {
    uint32_t k = 0xffffffffu;  // past the end: above every key
    if (j < len) {
      const int64_t t = tokens[start + j];
      const bool ok = t >= 0 && t < (int64_t)table_rows;
      k = ok ? (uint32_t)t : table_rows;
      bad += !ok && t != -1 && j >= i0 && j < i0 + BLOCK ? 1 : 0;
    }
    s_key[j] = k;
  }
  count_errors(bad, err);
  __syncthreads();
  const int lane = threadIdx.x % BLOCK, part = threadIdx.x / BLOCK;
  const int i = i0 + lane;
  const uint32_t key = i < len ? s_key[i] : 0u;
  const int quads = (len + 3) / 4;
  uint32_t count = 0;
  // the block's own tokens lie in quads [i0 / 4, i0 / 4 + BLOCK / 4)
  for (int q = part; q < quads; q += kParts) {
    const u32x4 k = s_key4[q];
    if (q < i0 / 4) {
      count += (k.x <= key) + (k.y <= key) + (k.z <= key) + (k.w <= key);
    } else if (q >= i0 / 4 + BLOCK / 4) {
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
  if (threadIdx.x >= BLOCK || i >= len) return;
  uint32_t place = 0;
#pragma unroll
  for (int p = 0; p < kParts; ++p) place += s_count[p][lane];
  keys[start + place] = key;
  vals[start + place] = (uint32_t)(start + i);
}

// Sorted pieces into one order: a token's place is its place in its piece, plus
// the tokens not above it in the pieces before and those below it in the pieces
// after, by binary search.  A block takes 64 tokens of a piece; its 8 wavefronts
// share out the other pieces, kMergeAhead searches at a time.
constexpr int kMergeThreads = 512, kMergeAhead = 4;
__global__ __launch_bounds__(kMergeThreads) void embed_merge_kernel(
    const uint32_t *__restrict__ in_keys, const uint32_t *__restrict__ in_vals, int64_t n,
    uint32_t *keys, uint32_t *vals) {
  __shared__ uint32_t s_count[kMergeThreads / kWave][kWave];
  const int lane = threadIdx.x & 63, wave = threadIdx.x / kWave;
  const int64_t at = (int64_t)blockIdx.x * kWave + lane;
  const bool on = at < n;
  const uint32_t key = in_keys[on ? at : 0];
  const int own = (int)((int64_t)blockIdx.x * kWave / kPieceTokens);
  const int pieces = (int)((n + kPieceTokens - 1) / kPieceTokens);
  uint32_t count = 0;
  for (int p0 = wave * kMergeAhead; p0 < pieces; p0 += kMergeThreads / kWave * kMergeAhead) {
    uint32_t low[kMergeAhead], size[kMergeAhead];
    const uint32_t *piece[kMergeAhead];
    uint32_t bound[kMergeAhead];  // counted are the keys below it
#pragma unroll
    for (int k = 0; k < kMergeAhead; ++k) {
      const int p = p0 + k;
      const bool other = p < pieces && p != own;
      const int64_t start = (int64_t)(other ? p : 0) * kPieceTokens;
      piece[k] = in_keys + start;
      low[k] = 0;
      size[k] = other ? (uint32_t)min(kPieceTokens, n - start) : 0u;
      bound[k] = p < own ? key + 1 : key;  // (keys are below 2^32 - 1)
    }
    // halves of [low, low + size) that hold the first key not below the bound
#pragma unroll 1
    for (int step = 0; step < 12; ++step) {
#pragma unroll
      for (int k = 0; k < kMergeAhead; ++k) {
        const uint32_t half = size[k] / 2;
        const bool below = size[k] > 0 && piece[k][low[k] + half] < bound[k];
        low[k] += below ? half + 1 : 0u;
        size[k] = below ? size[k] - half - 1 : half;
      }
    }
#pragma unroll
    for (int k = 0; k < kMergeAhead; ++k) count += low[k];
  }
  s_count[wave][lane] = count;
  __syncthreads();
  if (wave != 0 || !on) return;
  uint32_t place = (uint32_t)(at - (int64_t)own * kPieceTokens);
#pragma unroll
  for (int w = 0; w < kMergeThreads / kWave; ++w) place += s_count[w][lane];
  keys[place] = key;
  vals[place] = in_vals[at];
}
static_assert(kPieceTokens == 1 << 11, "12 halvings empty a piece");
static_assert(kPieceTokens % kPieceBlock == 0 && kPieceTokens % kWave == 0 &&
                  kPieceTokens <= kRankTokens && kRankTokens % kRankBlock == 0,
              "blocks do not straddle pieces");

template <class G, class OUT, bool ACCUMULATE>
__device__ __forceinline__ void write_row(const EmbedGradArgs &g, int64_t row, const Cols &c,
                                          const double (&sum)[8]) {
  OUT *dst = static_cast<OUT *>(g.out) + row * g.chunks * 8;
  float f[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) f[e] = (float)(sum[e] * (double)g.scale);
  if (ACCUMULATE) {
    const f32x4 *old = reinterpret_cast<const f32x4 *>(dst);
    const f32x4 x = old[c.a], y = old[c.on_b ? c.b : c.a];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      f[e] = x[e] + f[e];
      f[4 + e] = y[e] + f[4 + e];
    }
  }
  store_cols<G, OUT>(dst, c, f);
}

// A row of partial sums, in the thread's own order of columns.
__device__ __forceinline__ f64x2 *part_at(const EmbedGradArgs &g, int64_t walk, int which,
                                          int64_t quad) {
  return reinterpret_cast<f64x2 *>(g.partials + (walk * 2 + which) * g.chunks * 8) + quad * 2;
}
__device__ __forceinline__ void write_part(const EmbedGradArgs &g, int64_t walk, int which,
                                           const Cols &c, const double (&sum)[8]) {
  f64x2 *x = part_at(g, walk, which, c.a);
  x[0] = f64x2{sum[0], sum[1]};
  x[1] = f64x2{sum[2], sum[3]};
  if (!c.on_b) return;
  x = part_at(g, walk, which, c.b);
  x[0] = f64x2{sum[4], sum[5]};
  x[1] = f64x2{sum[6], sum[7]};
}

// A walker's chunk [a, b) of the sorted positions: its runs' sums.
template <class G, class OUT, bool ACCUMULATE>
__device__ void walk_chunk(const EmbedGradArgs &g, int64_t walk, int lane) {
  typedef RowIn<G, kSplitCols<G, OUT>> Row;
  constexpr int kAhead = Row::kAhead;
  const int64_t a = walk * g.walk_len, b = min(a + g.walk_len, g.n);
  const uint32_t before = a > 0 ? g.keys[a - 1] : 0xffffffffu;  // no key (they are smaller)
  const uint32_t after = b < g.n ? g.keys[b] : 0xffffffffu;
  const int64_t quads = g.chunks * 2;
  for (int64_t base = 0; base < quads; base += 2 * g.lanes) {
    const Cols c = cols_of<G, OUT>(base, lane, g.lanes, quads);
    if (c.a >= quads) break;
    double sum[8] = {0.0, 0.0, 0.0, 0.0, 0.0, 0.0, 0.0, 0.0};
    uint32_t run = g.keys[a];
    bool entered = run == before;
    for (int64_t i = a; i < b; i += kAhead) {
      uint32_t key[kAhead];
      typename Row::Raw v[kAhead];
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        const int64_t at = min(i + k, b - 1);
        key[k] = g.keys[at];
        v[k] = Row::load(g.grads, (int64_t)g.vals[at] * quads, c);
      }
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        if (i + k >= b) break;
        if (key[k] != run) {  // a run has ended in this chunk
          if (run < g.table_rows) {
            if (entered)
              write_part(g, walk, 0, c, sum);
            else
              write_row<G, OUT, ACCUMULATE>(g, run, c, sum);
          }
          run = key[k];
          entered = false;
#pragma unroll
          for (int e = 0; e < 8; ++e) sum[e] = 0.0;
        }
        float f[8];
        Row::unpack(v[k], f);
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
      write_row<G, OUT, ACCUMULATE>(g, run, c, sum);
  }
}

// Blocks below walk_blocks walk the sorted tokens; the others write the zeros
// of the rows without one.
template <class G, class OUT, bool ACCUMULATE>
__global__ __launch_bounds__(kEmbedThreads) void embed_grad_kernel(const EmbedGradArgs g) {
  if (!order_holds(g)) return;
  const int slots = kEmbedThreads / g.lanes;
  const int slot = threadIdx.x / g.lanes, lane = threadIdx.x % g.lanes;
  if (blockIdx.x < g.walk_blocks) {
    const int64_t walk = (int64_t)blockIdx.x * slots + slot;
    if (walk < g.walks) walk_chunk<G, OUT, ACCUMULATE>(g, walk, lane);
    return;
  }
  const int64_t r0 = ((int64_t)blockIdx.x - g.walk_blocks) * g.rows_per_block;
  const int64_t end = min(r0 + g.rows_per_block, g.table_rows);
  // 16 bytes a lane, side by side
  const int64_t words = g.chunks * (int64_t)(sizeof(OUT) / 2);
  for (int64_t r = r0 + slot; r < end; r += slots) {
    if (g.present != nullptr && g.present[r] != 0) continue;
    u32x4 *row = reinterpret_cast<u32x4 *>(static_cast<OUT *>(g.out) + r * g.chunks * 8);
    for (int64_t c = lane; c < words; c += g.lanes)
      __builtin_nontemporal_store(u32x4{0u, 0u, 0u, 0u}, row + c);
  }
}

// The runs that cross chunks: a block of the chunk that one begins in adds its
// parts.  It takes up to 64 chunks of 8 channels; its other threads share the
// parts out, so a frequent token's hundreds of them are on their way together,
// and their sums are added in order.
template <class G, class OUT, bool ACCUMULATE>
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
  const int64_t quads = g.chunks * 2, base = (blockIdx.x % col_blocks) * cols * 2;
  const Cols c = cols_of<G, OUT>(base, col, cols, quads);
  const bool on = c.a < quads;
  const int64_t qa = on ? c.a : 0, qb = on && c.on_b ? c.b : qa;
  double sum[8] = {0.0, 0.0, 0.0, 0.0, 0.0, 0.0, 0.0, 0.0};
  // part 0 begins with the run's first piece, the one that leaves `walk`
#pragma unroll 4
  for (int64_t q = walk + part; q <= last; q += parts) {
    const f64x2 *x = part_at(g, q, q == walk ? 1 : 0, qa);
    const f64x2 *y = part_at(g, q, q == walk ? 1 : 0, qb);
    const f64x2 v[4] = {x[0], x[1], y[0], y[1]};
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
  write_row<G, OUT, ACCUMULATE>(g, run, c, sum);
}

template <class G, class OUT, bool ACCUMULATE>
void launch_grad(const EmbedGradArgs &g, unsigned blocks, hipStream_t s) {
  const dim3 block(kEmbedThreads);
  hipLaunchKernelGGL((embed_grad_kernel<G, OUT, ACCUMULATE>), dim3(blocks), block, 0, s, g);
  if (g.walks > 1) {
    const int64_t col_blocks = ceil_div(g.chunks, 64);
    hipLaunchKernelGGL((embed_join_kernel<G, OUT, ACCUMULATE>),
                       dim3((unsigned)(g.walks * col_blocks)), block, 0, s, g, col_blocks);
  }
}
template <class G>
void launch_grad(const EmbedGradArgs &g, const EmbedGradCall &c, unsigned blocks, hipStream_t s) {
  if (c.accumulate)
    launch_grad<G, float, true>(g, blocks, s);
  else if (c.type == ENGRAM_F32)
    launch_grad<G, float, false>(g, blocks, s);
  else
    launch_grad<G, uint16_t, false>(g, blocks, s);
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
  if (out_type == ENGRAM_F32)
    hipLaunchKernelGGL(embed_kernel<float>, grid, block, 0, as_stream(stream), d_tokens, n,
                       d_table, table_rows, chunks, lanes, scale, static_cast<float *>(d_out),
                       d_err_count);
  else
    hipLaunchKernelGGL(embed_kernel<uint16_t>, grid, block, 0, as_stream(stream), d_tokens, n,
                       d_table, table_rows, chunks, lanes, scale, static_cast<uint16_t *>(d_out),
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
  // about 8 KB of rows a block of zeros (blocks that end soon keep the stores
  // that run together on one stretch of memory: 65,536 x 2048 into float 306 us,
  // with 16 KB 337, with 32 KB 352)
  const int64_t row_bytes = c.channels * (c.type == ENGRAM_F32 ? 4 : 2);
  g.rows_per_block = kEmbedThreads / g.lanes;
  // (and not more blocks than a launch holds, for tables past 64 GB)
  while (g.rows_per_block < (1 << 28) &&
         ((g.rows_per_block < 4096 && g.rows_per_block * row_bytes < (8 << 10)) ||
          ceil_div(c.table_rows, g.rows_per_block) > (1 << 23)))
    g.rows_per_block *= 2;
  g.walk_len = embed_chunk(c.n, c.channels);
  g.walks = ceil_div(c.n, g.walk_len);
  g.walk_blocks = ceil_div(g.walks, kEmbedThreads / g.lanes);
  const int64_t zero_blocks = c.accumulate ? 0 : ceil_div(c.table_rows, g.rows_per_block);
  const int64_t blocks = g.walk_blocks + zero_blocks;
  const int64_t mark_blocks = c.accumulate ? 0 : ceil_div(c.table_rows, kMarkRows);
  static_assert(kMarkRows == kEmbedMarkRows, "the workspace pads the marks to whole blocks");
  if (!grid_fits(blocks, kEmbedThreads) ||
      !grid_fits(mark_blocks + kRankTokens / kRankBlock, kRankThreads) ||
      !grid_fits(ceil_div(c.table_rows, kEmbedThreads), kEmbedThreads) ||
      !grid_fits(g.walks * ceil_div(g.chunks, 64), kEmbedThreads))
    return ENGRAM_EINVAL;
  if (c.n > 0) {
    const Views v = views_of(p, d_workspace);
    g.keys = v.sorted_keys;
    g.vals = v.sorted_vals;
    g.present = c.present;
    uint32_t *keys = const_cast<uint32_t *>(g.keys), *vals = const_cast<uint32_t *>(g.vals);
    if (c.n <= kRankTokens) {
      const int64_t rank_blocks = ceil_div(c.n, kRankBlock);
      hipLaunchKernelGGL(embed_rank_kernel<kRankBlock>,
                         dim3((unsigned)(rank_blocks + mark_blocks)), dim3(kRankThreads), 0, st,
                         c.tokens, c.n, (int)kRankTokens, (uint32_t)c.table_rows,
                         (uint32_t)rank_blocks, keys, vals, c.present, c.err);
    } else {
      if (c.n <= kMergeTokens) {
        uint32_t *piece_keys = keys == v.keys_a ? v.keys_b : v.keys_a;
        uint32_t *piece_vals = vals == v.vals_a ? v.vals_b : v.vals_a;
        const int64_t rank_blocks = ceil_div(c.n, kPieceBlock);
        hipLaunchKernelGGL(embed_rank_kernel<kPieceBlock>, dim3((unsigned)rank_blocks),
                           dim3(kRankThreads), 0, st, c.tokens, c.n, (int)kPieceTokens,
                           (uint32_t)c.table_rows, (uint32_t)rank_blocks, piece_keys, piece_vals,
                           nullptr, c.err);
        hipLaunchKernelGGL(embed_merge_kernel, dim3((unsigned)ceil_div(c.n, kWave)),
                           dim3(kMergeThreads), 0, st, piece_keys, piece_vals, c.n, keys, vals);
      } else {
        g.plan = v.scalars;
        const int rc =
            launch_sort_crowded(c.tokens, c.n, c.table_rows, p, d_workspace, c.err, stream);
        if (rc != ENGRAM_OK) return rc;
      }
      const dim3 marks((unsigned)ceil_div(c.table_rows, kEmbedThreads)), block(kEmbedThreads);
      if (mark_blocks > 0 && c.type == ENGRAM_F32)
        hipLaunchKernelGGL(embed_mark_kernel<float>, marks, block, 0, st, g, c.present);
      else if (mark_blocks > 0)
        hipLaunchKernelGGL(embed_mark_kernel<uint16_t>, marks, block, 0, st, g, c.present);
    }
    if (c.table_rows == 0) return launch_status();
  }
  if (c.grads_type == ENGRAM_F32)
    launch_grad<float>(g, c, (unsigned)blocks, st);
  else
    launch_grad<uint16_t>(g, c, (unsigned)blocks, st);
  return launch_status();
}
