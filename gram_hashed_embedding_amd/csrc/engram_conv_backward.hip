// engram_conv_backward.hip -- the gradients of the PLE causal dilated
// depthwise convolution, for gfx950.
//
// What is computed is stated with engram_ple_conv_backward in include/
// engram_layer.h: the transpose of the convolution of the NeMo AutoModel v0.7
// API page "qwen3_8_flash_next.engram", Qwen3_8_FlashNextPLELayer
// (_causal_short_conv, _segmented_conv), with the readings of
// engram_ple_conv.
//
// Mathematics.  Both sums run over the same pairs (p, t = p + j * dilation):
// grad_x[p] adds w_j * g[t] and grad_w_j adds g[t] * x[p], so a position needs
// its own x and the K values of g ahead of it.  A pair counts when t lies in
// the row and no segment begins in (p, t].
//
// Bound by HBM: 6 bytes a value (5 from an 8-bit checkpoint) against 17
// operations.  A wave owns 256 channels, 4 a lane, and a slice of a row's
// positions, which it walks from the end: the rows of g ahead of a position
// are those it has just passed, so they stay in registers and each row of g is
// read once (a slice reads (K-1) * dilation rows past its end).  The
// segments' bounds are the same for a whole wave: one ballot a tile gives a
// mask of the positions where a segment begins, and a tile without any takes
// the path without tests.  Sums over positions stay in registers; each slice
// leaves one fp32 row of them, which a second kernel adds in fp64.
//
// A tile's loads are straight-line code, at clamped addresses, and go out while
// the tile before is worked on: behind branches, even wave-uniform ones, each
// was waited for on its own (985 us for the encoding and the gradients below,
// 780 us so).  Registers bound the waves to two a SIMD up to dilation 4 (5 with x in
// bf16), and to one beyond (256 registers and accumulation registers).  As many
// slices as two a SIMD (2048 waves) were faster than twice as many (780 and 817 us),
// tiles of 8 positions than tiles of 4 (801 us), both at dilation 4.  Measured on
// MI355X, [8, 8192, 8192], packed segments: from the checkpoint at dilation 4 500 us
// (5.4 TB/s; 540 under the profiler), its sums joined in 7 us, at dilations 5, 6 and
// 8 584, 681 and 740; from bf16 at dilations 4 and 5 610 us (5.3 TB/s), at 6 and 8
// 648 and 717.  [2, 2053, 1032] with a halo: 23 us, bound by latency (about 14 of
// them for a wave's four tiles alone).  The kernel for other shapes reads every row
// of g K times for each of the two sums: 6.1 ms for [8, 8192, 8192] with 3 taps.
#include "engram_layer_dev.h"

namespace engram {
namespace {

constexpr int kConvWaves = 4;  // waves of a block, each on its own
constexpr int kConvBlock = kConvWaves * kWave;

struct ConvBackArgs {
  const u32x2 *g;  // grad_out [batch, seq, quads]
  const u32x2 *x;
  const uint32_t *codes;
  const float *scales;
  int64_t code_blocks, code_width;  // of a position
  const u32x2 *halo;
  const int64_t *seg;
  const uint16_t *w;
  u32x2 *gx, *ghalo;
  float *partials;  // [batch * slices][K + 1][channels], or null
  int64_t batch, seq, halo_len, quads, units;
  ConvBackwardShape s;
  int K, dil;
  bool want_w;
};

__device__ __forceinline__ void unpack4(const u32x2 &r, float (&f)[4]) {
  f[0] = bf16_lo(r.x); f[1] = bf16_hi(r.x);
  f[2] = bf16_lo(r.y); f[3] = bf16_hi(r.y);
}

// One wave's place: (batch row, slice, channel group), groups fastest.  The
// first `halo_slices` slices of a row are the halo's, the others the
// sequence's: a slice lies on one side of position 0.
struct ConvPlace {
  int64_t b, slice, quad0, first, last;  // positions [first, last); the wave's first quad
  uint32_t lane;                         // this lane's quad after quad0
  bool on, halo;
};
__device__ __forceinline__ ConvPlace conv_place(const ConvBackArgs &a, uint32_t unit) {
  ConvPlace p;  // (units fit 32 bits: the grid has four to a block of 256 threads)
  const uint32_t groups = (uint32_t)a.s.groups, slices = (uint32_t)a.s.slices;
  const uint32_t rest = unit / groups, grp = unit - rest * groups;
  const uint32_t row = rest / slices;
  p.slice = rest - row * slices;
  p.b = row;
  p.quad0 = grp * kWave;
  p.lane = threadIdx.x & 63;
  p.on = p.quad0 + p.lane < a.quads;
  if (!p.on) p.lane = 0;  // reads what another lane reads, writes nothing
  p.halo = p.slice < a.s.halo_slices;
  p.first = p.halo ? p.slice * a.s.slice - a.halo_len
                   : (p.slice - a.s.halo_slices) * a.s.slice;
  p.last = min(p.first + a.s.slice, p.halo ? 0 : a.seq);
  return p;
}

// x of a position: 4 values of this lane's channels, as bf16 or as codes.
struct XRow {
  u32x2 bits;
  float scale;  // codes only
};
// (Row addresses are the same for a wave: scalar registers; a lane adds its
// 32-bit offset.)
__device__ __forceinline__ XRow load_halo(const ConvBackArgs &a, const ConvPlace &p, int64_t pos) {
  const u32x2 *row = a.halo + (p.b * a.halo_len + a.halo_len + pos) * a.quads + p.quad0;
  return XRow{row[p.lane], 0.0f};
}
template <bool CODES>
__device__ __forceinline__ XRow load_x(const ConvBackArgs &a, const ConvPlace &p, int64_t pos,
                                       uint32_t scale_at) {
  const int64_t at = p.b * a.seq + pos;
  if (CODES) {
    const uint32_t *row = a.codes + at * a.quads + p.quad0;
    const float *scales = a.scales + at * a.code_blocks;
    return XRow{u32x2{row[p.lane], 0u}, scales[scale_at]};
  }
  const u32x2 *row = a.x + at * a.quads + p.quad0;
  return XRow{row[p.lane], 0.0f};
}
// The scale of a lane's channels among a position's.
__device__ __forceinline__ uint32_t scale_of(const ConvBackArgs &a, const ConvPlace &p) {
  const uint32_t c = (uint32_t)(p.quad0 + p.lane) * 4, width = (uint32_t)a.code_width;
  const uint32_t g = c / width;  // (channels are below 2^31)
  return g * ((width + 127) / 128) + (c - g * width) / 128;
}
// One row of the gradient of x or of the halo.
__device__ __forceinline__ void store_gx(const ConvBackArgs &a, const ConvPlace &p, int64_t t,
                                         bool halo, const u32x2 &v) {
  if (!halo) {
    if (a.gx == nullptr) return;
    u32x2 *row = a.gx + (p.b * a.seq + t) * a.quads + p.quad0;
    row[p.lane] = v;
  } else if (a.ghalo != nullptr) {
    u32x2 *row = a.ghalo + (p.b * a.halo_len + a.halo_len + t) * a.quads + p.quad0;
    row[p.lane] = v;
  }
}
template <bool CODES>
__device__ __forceinline__ void unpack_x(const XRow &r, bool halo, float (&f)[4]) {
  if (CODES && !halo) {
    code_values(r.bits.x, r.scale, f);
  } else {
    unpack4(r.bits, f);
  }
}

// The segment ids of the positions at + lane and before it (loaded ahead of
// their use), and from them the bits of the positions at .. at + 63 where a
// segment begins (bit 0 is not used) or the row has ended.
struct SegPair {
  int64_t here, before;
};
__device__ __forceinline__ SegPair load_seg(const ConvBackArgs &a, int64_t b, int64_t at) {
  // no branch (a load behind one is waited for at once): without ids, any words
  const int64_t low = -a.halo_len;
  const int64_t *p = reinterpret_cast<const int64_t *>(a.g);
  int64_t here = 0, before = 0;
  if (a.seg != nullptr) {
    p = a.seg + b * (a.halo_len + a.seq) + a.halo_len;
    here = min(max(at + (int64_t)(threadIdx.x & 63), low), a.seq - 1);
    before = max(here - 1, low);
  }
  return SegPair{p[here], p[before]};
}
__device__ __forceinline__ uint64_t begins_mask(const ConvBackArgs &a, const SegPair &s,
                                                int64_t at) {
  const int64_t pos = at + (threadIdx.x & 63);
  return __ballot(pos >= a.seq || (a.seg != nullptr && pos > -a.halo_len && s.here != s.before));
}

// The first position after `at` (of the slice's last position) where a segment
// begins or the row ends, or one past `reach` positions ahead if none does
// before; 64 positions a step, the same in every lane of the wave.
__device__ __forceinline__ int64_t run_end(const ConvBackArgs &a, const int64_t *seg, int64_t at,
                                           int64_t reach) {
  const int64_t end = min(a.seq, at + reach + 1);
  if (seg == nullptr) return end;
  for (int64_t from = at + 1; from < end; from += kWave) {
    const int64_t pos = from + (threadIdx.x & 63);
    const int64_t at_most = min(pos, end - 1);
    const uint64_t begins = __ballot(pos < end && seg[at_most] != seg[at_most - 1]);
    if (begins != 0) return from + __builtin_ctzll(begins);
  }
  return end;
}

// Any K up to kConvMaxKernel and any dilation: the same walk, each row of g
// read from memory.  `limit` is where the pairs of a position end: the next
// place a segment begins, which only moves down as the walk does.
template <bool CODES>
__global__ __launch_bounds__(kConvBlock) void conv_backward_generic_kernel(const ConvBackArgs a) {
  const uint32_t unit = blockIdx.x * kConvWaves + threadIdx.x / kWave;
  if (unit >= a.units) return;
  const ConvPlace p = conv_place(a, unit);
  const uint32_t scale_at = CODES ? scale_of(a, p) : 0u;
  const int64_t *seg =
      a.seg != nullptr ? a.seg + p.b * (a.halo_len + a.seq) + a.halo_len : nullptr;
  const int64_t quad = p.quad0 + p.lane;
  const u32x2 *g = a.g + p.b * a.seq * a.quads + quad;
  const int64_t end = run_end(a, seg, p.last - 1, (int64_t)(a.K - 1) * a.dil);
  float sum_b[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  int64_t limit = end;
  for (int64_t t = p.last - 1; t >= p.first; --t) {
    if (seg != nullptr && t + 1 < p.last && seg[t + 1] != seg[t]) limit = t + 1;
    float dx[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int j = 0; j < a.K; ++j) {
      const int64_t q = t + (int64_t)j * a.dil;
      if (q >= limit) break;
      if (q < 0) continue;
      float v[4];
      unpack4(g[q * a.quads], v);
      for (int c = 0; c < 4; ++c) {
        dx[c] += bf16_lo(a.w[(quad * 4 + c) * a.K + (a.K - 1 - j)]) * v[c];
        if (j == 0) sum_b[c] += v[c];
      }
    }
    if (!p.on) continue;
    store_gx(a, p, t, p.halo, u32x2{pack_bf16(dx[0], dx[1]), pack_bf16(dx[2], dx[3])});
  }
  if (a.partials == nullptr) return;
  f32x4 *dst = reinterpret_cast<f32x4 *>(a.partials) +
               (p.b * a.s.slices + p.slice) * (a.K + 1) * a.quads + quad;
  // one tap at a time for the weight's sums, so that K stays a run-time number
  for (int j = 0; j < a.K && a.want_w; ++j) {
    const int64_t back = (int64_t)j * a.dil;
    float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    limit = end;
    for (int64_t t = p.last - 1; t >= p.first; --t) {
      if (seg != nullptr && t + 1 < p.last && seg[t + 1] != seg[t]) limit = t + 1;
      const int64_t q = t + back;
      if (q >= limit || q < 0) continue;
      float v[4], x[4];
      unpack4(g[q * a.quads], v);
      unpack_x<CODES>(p.halo ? load_halo(a, p, t) : load_x<CODES>(a, p, t, scale_at), p.halo, x);
      for (int c = 0; c < 4; ++c) s[c] += v[c] * x[c];
    }
    if (p.on) dst[(a.K - 1 - j) * a.quads] = f32x4{s[0], s[1], s[2], s[3]};
  }
  if (p.on) dst[a.K * a.quads] = f32x4{sum_b[0], sum_b[1], sum_b[2], sum_b[3]};
}

// A tile's positions, from the last.  kClear: every pair counts; kTested: the
// slice's own positions' pairs that no boundary cuts; kHalo: the same of the
// halo's positions, which have x in bf16 and pairs with the sequence only.
enum Tile { kClear, kTested, kHalo };
template <int D, int T, bool CODES, bool WANT_W, Tile KIND>
__device__ __forceinline__ void conv_tile(const ConvBackArgs &a, const ConvPlace &p, int64_t t0,
                                          uint64_t begins, const u32x2 (&win)[T + 3 * D],
                                          const XRow (&xr)[T], const float (&w)[4][4],
                                          float (&sum_w)[4][4], float (&sum_b)[4]) {
  constexpr int K = 4;
  u32x2 o[T];
#pragma unroll
  for (int i = T - 1; i >= 0; --i) {
    const int64_t t = t0 + i;
    float dx[4] = {0.0f, 0.0f, 0.0f, 0.0f}, x[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    if (WANT_W) unpack_x<CODES>(xr[i], KIND == kHalo, x);
#pragma unroll
    for (int j = 0; j < K; ++j) {
      const uint64_t between = (((uint64_t)1 << (j * D)) - 1) << (i + 1);
      if (KIND == kClear || (t >= p.first && (begins & between) == 0 &&
                             (KIND != kHalo || t + j * D >= 0))) {
        float v[4];
        unpack4(win[i + j * D], v);
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          dx[c] += w[c][j] * v[c];
          if (WANT_W) sum_w[c][j] += v[c] * x[c];
          if (WANT_W && KIND != kHalo && j == 0) sum_b[c] += v[c];
        }
      }
    }
    o[i] = u32x2{pack_bf16(dx[0], dx[1]), pack_bf16(dx[2], dx[3])};
  }
  // (a lane past the last channel repeats another's values at its place)
  u32x2 *dst = KIND == kHalo ? a.ghalo : a.gx;
  if (dst == nullptr) return;
  dst += (KIND == kHalo ? (p.b + 1) * a.halo_len + t0 : p.b * a.seq + t0) * a.quads + p.quad0;
#pragma unroll
  for (int i = 0; i < T; ++i)
    if (KIND == kClear || t0 + i >= p.first)
      __builtin_nontemporal_store(o[i], dst + i * a.quads + p.lane);
}

// A slice's sums: a row of partials for each tap and the bias.
template <int K>
__device__ __forceinline__ void store_sums(const ConvBackArgs &a, const ConvPlace &p,
                                           const float (&sum_w)[4][K], const float (&sum_b)[4]) {
  if (!p.on) return;
  f32x4 *dst = reinterpret_cast<f32x4 *>(a.partials) +
               (p.b * a.s.slices + p.slice) * (K + 1) * a.quads + p.quad0 + p.lane;
#pragma unroll
  for (int j = 0; j < K; ++j)
    dst[(K - 1 - j) * a.quads] = f32x4{sum_w[0][j], sum_w[1][j], sum_w[2][j], sum_w[3][j]};
  dst[K * a.quads] = f32x4{sum_b[0], sum_b[1], sum_b[2], sum_b[3]};
}

template <int D, bool CODES, bool WANT_W>
__global__ __launch_bounds__(kConvBlock) void conv_backward_k4_kernel(const ConvBackArgs a) {
  constexpr int K = 4, H = (K - 1) * D;
  constexpr int T = 8;  // positions of a tile
  static_assert(T + H < 64, "a tile and the rows ahead of it fit one mask");
  const uint32_t unit =
      blockIdx.x * kConvWaves + __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  if (unit >= a.units) return;
  const ConvPlace p = conv_place(a, unit);
  const uint32_t scale_at = CODES ? scale_of(a, p) : 0u;
  float w[4][K];  // [channel][tap j back]
  {
    const u32x4 *wp = reinterpret_cast<const u32x4 *>(a.w) + (p.quad0 + p.lane) * 2;
    float f[8], h[8];
    unpack_bf16x8(wp[0], f);
    unpack_bf16x8(wp[1], h);
#pragma unroll
    for (int j = 0; j < K; ++j) {
      w[0][j] = f[K - 1 - j];
      w[1][j] = f[2 * K - 1 - j];
      w[2][j] = h[K - 1 - j];
      w[3][j] = h[2 * K - 1 - j];
    }
  }
  float sum_w[4][K], sum_b[4];
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    sum_b[c] = 0.0f;
#pragma unroll
    for (int j = 0; j < K; ++j) sum_w[c][j] = 0.0f;
  }
  const u32x2 *g = a.g + p.b * a.seq * a.quads + p.quad0;
  // row i of the window is position t0 + i: the tile, then the rows ahead
  u32x2 win[T + H];
  int64_t t0 = p.last - T;
  if (p.halo) {  // a few positions: each tile loads its whole window
    for (;; t0 -= T) {
      XRow xr[T] = {};
#pragma unroll
      for (int i = 0; i < T + H; ++i) {
        win[i] = (g + min(max(t0 + i, (int64_t)0), a.seq - 1) * a.quads)[p.lane];
        if (WANT_W && i < T) xr[i] = load_halo(a, p, max(t0 + i, p.first));
      }
      const uint64_t begins = begins_mask(a, load_seg(a, p.b, t0), t0);
      conv_tile<D, T, CODES, WANT_W, kHalo>(a, p, t0, begins, win, xr, w, sum_w, sum_b);
      if (t0 <= p.first) break;
    }
    if constexpr (WANT_W) store_sums<K>(a, p, sum_w, sum_b);
    return;
  }
#pragma unroll
  for (int i = 0; i < H; ++i) {
    // (past the row's end: its last row, not used)
    win[T + i] = (g + min(p.last + i, a.seq - 1) * a.quads)[p.lane];
  }
  // A tile's rows, all loads at once; rows below the slice repeat its first, and
  // their values are not used.  The next tile's are loaded while one is worked on
  // (after the last, the first rows once more).
  u32x2 next_g[T];
  XRow next_x[T] = {};
  auto load_tile = [&](int64_t at) {
#pragma unroll
    for (int i = 0; i < T; ++i) {
      const int64_t t = max(at + i, p.first);
      next_g[i] = (g + t * a.quads)[p.lane];
      if (WANT_W) next_x[i] = load_x<CODES>(a, p, t, scale_at);
    }
  };
  load_tile(t0);
  SegPair next_seg = load_seg(a, p.b, t0);
  for (;;) {
    XRow xr[T];
#pragma unroll
    for (int i = 0; i < T; ++i) {
      win[i] = next_g[i];
      xr[i] = next_x[i];
    }
    const uint64_t begins = begins_mask(a, next_seg, t0);
    load_tile(t0 - T);
    next_seg = load_seg(a, p.b, t0 - T);
    // every pair of the tile counts: the whole tile is the slice's own, inside
    // the row, and no segment begins in it or in the rows ahead
    const bool clear = t0 >= p.first &&
                       (begins & ((((uint64_t)1 << (T + H - 1)) - 1) << 1)) == 0;
    if (clear)
      conv_tile<D, T, CODES, WANT_W, kClear>(a, p, t0, begins, win, xr, w, sum_w, sum_b);
    else
      conv_tile<D, T, CODES, WANT_W, kTested>(a, p, t0, begins, win, xr, w, sum_w, sum_b);
    if (t0 <= p.first) break;
    t0 -= T;
    // the rows ahead of the next tile are this window's first H
    // (the compiler makes it a move of its own, which it then splits into registers)
    for (int i = H - 1; i >= 0; --i) win[T + i] = win[i];
  }
  if constexpr (WANT_W) store_sums<K>(a, p, sum_w, sum_b);
}

// The weight's and the bias's gradients from the slices' sums.
template <int COLUMNS>
__global__ __launch_bounds__(kJoinThreads) void conv_join_kernel(const float *partials,
                                                                 int64_t rows, int K,
                                                                 int64_t channels,
                                                                 float *grad_weight,
                                                                 float *grad_bias) {
  const int64_t col = (int64_t)blockIdx.x * COLUMNS + threadIdx.x % COLUMNS;
  const int64_t cols = (K + 1) * channels;
  const bool bias = col >= K * channels;
  const bool on = col < cols && (bias ? grad_bias : grad_weight) != nullptr;
  const double s = join_column<COLUMNS>(partials + col, rows, cols, on);
  if (threadIdx.x >= COLUMNS || !on) return;
  const int64_t k = col / channels, c = col % channels;
  if (bias)
    grad_bias[c] = (float)s;
  else
    grad_weight[c * K + k] = (float)s;
}

__global__ __launch_bounds__(256) void fill_zero_kernel(u32x4 *dst, int64_t n) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i < n) dst[i] = u32x4{0u, 0u, 0u, 0u};
}

template <bool CODES, bool WANT_W>
void launch_k4(const ConvBackArgs &a, dim3 grid, hipStream_t s) {
  switch (a.dil) {
#define ENGRAM_CONV_CASE(D)                                                                    \
  case D:                                                                                      \
    hipLaunchKernelGGL((conv_backward_k4_kernel<D, CODES, WANT_W>), grid, dim3(kConvBlock), 0, s, \
                       a);                                                                     \
    break;
    ENGRAM_CONV_CASE(1)
    ENGRAM_CONV_CASE(2)
    ENGRAM_CONV_CASE(3)
    ENGRAM_CONV_CASE(4)
    ENGRAM_CONV_CASE(5)
    ENGRAM_CONV_CASE(6)
    ENGRAM_CONV_CASE(7)
    ENGRAM_CONV_CASE(8)
#undef ENGRAM_CONV_CASE
  }
}

}  // namespace
}  // namespace engram

int engram::launch_conv_backward(const ConvBackwardCall &c, void *stream) {
  hipStream_t st = as_stream(stream);
  const bool empty = c.batch == 0 || c.seq == 0;
  const bool sums = c.grad_weight != nullptr || c.grad_bias != nullptr;
  const ConvBackwardShape s =
      conv_backward_shape(c.batch, c.seq, c.halo_len, c.channels, c.K, c.dilation);
  const int64_t units = c.batch * s.slices * s.groups;
  const int64_t blocks = ceil_div(units, kConvWaves);
  const int64_t cols = (c.K + 1) * c.channels;
  const int64_t halo_words = c.batch * c.halo_len * c.channels / 8;
  if (!grid_fits(blocks, kConvBlock) || !grid_fits(ceil_div(cols, 16), kJoinThreads) ||
      !grid_fits(ceil_div(halo_words, 256), 256))
    return ENGRAM_EINVAL;
  if (empty && c.grad_halo != nullptr && halo_words > 0)
    hipLaunchKernelGGL(fill_zero_kernel, dim3((unsigned)ceil_div(halo_words, 256)), dim3(256), 0,
                       st, static_cast<u32x4 *>(c.grad_halo), halo_words);
  if (!empty) {
    ConvBackArgs a = {};
    a.g = static_cast<const u32x2 *>(c.grad_out);
    a.x = static_cast<const u32x2 *>(c.x);
    a.codes = reinterpret_cast<const uint32_t *>(c.codes);
    a.scales = c.scales;
    a.code_width = c.code_width;
    a.code_blocks = c.channels / c.code_width * ceil_div(c.code_width, kActBlock);
    a.halo = static_cast<const u32x2 *>(c.halo);
    a.seg = c.seg;
    a.w = static_cast<const uint16_t *>(c.weight);
    a.gx = static_cast<u32x2 *>(c.grad_x);
    a.ghalo = static_cast<u32x2 *>(c.grad_halo);
    a.partials = sums ? c.partials : nullptr;
    a.batch = c.batch;
    a.seq = c.seq;
    a.halo_len = c.halo_len;
    a.quads = s.quads;
    a.units = units;
    a.s = s;
    a.K = c.K;
    a.dil = c.dilation;
    a.want_w = c.grad_weight != nullptr;
    const dim3 grid((unsigned)blocks);
    const bool codes = c.codes != nullptr;
    // the register-window kernel sums the weight's gradient with the bias's: a
    // bias alone (no x given) takes the plain one
    if (conv_windowed(c.K, c.dilation) && (a.want_w || !sums)) {
      if (!sums)
        launch_k4<false, false>(a, grid, st);
      else if (codes)
        launch_k4<true, true>(a, grid, st);
      else
        launch_k4<false, true>(a, grid, st);
    } else if (codes) {
      hipLaunchKernelGGL(conv_backward_generic_kernel<true>, grid, dim3(kConvBlock), 0, st, a);
    } else {
      hipLaunchKernelGGL(conv_backward_generic_kernel<false>, grid, dim3(kConvBlock), 0, st, a);
    }
  }
  if (sums) {
    const int64_t rows = empty ? 0 : c.batch * s.slices;
    const int columns = join_columns(rows);
    const dim3 grid((unsigned)ceil_div(cols, columns));
    if (columns == 64)
      hipLaunchKernelGGL(conv_join_kernel<64>, grid, dim3(kJoinThreads), 0, st, c.partials, rows,
                         c.K, c.channels, c.grad_weight, c.grad_bias);
    else
      hipLaunchKernelGGL(conv_join_kernel<16>, grid, dim3(kJoinThreads), 0, st, c.partials, rows,
                         c.K, c.channels, c.grad_weight, c.grad_bias);
  }
  return launch_status();
}
