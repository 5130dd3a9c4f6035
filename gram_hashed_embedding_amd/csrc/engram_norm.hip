// engram_norm.hip -- the residual norm and its backward, for gfx950.
//
// What is computed is stated with engram_residual_norm in include/
// engram_layer.h.  The norms and the branch follow the NeMo AutoModel v0.7
// API page "qwen3_8_flash_next.engram", Qwen3_8_FlashNextPLELayer
// (_apply_branch_norm, norm_query / norm_key / norm_conv: grouped RMS norms
// of a hyper-connection's branches); the order norm, gate, scale, add, norm is
// the reading taken, the page does not give one.
//
// Mathematics.  Everything is per group of n channels of a row: two means (of
// y^2 and out^2; in the backward of gx * xh and q * yh), each needed before
// the values after it.  One kernel holds a group in registers between its
// means, so each array crosses HBM once.  The gate's gradient needs no sum of
// its own: with one gate a group, sum(dR * scale * w * yh) * a * (1 - a) is
// (1 - a) times the sum the backward of the norm takes anyway.
//
// Bound by HBM: 9 to 21 bytes a value against 10 to 30 operations.
//
// Layout.  A lane holds chunks of 8 adjacent channels (16 bytes of bf16); a
// group of up to 512 channels is a power of two of lanes of one wavefront, so
// its means are DPP adds with no LDS and no barrier; wider groups take a
// wavefront with several chunks a lane, or a block (one LDS exchange a mean).
// A block keeps its columns and walks rows, so weights stay in registers and
// the backward's sums over rows accumulate there; each block leaves one fp32
// row of sums, which a second kernel adds in block order in fp64.
#include "engram_layer_dev.h"

namespace engram {
namespace {

struct NormArgs {
  NormShape s;
  const void *residual;
  const u32x4 *y;
  const void *gate;
  const u32x4 *w_post, *scale, *w_next;
  void *out;
  u32x4 *next;
  float *rstd_post, *rstd_next;
  u32x2 *y_codes;
  float *y_scales;
  u32x2 *next_codes;
  float *next_scales;
  const void *grad_out;
  const u32x4 *grad_next;
  void *grad_residual;
  u32x4 *grad_y;
  void *grad_gate;
  float *partials;  // [rowblocks][2][channels]: sums of dR a yh, of grad_next xh
  float *grad_w_post, *grad_scale, *grad_w_next;
  int64_t code_blocks;  // 8-bit blocks of a group
  float eps, alpha, inv_n;
  int gate_kind;  // 0 none, 1 one a group, 2 one a channel
};

// Eight values of a row of type RT (bf16 bits or float), chunk c.
template <class RT>
struct Row;
template <>
struct Row<uint16_t> {
  typedef u32x4 Raw;
  static __device__ __forceinline__ Raw load(const void *p, int64_t c) {
    return static_cast<const u32x4 *>(p)[c];
  }
  static __device__ __forceinline__ void unpack(const Raw &r, float (&f)[8]) {
    unpack_bf16x8(r, f);
  }
  // Rounds f to what is stored.
  static __device__ __forceinline__ void store(void *p, int64_t c, float (&f)[8]) {
    const u32x4 v = pack_bf16x8(f);
    static_cast<u32x4 *>(p)[c] = v;
    unpack_bf16x8(v, f);
  }
  static __device__ __forceinline__ Raw zero() { return Raw{0u, 0u, 0u, 0u}; }
};
template <>
struct Row<float> {
  struct Raw {
    f32x4 a, b;
  };
  static __device__ __forceinline__ Raw load(const void *p, int64_t c) {
    const f32x4 *q = static_cast<const f32x4 *>(p) + 2 * c;
    return Raw{q[0], q[1]};
  }
  static __device__ __forceinline__ void unpack(const Raw &r, float (&f)[8]) {
    f[0] = r.a.x; f[1] = r.a.y; f[2] = r.a.z; f[3] = r.a.w;
    f[4] = r.b.x; f[5] = r.b.y; f[6] = r.b.z; f[7] = r.b.w;
  }
  static __device__ __forceinline__ void store(void *p, int64_t c, float (&f)[8]) {
    f32x4 *q = static_cast<f32x4 *>(p) + 2 * c;
    q[0] = f32x4{f[0], f[1], f[2], f[3]};
    q[1] = f32x4{f[4], f[5], f[6], f[7]};
  }
  static __device__ __forceinline__ Raw zero() {
    return Raw{f32x4{0.f, 0.f, 0.f, 0.f}, f32x4{0.f, 0.f, 0.f, 0.f}};
  }
};

// A sum over a group's lanes: within a wavefront, or over a block through
// LDS (kWide: `part` has one slot a wavefront; consecutive calls alternate
// between two sets, so one barrier a call is enough).
template <int LANES>
__device__ __forceinline__ float group_sum(float v, float (*part)[16], int set) {
  if (LANES <= 64) return lanes_sum<(LANES <= 64 ? LANES : 64)>(v);
  v = lanes_sum<64>(v);
  if ((threadIdx.x & 63) == 0) part[set][threadIdx.x >> 6] = v;
  __syncthreads();
  float s = 0.0f;
#pragma unroll
  for (int w = 0; w < LANES / 64; ++w) s += part[set][w];
  return s;
}

// The gate and one minus it, from one exponential that cannot overflow.
__device__ __forceinline__ void sigmoid(float z, float &a, float &one_minus) {
  const float e = __expf(-fabsf(z));
  const float r = 1.0f / (1.0f + e);
  a = z >= 0.0f ? r : e * r;
  one_minus = z >= 0.0f ? e * r : r;
  if (z != z) a = one_minus = z;
}

__device__ __forceinline__ float gate_at(const void *gate, int64_t i) {
  return bf16_lo(static_cast<const uint16_t *>(gate)[i]);
}

// 8-bit codes of a lane's chunk `c8` of the row (chunk j of the group).  The
// 16 lanes (or the group's fewer) that share a block take its maximum.
template <int LANES>
__device__ __forceinline__ void store_codes(const float (&x)[8], bool ok, int64_t c8, int64_t j,
                                            int64_t unit, int64_t code_blocks, u32x2 *codes,
                                            float *scales) {
  const uint32_t m = lanes_max<(LANES < 16 ? LANES : 16)>(ok ? max_magnitude(x) : 0u);
  const CodeScale cs = code_scale(m);
  if (!ok) return;
  codes[c8] = code_bytes8(x, cs.inv);
  if ((j & 15) == 0) scales[unit * code_blocks + (j >> 4)] = cs.scale;
}

// Where a block's threads stand.
struct Place {
  int lane, trow;
  int64_t group, row0, row_end;
  bool group_ok;
};
template <int LANES, int THREADS>
__device__ __forceinline__ Place place_of(const NormShape &s) {
  Place p;
  const int slot = threadIdx.x / LANES;
  p.lane = threadIdx.x % LANES;
  p.trow = slot / s.gcols;
  const int64_t cb = blockIdx.x % s.colblocks, rb = blockIdx.x / s.colblocks;
  p.group = cb * s.gcols + slot % s.gcols;
  p.group_ok = p.group < s.groups;
  p.row0 = rb * s.per_block;
  p.row_end = min(p.row0 + s.per_block, s.rows);
  return p;
}

template <class RT, int LANES, int ITEMS, int THREADS>
__global__ __launch_bounds__(THREADS) void norm_forward_kernel(const NormArgs a) {
  __shared__ float part[2][16];
  const Place p = place_of<LANES, THREADS>(a.s);
  const int64_t row_chunks = a.s.channels / 8;
  const int64_t g0 = p.group * a.s.chunks;  // the group's first chunk of a row
  bool on[ITEMS];
  float sw[ITEMS][8];
  u32x4 wn[ITEMS];
#pragma unroll
  for (int i = 0; i < ITEMS; ++i) {
    const int64_t j = p.lane + (int64_t)i * LANES;
    on[i] = p.group_ok && j < a.s.chunks;
    const int64_t c = on[i] ? g0 + j : 0;
    float f[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) sw[i][e] = 1.0f;
    if (a.scale != nullptr) unpack_bf16x8(a.scale[c], sw[i]);
    if (a.w_post != nullptr) {
      unpack_bf16x8(a.w_post[c], f);
#pragma unroll
      for (int e = 0; e < 8; ++e) sw[i][e] *= f[e];
    }
    wn[i] = a.w_next != nullptr ? a.w_next[c] : u32x4{0u, 0u, 0u, 0u};
  }
  for (int64_t t0 = p.row0; t0 < p.row_end; t0 += a.s.trows) {
    const int64_t t = t0 + p.trow;
    const bool row_ok = t < p.row_end;
    const int64_t tt = row_ok ? t : p.row0;
    const int64_t unit = tt * a.s.groups + p.group;
    const int64_t base = tt * row_chunks + g0;
    typename Row<RT>::Raw r[ITEMS];
    u32x4 y[ITEMS], z[ITEMS];
    float zg = 0.0f;
    // every load of the row before the first use
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
      const int64_t c = base + p.lane + (int64_t)i * LANES;
      r[i] = on[i] ? Row<RT>::load(a.residual, c) : Row<RT>::zero();
      if (a.y != nullptr) y[i] = on[i] ? a.y[c] : u32x4{0u, 0u, 0u, 0u};
      if (a.gate_kind == 2)
        z[i] = on[i] ? static_cast<const u32x4 *>(a.gate)[c] : u32x4{0u, 0u, 0u, 0u};
    }
    if (a.gate_kind == 1 && p.group_ok) zg = gate_at(a.gate, unit);
    float o[ITEMS][8];
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) Row<RT>::unpack(r[i], o[i]);
    if (a.y != nullptr) {
      float sq = 0.0f;
#pragma unroll
      for (int i = 0; i < ITEMS; ++i) {
        float f[8];
        unpack_bf16x8(y[i], f);
#pragma unroll
        for (int e = 0; e < 8; ++e) sq += f[e] * f[e];
      }
      const float u = 1.0f / sqrtf(group_sum<LANES>(sq, part, 0) * a.inv_n + a.eps);
      float ag = 1.0f, unused;
      if (a.gate_kind == 1) sigmoid(zg, ag, unused);
      const float ua = u * ag;
#pragma unroll
      for (int i = 0; i < ITEMS; ++i) {
        float f[8];
        unpack_bf16x8(y[i], f);
        if (a.y_codes != nullptr)
          store_codes<LANES>(f, on[i] && row_ok, base + p.lane + (int64_t)i * LANES,
                             p.lane + (int64_t)i * LANES, unit, a.code_blocks, a.y_codes,
                             a.y_scales);
        if (a.gate_kind == 2) {
          float zf[8];
          unpack_bf16x8(z[i], zf);
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            float ac;
            sigmoid(zf[e], ac, unused);
            o[i][e] = a.alpha * o[i][e] + sw[i][e] * (ac * (f[e] * u));
          }
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e) o[i][e] = a.alpha * o[i][e] + sw[i][e] * (f[e] * ua);
        }
        if (on[i] && row_ok)
          Row<RT>::store(a.out, base + p.lane + (int64_t)i * LANES, o[i]);
      }
      if (a.rstd_post != nullptr && p.lane == 0 && p.group_ok && row_ok) a.rstd_post[unit] = u;
    }
    if (a.w_next != nullptr) {
      float sq = 0.0f;
#pragma unroll
      for (int i = 0; i < ITEMS; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e) sq += on[i] ? o[i][e] * o[i][e] : 0.0f;
      const float v = 1.0f / sqrtf(group_sum<LANES>(sq, part, 1) * a.inv_n + a.eps);
#pragma unroll
      for (int i = 0; i < ITEMS; ++i) {
        float w[8];
        unpack_bf16x8(wn[i], w);
#pragma unroll
        for (int e = 0; e < 8; ++e) w[e] *= o[i][e] * v;
        const u32x4 packed = pack_bf16x8(w);
        const int64_t j = p.lane + (int64_t)i * LANES;
        if (on[i] && row_ok) a.next[base + j] = packed;
        if (a.next_codes != nullptr) {
          unpack_bf16x8(packed, w);
          store_codes<LANES>(w, on[i] && row_ok, base + j, j, unit, a.code_blocks, a.next_codes,
                             a.next_scales);
        }
      }
      if (a.rstd_next != nullptr && p.lane == 0 && p.group_ok && row_ok) a.rstd_next[unit] = v;
    }
  }
}

template <class RT, int LANES, int ITEMS, int THREADS>
__global__ __launch_bounds__(THREADS) void norm_backward_kernel(const NormArgs a) {
  __shared__ float part[2][16];
  __shared__ float sums[THREADS == LANES ? 1 : THREADS * ITEMS * 8];
  const Place p = place_of<LANES, THREADS>(a.s);
  const int64_t row_chunks = a.s.channels / 8;
  const int64_t g0 = p.group * a.s.chunks;
  bool on[ITEMS];
  u32x4 wp[ITEMS], sc[ITEMS], wn[ITEMS];
  float sum_d[ITEMS][8], sum_n[ITEMS][8];
  const u32x4 ones = {0x3f803f80u, 0x3f803f80u, 0x3f803f80u, 0x3f803f80u};
#pragma unroll
  for (int i = 0; i < ITEMS; ++i) {
    const int64_t j = p.lane + (int64_t)i * LANES;
    on[i] = p.group_ok && j < a.s.chunks;
    const int64_t c = on[i] ? g0 + j : 0;
    wp[i] = a.w_post != nullptr ? a.w_post[c] : ones;
    sc[i] = a.scale != nullptr ? a.scale[c] : ones;
    wn[i] = a.w_next != nullptr ? a.w_next[c] : ones;
#pragma unroll
    for (int e = 0; e < 8; ++e) sum_d[i][e] = sum_n[i][e] = 0.0f;
  }
  const bool branch = a.y != nullptr || a.y_codes != nullptr;
  const u32x4 zero4 = {0u, 0u, 0u, 0u};
  for (int64_t t0 = p.row0; t0 < p.row_end; t0 += a.s.trows) {
    const int64_t t = t0 + p.trow;
    const bool row_ok = t < p.row_end;
    const int64_t tt = row_ok ? t : p.row0;
    const int64_t unit = tt * a.s.groups + p.group;
    const int64_t base = tt * row_chunks + g0 + p.lane;
    typename Row<RT>::Raw go[ITEMS], ro[ITEMS];
    u32x4 gn[ITEMS], y[ITEMS], z[ITEMS];
    u32x2 yc[ITEMS];
    float ys[ITEMS];
    bool live[ITEMS];
    float u = 0.0f, v = 0.0f, zg = 0.0f;
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
      const int64_t j = p.lane + (int64_t)i * LANES, c = base + (int64_t)i * LANES;
      live[i] = on[i] && row_ok;  // a lane without a value reads nothing and adds zeros
      go[i] = live[i] && a.grad_out != nullptr ? Row<RT>::load(a.grad_out, c) : Row<RT>::zero();
      if (a.grad_next != nullptr) {
        gn[i] = live[i] ? a.grad_next[c] : zero4;
        ro[i] = live[i] ? Row<RT>::load(a.out, c) : Row<RT>::zero();
      }
      if (a.y != nullptr) {
        y[i] = live[i] ? a.y[c] : zero4;
      } else if (a.y_codes != nullptr) {
        yc[i] = live[i] ? a.y_codes[c] : u32x2{0u, 0u};
        ys[i] = live[i] ? a.y_scales[unit * a.code_blocks + (j >> 4)] : 0.0f;
      }
      if (a.gate_kind == 2) z[i] = live[i] ? static_cast<const u32x4 *>(a.gate)[c] : zero4;
    }
    if (p.group_ok && row_ok) {
      if (branch) u = a.rstd_post[unit];
      if (a.grad_next != nullptr) v = a.rstd_next[unit];
      if (a.gate_kind == 1) zg = gate_at(a.gate, unit);
    }
    float dr[ITEMS][8];
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) Row<RT>::unpack(go[i], dr[i]);
    if (a.grad_next != nullptr) {
      float s = 0.0f;
#pragma unroll
      for (int i = 0; i < ITEMS; ++i) {
        float w[8], g[8], x[8];
        unpack_bf16x8(wn[i], w);
        unpack_bf16x8(gn[i], g);
        Row<RT>::unpack(ro[i], x);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float xh = x[e] * v;
          s += g[e] * w[e] * xh;
          sum_n[i][e] += g[e] * xh;
        }
      }
      const float m = group_sum<LANES>(s, part, 0) * a.inv_n;
#pragma unroll
      for (int i = 0; i < ITEMS; ++i) {
        float w[8], g[8], x[8];
        unpack_bf16x8(wn[i], w);
        unpack_bf16x8(gn[i], g);
        Row<RT>::unpack(ro[i], x);
#pragma unroll
        for (int e = 0; e < 8; ++e) dr[i][e] += v * (g[e] * w[e] - x[e] * v * m);
      }
    }
    if (branch) {
      float ag = 1.0f, bg = 0.0f, s = 0.0f;
      if (a.gate_kind == 1) sigmoid(zg, ag, bg);
      float q[ITEMS][8], yh[ITEMS][8];
#pragma unroll
      for (int i = 0; i < ITEMS; ++i) {
        float w[8], k[8];
        if (a.y != nullptr) {
          unpack_bf16x8(y[i], yh[i]);
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            yh[i][e] = code_value(yc[i].x, e, ys[i]);
            yh[i][4 + e] = code_value(yc[i].y, e, ys[i]);
          }
        }
        unpack_bf16x8(wp[i], w);
        unpack_bf16x8(sc[i], k);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          yh[i][e] *= u;
          q[i][e] = dr[i][e] * ag;
        }
        if (a.gate_kind == 2) {
          float zf[8];
          unpack_bf16x8(z[i], zf);
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            float ac, bc;
            sigmoid(zf[e], ac, bc);
            q[i][e] *= ac;
            zf[e] = bc * (q[i][e] * (w[e] * k[e])) * yh[i][e];
          }
          if (a.grad_gate != nullptr && live[i])
            static_cast<u32x4 *>(a.grad_gate)[base + (int64_t)i * LANES] = pack_bf16x8(zf);
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          sum_d[i][e] += q[i][e] * yh[i][e];
          q[i][e] *= w[e] * k[e];
          s += q[i][e] * yh[i][e];
        }
      }
      s = group_sum<LANES>(s, part, 1);
      const float m = s * a.inv_n;
      if (a.grad_y != nullptr) {
#pragma unroll
        for (int i = 0; i < ITEMS; ++i) {
#pragma unroll
          for (int e = 0; e < 8; ++e) q[i][e] = u * (q[i][e] - yh[i][e] * m);
          if (live[i]) a.grad_y[base + (int64_t)i * LANES] = pack_bf16x8(q[i]);
        }
      }
      if (a.gate_kind == 1 && a.grad_gate != nullptr && p.lane == 0 && p.group_ok && row_ok)
        static_cast<uint16_t *>(a.grad_gate)[unit] = (uint16_t)pack_bf16(bg * s, 0.0f);
    }
    if (a.grad_residual != nullptr) {
#pragma unroll
      for (int i = 0; i < ITEMS; ++i) {
#pragma unroll
        for (int e = 0; e < 8; ++e) dr[i][e] *= a.alpha;
        if (live[i]) Row<RT>::store(a.grad_residual, base + (int64_t)i * LANES, dr[i]);
      }
    }
  }
  if (a.partials == nullptr) return;
  // one row of sums a block: the rows a block works on side by side are added
  // first, in order
  const int64_t rb = blockIdx.x / a.s.colblocks;
#pragma unroll
  for (int which = 0; which < 2; ++which) {
    float(&mine)[ITEMS][8] = which == 0 ? sum_d : sum_n;
    if (THREADS != LANES && a.s.trows > 1) {
      __syncthreads();
#pragma unroll
      for (int i = 0; i < ITEMS; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e) sums[(i * 8 + e) * THREADS + threadIdx.x] = mine[i][e];
      __syncthreads();
      if (p.trow == 0) {
        for (int r = 1; r < a.s.trows; ++r)
#pragma unroll
          for (int i = 0; i < ITEMS; ++i)
#pragma unroll
            for (int e = 0; e < 8; ++e)
              mine[i][e] += sums[(i * 8 + e) * THREADS + threadIdx.x + r * a.s.gcols * LANES];
      }
    }
    if (p.trow == 0) {
#pragma unroll
      for (int i = 0; i < ITEMS; ++i) {
        const int64_t j = p.lane + (int64_t)i * LANES;
        if (!on[i]) continue;
        f32x4 *dst = reinterpret_cast<f32x4 *>(a.partials + (rb * 2 + which) * a.s.channels) +
                     2 * (g0 + j);
        dst[0] = f32x4{mine[i][0], mine[i][1], mine[i][2], mine[i][3]};
        dst[1] = f32x4{mine[i][4], mine[i][5], mine[i][6], mine[i][7]};
      }
    }
  }
}

// The weights' gradients from the row blocks' sums: a block takes 64
// channels, each of its 16 wavefronts every 16th row block, in fp64.
constexpr int kJoinThreads = 1024;
__global__ __launch_bounds__(kJoinThreads) void norm_join_kernel(const NormArgs a) {
  __shared__ double part[2][16][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t c = (int64_t)blockIdx.x * 64 + lane;
  double d = 0.0, n = 0.0;
  if (c < a.s.channels && a.s.rows > 0) {
#pragma unroll 4
    for (int64_t rb = wave; rb < a.s.rowblocks; rb += 16) {
      d += a.partials[(rb * 2) * a.s.channels + c];
      n += a.partials[(rb * 2 + 1) * a.s.channels + c];
    }
  }
  part[0][wave][lane] = d;
  part[1][wave][lane] = n;
  __syncthreads();
  if (wave != 0 || c >= a.s.channels) return;
  d = n = 0.0;
#pragma unroll
  for (int w = 0; w < 16; ++w) {
    d += part[0][w][lane];
    n += part[1][w][lane];
  }
  const uint16_t *wp = reinterpret_cast<const uint16_t *>(a.w_post);
  const uint16_t *sc = reinterpret_cast<const uint16_t *>(a.scale);
  if (a.grad_w_post != nullptr) a.grad_w_post[c] = (float)(d * (sc ? bf16_lo(sc[c]) : 1.0f));
  if (a.grad_scale != nullptr) a.grad_scale[c] = (float)(d * (wp ? bf16_lo(wp[c]) : 1.0f));
  if (a.grad_w_next != nullptr) a.grad_w_next[c] = (float)n;
}

NormArgs norm_args(const engram_norm_args &c, const NormShape &s) {
  NormArgs a = {};
  a.s = s;
  a.residual = c.d_residual;
  a.y = static_cast<const u32x4 *>(c.d_y);
  a.gate = c.d_gate;
  a.w_post = static_cast<const u32x4 *>(c.d_w_post);
  a.scale = static_cast<const u32x4 *>(c.d_scale);
  a.w_next = static_cast<const u32x4 *>(c.d_w_next);
  a.out = c.d_out;
  a.next = static_cast<u32x4 *>(c.d_next);
  a.rstd_post = c.d_rstd_post;
  a.rstd_next = c.d_rstd_next;
  a.y_codes = reinterpret_cast<u32x2 *>(c.d_y_codes);
  a.y_scales = c.d_y_scales;
  a.next_codes = reinterpret_cast<u32x2 *>(c.d_next_codes);
  a.next_scales = c.d_next_scales;
  a.grad_out = c.d_grad_out;
  a.grad_next = static_cast<const u32x4 *>(c.d_grad_next);
  a.grad_residual = c.d_grad_residual;
  a.grad_y = static_cast<u32x4 *>(c.d_grad_y);
  a.grad_gate = c.d_grad_gate;
  a.grad_w_post = c.d_grad_w_post;
  a.grad_scale = c.d_grad_scale;
  a.grad_w_next = c.d_grad_w_next;
  if (c.d_grad_w_post != nullptr || c.d_grad_scale != nullptr || c.d_grad_w_next != nullptr)
    a.partials = static_cast<float *>(c.d_workspace);
  a.code_blocks = ceil_div(s.chunks * 8, kActBlock);
  a.eps = c.eps;
  a.alpha = c.residual_scale;
  a.inv_n = 1.0f / (float)(s.chunks * 8);
  a.gate_kind = c.gate_width == 0 ? 0 : c.gate_width == c.groups ? 1 : 2;
  return a;
}

}  // namespace
}  // namespace engram

// Every (lanes, items, threads) norm_shape gives a kernel of at most MAX items.
#define ENGRAM_NORM_COMMON(CASE) \
  CASE(4, 1, 256) CASE(8, 1, 256) CASE(16, 1, 256) CASE(32, 1, 256) CASE(64, 1, 256) \
  CASE(64, 2, 256) CASE(256, 1, 256) CASE(256, 2, 256) CASE(1024, 1, 1024) CASE(1024, 2, 1024)

int engram::launch_residual_norm(const engram_norm_args &c) {
  const NormShape s =
      norm_shape(c.rows, c.channels, c.groups, kNormForwardItems, kNormForwardBlocks);
  const NormArgs a = norm_args(c, s);
  if (!grid_fits(s.colblocks * s.rowblocks, s.threads)) return ENGRAM_EINVAL;
  const dim3 grid((unsigned)(s.colblocks * s.rowblocks)), block(s.threads);
  hipStream_t st = as_stream(c.stream);
  switch (s.lanes * 8 + s.items) {
#define ENGRAM_NORM_CASE(L, I, T)                                                           \
  case L * 8 + I:                                                                           \
    if (c.residual_type == ENGRAM_F32)                                                      \
      hipLaunchKernelGGL((norm_forward_kernel<float, L, I, T>), grid, block, 0, st, a);     \
    else                                                                                    \
      hipLaunchKernelGGL((norm_forward_kernel<uint16_t, L, I, T>), grid, block, 0, st, a);  \
    break;
    ENGRAM_NORM_COMMON(ENGRAM_NORM_CASE)
    ENGRAM_NORM_CASE(64, 4, 256)
    ENGRAM_NORM_CASE(256, 4, 256)
#undef ENGRAM_NORM_CASE
    default: return ENGRAM_EINVAL;
  }
  return launch_status();
}

int engram::launch_residual_norm_backward(const engram_norm_args &c) {
  const NormShape s = norm_backward_shape(c.rows, c.channels, c.groups);
  const NormArgs a = norm_args(c, s);
  if (!grid_fits(s.colblocks * s.rowblocks, s.threads) ||
      !grid_fits(ceil_div(c.channels, 64), kJoinThreads))
    return ENGRAM_EINVAL;
  hipStream_t st = as_stream(c.stream);
  if (c.rows > 0) {
    const dim3 grid((unsigned)(s.colblocks * s.rowblocks)), block(s.threads);
    switch (s.lanes * 8 + s.items) {
#define ENGRAM_NORM_CASE(L, I, T)                                                           \
  case L * 8 + I:                                                                           \
    if (c.residual_type == ENGRAM_F32)                                                      \
      hipLaunchKernelGGL((norm_backward_kernel<float, L, I, T>), grid, block, 0, st, a);    \
    else                                                                                    \
      hipLaunchKernelGGL((norm_backward_kernel<uint16_t, L, I, T>), grid, block, 0, st, a); \
    break;
      ENGRAM_NORM_COMMON(ENGRAM_NORM_CASE)
#undef ENGRAM_NORM_CASE
      default: return ENGRAM_EINVAL;
    }
  }
  if (a.grad_w_post != nullptr || a.grad_scale != nullptr || a.grad_w_next != nullptr)
    hipLaunchKernelGGL(norm_join_kernel, dim3((unsigned)ceil_div(c.channels, 64)),
                       dim3(kJoinThreads), 0, st, a);
  return launch_status();
}
