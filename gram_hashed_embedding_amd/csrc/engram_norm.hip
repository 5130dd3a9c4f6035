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
// Bound by HBM: 9 to 21 bytes a value against 10 to 30 operations; a few rows
// by latency.  Measured on MI355X, 65,536 rows of 24 groups of 256, float
// stream, one gate a group, 8-bit checkpoint of y: forward 945 us (5.6 TB/s),
// backward 1236 us (5.5 TB/s), where a streaming copy reaches 6.5 TB/s.  8 rows
// of one group of 6144: 5.2 us.  One group a row: [8192, 6144] forward 120 us (5.0
// TB/s), backward 213 (4.2 TB/s); the norm alone of [16384, 4096] in bf16 54 and 125
// us.  Two to four chunks a lane take 128 to 246 registers, which leaves 2 or 3
// wavefronts a SIMD; the 1024-thread backward of two chunks (groups past 8192
// channels) spills 290 to 390 bytes a lane ([2048, 16384]: 276 us, 1.5 TB/s), that of
// one chunk with a float stream 20.
//
// Layout.  A lane holds chunks of 8 adjacent channels (16 bytes of bf16); a
// group of up to 512 channels is a power of two of lanes of one wavefront, so
// its means are DPP adds with no LDS and no barrier; wider groups take a
// wavefront with several chunks a lane, or a block (one LDS exchange a mean).
// A block keeps its columns and takes rows in turn, so weights stay in registers
// and the backward's sums over rows accumulate there; each block leaves one fp32
// row of sums, which a second kernel adds in block order in fp64.  Two chunks a
// lane where one does was slower (groups of 256 on 16 lanes: forward 1079 us,
// backward 1710); so was holding the backward to 128 registers for a fourth
// wavefront a SIMD (1993 us: it spills).
#include "engram_layer_dev.h"

namespace engram {
namespace {

struct NormArgs {
  NormShape s;
  const void *residual;
  const void *y, *gate, *w_post, *scale, *w_next;
  void *out, *next;
  float *rstd_post, *rstd_next;
  int8_t *y_codes;
  float *y_scales;
  int8_t *next_codes;
  float *next_scales;
  const void *grad_out, *grad_next;
  void *grad_residual, *grad_y, *grad_gate;
  float *partials;  // [rowblocks][2][channels]: sums of dR a yh, of grad_next xh
  float *grad_w_post, *grad_scale, *grad_w_next;
  int64_t code_blocks;  // 8-bit blocks of a group
  float eps, alpha, inv_n;
  int gate_kind;  // 0 none, 1 one a group, 2 one a channel
};

// A lane's eight values of a group are two runs of four channels, at the
// offsets a and b of the group.  With a bf16 stream they are adjacent (16
// bytes a lane).  With a float stream they are LANES runs apart, so that a
// wavefront's 16-byte accesses of the stream are side by side too (32 bytes a
// lane in two halves touch every line twice: the training step above took
// 2415 us so and 2320 us split).
struct Span {
  int a, b;
  bool on_a, on_b;
};
template <class RT>
constexpr bool kSplit = sizeof(RT) == 4;

template <class RT, int LANES>
__device__ __forceinline__ Span span_of(int lane, int item, int n, bool ok) {
  Span p;
  if (kSplit<RT>) {
    p.a = (lane + 2 * item * LANES) * 4;
    p.b = p.a + LANES * 4;
  } else {
    p.a = (lane + item * LANES) * 8;
    p.b = p.a + 4;
  }
  p.on_a = ok && p.a < n;
  p.on_b = ok && p.b < n;
  return p;
}

// bf16 arrays: eight values as four words, zero where there is none.
template <class RT>
__device__ __forceinline__ u32x4 load_bf16(const void *base, int64_t at, const Span &p,
                                           bool live) {
  const uint16_t *q = static_cast<const uint16_t *>(base) + at;
  u32x4 v = {0u, 0u, 0u, 0u};
  if (kSplit<RT>) {
    if (p.on_a && live) {
      const u32x2 h = *reinterpret_cast<const u32x2 *>(q + p.a);
      v.x = h.x;
      v.y = h.y;
    }
    if (p.on_b && live) {
      const u32x2 h = *reinterpret_cast<const u32x2 *>(q + p.b);
      v.z = h.x;
      v.w = h.y;
    }
  } else if (p.on_a && live) {
    v = *reinterpret_cast<const u32x4 *>(q + p.a);
  }
  return v;
}
template <class RT>
__device__ __forceinline__ void store_bf16(void *base, int64_t at, const Span &p, bool live,
                                           const u32x4 &v) {
  uint16_t *q = static_cast<uint16_t *>(base) + at;
  if (kSplit<RT>) {
    if (p.on_a && live)
      __builtin_nontemporal_store(u32x2{v.x, v.y}, reinterpret_cast<u32x2 *>(q + p.a));
    if (p.on_b && live)
      __builtin_nontemporal_store(u32x2{v.z, v.w}, reinterpret_cast<u32x2 *>(q + p.b));
  } else if (p.on_a && live) {
    __builtin_nontemporal_store(v, reinterpret_cast<u32x4 *>(q + p.a));
  }
}

// Rows of the stream: bf16 bits (uint16_t) or float.
template <class RT>
struct Row;
template <>
struct Row<uint16_t> {
  typedef u32x4 Raw;
  static __device__ __forceinline__ Raw load(const void *base, int64_t at, const Span &p,
                                             bool live) {
    return load_bf16<uint16_t>(base, at, p, live);
  }
  static __device__ __forceinline__ void unpack(const Raw &r, float (&f)[8]) {
    unpack_bf16x8(r, f);
  }
  // Rounds f to what is stored.
  static __device__ __forceinline__ void store(void *base, int64_t at, const Span &p, bool live,
                                               float (&f)[8]) {
    const u32x4 v = pack_bf16x8(f);
    store_bf16<uint16_t>(base, at, p, live, v);
    unpack_bf16x8(v, f);
  }
};
template <>
struct Row<float> {
  struct Raw {
    f32x4 a, b;
  };
  static __device__ __forceinline__ Raw load(const void *base, int64_t at, const Span &p,
                                             bool live) {
    const float *q = static_cast<const float *>(base) + at;
    Raw r = {f32x4{0.f, 0.f, 0.f, 0.f}, f32x4{0.f, 0.f, 0.f, 0.f}};
    if (p.on_a && live) r.a = *reinterpret_cast<const f32x4 *>(q + p.a);
    if (p.on_b && live) r.b = *reinterpret_cast<const f32x4 *>(q + p.b);
    return r;
  }
  static __device__ __forceinline__ void unpack(const Raw &r, float (&f)[8]) {
    f[0] = r.a.x; f[1] = r.a.y; f[2] = r.a.z; f[3] = r.a.w;
    f[4] = r.b.x; f[5] = r.b.y; f[6] = r.b.z; f[7] = r.b.w;
  }
  static __device__ __forceinline__ void store(void *base, int64_t at, const Span &p, bool live,
                                               float (&f)[8]) {
    float *q = static_cast<float *>(base) + at;
    if (p.on_a && live)
      __builtin_nontemporal_store(f32x4{f[0], f[1], f[2], f[3]},
                                  reinterpret_cast<f32x4 *>(q + p.a));
    if (p.on_b && live)
      __builtin_nontemporal_store(f32x4{f[4], f[5], f[6], f[7]},
                                  reinterpret_cast<f32x4 *>(q + p.b));
  }
};

// A sum over a group's lanes: within a wavefront, or over a block through
// LDS (`part` has one slot a wavefront).  One barrier a call is enough because
// each call takes the other set than the call before it, whichever means the
// rows have (`set`, alike in the whole block, is carried from call to call and
// from row to row): a set is written again after the barrier of the call
// between, which every wavefront reaches after its reads of that set.
template <int LANES>
__device__ __forceinline__ float group_sum(float v, float (*part)[16], int &set) {
  if (LANES <= 64) return lanes_sum<(LANES <= 64 ? LANES : 64)>(v);
  v = lanes_sum<64>(v);
  set ^= 1;
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

// The 8-bit codes of a lane's eight values.  The lanes whose values lie in one
// block of 128 channels take their maximum together: 16 lanes of adjacent
// values; 32 of split ones (a run each), or, in a group of at most 128
// channels, all its lanes with both runs.
template <class RT, int LANES>
__device__ __forceinline__ void store_codes(const float (&x)[8], const Span &p, bool live,
                                            int64_t at, int64_t unit, int64_t code_blocks,
                                            int8_t *codes, float *scales) {
  uint32_t ma = 0u, mb = 0u;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const uint32_t xa = __float_as_uint(x[e]) & 0x7fffffffu;
    const uint32_t xb = __float_as_uint(x[4 + e]) & 0x7fffffffu;
    ma = xa > ma ? xa : ma;
    mb = xb > mb ? xb : mb;
  }
  ma = p.on_a && live ? ma : 0u;
  mb = p.on_b && live ? mb : 0u;
  float *scale = scales + unit * code_blocks;
  if (kSplit<RT> && LANES >= 32) {
    const CodeScale ca = code_scale(lanes_max<32>(ma)), cb = code_scale(lanes_max<32>(mb));
    if (p.on_a && live) {
      *reinterpret_cast<uint32_t *>(codes + at + p.a) = code_bytes(x, ca.inv);
      if (p.a % 128 == 0) scale[p.a / 128] = ca.scale;
    }
    if (p.on_b && live) {
      *reinterpret_cast<uint32_t *>(codes + at + p.b) = code_bytes(x + 4, cb.inv);
      if (p.b % 128 == 0) scale[p.b / 128] = cb.scale;
    }
    return;
  }
  const CodeScale c = code_scale(lanes_max<(LANES < 16 ? LANES : 16)>(ma > mb ? ma : mb));
  if (kSplit<RT>) {
    if (p.on_a && live) *reinterpret_cast<uint32_t *>(codes + at + p.a) = code_bytes(x, c.inv);
    if (p.on_b && live) *reinterpret_cast<uint32_t *>(codes + at + p.b) = code_bytes(x + 4, c.inv);
  } else if (p.on_a && live) {
    *reinterpret_cast<u32x2 *>(codes + at + p.a) = code_bytes8(x, c.inv);
  }
  if (p.on_a && live && p.a % 128 == 0) scale[p.a / 128] = c.scale;
}

// Eight codes and their scales, zero where there is none.
struct Codes {
  u32x2 words;
  float scale_a, scale_b;
};
template <class RT>
__device__ __forceinline__ Codes load_codes(const int8_t *codes, const float *scales, int64_t at,
                                            int64_t unit, int64_t code_blocks, const Span &p,
                                            bool live) {
  Codes c = {u32x2{0u, 0u}, 0.0f, 0.0f};
  const float *scale = scales + unit * code_blocks;
  if (kSplit<RT>) {
    if (p.on_a && live) {
      c.words.x = *reinterpret_cast<const uint32_t *>(codes + at + p.a);
      c.scale_a = scale[p.a / 128];
    }
    if (p.on_b && live) {
      c.words.y = *reinterpret_cast<const uint32_t *>(codes + at + p.b);
      c.scale_b = scale[p.b / 128];
    }
  } else if (p.on_a && live) {
    c.words = *reinterpret_cast<const u32x2 *>(codes + at + p.a);
    c.scale_a = c.scale_b = scale[p.a / 128];
  }
  return c;
}

// Where a block's threads stand.
struct Place {
  int lane, trow;
  int64_t group, row0, stride;  // rows row0, row0 + stride, ...
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
  p.row0 = rb * s.trows;
  p.stride = s.rowblocks * s.trows;
  return p;
}

template <class RT, int LANES, int ITEMS, int THREADS>
__global__ __launch_bounds__(THREADS) void norm_forward_kernel(const NormArgs a) {
  __shared__ float part[2][16];
  int set = 0;  // of part, the last one written
  const Place p = place_of<LANES, THREADS>(a.s);
  const int n = (int)a.s.chunks * 8;
  const int64_t g0 = p.group * n;  // the group's first channel
  Span sp[ITEMS];
  float sw[ITEMS][8];
  u32x4 wn[ITEMS];
#pragma unroll
  for (int i = 0; i < ITEMS; ++i) {
    sp[i] = span_of<RT, LANES>(p.lane, i, n, p.group_ok);
#pragma unroll
    for (int e = 0; e < 8; ++e) sw[i][e] = 1.0f;
    if (a.scale != nullptr) unpack_bf16x8(load_bf16<RT>(a.scale, g0, sp[i], true), sw[i]);
    if (a.w_post != nullptr) {
      float f[8];
      unpack_bf16x8(load_bf16<RT>(a.w_post, g0, sp[i], true), f);
#pragma unroll
      for (int e = 0; e < 8; ++e) sw[i][e] *= f[e];
    }
    wn[i] = u32x4{0u, 0u, 0u, 0u};
    if (a.w_next != nullptr) wn[i] = load_bf16<RT>(a.w_next, g0, sp[i], true);
  }
  for (int64_t t0 = p.row0; t0 < a.s.rows; t0 += p.stride) {
    const int64_t t = t0 + p.trow;
    const bool row_ok = t < a.s.rows;
    const int64_t unit = t * a.s.groups + p.group;
    const int64_t at = t * a.s.channels + g0;
    typename Row<RT>::Raw r[ITEMS];
    u32x4 y[ITEMS], z[ITEMS];
    float zg = 0.0f;
    // every load of the row before the first use
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
      r[i] = Row<RT>::load(a.residual, at, sp[i], row_ok);
      if (a.y != nullptr) y[i] = load_bf16<RT>(a.y, at, sp[i], row_ok);
      if (a.gate_kind == 2) z[i] = load_bf16<RT>(a.gate, at, sp[i], row_ok);
    }
    if (a.gate_kind == 1 && p.group_ok && row_ok) zg = gate_at(a.gate, unit);
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
      const float u = 1.0f / sqrtf(group_sum<LANES>(sq, part, set) * a.inv_n + a.eps);
      float ag = 1.0f, unused;
      if (a.gate_kind == 1) sigmoid(zg, ag, unused);
      const float ua = u * ag;
#pragma unroll
      for (int i = 0; i < ITEMS; ++i) {
        float f[8];
        unpack_bf16x8(y[i], f);
        if (a.y_codes != nullptr)
          store_codes<RT, LANES>(f, sp[i], row_ok, at, unit, a.code_blocks, a.y_codes,
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
        Row<RT>::store(a.out, at, sp[i], row_ok, o[i]);
      }
      if (a.rstd_post != nullptr && p.lane == 0 && p.group_ok && row_ok) a.rstd_post[unit] = u;
    }
    if (a.w_next != nullptr) {
      float sq = 0.0f;
#pragma unroll
      for (int i = 0; i < ITEMS; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e)
          sq += (e < 4 ? sp[i].on_a : sp[i].on_b) ? o[i][e] * o[i][e] : 0.0f;
      const float v = 1.0f / sqrtf(group_sum<LANES>(sq, part, set) * a.inv_n + a.eps);
#pragma unroll
      for (int i = 0; i < ITEMS; ++i) {
        float w[8];
        unpack_bf16x8(wn[i], w);
#pragma unroll
        for (int e = 0; e < 8; ++e) w[e] *= o[i][e] * v;
        const u32x4 packed = pack_bf16x8(w);
        store_bf16<RT>(a.next, at, sp[i], row_ok, packed);
        if (a.next_codes != nullptr) {
          unpack_bf16x8(packed, w);
          store_codes<RT, LANES>(w, sp[i], row_ok, at, unit, a.code_blocks, a.next_codes,
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
  int set = 0;  // of part, the last one written
  __shared__ float sums[THREADS == LANES ? 1 : THREADS * ITEMS * 8];
  const Place p = place_of<LANES, THREADS>(a.s);
  const int n = (int)a.s.chunks * 8;
  const int64_t g0 = p.group * n;
  Span sp[ITEMS];
  u32x4 wp[ITEMS], sc[ITEMS], wn[ITEMS];
  float sum_d[ITEMS][8], sum_n[ITEMS][8];
#pragma unroll
  for (int i = 0; i < ITEMS; ++i) {
    sp[i] = span_of<RT, LANES>(p.lane, i, n, p.group_ok);
    const u32x4 ones = {0x3f803f80u, 0x3f803f80u, 0x3f803f80u, 0x3f803f80u};
    wp[i] = sc[i] = wn[i] = ones;
    if (a.w_post != nullptr) wp[i] = load_bf16<RT>(a.w_post, g0, sp[i], true);
    if (a.scale != nullptr) sc[i] = load_bf16<RT>(a.scale, g0, sp[i], true);
    if (a.w_next != nullptr) wn[i] = load_bf16<RT>(a.w_next, g0, sp[i], true);
#pragma unroll
    for (int e = 0; e < 8; ++e) sum_d[i][e] = sum_n[i][e] = 0.0f;
  }
  const bool branch = a.y != nullptr || a.y_codes != nullptr;
  for (int64_t t0 = p.row0; t0 < a.s.rows; t0 += p.stride) {
    const int64_t t = t0 + p.trow;
    const bool row_ok = t < a.s.rows;  // a lane without a value reads nothing and adds zeros
    const int64_t unit = t * a.s.groups + p.group;
    const int64_t at = t * a.s.channels + g0;
    typename Row<RT>::Raw go[ITEMS], ro[ITEMS];
    u32x4 gn[ITEMS], y[ITEMS], z[ITEMS];
    Codes yc[ITEMS];
    float u = 0.0f, v = 0.0f, zg = 0.0f;
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
      go[i] = Row<RT>::load(a.grad_out, at, sp[i], row_ok && a.grad_out != nullptr);
      if (a.grad_next != nullptr) {
        gn[i] = load_bf16<RT>(a.grad_next, at, sp[i], row_ok);
        ro[i] = Row<RT>::load(a.out, at, sp[i], row_ok);
      }
      if (a.y != nullptr)
        y[i] = load_bf16<RT>(a.y, at, sp[i], row_ok);
      else if (a.y_codes != nullptr)
        yc[i] = load_codes<RT>(a.y_codes, a.y_scales, at, unit, a.code_blocks, sp[i], row_ok);
      if (a.gate_kind == 2) z[i] = load_bf16<RT>(a.gate, at, sp[i], row_ok);
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
      const float m = group_sum<LANES>(s, part, set) * a.inv_n;
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
          code_values(yc[i].words.x, yc[i].scale_a, yh[i]);
          code_values(yc[i].words.y, yc[i].scale_b, yh[i] + 4);
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
          if (a.grad_gate != nullptr)
            store_bf16<RT>(a.grad_gate, at, sp[i], row_ok, pack_bf16x8(zf));
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          sum_d[i][e] += q[i][e] * yh[i][e];
          q[i][e] *= w[e] * k[e];
          s += q[i][e] * yh[i][e];
        }
      }
      s = group_sum<LANES>(s, part, set);
      const float m = s * a.inv_n;
      if (a.grad_y != nullptr) {
#pragma unroll
        for (int i = 0; i < ITEMS; ++i) {
#pragma unroll
          for (int e = 0; e < 8; ++e) q[i][e] = u * (q[i][e] - yh[i][e] * m);
          store_bf16<RT>(a.grad_y, at, sp[i], row_ok, pack_bf16x8(q[i]));
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
        Row<RT>::store(a.grad_residual, at, sp[i], row_ok, dr[i]);
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
      float *dst = a.partials + (rb * 2 + which) * a.s.channels + g0;
#pragma unroll
      for (int i = 0; i < ITEMS; ++i) {
        if (sp[i].on_a)
          *reinterpret_cast<f32x4 *>(dst + sp[i].a) =
              f32x4{mine[i][0], mine[i][1], mine[i][2], mine[i][3]};
        if (sp[i].on_b)
          *reinterpret_cast<f32x4 *>(dst + sp[i].b) =
              f32x4{mine[i][4], mine[i][5], mine[i][6], mine[i][7]};
      }
    }
  }
}

// The weights' gradients from the row blocks' sums.
template <int COLUMNS>
__global__ __launch_bounds__(kJoinThreads) void norm_join_kernel(const NormArgs a) {
  const int64_t c = (int64_t)blockIdx.x * COLUMNS + threadIdx.x % COLUMNS;
  const bool on = c < a.s.channels && a.s.rows > 0;
  const int64_t stride = 2 * a.s.channels;
  const double d = join_column<COLUMNS>(a.partials + c, a.s.rowblocks, stride, on);
  const double n =
      join_column<COLUMNS>(a.partials + a.s.channels + c, a.s.rowblocks, stride, on);
  if (threadIdx.x >= COLUMNS || c >= a.s.channels) return;
  const uint16_t *wp = static_cast<const uint16_t *>(a.w_post);
  const uint16_t *sc = static_cast<const uint16_t *>(a.scale);
  if (a.grad_w_post != nullptr) a.grad_w_post[c] = (float)(d * (sc ? bf16_lo(sc[c]) : 1.0f));
  if (a.grad_scale != nullptr) a.grad_scale[c] = (float)(d * (wp ? bf16_lo(wp[c]) : 1.0f));
  if (a.grad_w_next != nullptr) a.grad_w_next[c] = (float)n;
}

NormArgs norm_args(const engram_norm_args &c, const NormShape &s) {
  NormArgs a = {};
  a.s = s;
  a.residual = c.d_residual;
  a.y = c.d_y;
  a.gate = c.d_gate;
  a.w_post = c.d_w_post;
  a.scale = c.d_scale;
  a.w_next = c.d_w_next;
  a.out = c.d_out;
  a.next = c.d_next;
  a.rstd_post = c.d_rstd_post;
  a.rstd_next = c.d_rstd_next;
  a.y_codes = c.d_y_codes;
  a.y_scales = c.d_y_scales;
  a.next_codes = c.d_next_codes;
  a.next_scales = c.d_next_scales;
  a.grad_out = c.d_grad_out;
  a.grad_next = c.d_grad_next;
  a.grad_residual = c.d_grad_residual;
  a.grad_y = c.d_grad_y;
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
  const NormShape s = norm_forward_shape(c.rows, c.channels, c.groups);
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
    ENGRAM_NORM_CASE(64, 3, 256)
    ENGRAM_NORM_CASE(64, 4, 256)
    ENGRAM_NORM_CASE(256, 3, 256)
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
      !grid_fits(ceil_div(c.channels, 16), kJoinThreads))
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
  if (a.grad_w_post != nullptr || a.grad_scale != nullptr || a.grad_w_next != nullptr) {
    const int columns = join_columns(c.rows > 0 ? s.rowblocks : 0);
    const dim3 grid((unsigned)ceil_div(c.channels, columns));
    if (columns == 64)
      hipLaunchKernelGGL(norm_join_kernel<64>, grid, dim3(kJoinThreads), 0, st, a);
    else
      hipLaunchKernelGGL(norm_join_kernel<16>, grid, dim3(kJoinThreads), 0, st, a);
  }
  return launch_status();
}
