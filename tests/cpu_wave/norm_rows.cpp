// norm_rows.cpp -- the residual norm's kernels on the CPU, in the worst order of
// the wavefronts, with blocks that take several rows: every form of the call has to
// give, bit for bit, what blocks of one row each give (where no LDS is used twice).
// Prints one line a form; the exit status is the number of forms that differ.
#include "engram_norm.hip"

namespace {
int64_t rows_a_block = 1;
int lanes, items;
}  // namespace

namespace engram {
// The launch's shape, as this test wants it: one group a row, held by a whole block.
NormShape norm_shape(int64_t rows, int64_t channels, int64_t groups, int, int64_t, bool) {
  NormShape s = {};
  s.rows = rows;
  s.channels = channels;
  s.groups = groups;
  s.chunks = channels / groups / 8;
  s.lanes = s.threads = lanes;
  s.items = items;
  s.gcols = s.trows = 1;
  s.colblocks = groups;
  s.rowblocks = (rows + rows_a_block - 1) / rows_a_block;
  return s;
}
}  // namespace engram

namespace {

using namespace engram;

constexpr int64_t kRows = 5;

struct Random {
  uint64_t s;
  float next() {  // about [-1, 1)
    s = s * 6364136223846793005ull + 1442695040888963407ull;
    return (float)(int32_t)(s >> 32) * 0x1p-31f;
  }
};
// 16-byte aligned values: floats, or bf16 bits
template <class T>
std::vector<T> draw(int64_t n, uint64_t seed) {
  Random r = {seed};
  std::vector<T> v(n + 16);
  for (T &x : v) {
    const float f = r.next();
    if (sizeof(T) == 4) memcpy(&x, &f, 4);
    else x = (T)(__float_as_uint(f) >> 16);
  }
  return v;
}
template <class T>
T *aligned(std::vector<T> &v) {
  return reinterpret_cast<T *>((reinterpret_cast<uintptr_t>(v.data()) + 15) & ~(uintptr_t)15);
}

// Everything a call writes.
struct Result {
  std::vector<float> out, grad_residual, rstd_post, rstd_next;
  std::vector<uint16_t> next, grad_y, grad_gate;
  bool operator==(const Result &o) const {
    return same(out, o.out) && same(grad_residual, o.grad_residual) &&
           same(rstd_post, o.rstd_post) && same(rstd_next, o.rstd_next) && next == o.next &&
           grad_y == o.grad_y && grad_gate == o.grad_gate;
  }
  static bool same(const std::vector<float> &a, const std::vector<float> &b) {
    return a.size() == b.size() && memcmp(a.data(), b.data(), a.size() * 4) == 0;
  }
};

Result call(int64_t channels, bool branch, bool next, bool backward) {
  const int64_t n = kRows * channels;
  std::vector<float> residual = draw<float>(n, 1), grad_out = draw<float>(n, 2);
  std::vector<uint16_t> y = draw<uint16_t>(n, 3), grad_next = draw<uint16_t>(n, 4);
  std::vector<uint16_t> gate = draw<uint16_t>(kRows, 5), w_post = draw<uint16_t>(channels, 6);
  std::vector<uint16_t> w_next = draw<uint16_t>(channels, 7);
  // each row of another size, so that a mean of another row shows
  float *r = aligned(residual);
  for (int64_t t = 0; t < kRows; ++t)
    for (int64_t c = 0; c < channels; ++c) {
      r[t * channels + c] *= (float)(1 << t);
      uint16_t &v = aligned(y)[t * channels + c];
      v = (uint16_t)(__float_as_uint(__uint_as_float((uint32_t)v << 16) * (float)(1 << t)) >> 16);
    }
  std::vector<float> out(n + 16), grad_residual(n + 16), post(kRows), nxt(kRows);
  std::vector<uint16_t> next_out(n + 16), grad_y(n + 16), grad_gate(kRows);
  engram_norm_args a = {};
  a.rows = kRows;
  a.channels = channels;
  a.groups = 1;
  a.eps = 1e-5f;
  a.residual_scale = branch ? 0.75f : 1.0f;
  a.residual_type = ENGRAM_F32;
  if (branch) {
    a.gate_width = 1;
    a.d_gate = gate.data();
    a.d_y = aligned(y);
    a.d_w_post = aligned(w_post);
    a.d_rstd_post = post.data();
  }
  if (next) {
    a.d_w_next = aligned(w_next);
    a.d_rstd_next = nxt.data();
  }
  if (backward) {
    for (int64_t t = 0; t < kRows; ++t) post[t] = nxt[t] = 1.0f / (float)(1 << t);
    a.d_out = r;
    a.d_grad_out = aligned(grad_out);
    if (next) a.d_grad_next = aligned(grad_next);
    a.d_grad_residual = aligned(grad_residual);
    if (branch) {
      a.d_grad_y = aligned(grad_y);
      a.d_grad_gate = grad_gate.data();
    }
    launch_residual_norm_backward(a);
  } else {
    a.d_residual = r;
    if (branch) a.d_out = aligned(out);
    if (next) a.d_next = aligned(next_out);
    launch_residual_norm(a);
  }
  Result res;
  res.out.assign(aligned(out), aligned(out) + n);
  res.grad_residual.assign(aligned(grad_residual), aligned(grad_residual) + n);
  res.rstd_post = post;
  res.rstd_next = nxt;
  res.next.assign(aligned(next_out), aligned(next_out) + n);
  res.grad_y.assign(aligned(grad_y), aligned(grad_y) + n);
  res.grad_gate = grad_gate;
  return res;
}

}  // namespace

int main() {
  int differ = 0;
  const struct {
    int64_t channels;
    int lanes, items;
  } shapes[] = {{2048, 256, 1}, {4096, 256, 2}, {8192, 1024, 1}};
  for (const auto &s : shapes)
    for (int form = 0; form < 6; ++form)
      for (int order = 0; order < 2; ++order) {
        const bool backward = form >= 3, branch = form % 3 != 1, next = form % 3 != 2;
        lanes = s.lanes;
        items = s.items;
        cpu_wave::descending = order == 1;
        rows_a_block = 1;
        const Result want = call(s.channels, branch, next, backward);
        rows_a_block = kRows;
        const bool ok = call(s.channels, branch, next, backward) == want;
        printf("%s %lld channels, %s%s, wavefronts %s: %s\n", backward ? "backward" : "forward",
               (long long)s.channels, branch ? "branch" : "no branch",
               next ? ", next norm" : ", no next norm", order ? "from the last" : "from the first",
               ok ? "same" : "DIFFERENT");
        differ += !ok;
      }
  return differ;
}
