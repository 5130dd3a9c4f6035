// embed_stall.cpp -- the embedding's gradient of more tokens than are sorted by
// counting, on the CPU, with a sort that stands in for the library's: one that is
// right, and one that says that a wait of its own has expired.  A table that such
// an order cannot fill must not be left as it was found.  The exit status is the
// number of checks that fail.
#include "engram_embed.hip"

#include <algorithm>
#include <numeric>

namespace {
bool stalls = false;
int failed = 0;

void check(bool ok, const char *what) {
  printf("%s: %s\n", what, ok ? "ok" : "FAILED");
  failed += !ok;
}
}  // namespace

namespace engram {
int launch_sort_crowded(const int64_t *tokens, int64_t n, int64_t table_rows, const Plan &p,
                        void *workspace, int64_t *err, void *) {
  const Views v = views_of(p, workspace);
  uint32_t *keys = const_cast<uint32_t *>(v.sorted_keys);
  uint32_t *vals = const_cast<uint32_t *>(v.sorted_vals);
  v.scalars->stalled = stalls ? 1 : 0;
  if (stalls) {  // what the buffers held before
    std::fill(keys, keys + n, 0xdeadbeefu);
    std::fill(vals, vals + n, 0xdeadbeefu);
    add_mark(err, kStallMark);
    return ENGRAM_OK;
  }
  auto key = [&](uint32_t i) {
    return (uint32_t)(tokens[i] >= 0 && tokens[i] < table_rows ? tokens[i] : table_rows);
  };
  std::iota(vals, vals + n, 0u);
  std::stable_sort(vals, vals + n, [&](uint32_t a, uint32_t b) { return key(a) < key(b); });
  for (int64_t i = 0; i < n; ++i) keys[i] = key(vals[i]);
  return ENGRAM_OK;
}
}  // namespace engram

namespace {

using namespace engram;

constexpr int64_t kTokens = kMergeTokens + 3, kRows = 300, kChannels = 8;

template <class T>
T *aligned(std::vector<T> &v) {
  return reinterpret_cast<T *>((reinterpret_cast<uintptr_t>(v.data()) + 15) & ~(uintptr_t)15);
}

// The table after the call, from one that holds `before` everywhere.
template <class T>
std::vector<T> gradient(T before, bool accumulate, int64_t *err) {
  std::vector<int64_t> tokens(kTokens);
  std::vector<uint16_t> grads(kTokens * kChannels + 16, (uint16_t)0x3f80);  // ones
  for (int64_t i = 0; i < kTokens; ++i) tokens[i] = (i * i) % 7 == 0 ? 5 : (i * 31) % 200 - 1;
  Plan p;
  if (!make_plan(kTokens, kRows, 8, &p)) abort();
  std::vector<char> workspace(p.total + 64);
  const int64_t chunks = ceil_div(kTokens, embed_chunk(kTokens, kChannels));
  std::vector<double> partials(chunks * 2 * kChannels + 16);
  std::vector<uint8_t> present(kEmbedMarkRows);
  std::vector<T> table(kRows * kChannels + 16, before);
  const EmbedGradCall c = {tokens.data(), kTokens, aligned(grads), ENGRAM_BF16, kChannels, 0.5f,
                           kRows, sizeof(T) == 4 ? ENGRAM_F32 : ENGRAM_BF16, accumulate,
                           aligned(table), aligned(partials), present.data(), err};
  if (launch_embed_grad(c, p, aligned(workspace), nullptr) != ENGRAM_OK) abort();
  std::vector<T> res(aligned(table), aligned(table) + kRows * kChannels);
  if (!stalls && sizeof(T) == 4 && !accumulate) {
    std::vector<double> want(kRows, 0.0);
    for (int64_t t : tokens)
      if (t >= 0) want[t] += 0.5;
    bool same = true;
    for (int64_t i = 0; i < kRows * kChannels; ++i) same &= (double)res[i] == want[i / kChannels];
    check(same, "sums of a sort that holds");
  }
  return res;
}

template <class T>
bool all(const std::vector<T> &v, bool (*is)(T)) {
  return std::all_of(v.begin(), v.end(), is);
}

}  // namespace

int main() {
  int64_t err = 0;
  gradient<float>(7.0f, false, &err);
  check(err == 0, "no mark of a sort that holds");
  stalls = true;
  check(all<float>(gradient<float>(7.0f, false, &err), [](float x) { return x != x; }),
        "every float is NaN after a stalled sort");
  check(err == ENGRAM_ERR_STALLED, "the counter has the mark");
  check(all<uint16_t>(gradient<uint16_t>(0x3f80, false, nullptr),
                      [](uint16_t x) { return (x & 0x7fff) > 0x7f80; }),
        "every bf16 is NaN after a stalled sort, without a counter");
  check(all<float>(gradient<float>(7.0f, true, nullptr), [](float x) { return x == 7.0f; }),
        "a table accumulated into stays as it was");
  return failed;
}
