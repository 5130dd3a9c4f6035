// beam_choice.cpp -- a beam search's selection on the CPU, through its entry point.  The
// argument names the check; the exit status is the number of those that fail.
#include "vocab_wave.h"

#include "engram_beam.hip"

#include <sys/mman.h>

#include <algorithm>
#include <numeric>
#include <string>

namespace engram {
int launch_distill(const engram_distill_args &) { abort(); }
int launch_distill_backward(const engram_distill_args &) { abort(); }
}  // namespace engram

namespace {

using namespace engram;

int failed = 0;
void check(bool ok, const std::string &what) {
  printf("%s: %s\n", what.c_str(), ok ? "ok" : "FAILED");
  failed += !ok;
}

constexpr size_t kPage = 4096;

// Rows of logits of T that begin `first` bytes behind a page each, with pages that can be
// taken away from under a row.
template <class T>
struct Logits {
  size_t pages;
  int64_t rows, vocab, stride;
  char *memory;
  T *first;
  Logits(int64_t rows_, int64_t vocab_, size_t at)
      : pages((at + vocab_ * sizeof(T) + kPage - 1) / kPage), rows(rows_), vocab(vocab_),
        stride(pages * kPage / sizeof(T)) {
    memory = static_cast<char *>(mmap(nullptr, rows * pages * kPage, PROT_READ | PROT_WRITE,
                                      MAP_PRIVATE | MAP_ANONYMOUS, -1, 0));
    if (memory == MAP_FAILED) abort();
    first = reinterpret_cast<T *>(memory + at);
  }
  ~Logits() { munmap(memory, rows * pages * kPage); }
  T *row(int64_t r) { return first + r * stride; }
  void take(int64_t r) { mprotect(memory + r * pages * kPage, pages * kPage, PROT_NONE); }
};
template <class T>
T value(float v) {
  if constexpr (sizeof(T) == 2) return (uint16_t)(__float_as_uint(v) >> 16);
  else return v;
}

uint32_t state = 1;
float draw() {  // -4 to 4, of 16 bits
  state = state * 1664525u + 1013904223u;
  return (float)(state >> 16) * 0x1p-13f - 4.0f;
}

struct Chosen {
  std::vector<float> scores;
  std::vector<int64_t> parents, tokens;
  std::vector<uint8_t> finished;
};
template <class T>
Chosen choose(const T *logits, int64_t stride, const std::vector<float> &scores,
              const std::vector<uint8_t> &finished, int64_t eos, int64_t beams, int64_t vocab,
              int64_t count) {
  const int64_t batch = (int64_t)scores.size() / beams;
  const size_t need = engram_beam_select_workspace(batch, beams, vocab);
  std::vector<char> space(need + 16, (char)0x7f);
  void *workspace =
      reinterpret_cast<void *>((reinterpret_cast<uintptr_t>(space.data()) + 15) & ~(uintptr_t)15);
  Chosen c;
  c.scores.resize(batch * count);
  c.parents.resize(batch * count);
  c.tokens.resize(batch * count);
  c.finished.resize(batch * count);
  if (engram_beam_select(logits, sizeof(T) == 2 ? ENGRAM_BF16 : ENGRAM_F32, stride, scores.data(),
                         finished.empty() ? nullptr : finished.data(), eos, batch, beams, vocab,
                         count, c.scores.data(), c.parents.data(), c.tokens.data(),
                         c.finished.data(), workspace, need, nullptr) != ENGRAM_OK)
    abort();
  return c;
}

// A finished beam's logits are not read: none of its memory is there.
template <class T>
void finished_rows(int64_t vocab, size_t at) {
  Logits<T> z(4, vocab, at);
  for (int64_t r = 0; r < 4; ++r)
    for (int64_t v = 0; v < vocab; ++v) z.row(r)[v] = value<T>(draw());
  z.take(1);
  z.take(3);
  const Chosen c = choose(z.first, z.stride, {-30.0f, -1.0f, -30.0f, -2.0f}, {0, 1, 0, 1}, 2, 4,
                          vocab, 6);
  check(c.parents[0] == 1 && c.tokens[0] == 2 && c.scores[0] == -1.0f && c.finished[0] &&
            c.parents[1] == 3 && c.tokens[1] == 2 && c.scores[1] == -2.0f && c.finished[1] &&
            c.parents[2] % 2 == 0 && c.scores[2] < -30.0f,
        "finished beams, " + std::to_string(vocab) + " values, " + std::to_string(at));
}

// Beams whose logits are all a mask's lowest value: each id has 1 / vocab of the probability,
// below what the other beam offers, equal ones by place.
template <class T>
void masked_beams(int64_t vocab, float mask) {
  Logits<T> z(3, vocab, 0);
  for (int64_t v = 0; v < vocab; ++v) {
    z.row(0)[v] = z.row(2)[v] = value<T>(mask);
    z.row(1)[v] = value<T>(v == vocab / 2 ? 9.0f : v == 1 ? 8.0f : 0.0f);
  }
  const Chosen c = choose(z.first, z.stride, {-5.0f, -5.5f, -5.25f}, {}, -1, 3, vocab, 5);
  const double log = ::log((double)vocab);
  bool ok = c.parents[0] == 1 && c.tokens[0] == vocab / 2 && c.parents[1] == 1 && c.tokens[1] == 1;
  for (int k = 2; k < 5; ++k)
    ok &= c.parents[k] == 0 && c.tokens[k] == k - 2 &&
          fabs((double)c.scores[k] + 5.0 + log) < 1e-5;
  check(ok, "masked beams, " + std::to_string(vocab) + " values at " + std::to_string(mask));
}

// Beams that are copies of one another, each at another place in a cache line, with equal
// scores: equal logits have equal values, in the order of beams and then of ids.
template <class T>
void equal_beams(int64_t vocab) {
  const int64_t stride = vocab + 3;
  std::vector<T> memory(5 * stride + 64);
  for (size_t at : {0, 1, 13}) {
    for (int64_t v = 0; v < vocab; ++v) {
      const T x = value<T>(draw());
      for (int64_t w = 0; w < 5; ++w) memory[at + w * stride + v] = x;
    }
    const Chosen c = choose(memory.data() + at, stride, std::vector<float>(5, -7.0f), {}, -1, 5,
                            vocab, 10);
    std::vector<int64_t> order(5 * vocab);
    std::iota(order.begin(), order.end(), 0);
    std::stable_sort(order.begin(), order.end(), [&](int64_t i, int64_t j) {
      return Chunk<T>::one(memory[at + i % vocab]) > Chunk<T>::one(memory[at + j % vocab]);
    });
    bool ok = true;
    for (int k = 0; k < 10; ++k)
      ok &= c.parents[k] == order[k] / vocab && c.tokens[k] == order[k] % vocab;
    check(ok, "equal beams, " + std::to_string(vocab) + " values from " + std::to_string(at));
  }
}

}  // namespace

int main(int, char **argv) {
  const std::string which = argv[1];
  if (which == "finished")
    for (int64_t vocab : {3, 100, 5000})
      for (size_t at : {0, 4, 100, 124}) {
        finished_rows<uint16_t>(vocab, at);
        finished_rows<float>(vocab, at);
      }
  if (which == "masked")
    for (int64_t vocab : {1000, 9000}) {
      masked_beams<uint16_t>(vocab, __uint_as_float(0xff7f0000u));
      masked_beams<float>(vocab, __uint_as_float(0xff7fffffu));
      masked_beams<float>(vocab, -1e30f);
      masked_beams<float>(vocab, -1e9f);
    }
  if (which == "equal")
    for (int64_t vocab : {700, 1003, 5001, 20011}) {
      equal_beams<uint16_t>(vocab);
      equal_beams<float>(vocab);
    }
  return failed;
}
