// Which products run on realigned copies of their operands, over the fake runtime: those launch the copies first, the
// general kernel is one launch.
#include <cstdio>

#include "fake_cudart.h"
#include "hoc_layer.h"

namespace hoc {
void set_error_detail(const char*) {}
}  // namespace hoc

int main() {
  static char at[256];
  char* a = at + (64 - reinterpret_cast<size_t>(at) % 64);
  int32_t* status = reinterpret_cast<int32_t*>(a + 64);
  const void* c[1] = {a};
  void* p[1] = {a};
  struct Case {
    int experts, rows, in, out;  // experts 0: a linear layer
    bool copies[3];              // forward, data gradient, weight gradient
  };
  const Case cases[] = {
      {0, 1, 257, 255, {true, true, false}},     // long contractions of a few rows
      {0, 1, 2047, 31, {true, false, false}},
      {0, 1, 31, 2047, {false, true, false}},
      {0, 64, 257, 255, {true, true, false}},    // a weight gradient over few rows
      {0, 256, 257, 255, {true, true, true}},
      {0, 2000, 65, 67, {true, true, true}},     // over many, few tiles
      {0, 16000, 33, 31, {true, true, true}},
      {0, 1, 65, 63, {false, false, false}},     // small
      {0, 16, 33, 31, {false, false, false}},
      {8, 1000, 9, 7, {false, false, false}},    // 125 rows to an expert
      {1, 1000, 9, 7, {false, false, true}},
      {0, 4096, 2047, 2047, {true, true, true}}, // large
      {0, 4096, 64, 128, {false, false, false}}, // whole vectors
  };
  int bad = 0;
  for (const Case& k : cases)
    for (int mode = 0; mode < 3; ++mode) {
      int64_t seg[9] = {};
      const size_t capacity[1] = {size_t(k.rows)};
      const hocRowGroups_t g = {1, k.experts, 1, seg, capacity};
      const int before = fake::launches;
      int r;
      if (mode == 0)
        r = k.experts ? hoc_expert_mm(&g, c, c, nullptr, k.in, k.out, 0, p, nullptr, status, nullptr)
                      : hoc_linear(k.rows, a, k.in, a, nullptr, nullptr, 0, k.in, k.out, 0, a, k.out, nullptr, status, nullptr);
      else if (mode == 1)
        r = k.experts ? hoc_expert_mm_dgrad(&g, c, c, k.in, k.out, 0, nullptr, p, status, nullptr)
                      : hoc_linear_dgrad(k.rows, a, k.out, a, k.in, k.out, 0, nullptr, a, status, nullptr);
      else
        r = k.experts ? hoc_expert_mm_wgrad(&g, c, c, k.in, k.out, HOC_FLOAT32, 0, p, nullptr, status, nullptr)
                      : hoc_linear_wgrad(k.rows, a, k.out, a, k.in, k.in, k.out, HOC_FLOAT32, 0, a, nullptr, status, nullptr);
      const int n = fake::launches - before;
      if (r == HOC_SUCCESS && n == (k.copies[mode] ? 3 : 1)) continue;
      ++bad;
      printf("FAIL product %d of %d rows, %d -> %d, %d experts: result %d, %d launches\n", mode, k.rows, k.in, k.out,
             k.experts, r, n);
    }
  printf(bad ? "%d WRONG\n" : "REALIGN OK\n", bad);
  return bad != 0;
}
