// Entry points of hoc_layer.h over the fake runtime: which errors they report.  Device memory is the heap here, and no
// kernel runs.
#include <cstdio>
#include <functional>
#include <utility>
#include <vector>

#include "fake_cudart.h"
#include "hoc_layer.h"

namespace hoc {
void set_error_detail(const char*) {}
}  // namespace hoc

int main() {
  static char at[1 << 16];
  char* a = at + (64 - reinterpret_cast<size_t>(at) % 64);
  void* p[1] = {a};
  const void* c[1] = {a};
  const int32_t* ids[1] = {reinterpret_cast<const int32_t*>(a)};
  int64_t seg[9] = {};
  const size_t capacity[1] = {40};
  const hocRowGroups_t groups = {1, 2, 1, seg, capacity};
  int32_t* status = reinterpret_cast<int32_t*>(a + 1024);
  using Call = std::pair<const char*, std::function<int()>>;
  std::vector<Call> calls;
  for (int width : {64, 61, 701})  // whole vectors; the general kernel; realigned copies
    for (int rows : {4, 40}) {
      calls.push_back({"linear", [=] { return hoc_linear(rows, a, width, a, a, a, width, width, width, HOC_ACT_GELU, a, width, a, status, nullptr); }});
      calls.push_back({"linear_dgrad", [=] { return hoc_linear_dgrad(rows, a, width, a, width, width, HOC_ACT_SILU, a, a, status, nullptr); }});
      calls.push_back({"linear_wgrad", [=] { return hoc_linear_wgrad(rows, a, width, a, width, width, width, HOC_FLOAT32, 1, a, a, status, nullptr); }});
      calls.push_back({"expert_mm", [=, &groups] { return hoc_expert_mm(&groups, c, c, c, width, width, 0, p, p, status, nullptr); }});
      calls.push_back({"expert_mm_dgrad", [=, &groups] { return hoc_expert_mm_dgrad(&groups, c, c, width, width, 1, c, p, status, nullptr); }});
      calls.push_back({"expert_mm_wgrad", [=, &groups] { return hoc_expert_mm_wgrad(&groups, c, c, width, width, HOC_BFLOAT16, 0, p, p, status, nullptr); }});
      calls.push_back({"act_grad", [=] { return hoc_act_grad(rows, width, HOC_ACT_RELU, a, a, a, nullptr); }});
    }
  calls.push_back({"ep_segments", [=, &seg] { return hoc_ep_segments(1, ids, 4, 2, 8, seg, nullptr); }});
  int bad = 0;
  auto check = [&](bool ok, const Call& c, const char* what) {
    if (!ok && bad++ < 10) printf("FAIL %s: %s\n", c.first, what);
  };
  const int earlier = 101;  // an error that somebody else has not read yet
  for (const Call& c : calls) {
    fake::refuse = false;
    fake::last = 0;
    const int before = fake::launches;
    check(c.second() == HOC_SUCCESS && fake::launches > before, c, "does not run");
    check(fake::last == 0, c, "left an error");
    fake::last = earlier;
    check(c.second() == HOC_SUCCESS, c, "an earlier error is reported as its own");
    check(fake::last == earlier, c, "an earlier error was cleared");
    fake::refuse = true;
    fake::last = 0;
    check(c.second() == HOC_ERR_CUDA, c, "a failed launch is not reported");
    check(fake::last == 0, c, "left its own error to be read by the next call");
  }
  // the most pairs that ep_segments takes, 2048 to a CTA
  fake::refuse = false;
  fake::widest = 0;
  const Call most = {"ep_segments", [&] { return hoc_ep_segments(1, ids, 0x7FFFFFFF, 1, 8, seg, nullptr); }};
  check(most.second() == HOC_SUCCESS && fake::widest == 1u << 20, most, "a grid that does not fit the pairs");
  printf(bad ? "%d WRONG\n" : "LAUNCHES OK\n", bad);
  return bad != 0;
}
