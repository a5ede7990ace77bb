// Which products the tensor-core kernel's epilogue moves value by value, asked of the rule itself (no GPU): one launch
// of a call that is split over its rank buffers looks at the buffers of that launch.
#include <cstdio>

#include "mm.h"

using namespace hoc;

static MmParams params(int part0, int parts) {
  MmParams P{};
  P.part0 = part0;
  P.parts = parts;
  P.groups = P.experts = 1024;
  P.in = P.out = 64;
  P.ld_rows = P.ld_dy = P.ld_y = P.ld_res = P.ld_w = 64;
  for (int p = 0; p < kMaxRanks; ++p) {
    const char* at = reinterpret_cast<const char*>(size_t(p + 1) << 20);
    P.cap[p] = 8;
    P.y[p] = const_cast<char*>(at);
    P.pre[p] = P.res[p] = reinterpret_cast<const __nv_bfloat16*>(at + 4096);
    P.pre_out[p] = const_cast<char*>(at + 8192);
  }
  return P;
}

template <class T>
static void move_by_2(T*& p) { p = reinterpret_cast<T*>(reinterpret_cast<uintptr_t>(p) + 2); }

int main() {
  int bad = 0;
  for (int part0 = 0; part0 < kMaxRanks; ++part0)
    for (int parts = 1; part0 + parts <= kMaxRanks; ++parts)
      for (int off = -1; off < kMaxRanks; ++off)
        for (int what = 0; what < 4; ++what)
          for (int mode = 0; mode < 3; ++mode) {
            MmParams P = params(part0, parts);
            if (off >= 0) {
              if (what == 0) P.y[off] = static_cast<char*>(P.y[off]) + 2;
              if (what == 1) move_by_2(P.pre[off]);
              if (what == 2) move_by_2(P.res[off]);
              if (what == 3) P.pre_out[off] = static_cast<char*>(P.pre_out[off]) + 2;
            }
            // the bias gradient, which is what pre_out is of a weight gradient, is not the epilogue's
            const bool here = off >= part0 && off < part0 + parts && (what != 3 || mode == kForward);
            if (mm_tc_loose(P, mode) == here) continue;
            if (bad++ < 5)
              printf("launch of buffers %d..%d, tensor %d of buffer %d misaligned, product %d: want %d\n", part0,
                     part0 + parts - 1, what, off, mode, int(here));
          }
  printf(bad ? "%d WRONG\n" : "LOOSE OK\n", bad);
  return bad != 0;
}
