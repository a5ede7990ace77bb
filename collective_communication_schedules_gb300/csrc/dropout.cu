// Dropout from a counter-based generator, with the residual's addition (hoc_block.h).
//
// Element i's 16 random bits are a part of Philox4x32-10 of the counter i / 8, so that
// nothing of the mask is stored and the gradient draws it again.  Bound by its bytes:
// 32,768 x 4096 bf16 with the residual take 121 us, 0.98 of the copy rate.  Ten rounds for eight elements
// are about 8 integer operations an element, so the rest is kept short: a word's upper half
// is compared as it stands, elements are dropped by a choice before the multiply-add, and rows that
// lie together are one run, without a division (188 us before that).
#include "block.h"

namespace hoc {
namespace {

using namespace block;

struct DropArgs {
  const void *x, *r;
  void* y;
  const int64_t* seed;
  int64_t ldx, ldr, ldy, total;  // total: rows * width
  int64_t width;
  unsigned t;                    // dropped where the element's bits are below this
  float keep;                    // 65536 / (65536 - t)
  // i / width of i below 2^31 as (umulhi(magic, i) + i) >> shift (Granlund and Montgomery, 1994)
  unsigned magic, shift;
};

// Philox4x32 with 10 rounds (Salmon, Moraes, Dror, Shaw, 2011).
__device__ __forceinline__ uint4 philox(uint4 c, uint32_t k0, uint32_t k1) {
#pragma unroll
  for (int i = 0; i < 10; ++i) {
    const uint64_t a = uint64_t(0xD2511F53u) * c.x, b = uint64_t(0xCD9E8D57u) * c.z;
    c = make_uint4(uint32_t(b >> 32) ^ c.y ^ k0, uint32_t(b), uint32_t(a >> 32) ^ c.w ^ k1, uint32_t(a));
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
  return c;
}

constexpr int kDropThreads = 256, kDropAhead = 2;

// How rows lie: one after the other, so that they are one run, of which only the last group
// may be short; in rows of whole groups; or anyhow.  The first two start on 16-byte boundaries.
enum Lie { kRun, kRows, kAnyhow };

// A thread takes kDropAhead groups of eight elements.
template <class T, int LIE, bool RES>
__global__ void __launch_bounds__(kDropThreads) dropout_kernel(const __grid_constant__ DropArgs A) {
  after_the_last();
  constexpr int N = 16 / sizeof(T), Q = 8 / N;
  const T *x = static_cast<const T*>(A.x), *r = static_cast<const T*>(A.r);
  T* y = static_cast<T*>(A.y);
  const uint64_t key = A.t ? uint64_t(A.seed[0]) : 0, call = A.t ? uint64_t(A.seed[1]) : 0;
  const int64_t first = int64_t(blockIdx.x) * kDropThreads * kDropAhead + threadIdx.x;
  const int64_t groups = (A.total + 7) / 8;
  const uint32_t t = A.t << 16;
  Vec<T, N> v[kDropAhead][Q], w[kDropAhead][Q];
  int64_t row[kDropAhead] = {}, col[kDropAhead];
#pragma unroll
  for (int u = 0; u < kDropAhead; ++u) {
    const int64_t i = (first + u * kDropThreads) * 8;
    if (LIE != kRun) row[u] = A.total < (int64_t(1) << 31) ? int64_t((__umulhi(A.magic, unsigned(i)) + unsigned(i)) >> A.shift) : i / A.width;
    col[u] = LIE == kRun ? i : i - row[u] * A.width;
    if (LIE != kAnyhow && i + 8 <= A.total) {
#pragma unroll
      for (int q = 0; q < Q; ++q) {
        v[u][q] = *reinterpret_cast<const Vec<T, N>*>(x + (LIE == kRun ? 0 : row[u] * A.ldx) + col[u] + q * N);
        if (RES) w[u][q] = *reinterpret_cast<const Vec<T, N>*>(r + (LIE == kRun ? 0 : row[u] * A.ldr) + col[u] + q * N);
      }
    }
  }
#pragma unroll
  for (int u = 0; u < kDropAhead; ++u) {
    const int64_t g = first + u * kDropThreads;
    if (g >= groups) break;
    uint32_t bits[4] = {};
    if (A.t) {
      const uint4 c = philox(make_uint4(uint32_t(g), uint32_t(uint64_t(g) >> 32), uint32_t(call), uint32_t(call >> 32)),
                             uint32_t(key), uint32_t(key >> 32));
      bits[0] = c.x, bits[1] = c.y, bits[2] = c.z, bits[3] = c.w;
    }
    auto result = [&](int e, T xv, T rv) {  // (the other half of the word does not change how its upper half compares)
      const float f = (e & 1 ? bits[e >> 1] : bits[e >> 1] << 16) >= t ? widen(xv) : 0.f;
      return narrow<T>(RES ? fmaf(f, A.keep, widen(rv)) : f * A.keep);
    };
    if (LIE == kRows || (LIE == kRun && g * 8 + 8 <= A.total)) {
#pragma unroll
      for (int q = 0; q < Q; ++q) {
        Vec<T, N> o;
#pragma unroll
        for (int e = 0; e < N; ++e) o.v[e] = result(q * N + e, v[u][q].v[e], w[u][q].v[e]);
        *reinterpret_cast<Vec<T, N>*>(y + (LIE == kRun ? 0 : row[u] * A.ldy) + col[u] + q * N) = o;
      }
    } else {
      int64_t at = row[u], c = col[u];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        if (g * 8 + e >= A.total) break;
        y[at * A.ldy + c] = result(e, x[at * A.ldx + c], RES ? r[at * A.ldr + c] : narrow<T>(0.f));
        if (++c == A.width) {
          c = 0;
          ++at;
        }
      }
    }
  }
}

template <class T>
void (*drop_pick(int lie, bool res))(DropArgs) {
  if (lie == kRun) return res ? dropout_kernel<T, kRun, true> : dropout_kernel<T, kRun, false>;
  if (lie == kRows) return res ? dropout_kernel<T, kRows, true> : dropout_kernel<T, kRows, false>;
  return res ? dropout_kernel<T, kAnyhow, true> : dropout_kernel<T, kAnyhow, false>;
}

}  // namespace

cudaError_t dropout_preload() {
  for (int lie : {kRun, kRows, kAnyhow})
    for (bool res : {false, true})
      for (auto kernel : {drop_pick<float>(lie, res), drop_pick<__nv_bfloat16>(lie, res)}) {
        cudaFuncAttributes a;
        const cudaError_t e = cudaFuncGetAttributes(&a, reinterpret_cast<const void*>(kernel));
        if (e != cudaSuccess) return e;
      }
  return cudaSuccess;
}

}  // namespace hoc

using namespace hoc;
using namespace hoc::block;

extern "C" hocResult_t hoc_dropout(size_t rows, int width, hocDataType_t dtype, const void* x, size_t ldx,
                                   const void* residual, size_t ldr, const double* p, const int64_t* seed, void* y, size_t ldy,
                                   void* stream) {
  const char* who = "hoc_dropout";
  constexpr size_t kMost = size_t(0x7FFFFFFF) * 8 * kDropThreads * kDropAhead;  // what a grid reaches
  if (width < 0 || rows > kMost / size_t(width > 1 ? width : 1)) return refuse(who, "rows or width out of range");
  if (!row_dtype(dtype)) return refuse(who, "dtype must be HOC_FLOAT32 or HOC_BFLOAT16");
  if (!p || !(*p >= 0.0 && *p < 1.0)) return refuse(who, "p must be given, at least 0 and below 1");
  const bool none = rows == 0 || width == 0;
  const int64_t n = int64_t(rows);
  const size_t b = bytes_of(dtype);
  const char* bad = bad_rows(x, ldx, n, width, b, none);
  if (!bad) bad = bad_rows(residual, ldr, n, width, b, true);
  if (!bad) bad = bad_rows(y, ldy, n, width, b, none);
  if (!bad && (!seed || !aligned(seed, 8))) bad = "seed must be given, aligned to its elements";
  if (bad) return refuse(who, bad);
  if (none) return HOC_SUCCESS;
  const int64_t total = n * width;
  const int t = int(*p * 65536 + 0.5) < 65535 ? int(*p * 65536 + 0.5) : 65535;
  unsigned shift = 0;
  while ((int64_t(1) << shift) < width) ++shift;
  const unsigned magic = unsigned(((uint64_t(1) << 32) * ((uint64_t(1) << shift) - uint64_t(width))) / uint64_t(width) + 1);
  const DropArgs A{x, residual, y, seed, int64_t(ldx), int64_t(ldr), int64_t(ldy), total, width, unsigned(t),
                   65536.f / float(65536 - t), magic, shift};
  const int64_t ctas = ((total + 7) / 8 + kDropThreads * kDropAhead - 1) / (kDropThreads * kDropAhead);
  const bool vec = vector_rows(x, ldx, b) && (!residual || vector_rows(residual, ldr, b)) && vector_rows(y, ldy, b);
  const bool together = rows == 1 || (ldx == size_t(width) && ldy == size_t(width) && (!residual || ldr == size_t(width)));
  const bool starts = aligned(x, 16) && aligned(residual, 16) && aligned(y, 16);
  const int lie = starts && together ? kRun : vec && width % 8 == 0 ? kRows : kAnyhow;
  const auto kernel = dtype == HOC_FLOAT32 ? drop_pick<float>(lie, residual) : drop_pick<__nv_bfloat16>(lie, residual);
  return launched(who, launch(kernel, dim3(unsigned(ctas)), dim3(kDropThreads), 0, static_cast<cudaStream_t>(stream), A));
}
