// Root-mean-square norm with the residual's addition, its gradient, and rows of 8
// bits (hoc_block.h).
//
// All are bound by their bytes.  A row is read once and stays in registers between
// its sum of squares and its result.  Narrow rows take a run of lanes of a warp, so that
// nothing but the warp has to wait; wide ones take a CTA.  Rows that are not whole
// 16-byte vectors are read element by element.
#include <atomic>

#include <cuda_fp8.h>

#include "block.h"
#include "f32x2.cuh"

namespace hoc {
namespace {

using namespace block;

constexpr int kGroup = 128;  // columns that share a scale
constexpr float kE4m3Most = 448.f;
constexpr float kLeastScale = 0x1p-100f;
constexpr int kMaxWidth = HOC_NORM_MAX_WIDTH;

__host__ __device__ constexpr int scales_at(int width) { return (width + 15) / 16 * 16; }
__host__ __device__ constexpr int wire_bytes(int width) {
  return scales_at(width) + ((width + kGroup - 1) / kGroup * 4 + 15) / 16 * 16;
}

struct NormArgs {
  const void *x, *r, *w;
  void *h, *y;
  uint8_t* wire;
  int64_t ldx, ldr, ldh, ldy;
  int rows, width;
  float eps;
  int w32;  // weights are binary32
  int log;  // 2^log lanes take a row; -1: a CTA does
};

// The threads of a row: `count` of them, of which this is number `at`.
struct RowThreads {
  int64_t row;
  int at, count;
};
__device__ __forceinline__ RowThreads row_threads_of(int log) {
  const int t = threadIdx.x;
  if (log < 0) return {int64_t(blockIdx.x), t, int(blockDim.x)};
  return {(int64_t(blockIdx.x) * blockDim.x + t) >> log, t & ((1 << log) - 1), 1 << log};
}

// N weights from column c on.
template <int N>
__device__ __forceinline__ void load_weights(const void* w, int w32, int c, float (&to)[N]) {
  if (w32) {
    constexpr int M = N < 4 ? N : 4;
#pragma unroll
    for (int i = 0; i < N; i += M) {
      const Vec<float, M> a = *reinterpret_cast<const Vec<float, M>*>(static_cast<const float*>(w) + c + i);
#pragma unroll
      for (int e = 0; e < M; ++e) to[i + e] = a.v[e];
    }
  } else {
    const Vec<__nv_bfloat16, N> a =
        *reinterpret_cast<const Vec<__nv_bfloat16, N>*>(static_cast<const __nv_bfloat16*>(w) + c);
#pragma unroll
    for (int e = 0; e < N; ++e) to[e] = __bfloat162float(a.v[e]);
  }
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int off = 16; off; off >>= 1) v += __shfl_xor_sync(kAll, v, off);
  return v;
}

// The sum over the row's threads: 2^log lanes, or the CTA (sh: one entry per warp).
__device__ __forceinline__ float row_sum(float v, int log, float* sh) {
  if (log >= 0) {
    for (int off = 1 << log >> 1; off; off >>= 1) v += __shfl_xor_sync(kAll, v, off);
    return v;
  }
  v = warp_sum(v);
  if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = v;
  __syncthreads();
  const int warps = blockDim.x >> 5, lane = threadIdx.x & 31;
  return warp_sum(lane < warps ? sh[lane] : 0.f);  // in the same order in every warp
}

__device__ __forceinline__ unsigned e4m3x2(float a, float b) {
  return __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
}

// v / scale, inv being the rounded 1 / scale: their product is off by up to 2^-23 of itself, which moves a quotient on a tie of
// e4m3 to one side of it.  Adding what is left of v, divided likewise, gives the quotient rounded once (Markstein, 1990), but
// where it lies within 2^-46 of itself of the middle of two binary32 numbers.
__device__ __forceinline__ float quotient(float v, float scale, float inv) {
  const float q = v * inv;
  return fmaf(fmaf(-q, scale, v), inv, q);
}

__device__ __forceinline__ unsigned long long mul_f32x2(unsigned long long a, unsigned long long b) {
  unsigned long long d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

// Two of them, packed, in e4m3.
__device__ __forceinline__ unsigned quotients(float a, float b, float scale, float inv) {
  const unsigned long long v = pack_f32x2(a, b), r = pack_f32x2(inv, inv), minus = pack_f32x2(-scale, -scale);
  unsigned long long q = mul_f32x2(v, r), rest;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(rest) : "l"(q), "l"(minus), "l"(v));
  asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(q) : "l"(rest), "l"(r));
  return e4m3x2(lo_f32(q), hi_f32(q));
}

// V vectors of 16 bytes of each operand to a thread, all on their way before the first is used.
// Bound by its bytes: 32,768 x 2048 bf16 with the residual, h, y and rows of 8 bits 91 us (6.7 TB/s,
// 0.98 of the copy rate; 95 with products one by one), without the rows of 8 bits 78 us.
template <class T, int V, bool RES, bool WIRE>
__global__ void __launch_bounds__(1024) norm_kernel(const __grid_constant__ NormArgs A) {
  constexpr int N = 16 / sizeof(T);
  __shared__ float sh[32];
  after_the_last();
  const RowThreads R = row_threads_of(A.log);
  const bool there = R.row < A.rows;
  auto column = [&](int j) { return (j * R.count + R.at) * N; };
  Vec<T, N> x[V], r[V];
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const int c = column(j);
    if (there && c < A.width) {
      x[j] = *reinterpret_cast<const Vec<T, N>*>(static_cast<const T*>(A.x) + R.row * A.ldx + c);
      if (RES) r[j] = *reinterpret_cast<const Vec<T, N>*>(static_cast<const T*>(A.r) + R.row * A.ldr + c);
    } else {
#pragma unroll
      for (int e = 0; e < N; ++e) x[j].v[e] = r[j].v[e] = narrow<T>(0.f);
    }
  }
  float sum = 0.f;
#pragma unroll
  for (int j = 0; j < V; ++j)
#pragma unroll
    for (int e = 0; e < N; ++e) {
      if (RES) x[j].v[e] = narrow<T>(widen(x[j].v[e]) + widen(r[j].v[e]));
      const float f = widen(x[j].v[e]);
      sum = fmaf(f, f, sum);
    }
  if (RES && A.h) {
#pragma unroll
    for (int j = 0; j < V; ++j)
      if (there && column(j) < A.width)
        *reinterpret_cast<Vec<T, N>*>(static_cast<T*>(A.h) + R.row * A.ldh + column(j)) = x[j];
  }
  sum = row_sum(sum, A.log, sh);
  const float s = rsqrtf(sum / float(A.width) + A.eps);
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const int c = column(j), i = c / N;
    const bool in = there && c < A.width;
    float w[N], y[N];
    if (in) load_weights<N>(A.w, A.w32, c, w);
#pragma unroll
    for (int e = 0; e < N; e += 2) {
      const unsigned long long v = mul_f32x2(mul_f32x2(pack_f32x2(widen(x[j].v[e]), widen(x[j].v[e + 1])), pack_f32x2(s, s)),
                                             pack_f32x2(w[e], w[e + 1]));
      y[e] = in ? lo_f32(v) : 0.f;
      y[e + 1] = in ? hi_f32(v) : 0.f;
    }
    if (in && A.y) {
      Vec<T, N> o;
#pragma unroll
      for (int e = 0; e < N; ++e) o.v[e] = narrow<T>(y[e]);
      *reinterpret_cast<Vec<T, N>*>(static_cast<T*>(A.y) + R.row * A.ldy + c) = o;
    }
    if (WIRE) {  // a group is kGroup / N neighbouring lanes, or the whole of a narrower row
      float most = 0.f;
#pragma unroll
      for (int e = 0; e < N; ++e) most = fmaxf(most, fabsf(y[e]));
#pragma unroll
      for (int off = kGroup / N / 2; off; off >>= 1)
        if (off < R.count) most = fmaxf(most, __shfl_xor_sync(kAll, most, off));
      const float scale = fmaxf(most / kE4m3Most, kLeastScale), inv = 1.f / scale;
      if (in) {
        uint8_t* to = A.wire + R.row * wire_bytes(A.width);
        if (i % (kGroup / N) == 0) *reinterpret_cast<float*>(to + scales_at(A.width) + i / (kGroup / N) * 4) = scale;
        uint32_t q[N / 4];
#pragma unroll
        for (int e = 0; e < N / 4; ++e)
          q[e] = quotients(y[4 * e], y[4 * e + 1], scale, inv) | quotients(y[4 * e + 2], y[4 * e + 3], scale, inv) << 16;
        if (N == 8) *reinterpret_cast<uint2*>(to + c) = make_uint2(q[0], q[N / 4 - 1]);
        else *reinterpret_cast<uint32_t*>(to + c) = q[0];
      }
    }
  }
}

// Any width and alignment.  A row's warp w has the groups w, w + warps, .., U of them at most, a
// lane the columns lane, lane + 32, .. of a group.
template <class T, int U, int THREADS>
__global__ void __launch_bounds__(THREADS) norm_any_kernel(const __grid_constant__ NormArgs A) {
  __shared__ float sh[32];
  after_the_last();
  const RowThreads R = row_threads_of(A.log);
  const bool there = R.row < A.rows;
  const int warp = R.at >> 5, lane = R.at & 31, warps = R.count >> 5;
  const T* x = static_cast<const T*>(A.x) + R.row * A.ldx;
  const T* r = static_cast<const T*>(A.r) + R.row * A.ldr;
  T v[U][4], rv[U][4];
#pragma unroll
  for (int u = 0; u < U; ++u)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int c = (warp + u * warps) * kGroup + e * 32 + lane;
      const bool in = there && c < A.width;
      v[u][e] = in ? x[c] : narrow<T>(0.f);
      rv[u][e] = in && A.r ? r[c] : narrow<T>(0.f);
    }
  if (A.r) {
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int e = 0; e < 4; ++e) v[u][e] = narrow<T>(widen(v[u][e]) + widen(rv[u][e]));
  }
  float sum = 0.f;
#pragma unroll
  for (int u = 0; u < U; ++u)
#pragma unroll
    for (int e = 0; e < 4; ++e) sum = fmaf(widen(v[u][e]), widen(v[u][e]), sum);
  sum = row_sum(sum, A.log, sh);
  const float s = rsqrtf(sum / float(A.width) + A.eps);
  if (!there) return;  // (a warp of its own)
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int g = warp + u * warps;
    if (g * kGroup >= A.width) break;
    float y[4], most = 0.f;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int c = g * kGroup + e * 32 + lane;
      y[e] = 0.f;
      if (c < A.width) {
        const float w = A.w32 ? static_cast<const float*>(A.w)[c] : widen(static_cast<const __nv_bfloat16*>(A.w)[c]);
        y[e] = widen(v[u][e]) * s * w;
        if (A.h) static_cast<T*>(A.h)[R.row * A.ldh + c] = v[u][e];
        if (A.y) static_cast<T*>(A.y)[R.row * A.ldy + c] = narrow<T>(y[e]);
      }
      most = fmaxf(most, fabsf(y[e]));
    }
    if (!A.wire) continue;
#pragma unroll
    for (int off = 16; off; off >>= 1) most = fmaxf(most, __shfl_xor_sync(kAll, most, off));
    const float scale = fmaxf(most / kE4m3Most, kLeastScale), inv = 1.f / scale;
    uint8_t* to = A.wire + R.row * wire_bytes(A.width);
    if (lane == 0) *reinterpret_cast<float*>(to + scales_at(A.width) + g * 4) = scale;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int c = g * kGroup + e * 32 + lane;
      if (c < A.width) to[c] = uint8_t(e4m3x2(quotient(y[e], scale, inv), 0.f));
    }
  }
}

// ------------------------------------------------------------------ gradient
constexpr int kGradThreads = 512;  // at most

struct NormGradArgs {
  const void *dy, *dy2, *h, *w, *dres;
  void* dx;
  float* part;  // [parts][width]: sums of d h s over a CTA's rows; NULL: not wanted
  int64_t lddy, lddy2, ldh, lddres, lddx;
  int rows, width;
  float eps;
  int w32;
  int log;  // 2^log lanes take a row; -1: a CTA does
};

// The sums of two values over the row's threads.  In a CTA both go through one tree: the
// lower half of a warp adds up the first, the upper the second.  sh: [2][16], an entry per
// warp for each, 0 for the warps there are none of.
__device__ __forceinline__ float2 row_sum2(float a, float b, int log, float* sh) {
  if (log >= 0) {
    for (int off = 1 << log >> 1; off; off >>= 1) {
      a += __shfl_xor_sync(kAll, a, off);
      b += __shfl_xor_sync(kAll, b, off);
    }
    return make_float2(a, b);
  }
  const int lane = threadIdx.x & 31;
  const bool low = lane < 16;
  float v = (low ? a : b) + __shfl_xor_sync(kAll, low ? b : a, 16);
#pragma unroll
  for (int off = 8; off; off >>= 1) v += __shfl_xor_sync(kAll, v, off);
  if ((lane & 15) == 0) sh[lane + (threadIdx.x >> 5)] = v;
  __syncthreads();
  v = sh[lane];
#pragma unroll
  for (int off = 8; off; off >>= 1) v += __shfl_xor_sync(kAll, v, off);
  const float w = __shfl_xor_sync(kAll, v, 16);
  return low ? make_float2(v, w) : make_float2(w, v);
}

// N sums, in vectors of 16 bytes where there are more than one.
template <int N>
__device__ __forceinline__ void store_sums(float* to, const float (&v)[N]) {
  if constexpr (N == 1) {
    *to = v[0];
  } else {
#pragma unroll
    for (int e = 0; e < N; e += 4) *reinterpret_cast<float4*>(to + e) = make_float4(v[e], v[e + 1], v[e + 2], v[e + 3]);
  }
}

__device__ __forceinline__ void copy_ahead(void* to, const void* from) {  // 16 bytes, past L1
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(uint32_t(__cvta_generic_to_shared(to))), "l"(from) : "memory");
}

// A row takes 2^log lanes or a CTA; rows are handed out in turn, and a thread has the same
// columns of each, so that it sums the weight gradient over them in registers.  Rows of whole
// vectors (N values): the next S - 1 rows are on their way into shared memory while one is
// worked on; a thread fetches what it reads itself, so that nothing but its own copies
// has to be waited for.  Other rows: N = 1, S = 0, everything of a row is loaded at once.
// Bound by its bytes: 32,768 x 2048 bf16 with dy2 and dres 104 us (6.4 TB/s; the sum over the parts
// behind it 5 us more).  With the next row in registers instead, too few of them left room for
// other rows: 178 us.
template <class T, int N, int V, int S, int THREADS>
__global__ void __launch_bounds__(THREADS) norm_grad_kernel(const __grid_constant__ NormGradArgs A) {
  using Q = Vec<T, N>;
  extern __shared__ uint4 ring[];  // [S][arrays][V][threads]
  __shared__ float sh[2][32];
  for (int i = threadIdx.x; i < 64; i += blockDim.x) sh[i >> 5][i & 31] = 0.f;
  __syncthreads();
  after_the_last();
  const int threads = blockDim.x, two = A.dy2 != nullptr, arrays = 2 + two + (A.dres != nullptr);
  const RowThreads R = row_threads_of(A.log);
  const int64_t step = A.log < 0 ? int64_t(gridDim.x) : int64_t(gridDim.x) * threads >> A.log;
  auto column = [&](int j) { return (j * R.count + R.at) * N; };
  float w[V][N], acc[V][N];
  auto weights = [&]() {
#pragma unroll
    for (int j = 0; j < V; ++j) {
#pragma unroll
      for (int e = 0; e < N; ++e) w[j][e] = 0.f;
      if (column(j) < A.width) load_weights<N>(A.w, A.w32, column(j), w[j]);
    }
  };
  if (N > 1) weights();
#pragma unroll
  for (int j = 0; j < V; ++j)
#pragma unroll
    for (int e = 0; e < N; ++e) acc[j][e] = 0.f;
  auto at = [&](const void* base, int64_t ld, int64_t row, int j) {
    return reinterpret_cast<const Q*>(static_cast<const T*>(base) + row * ld + column(j));
  };
  auto fetch = [&](int64_t row, int stage) {
    uint4* to = ring + size_t(stage) * arrays * V * threads + threadIdx.x;
    if (row < A.rows) {
#pragma unroll
      for (int j = 0; j < V; ++j) {
        if (column(j) >= A.width) continue;
        copy_ahead(to + j * threads, at(A.dy, A.lddy, row, j));
        copy_ahead(to + (V + j) * threads, at(A.h, A.ldh, row, j));
        if (A.dy2) copy_ahead(to + (2 * V + j) * threads, at(A.dy2, A.lddy2, row, j));
        if (A.dres) copy_ahead(to + ((2 + two) * V + j) * threads, at(A.dres, A.lddres, row, j));
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  if constexpr (S > 0) {
#pragma unroll
    for (int i = 0; i < S - 1; ++i) fetch(R.row + i * step, i);
  }
  const float inv = 1.f / float(A.width);
  int turn = 0, stage = 0;
  // (a warp's lanes go round together, also those whose rows have ended)
  auto any_left = [&](int64_t row) { return A.log < 0 ? row < A.rows : bool(__any_sync(kAll, row < A.rows)); };
  for (int64_t row = R.row; any_left(row); row += step, turn ^= 1) {
    const bool there = row < A.rows;
    float d[V][N], h[V][N];
    Q dres[V];
    if constexpr (S > 0) {
      fetch(row + (S - 1) * step, stage == 0 ? S - 1 : stage - 1);  // (read a turn ago, by this thread)
      asm volatile("cp.async.wait_group %0;" ::"n"(S > 0 ? S - 1 : 0) : "memory");
      const uint4* from = ring + size_t(stage) * arrays * V * threads + threadIdx.x;
      Q x2[V];
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const bool in = there && column(j) < A.width;
        const uint4 zero = make_uint4(0, 0, 0, 0);
        const uint4 qx = in ? from[j * threads] : zero, qh = in ? from[(V + j) * threads] : zero;
        const uint4 q2 = in && A.dy2 ? from[(2 * V + j) * threads] : zero;
        const uint4 qr = in && A.dres ? from[((2 + two) * V + j) * threads] : zero;
        x2[j] = *reinterpret_cast<const Q*>(&q2);
        dres[j] = *reinterpret_cast<const Q*>(&qr);
#pragma unroll
        for (int e = 0; e < N; ++e) {
          d[j][e] = widen(reinterpret_cast<const Q*>(&qx)->v[e]);
          h[j][e] = widen(reinterpret_cast<const Q*>(&qh)->v[e]);
        }
      }
      if (A.dy2) {
#pragma unroll
        for (int j = 0; j < V; ++j)
#pragma unroll
          for (int e = 0; e < N; ++e) d[j][e] += widen(x2[j].v[e]);
      }
      stage = stage == S - 1 ? 0 : stage + 1;
    } else {
      T x[V], y[V], x2[V];
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const bool in = there && column(j) < A.width;
        x[j] = in ? at(A.dy, A.lddy, row, j)->v[0] : narrow<T>(0.f);
        y[j] = in ? at(A.h, A.ldh, row, j)->v[0] : narrow<T>(0.f);
        x2[j] = in && A.dy2 ? at(A.dy2, A.lddy2, row, j)->v[0] : narrow<T>(0.f);
      }
      weights();
#pragma unroll
      for (int j = 0; j < V; ++j) {
        d[j][0] = A.dy2 ? widen(x[j]) + widen(x2[j]) : widen(x[j]);
        h[j][0] = widen(y[j]);
      }
    }
    float a = 0.f, b = 0.f;
#pragma unroll
    for (int j = 0; j < V; ++j)
#pragma unroll
      for (int e = 0; e < N; ++e) {
        a = fmaf(h[j][e], h[j][e], a);
        b = fmaf(d[j][e] * w[j][e], h[j][e], b);
      }
    const float2 t = row_sum2(a, b, A.log, sh[turn]);  // (two sets of entries: one barrier a row)
    const float s = rsqrtf(t.x * inv + A.eps), k = -s * (s * (t.y * inv));  // (s * s of a tiny row may be no binary32 number)
    if constexpr (S == 0) {
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const bool in = there && column(j) < A.width && A.dres;
        dres[j].v[0] = in ? at(A.dres, A.lddres, row, j)->v[0] : narrow<T>(0.f);
      }
    }
#pragma unroll
    for (int j = 0; j < V; ++j) {
      Q o;
#pragma unroll
      for (int e = 0; e < N; ++e) {
        const float hs = h[j][e] * s;
        acc[j][e] = fmaf(d[j][e], there ? hs : 0.f, acc[j][e]);
        o.v[e] = narrow<T>(fmaf(s, d[j][e] * w[j][e], fmaf(hs, k, widen(dres[j].v[e]))));
      }
      if (there && column(j) < A.width) *reinterpret_cast<Q*>(static_cast<T*>(A.dx) + row * A.lddx + column(j)) = o;
    }
  }
  if (!A.part) return;
  float* part = A.part + int64_t(blockIdx.x) * A.width;
  if (A.log < 0) {
#pragma unroll
    for (int j = 0; j < V; ++j) {
      if (column(j) < A.width) store_sums<N>(part + column(j), acc[j]);
    }
    return;
  }
  // the lanes that have the same columns, then the warps, one after the other
  float* sums = reinterpret_cast<float*>(ring);  // [width]; nothing is on its way any more
  asm volatile("cp.async.wait_all;" ::: "memory");
#pragma unroll
  for (int j = 0; j < V; ++j)
#pragma unroll
    for (int e = 0; e < N; ++e)
      for (int off = R.count; off < 32; off <<= 1) acc[j][e] += __shfl_xor_sync(kAll, acc[j][e], off);
  for (int warp = 0; warp < threads >> 5; ++warp) {
    __syncthreads();
    if (int(threadIdx.x) >> 5 != warp || (int(threadIdx.x) & 31) >= R.count) continue;
#pragma unroll
    for (int j = 0; j < V; ++j)
#pragma unroll
      for (int e = 0; e < N; ++e)
        if (column(j) < A.width) sums[column(j) + e] = warp ? sums[column(j) + e] + acc[j][e] : acc[j][e];
  }
  __syncthreads();
  for (int c = threadIdx.x; c < A.width; c += threads) part[c] = sums[c];
}

// Rows that do not fit the registers of a CTA's threads: read twice, the second time from L2.  V
// vectors of N values to a thread.
constexpr int kWideThreads = 1024;
template <class T, int N, int V>
__global__ void __launch_bounds__(kWideThreads) norm_grad_wide_kernel(const __grid_constant__ NormGradArgs A) {
  using Q = Vec<T, N>;
  __shared__ float sh[32];
  after_the_last();
  float acc[V][N] = {};
  const float inv = 1.f / float(A.width);
  for (int64_t row = blockIdx.x; row < A.rows; row += gridDim.x) {
    const T* dy = static_cast<const T*>(A.dy) + row * A.lddy;
    const T* dy2 = static_cast<const T*>(A.dy2) + row * A.lddy2;
    const T* hh = static_cast<const T*>(A.h) + row * A.ldh;
    const T* dres = static_cast<const T*>(A.dres) + row * A.lddres;
    T* dx = static_cast<T*>(A.dx) + row * A.lddx;
    float a = 0.f, b = 0.f;
    auto load = [&](int c, float (&d)[N], float (&h)[N], float (&w)[N]) {
      const Q x = *reinterpret_cast<const Q*>(dy + c), y = *reinterpret_cast<const Q*>(hh + c);
      load_weights<N>(A.w, A.w32, c, w);
#pragma unroll
      for (int e = 0; e < N; ++e) {
        d[e] = widen(x.v[e]);
        h[e] = widen(y.v[e]);
      }
      if (A.dy2) {
        const Q x2 = *reinterpret_cast<const Q*>(dy2 + c);
#pragma unroll
        for (int e = 0; e < N; ++e) d[e] += widen(x2.v[e]);
      }
    };
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int c = (j * kWideThreads + int(threadIdx.x)) * N;
      if (c >= A.width) continue;
      float d[N], h[N], w[N];
      load(c, d, h, w);
#pragma unroll
      for (int e = 0; e < N; ++e) {
        a = fmaf(h[e], h[e], a);
        b = fmaf(d[e] * w[e], h[e], b);
      }
    }
    __syncthreads();  // sh is read no more
    const float ta = row_sum(a, -1, sh);
    __syncthreads();
    const float tb = row_sum(b, -1, sh);
    const float s = rsqrtf(ta * inv + A.eps), k = -s * (s * (tb * inv));
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int c = (j * kWideThreads + int(threadIdx.x)) * N;
      if (c >= A.width) continue;
      float d[N], h[N], w[N];
      load(c, d, h, w);
      Q r = {}, o;
      if (A.dres) r = *reinterpret_cast<const Q*>(dres + c);
#pragma unroll
      for (int e = 0; e < N; ++e) {
        const float hs = h[e] * s;
        acc[j][e] = fmaf(d[e], hs, acc[j][e]);
        o.v[e] = narrow<T>(fmaf(s, d[e] * w[e], fmaf(hs, k, A.dres ? widen(r.v[e]) : 0.f)));
      }
      *reinterpret_cast<Q*>(dx + c) = o;
    }
  }
  if (!A.part) return;
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const int c = (j * kWideThreads + int(threadIdx.x)) * N;
    if (c < A.width) store_sums<N>(A.part + int64_t(blockIdx.x) * A.width + c, acc[j]);
  }
}

// dw (+)= sum over the parts, kSumCols columns a CTA, in an order that depends on the parts
// alone.  They are still being written when this kernel starts, and so not what __restrict__ would call them: read-only
// while it runs.  Bound by its latency: a thread's parts are all on their way at once, and there are
// twice as many CTAs as with 32 columns each (509 x 1408 binary32, both kernels: 6.6 us, 7.1 with 32).
constexpr int kSumCols = 16, kSumRows = 64;
template <class T>
__global__ void __launch_bounds__(kSumCols * kSumRows) norm_weight_kernel(const float* part, int parts, int width, T* dw,
                                                                          int accumulate) {
  __shared__ float sh[kSumRows][kSumCols + 1];
  after_the_last();
  const int c = blockIdx.x * kSumCols + int(threadIdx.x);
  constexpr int kAhead = 8;
  float sum = 0.f;
  if (c < width) {
    for (int p0 = threadIdx.y; p0 < parts; p0 += kAhead * kSumRows) {
      float v[kAhead];
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        const int p = p0 + u * kSumRows;
        v[u] = p < parts ? part[int64_t(p) * width + c] : 0.f;
      }
      sum += ((v[0] + v[1]) + (v[2] + v[3])) + ((v[4] + v[5]) + (v[6] + v[7]));
    }
  }
  sh[threadIdx.y][threadIdx.x] = sum;
  __syncthreads();
  if (threadIdx.y < 8) {
    sum = 0.f;
#pragma unroll
    for (int r = 0; r < kSumRows; r += 8) sum += sh[r + threadIdx.y][threadIdx.x];
    sh[threadIdx.y][threadIdx.x] = sum;  // (this row is this thread's own by now)
  }
  __syncthreads();
  if (threadIdx.y == 0 && c < width) {
    float v = 0.f;
#pragma unroll
    for (int r = 0; r < 8; ++r) v += sh[r][threadIdx.x];
    dw[c] = narrow<T>(accumulate ? widen(dw[c]) + v : v);
  }
}

// ------------------------------------------------------------------ rows of 8 bits
struct WidenArgs {
  const uint8_t* wire[kMaxRanks];
  __nv_bfloat16* y[kMaxRanks];
  int64_t cap[kMaxRanks];
  const int64_t* seg;
  uint64_t* counts;
  int64_t segs;  // entries of one rank
  int ranks, width, log;
};

constexpr int kWidenThreads = 256, kWidenCtas = kSms * 8;
constexpr int kWidenAhead = 2;  // steps a thread has in flight; one where a step is one value (1001 wide: 159 us, 199 with two)

// Bound by its stores: 8 x 18,432 rows of 2048 in 159 us are 3.8 TB/s of them beside 1.9 of loads,
// and writing alone (a memset of as many bytes) takes this memory to 3.9.  Steps of 8 values take
// 230 us; rows of 1000, which are not whole vectors of 32 bytes, 90 us with steps of 16 and 106 with 8.
// A step is E values: 16 where rows are whole vectors of 16 bytes (WIDE: of 32, and stored so; the
// last step of a row may be half a one otherwise), else 1.  2^log neighbouring lanes take a
// row, as many as it has steps, a warp at most; the rows of all ranks are one run, handed out in turn.
static_assert(kMaxRanks * kMaxRanks <= kWidenThreads, "a thread for each count");
template <int E, bool WIDE>
__global__ void __launch_bounds__(kWidenThreads) widen_kernel(const __grid_constant__ WidenArgs A) {
  constexpr int kAhead = E == 1 ? 1 : kWidenAhead;
  __shared__ int64_t ends[kMaxRanks];
  after_the_last();
  if (threadIdx.x < 32) {
    int64_t n = 0;
    if (int(threadIdx.x) < A.ranks) {
      n = A.seg[(int64_t(threadIdx.x) + 1) * A.segs - 1];
      n = n < 0 ? 0 : n < A.cap[threadIdx.x] ? n : A.cap[threadIdx.x];
    }
    for (int off = 1; off < kMaxRanks; off <<= 1) {
      const int64_t v = __shfl_up_sync(kAll, n, off);
      if (int(threadIdx.x) >= off) n += v;
    }
    if (int(threadIdx.x) < kMaxRanks) ends[threadIdx.x] = n;
  }
  if (A.counts && blockIdx.x == 0 && int(threadIdx.x) < A.ranks * A.ranks)
    A.counts[threadIdx.x] = A.counts[threadIdx.x] / uint64_t(wire_bytes(A.width) / 2) * uint64_t(A.width);
  __syncthreads();
  struct alignas(E) In {
    uint8_t v[E];
  };
  const int64_t total = ends[A.ranks - 1];
  const int row_bytes = wire_bytes(A.width), at = scales_at(A.width), span = E << A.log;
  const int first = (int(threadIdx.x) & ((1 << A.log) - 1)) * E;
  int d = 0;
  for (int64_t row = (int64_t(blockIdx.x) * kWidenThreads + threadIdx.x) >> A.log; row < total;
       row += int64_t(gridDim.x) * kWidenThreads >> A.log) {
    while (row >= ends[d]) ++d;
    const int64_t k = row - (d ? ends[d - 1] : 0);
    const uint8_t* from = A.wire[d] + k * row_bytes;
    __nv_bfloat16* to = A.y[d] + k * A.width;
    for (int c0 = first; c0 < A.width; c0 += span * kAhead) {
      In q[kAhead];
      float scale[kAhead];
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        const int c = c0 + u * span;
        if (c >= A.width) continue;
        q[u] = *reinterpret_cast<const In*>(from + c);
        scale[u] = *reinterpret_cast<const float*>(from + at + c / kGroup * 4);
      }
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        const int c = c0 + u * span;
        if (c >= A.width) continue;
        if constexpr (E == 1) {
          to[c] = __float2bfloat16_rn(__half2float(__half(__nv_cvt_fp8_to_halfraw(q[u].v[0], __NV_E4M3))) * scale[u]);
        } else {
          uint32_t o[E / 2];
#pragma unroll
          for (int e = 0; e < E; e += 2) {
            const __half2_raw f = __nv_cvt_fp8x2_to_halfraw2(__nv_fp8x2_storage_t(q[u].v[e] | q[u].v[e + 1] << 8), __NV_E4M3);
            const float2 v = __half22float2(__half2(f));
            const __nv_bfloat162 p = __floats2bfloat162_rn(v.x * scale[u], v.y * scale[u]);
            o[e / 2] = *reinterpret_cast<const uint32_t*>(&p);
          }
          if constexpr (E == 16 && WIDE) {
            asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(to + c), "r"(o[0]), "r"(o[1]),
                         "r"(o[2]), "r"(o[3]), "r"(o[4]), "r"(o[5]), "r"(o[6]), "r"(o[7])
                         : "memory");
          } else {  // (the last step of a row may be half a one)
            *reinterpret_cast<uint4*>(to + c) = make_uint4(o[0], o[1], o[2], o[3]);
            if (c + 8 < A.width) *reinterpret_cast<uint4*>(to + c + 8) = make_uint4(o[4], o[5], o[6], o[7]);
          }
        }
      }
    }
  }
}

// ------------------------------------------------------------------ host side
// Whole warps for a row that is `n` pieces, v to a thread.
int row_threads(int n, int v) { return (n + 32 * v - 1) / (32 * v) * 32; }

// The lanes that n pieces take, v to a lane, as a power of two; -1: more than a warp.
int row_log(int n, int v) {
  int log = 0;
  while (log < 5 && (v << log) < n) ++log;
  return (v << log) < n ? -1 : log;
}

constexpr int kNarrowThreads = 256;  // of a CTA whose rows take lanes

// CTAs for `rows` rows.
dim3 row_grid(int rows, int log, int threads) {
  return dim3(unsigned(log < 0 ? rows : ((int64_t(rows) << log) + threads - 1) / threads));
}

template <class T, int V>
cudaError_t launch_norm(NormArgs A, cudaStream_t s) {
  const int nvec = A.width / int(16 / sizeof(T));
  A.log = row_log(nvec, V);
  const int threads = A.log < 0 ? row_threads(nvec, V) : kNarrowThreads;
  const auto kernel = A.r ? A.wire ? norm_kernel<T, V, true, true> : norm_kernel<T, V, true, false>
                          : A.wire ? norm_kernel<T, V, false, true> : norm_kernel<T, V, false, false>;
  return launch(kernel, row_grid(A.rows, A.log, threads), dim3(threads), 0, s, A);
}

template <class T, int U, int THREADS>
cudaError_t launch_norm_any(NormArgs A, cudaStream_t s) {
  const int groups = (A.width + kGroup - 1) / kGroup, warps = (groups + U - 1) / U;
  A.log = warps > 1 ? -1 : 5;
  const int threads = warps > 1 ? warps * 32 : kNarrowThreads;
  return launch(norm_any_kernel<T, U, THREADS>, row_grid(A.rows, A.log, threads), dim3(threads), 0, s, A);
}

template <class T>
cudaError_t start_norm(const NormArgs& A, bool vec, cudaStream_t s) {
  const int nvec = A.width / int(16 / sizeof(T));
  if (vec && nvec <= 4096) {
    if (nvec <= 32) return launch_norm<T, 1>(A, s);
    // Two vectors a thread keep enough bytes on their way: 16,384 x 4096 bf16 without a residual 50 us,
    // with one 63; with a residual 81 and 84.  Up to 128 vectors a row stays in a warp.
    if (nvec <= 64 || (nvec > 128 && nvec <= 2048)) return launch_norm<T, 2>(A, s);
    return launch_norm<T, 4>(A, s);
  }
  const int groups = (A.width + kGroup - 1) / kGroup;
  if (groups <= 1) return launch_norm_any<T, 1, kNarrowThreads>(A, s);
  if (groups <= 4) return launch_norm_any<T, 4, kNarrowThreads>(A, s);
  // 65,536 x 1001 bf16: 159 us with two groups a warp, 164 with one, 213 with eight (a warp a row)
  if (groups <= 64) return launch_norm_any<T, 2, 1024>(A, s);
  if (groups <= 128) return launch_norm_any<T, 4, 1024>(A, s);
  return launch_norm_any<T, 8, 1024>(A, s);
}

constexpr int kMostParts = kSms * 8;

// CTAs of the gradient's kernel: what is resident at once, `resident` threads of an SM by their
// registers.
int grad_parts(int rows, int log, int threads, size_t smem, int resident) {
  int each = int(size_t(220) * 1024 / (smem + 2048)), regs = resident / threads;
  each = each < regs ? each : regs;
  const int most = kSms * (each > 8 ? 8 : each < 1 ? 1 : each);
  const int want = log < 0 ? rows : int(((int64_t(rows) << log) + threads - 1) / threads);
  return want < most ? want < 1 ? 1 : want : most;
}

// More shared memory than a kernel has without asking (48 KiB, its own variables among them), once
// per device.
constexpr size_t kSmemAsIs = 47 * 1024;
template <class Kernel>
cudaError_t opt_in(Kernel kernel, size_t smem, std::atomic<uint64_t>& done) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess || (dev < 64 && done.load() >> dev & 1)) return e;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, int(smem));
  if (e == cudaSuccess && dev < 64) done.fetch_or(uint64_t(1) << dev);
  return e;
}

constexpr size_t kMostRing = 200 * 1024;
constexpr int kGradNarrow = 128;  // threads of a CTA whose rows take lanes

template <class T, int N, int V, int S, int THREADS = kGradThreads>
cudaError_t launch_grad(NormGradArgs A, cudaStream_t s, int* parts) {
  static std::atomic<uint64_t> done{0};
  const int pieces = (A.width + N - 1) / N;
  A.log = row_log(pieces, V);
  const int threads = A.log < 0 ? row_threads(pieces, V) : kGradNarrow;
  size_t smem = size_t(S) * (2 + (A.dy2 != nullptr) + (A.dres != nullptr)) * V * threads * 16;
  if (A.log >= 0 && smem < A.width * sizeof(float)) smem = A.width * sizeof(float);  // for the sums at the end
  *parts = grad_parts(A.rows, A.log, threads, smem, N == 1 ? V <= 4 ? 1536 : V <= 9 ? 768 : 512 : 640);
  if (smem > kSmemAsIs) {
    const cudaError_t e = opt_in(norm_grad_kernel<T, N, V, S, THREADS>, kMostRing, done);
    if (e != cudaSuccess) return e;
  }
  return launch(norm_grad_kernel<T, N, V, S, THREADS>, dim3(*parts), dim3(threads), smem, s, A);
}

template <class T, int N, int V>
cudaError_t launch_grad_wide(const NormGradArgs& A, cudaStream_t s, int* parts) {
  *parts = A.rows < kSms ? A.rows < 1 ? 1 : A.rows : kSms;
  return launch(norm_grad_wide_kernel<T, N, V>, dim3(*parts), dim3(kWideThreads), 0, s, A);
}

template <class T>
cudaError_t start_grad(const NormGradArgs& A, bool vec, cudaStream_t s, int* parts) {
  constexpr int N = 16 / sizeof(T);
  const int nvec = A.width / N;
  if (vec) {
    if (nvec <= 32) return launch_grad<T, N, 1, 4>(A, s, parts);
    if (nvec <= 256) return launch_grad<T, N, 2, 4>(A, s, parts);
    if (nvec <= 2 * kGradThreads) return launch_grad<T, N, 2, 3>(A, s, parts);
    if (nvec <= 4 * kWideThreads) return launch_grad_wide<T, N, 4>(A, s, parts);
    return launch_grad_wide<T, N, kMaxWidth / (N * kWideThreads)>(A, s, parts);
  }
  // few columns to a thread and many rows at once: 65,536 x 1001 bf16 311 us with 2 columns, 321 with 4, 498
  // with 8; 443 with two rows an SM instead of three
  if (A.width <= 128) return launch_grad<T, 1, 4, 0, kGradNarrow>(A, s, parts);
  if (A.width <= 2 * kGradThreads) return launch_grad<T, 1, 2, 0>(A, s, parts);
  if (A.width <= 4 * kGradThreads) return launch_grad<T, 1, 4, 0>(A, s, parts);
  if (A.width <= 9 * kGradThreads) return launch_grad<T, 1, 9, 0>(A, s, parts);
  if (A.width <= 16 * kGradThreads) return launch_grad<T, 1, 16, 0>(A, s, parts);
  return launch_grad_wide<T, 1, 32>(A, s, parts);
}

}  // namespace

cudaError_t norm_preload() {
  const void* fns[] = {
      reinterpret_cast<const void*>(&widen_kernel<16, true>), reinterpret_cast<const void*>(&widen_kernel<16, false>),
      reinterpret_cast<const void*>(&widen_kernel<1, false>), reinterpret_cast<const void*>(&norm_weight_kernel<float>),
      reinterpret_cast<const void*>(&norm_weight_kernel<__nv_bfloat16>),
#define HOC_FN(...) reinterpret_cast<const void*>(&__VA_ARGS__)
#define HOC_NORM_V(T, V)                                                                                    \
  HOC_FN(norm_kernel<T, V, false, false>), HOC_FN(norm_kernel<T, V, false, true>),                          \
      HOC_FN(norm_kernel<T, V, true, false>), HOC_FN(norm_kernel<T, V, true, true>)
#define HOC_NORM_OF(T, N)                                                                                        \
  HOC_NORM_V(T, 1), HOC_NORM_V(T, 2), HOC_NORM_V(T, 4), HOC_FN(norm_any_kernel<T, 1, kNarrowThreads>),               \
      HOC_FN(norm_any_kernel<T, 4, kNarrowThreads>), HOC_FN(norm_any_kernel<T, 2, 1024>),                               \
      HOC_FN(norm_any_kernel<T, 4, 1024>), HOC_FN(norm_any_kernel<T, 8, 1024>),                                       \
       HOC_FN(norm_grad_kernel<T, N, 1, 4, kGradThreads>),                                                           \
      HOC_FN(norm_grad_kernel<T, N, 2, 4, kGradThreads>), HOC_FN(norm_grad_kernel<T, N, 2, 3, kGradThreads>),           \
      HOC_FN(norm_grad_kernel<T, 1, 4, 0, kGradNarrow>), HOC_FN(norm_grad_kernel<T, 1, 2, 0, kGradThreads>),            \
      HOC_FN(norm_grad_kernel<T, 1, 4, 0, kGradThreads>), HOC_FN(norm_grad_kernel<T, 1, 9, 0, kGradThreads>),           \
      HOC_FN(norm_grad_kernel<T, 1, 16, 0, kGradThreads>),                                                              \
      HOC_FN(norm_grad_wide_kernel<T, N, 4>), HOC_FN(norm_grad_wide_kernel<T, N, kMaxWidth / (N * kWideThreads)>), \
      HOC_FN(norm_grad_wide_kernel<T, 1, 32>)
      HOC_NORM_OF(float, 4), HOC_NORM_OF(__nv_bfloat16, 8)};
#undef HOC_NORM_OF
#undef HOC_NORM_V
#undef HOC_FN
  for (const void* f : fns) {
    cudaFuncAttributes a;
    const cudaError_t e = cudaFuncGetAttributes(&a, f);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace hoc

using namespace hoc;
using namespace hoc::block;

extern "C" hocResult_t hoc_wire8_row(int width, size_t* bytes, size_t* at) {
  if (width < 1 || width > kMaxWidth || !bytes || !at) return refuse("hoc_wire8_row", "width out of range, or a NULL result");
  *bytes = size_t(wire_bytes(width));
  *at = size_t(scales_at(width));
  return HOC_SUCCESS;
}

extern "C" hocResult_t hoc_rms_norm(int rows, int width, hocDataType_t dtype, const void* x, size_t ldx,
                                    const void* residual, size_t ldr, const void* weight, hocDataType_t weight_dtype,
                                    const float* eps, void* h, size_t ldh, void* y, size_t ldy, void* wire, void* stream) {
  const char* who = "hoc_rms_norm";
  if (rows < 0 || width < 1 || width > kMaxWidth) return refuse(who, "rows or width out of range");
  if (!row_dtype(dtype) || !row_dtype(weight_dtype)) return refuse(who, "dtypes must be HOC_FLOAT32 or HOC_BFLOAT16");
  if (!eps || !(*eps >= 0.f)) return refuse(who, "eps must be given, and at least 0");
  if (rows > 0 && !y && !wire) return refuse(who, "y or wire must be given");
  if (h && !residual) return refuse(who, "h is given where a residual is added");
  const size_t b = bytes_of(dtype);
  const char* bad = bad_rows(x, ldx, rows, width, b, rows == 0);
  if (!bad) bad = bad_rows(residual, ldr, rows, width, b, true);
  if (!bad) bad = bad_rows(h, ldh, rows, width, b, true);
  if (!bad) bad = bad_rows(y, ldy, rows, width, b, true);
  if (!bad && (!weight || !aligned(weight, bytes_of(weight_dtype)))) bad = "weight must be given, aligned to its elements";
  if (!bad && !aligned(wire, 16)) bad = "wire must be aligned to 16 bytes";
  if (bad) return refuse(who, bad);
  if (rows == 0) return HOC_SUCCESS;
  const NormArgs A{x,           residual,     weight,       h,    y,     static_cast<uint8_t*>(wire), int64_t(ldx), int64_t(ldr),
                   int64_t(ldh), int64_t(ldy), rows, width, *eps, weight_dtype == HOC_FLOAT32, -1};
  const bool vec = width * b % 16 == 0 && vector_rows(x, ldx, b) && (!residual || vector_rows(residual, ldr, b)) &&
                   (!h || vector_rows(h, ldh, b)) && (!y || vector_rows(y, ldy, b)) && aligned(weight, 16);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return launched(who, dtype == HOC_FLOAT32 ? start_norm<float>(A, vec, s) : start_norm<__nv_bfloat16>(A, vec, s));
}

extern "C" hocResult_t hoc_rms_norm_workspace(int rows, int width, size_t* ints) {
  if (rows < 0 || width < 1 || width > kMaxWidth || !ints)
    return refuse("hoc_rms_norm_workspace", "rows or width out of range, or a NULL result");
  *ints = size_t(width) * size_t(rows < 1 ? 1 : rows < kMostParts ? rows : kMostParts);
  return HOC_SUCCESS;
}

extern "C" hocResult_t hoc_rms_norm_grad(int rows, int width, hocDataType_t dtype, const void* dy, size_t lddy,
                                         const void* dy2, size_t lddy2, const void* h, size_t ldh, const void* weight,
                                         hocDataType_t weight_dtype, const float* eps, const void* dres, size_t lddres,
                                         void* dx, size_t lddx, void* dw, hocDataType_t dw_dtype, int accumulate,
                                         int32_t* workspace, size_t workspace_ints, void* stream) {
  const char* who = "hoc_rms_norm_grad";
  if (rows < 0 || width < 1 || width > kMaxWidth) return refuse(who, "rows or width out of range");
  if (!row_dtype(dtype) || !row_dtype(weight_dtype) || (dw && !row_dtype(dw_dtype)))
    return refuse(who, "dtypes must be HOC_FLOAT32 or HOC_BFLOAT16");
  if (!eps || !(*eps >= 0.f)) return refuse(who, "eps must be given, and at least 0");
  const size_t b = bytes_of(dtype);
  const char* bad = bad_rows(dy, lddy, rows, width, b, rows == 0);
  if (!bad) bad = bad_rows(dy2, lddy2, rows, width, b, true);
  if (!bad) bad = bad_rows(h, ldh, rows, width, b, rows == 0);
  if (!bad) bad = bad_rows(dres, lddres, rows, width, b, true);
  if (!bad) bad = bad_rows(dx, lddx, rows, width, b, rows == 0);
  if (!bad && (!weight || !aligned(weight, bytes_of(weight_dtype)))) bad = "weight must be given, aligned to its elements";
  if (!bad && dw && !aligned(dw, bytes_of(dw_dtype))) bad = "dw must be aligned to its elements";
  if (!bad && dw) {
    size_t need = 0;
    hoc_rms_norm_workspace(rows, width, &need);
    if (!workspace || workspace_ints < need) bad = "workspace smaller than hoc_rms_norm_workspace() asks for";
    else if (!aligned(workspace, 16)) bad = "workspace must be aligned to 16 bytes";
  }
  if (bad) return refuse(who, bad);
  if (rows == 0 && !dw) return HOC_SUCCESS;
  const NormGradArgs A{dy, dy2, h, weight, dres, dx, dw ? reinterpret_cast<float*>(workspace) : nullptr, int64_t(lddy),
                       int64_t(lddy2), int64_t(ldh), int64_t(lddres), int64_t(lddx), rows, width, *eps,
                       weight_dtype == HOC_FLOAT32, -1};
  const bool vec = width * b % 16 == 0 && vector_rows(dy, lddy, b) && (!dy2 || vector_rows(dy2, lddy2, b)) &&
                   vector_rows(h, ldh, b) && (!dres || vector_rows(dres, lddres, b)) && vector_rows(dx, lddx, b) &&
                   aligned(weight, 16);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  int parts = 1;
  cudaError_t e = dtype == HOC_FLOAT32 ? start_grad<float>(A, vec, s, &parts) : start_grad<__nv_bfloat16>(A, vec, s, &parts);
  if (e == cudaSuccess && dw) {
    const dim3 grid((width + kSumCols - 1) / kSumCols), cta(kSumCols, kSumRows);
    const float* part = A.part;
    e = dw_dtype == HOC_FLOAT32
            ? launch(norm_weight_kernel<float>, grid, cta, 0, s, part, parts, width, static_cast<float*>(dw), int(accumulate != 0))
            : launch(norm_weight_kernel<__nv_bfloat16>, grid, cta, 0, s, part, parts, width, static_cast<__nv_bfloat16*>(dw),
                     int(accumulate != 0));
  }
  return launched(who, e);
}

extern "C" hocResult_t hoc_expert_widen(const hocRowGroups_t* G, const void* const* wire, int width, void* const* y,
                                        uint64_t* counts, void* stream) {
  const char* who = "hoc_expert_widen";
  if (!G || !G->seg || !G->capacity || !wire || !y) return refuse(who, "groups, its seg and its capacity, wire and y must be given");
  if (G->nranks < 1 || G->nranks > kMaxRanks || G->experts < 1 || G->sources < 1)
    return refuse(who, "rank, expert or source count out of range");
  if (width < 1 || width > kMaxWidth) return refuse(who, "width out of range");
  if (!aligned(G->seg, 8) || !aligned(counts, 8)) return refuse(who, "seg and counts must be aligned to 8 bytes");
  WidenArgs A{};
  A.seg = G->seg;
  A.counts = counts;
  A.segs = int64_t(G->experts) * G->sources + 1;
  A.ranks = G->nranks;
  A.width = width;
  size_t most = 0;
  bool vec = true, wide = true;
  for (int d = 0; d < G->nranks; ++d) {
    const size_t cap = G->capacity[d];
    if (cap > (size_t(1) << 30)) return refuse(who, "a buffer of more than 2^30 rows");
    if (cap && (!wire[d] || !y[d])) return refuse(who, "a NULL buffer");
    if (!aligned(wire[d], 16) || !aligned(y[d], 2)) return refuse(who, "wire must be aligned to 16 bytes, y to its elements");
    A.wire[d] = static_cast<const uint8_t*>(wire[d]);
    A.y[d] = static_cast<__nv_bfloat16*>(y[d]);
    A.cap[d] = int64_t(cap);
    vec = vec && aligned(y[d], 16);
    wide = wide && aligned(y[d], 32);
    most += cap;
  }
  if (most == 0 && !counts) return HOC_SUCCESS;
  const int e = vec && width % 8 == 0 ? 16 : 1;
  wide = wide && width % 16 == 0;
  while (A.log < 5 && (e << A.log) < width) ++A.log;
  const size_t want = ((most << A.log) + kWidenThreads) / kWidenThreads;  // one at least
  return launched(who, launch(e == 1 ? widen_kernel<1, false> : wide ? widen_kernel<16, true> : widen_kernel<16, false>,
                              dim3(unsigned(want < size_t(kWidenCtas) ? want : size_t(kWidenCtas))), dim3(kWidenThreads), 0,
                              static_cast<cudaStream_t>(stream), A));
}
