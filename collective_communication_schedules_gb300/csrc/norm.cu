// Root-mean-square norm with the residual's addition, its gradient, and rows of 8
// bits (hoc_block.h).
//
// All are bound by their bytes.  A row is read once and stays in registers between
// its sum of squares and its result: a thread has V vectors of 16 bytes of it, so a
// row takes width / (V * values of a vector) threads, a warp or a CTA of its own.
// Rows that are not whole vectors are held element by element, four of a group of 128
// columns to a lane.
#include <atomic>

#include <cuda_fp8.h>

#include "block.h"

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
};

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

// The sum over the row's threads: a warp, or the CTA (sh: one entry per warp).
__device__ __forceinline__ float row_sum(float v, float* sh) {
  v = warp_sum(v);
  if (blockDim.x == 32) return v;
  if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = v;
  __syncthreads();
  const int warps = blockDim.x >> 5, lane = threadIdx.x & 31;
  return warp_sum(lane < warps ? sh[lane] : 0.f);  // in the same order in every warp
}

__device__ __forceinline__ unsigned e4m3x2(float a, float b) {
  return __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
}

// One row a warp (blockDim (32, rows)) or a CTA.
template <class T, int V, bool RES, bool WIRE>
__global__ void __launch_bounds__(1024) norm_kernel(const __grid_constant__ NormArgs A) {
  constexpr int N = 16 / sizeof(T);
  __shared__ float sh[32];
  after_the_last();
  const int64_t row = int64_t(blockIdx.x) * blockDim.y + threadIdx.y;
  if (row >= A.rows) return;  // (a warp of its own: there is no barrier)
  const int nvec = A.width / N, tpr = blockDim.x;
  Vec<T, N> x[V], r[V];
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const int c = (j * tpr + int(threadIdx.x)) * N;
    if (c < A.width) {
      x[j] = *reinterpret_cast<const Vec<T, N>*>(static_cast<const T*>(A.x) + row * A.ldx + c);
      if (RES) r[j] = *reinterpret_cast<const Vec<T, N>*>(static_cast<const T*>(A.r) + row * A.ldr + c);
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
    for (int j = 0; j < V; ++j) {
      const int c = (j * tpr + int(threadIdx.x)) * N;
      if (c < A.width) *reinterpret_cast<Vec<T, N>*>(static_cast<T*>(A.h) + row * A.ldh + c) = x[j];
    }
  }
  sum = row_sum(sum, sh);
  const float s = rsqrtf(sum / float(A.width) + A.eps);
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const int i = j * tpr + int(threadIdx.x), c = i * N;
    const bool in = i < nvec;
    float w[N], y[N];
    if (in) load_weights<N>(A.w, A.w32, c, w);
#pragma unroll
    for (int e = 0; e < N; ++e) y[e] = in ? widen(x[j].v[e]) * s * w[e] : 0.f;
    if (in && A.y) {
      Vec<T, N> o;
#pragma unroll
      for (int e = 0; e < N; ++e) o.v[e] = narrow<T>(y[e]);
      *reinterpret_cast<Vec<T, N>*>(static_cast<T*>(A.y) + row * A.ldy + c) = o;
    }
    if (WIRE) {  // a group is kGroup / N neighbouring lanes: rows of threads are whole warps
      float most = 0.f;
#pragma unroll
      for (int e = 0; e < N; ++e) most = fmaxf(most, fabsf(y[e]));
#pragma unroll
      for (int off = kGroup / N / 2; off; off >>= 1) most = fmaxf(most, __shfl_xor_sync(kAll, most, off));
      const float scale = fmaxf(most / kE4m3Most, kLeastScale), inv = 1.f / scale;
      if (in) {
        uint8_t* to = A.wire + row * wire_bytes(A.width);
        if (i % (kGroup / N) == 0) *reinterpret_cast<float*>(to + scales_at(A.width) + i / (kGroup / N) * 4) = scale;
        uint32_t q[N / 4];
#pragma unroll
        for (int e = 0; e < N / 4; ++e)
          q[e] = e4m3x2(y[4 * e] * inv, y[4 * e + 1] * inv) | e4m3x2(y[4 * e + 2] * inv, y[4 * e + 3] * inv) << 16;
        if (N == 8) *reinterpret_cast<uint2*>(to + c) = make_uint2(q[0], q[N / 4 - 1]);
        else *reinterpret_cast<uint32_t*>(to + c) = q[0];
      }
    }
  }
}

// Any width and alignment, one row a CTA: warp w has the groups w, w + warps, .., U of
// them at most, a lane the columns lane, lane + 32, .. of a group.
template <class T, int U>
__global__ void __launch_bounds__(1024) norm_any_kernel(const __grid_constant__ NormArgs A) {
  __shared__ float sh[32];
  after_the_last();
  const int64_t row = blockIdx.x;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  const T* x = static_cast<const T*>(A.x) + row * A.ldx;
  const T* r = static_cast<const T*>(A.r) + row * A.ldr;
  T v[U][4];
#pragma unroll
  for (int u = 0; u < U; ++u)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int c = (warp + u * warps) * kGroup + e * 32 + lane;
      v[u][e] = c < A.width ? x[c] : narrow<T>(0.f);
      if (A.r && c < A.width) v[u][e] = narrow<T>(widen(v[u][e]) + widen(r[c]));
    }
  float sum = 0.f;
#pragma unroll
  for (int u = 0; u < U; ++u)
#pragma unroll
    for (int e = 0; e < 4; ++e) sum = fmaf(widen(v[u][e]), widen(v[u][e]), sum);
  sum = row_sum(sum, sh);
  const float s = rsqrtf(sum / float(A.width) + A.eps);
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
        if (A.h) static_cast<T*>(A.h)[row * A.ldh + c] = v[u][e];
        if (A.y) static_cast<T*>(A.y)[row * A.ldy + c] = narrow<T>(y[e]);
      }
      most = fmaxf(most, fabsf(y[e]));
    }
    if (!A.wire) continue;
#pragma unroll
    for (int off = 16; off; off >>= 1) most = fmaxf(most, __shfl_xor_sync(kAll, most, off));
    const float scale = fmaxf(most / kE4m3Most, kLeastScale), inv = 1.f / scale;
    uint8_t* to = A.wire + row * wire_bytes(A.width);
    if (lane == 0) *reinterpret_cast<float*>(to + scales_at(A.width) + g * 4) = scale;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int c = g * kGroup + e * 32 + lane;
      if (c < A.width) to[c] = uint8_t(e4m3x2(y[e] * inv, 0.f));
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
};

// The sums of two values over the row's threads.  Both go through one tree: the lower half
// of a warp adds up the first, the upper the second.  sh: [2][16], an entry per warp for each,
// 0 for the warps there are none of.
__device__ __forceinline__ float2 row_sum2(float a, float b, float* sh) {
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

// A thread's part of a row: dy + dy2 and h widened, dres as it came.
template <class T, int V>
struct GradRow {
  static constexpr int N = 16 / sizeof(T);
  float d[V][N], h[V][N];
  Vec<T, N> dres[V];
};

__device__ __forceinline__ void copy_ahead(void* to, const void* from) {  // 16 bytes, past L1
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(uint32_t(__cvta_generic_to_shared(to))), "l"(from) : "memory");
}

// A CTA takes the rows blockIdx.x, + gridDim.x, ..; a thread has the same columns of
// each, so that it sums the weight gradient over them in registers.  With S > 0 the next S - 1
// rows are on their way into shared memory while one is worked on: a thread fetches
// what it reads itself, so that nothing but its own copies has to be waited for.
template <class T, int V, int S>
__global__ void __launch_bounds__(kGradThreads) norm_grad_kernel(const __grid_constant__ NormGradArgs A) {
  constexpr int N = 16 / sizeof(T);
  using Q = Vec<T, N>;
  extern __shared__ uint4 ring[];  // [S][arrays][V][threads]
  __shared__ float sh[2][32];
  if (threadIdx.x < 64) sh[threadIdx.x >> 5][threadIdx.x & 31] = 0.f;
  if (blockDim.x < 64) sh[1][threadIdx.x] = 0.f;
  __syncthreads();
  after_the_last();
  const int threads = blockDim.x, two = A.dy2 != nullptr, arrays = 2 + two + (A.dres != nullptr);
  auto column = [&](int j) { return (j * threads + int(threadIdx.x)) * N; };
  float w[V][N], acc[V][N];
#pragma unroll
  for (int j = 0; j < V; ++j) {
#pragma unroll
    for (int e = 0; e < N; ++e) w[j][e] = acc[j][e] = 0.f;
    if (column(j) < A.width) load_weights<N>(A.w, A.w32, column(j), w[j]);
  }
  auto at = [&](const void* base, int64_t ld, int64_t row, int j) { return static_cast<const T*>(base) + row * ld + column(j); };
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
  int64_t row = blockIdx.x;
  if constexpr (S > 0) {
#pragma unroll
    for (int i = 0; i < S - 1; ++i) fetch(row + int64_t(i) * gridDim.x, i);
  }
  const float inv = 1.f / float(A.width);
  int turn = 0, stage = 0;
  for (; row < A.rows; row += gridDim.x, turn ^= 1) {
    GradRow<T, V> R;
    Q x[V], y[V], x2[V];
    if constexpr (S > 0) {
      fetch(row + int64_t(S - 1) * gridDim.x, stage == 0 ? S - 1 : stage - 1);  // (read a turn ago, by this thread)
      asm volatile("cp.async.wait_group %0;" ::"n"(S > 0 ? S - 1 : 0) : "memory");
      const uint4* from = ring + size_t(stage) * arrays * V * threads + threadIdx.x;
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const bool in = column(j) < A.width;
        const uint4 zero = make_uint4(0, 0, 0, 0);
        const uint4 a = in ? from[j * threads] : zero, b = in ? from[(V + j) * threads] : zero;
        const uint4 c = in && A.dy2 ? from[(2 * V + j) * threads] : zero;
        const uint4 d = in && A.dres ? from[((2 + two) * V + j) * threads] : zero;
        x[j] = *reinterpret_cast<const Q*>(&a);
        y[j] = *reinterpret_cast<const Q*>(&b);
        x2[j] = *reinterpret_cast<const Q*>(&c);
        R.dres[j] = *reinterpret_cast<const Q*>(&d);
      }
      stage = stage == S - 1 ? 0 : stage + 1;
    } else {
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const uint4 zero = make_uint4(0, 0, 0, 0);
        x[j] = y[j] = x2[j] = R.dres[j] = *reinterpret_cast<const Q*>(&zero);
        if (column(j) >= A.width) continue;
        x[j] = *reinterpret_cast<const Q*>(at(A.dy, A.lddy, row, j));
        y[j] = *reinterpret_cast<const Q*>(at(A.h, A.ldh, row, j));
        if (A.dy2) x2[j] = *reinterpret_cast<const Q*>(at(A.dy2, A.lddy2, row, j));
        if (A.dres) R.dres[j] = *reinterpret_cast<const Q*>(at(A.dres, A.lddres, row, j));
      }
    }
    float a = 0.f, b = 0.f;
#pragma unroll
    for (int j = 0; j < V; ++j)
#pragma unroll
      for (int e = 0; e < N; ++e) {
        R.h[j][e] = widen(y[j].v[e]);
        R.d[j][e] = widen(x[j].v[e]);
      }
    if (A.dy2) {
#pragma unroll
      for (int j = 0; j < V; ++j)
#pragma unroll
        for (int e = 0; e < N; ++e) R.d[j][e] += widen(x2[j].v[e]);
    }
#pragma unroll
    for (int j = 0; j < V; ++j)
#pragma unroll
      for (int e = 0; e < N; ++e) {
        a = fmaf(R.h[j][e], R.h[j][e], a);
        b = fmaf(R.d[j][e] * w[j][e], R.h[j][e], b);
      }
    const float2 t = row_sum2(a, b, sh[turn]);  // (two sets of entries: one barrier a row)
    const float s = rsqrtf(t.x * inv + A.eps), k = -s * s * (t.y * inv);
#pragma unroll
    for (int j = 0; j < V; ++j) {
      if (column(j) >= A.width) continue;
      Q o;
#pragma unroll
      for (int e = 0; e < N; ++e) {
        const float hs = R.h[j][e] * s;
        acc[j][e] = fmaf(R.d[j][e], hs, acc[j][e]);
        o.v[e] = narrow<T>(fmaf(s, R.d[j][e] * w[j][e], fmaf(hs, k, widen(R.dres[j].v[e]))));
      }
      *reinterpret_cast<Q*>(static_cast<T*>(A.dx) + row * A.lddx + column(j)) = o;
    }
  }
  if (!A.part) return;
#pragma unroll
  for (int j = 0; j < V; ++j) {
    if (column(j) >= A.width) continue;
#pragma unroll
    for (int e = 0; e < N; e += 4)
      *reinterpret_cast<float4*>(A.part + int64_t(blockIdx.x) * A.width + column(j) + e) =
          make_float4(acc[j][e], acc[j][e + 1], acc[j][e + 2], acc[j][e + 3]);
  }
}

// Any width and alignment: a thread has the columns threadIdx.x, + blockDim.x, .. and reads
// them again for the second use; its sums for the weight gradient are in shared memory.
template <class T>
__global__ void __launch_bounds__(kGradThreads) norm_grad_any_kernel(const __grid_constant__ NormGradArgs A) {
  extern __shared__ float acc[];  // [width]; none where the weight gradient is not wanted
  __shared__ float sh[2][32];
  if (threadIdx.x < 64) sh[threadIdx.x >> 5][threadIdx.x & 31] = 0.f;
  if (blockDim.x < 64) sh[1][threadIdx.x] = 0.f;
  __syncthreads();
  after_the_last();
  const int step = blockDim.x;
  if (A.part)
    for (int c = threadIdx.x; c < A.width; c += step) acc[c] = 0.f;
  auto weight = [&](int c) {
    return A.w32 ? static_cast<const float*>(A.w)[c] : widen(static_cast<const __nv_bfloat16*>(A.w)[c]);
  };
  int turn = 0;
  for (int64_t row = blockIdx.x; row < A.rows; row += gridDim.x, turn ^= 1) {
    const T* dy = static_cast<const T*>(A.dy) + row * A.lddy;
    const T* dy2 = static_cast<const T*>(A.dy2) + row * A.lddy2;
    const T* hh = static_cast<const T*>(A.h) + row * A.ldh;
    const T* dres = static_cast<const T*>(A.dres) + row * A.lddres;
    T* dx = static_cast<T*>(A.dx) + row * A.lddx;
    float a = 0.f, b = 0.f;
#pragma unroll 4
    for (int c = threadIdx.x; c < A.width; c += step) {
      const float h = widen(hh[c]), d = widen(dy[c]) + (A.dy2 ? widen(dy2[c]) : 0.f);
      a = fmaf(h, h, a);
      b = fmaf(d * weight(c), h, b);
    }
    const float2 t = row_sum2(a, b, sh[turn]);
    const float s = rsqrtf(t.x / float(A.width) + A.eps), k = s * s * (t.y / float(A.width));
#pragma unroll 4
    for (int c = threadIdx.x; c < A.width; c += step) {
      const float h = widen(hh[c]), d = widen(dy[c]) + (A.dy2 ? widen(dy2[c]) : 0.f);
      if (A.part) acc[c] = fmaf(d, h * s, acc[c]);
      float g = s * (d * weight(c) - h * k);
      if (A.dres) g += widen(dres[c]);
      dx[c] = narrow<T>(g);
    }
  }
  if (A.part)
    for (int c = threadIdx.x; c < A.width; c += step) A.part[int64_t(blockIdx.x) * A.width + c] = acc[c];
}

// dw (+)= sum over the parts, 32 columns a CTA, in an order that depends on the parts
// alone.
constexpr int kSumRows = 32;
template <class T>
__global__ void __launch_bounds__(32 * kSumRows) norm_weight_kernel(const float* __restrict__ part, int parts, int width,
                                                                    T* dw, int accumulate) {
  __shared__ float sh[kSumRows][33];
  after_the_last();
  const int c = blockIdx.x * 32 + int(threadIdx.x);
  float sum[4] = {};
  if (c < width) {
    int p = threadIdx.y;
    for (; p + 3 * kSumRows < parts; p += 4 * kSumRows)
#pragma unroll
      for (int u = 0; u < 4; ++u) sum[u] += part[int64_t(p + u * kSumRows) * width + c];
    for (; p < parts; p += kSumRows) sum[0] += part[int64_t(p) * width + c];
  }
  sh[threadIdx.y][threadIdx.x] = (sum[0] + sum[1]) + (sum[2] + sum[3]);
  __syncthreads();
  if (threadIdx.y == 0 && c < width) {
    float v = 0.f;
#pragma unroll
    for (int r = 0; r < kSumRows; ++r) v += sh[r][threadIdx.x];
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
constexpr int kWidenAhead = 2;  // steps a thread has in flight

// A step is E values: 16 where rows of y are whole 32 bytes, else 8, else 1.  2^log neighbouring
// lanes take a row, as many as it has steps, a warp at most; the rows of all ranks are one run,
// handed out in turn.
static_assert(kMaxRanks * kMaxRanks <= kWidenThreads, "a thread for each count");
template <int E>
__global__ void __launch_bounds__(kWidenThreads) widen_kernel(const __grid_constant__ WidenArgs A) {
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
    for (int c0 = first; c0 < A.width; c0 += span * kWidenAhead) {
      In q[kWidenAhead];
      float scale[kWidenAhead];
#pragma unroll
      for (int u = 0; u < kWidenAhead; ++u) {
        const int c = c0 + u * span;
        if (c >= A.width) continue;
        q[u] = *reinterpret_cast<const In*>(from + c);
        scale[u] = *reinterpret_cast<const float*>(from + at + c / kGroup * 4);
      }
#pragma unroll
      for (int u = 0; u < kWidenAhead; ++u) {
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
          if constexpr (E == 16)
            asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(to + c), "r"(o[0]), "r"(o[1]),
                         "r"(o[2]), "r"(o[3]), "r"(o[4]), "r"(o[5]), "r"(o[6]), "r"(o[7])
                         : "memory");
          else
            *reinterpret_cast<uint4*>(to + c) = make_uint4(o[0], o[1], o[2], o[3]);
        }
      }
    }
  }
}

// ------------------------------------------------------------------ host side
// Threads of a row that is `nvec` vectors, V to a thread: a warp, or whole warps.
int row_threads(int nvec, int v) { return (nvec + 32 * v - 1) / (32 * v) * 32; }

template <class T, int V>
cudaError_t launch_norm(const NormArgs& A, cudaStream_t s) {
  const int tpr = row_threads(A.width / int(16 / sizeof(T)), V);
  const dim3 cta = tpr > 32 ? dim3(tpr, 1) : dim3(32, 8);
  const dim3 grid(unsigned((int64_t(A.rows) + cta.y - 1) / cta.y));
  const auto kernel = A.r ? A.wire ? norm_kernel<T, V, true, true> : norm_kernel<T, V, true, false>
                          : A.wire ? norm_kernel<T, V, false, true> : norm_kernel<T, V, false, false>;
  return launch(kernel, grid, cta, 0, s, A);
}

template <class T>
cudaError_t start_norm(const NormArgs& A, bool vec, cudaStream_t s) {
  const int nvec = A.width / int(16 / sizeof(T));
  if (vec && nvec <= 4096) {
    if (nvec <= 1024) return launch_norm<T, 1>(A, s);
    return launch_norm<T, 4>(A, s);
  }
  const int groups = (A.width + kGroup - 1) / kGroup;
  const dim3 grid{unsigned(A.rows)};
  if (groups <= 32) return launch(norm_any_kernel<T, 1>, grid, dim3(groups * 32), 0, s, A);
  return launch(norm_any_kernel<T, 8>, grid, dim3(1024), 0, s, A);
}

constexpr int kMostParts = kSms * 8;

// CTAs of the gradient's kernel: what is resident at once.
int grad_parts(int rows, int threads, size_t smem) {
  int each = int(size_t(220) * 1024 / (smem + 2048)), regs = 640 / threads;  // (up to 100 registers a thread)
  each = each < regs ? each : regs;
  const int most = kSms * (each > 8 ? 8 : each < 1 ? 1 : each);
  return rows < most ? rows < 1 ? 1 : rows : most;
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

template <class T, int V, int S>
cudaError_t launch_grad(const NormGradArgs& A, cudaStream_t s, int* parts) {
  static std::atomic<uint64_t> done{0};
  const int threads = row_threads(A.width / int(16 / sizeof(T)), V);
  const size_t smem = size_t(S) * (2 + (A.dy2 != nullptr) + (A.dres != nullptr)) * V * threads * 16;
  *parts = grad_parts(A.rows, threads, smem);
  if (smem > kSmemAsIs) {
    const cudaError_t e = opt_in(norm_grad_kernel<T, V, S>, kMostRing, done);
    if (e != cudaSuccess) return e;
  }
  return launch(norm_grad_kernel<T, V, S>, dim3(*parts), dim3(threads), smem, s, A);
}

template <class T>
cudaError_t start_grad(const NormGradArgs& A, bool vec, cudaStream_t s, int* parts) {
  const int nvec = A.width / int(16 / sizeof(T));
  if (vec && nvec <= 4 * kGradThreads) {
    if (nvec <= 256) return launch_grad<T, 2, 4>(A, s, parts);
    if (nvec <= 2 * kGradThreads) return launch_grad<T, 2, 3>(A, s, parts);
    return launch_grad<T, 4, 0>(A, s, parts);
  }
  const int threads = A.width >= kGradThreads ? kGradThreads : (A.width + 31) / 32 * 32;
  const size_t smem = A.part ? size_t(A.width) * sizeof(float) : 0;
  *parts = grad_parts(A.rows, threads, smem);
  if (smem > kSmemAsIs) {
    static std::atomic<uint64_t> done{0};
    const cudaError_t e = opt_in(norm_grad_any_kernel<T>, size_t(kMaxWidth) * sizeof(float), done);
    if (e != cudaSuccess) return e;
  }
  return launch(norm_grad_any_kernel<T>, dim3(*parts), dim3(threads), smem, s, A);
}

}  // namespace

cudaError_t norm_preload() {
  const void* fns[] = {
      reinterpret_cast<const void*>(&widen_kernel<16>), reinterpret_cast<const void*>(&widen_kernel<8>),
      reinterpret_cast<const void*>(&widen_kernel<1>), reinterpret_cast<const void*>(&norm_weight_kernel<float>),
      reinterpret_cast<const void*>(&norm_weight_kernel<__nv_bfloat16>),
#define HOC_NORM_OF(T)                                                                                               \
  reinterpret_cast<const void*>(&norm_any_kernel<T, 1>), reinterpret_cast<const void*>(&norm_any_kernel<T, 8>),      \
      reinterpret_cast<const void*>(&norm_grad_kernel<T, 2, 4>), reinterpret_cast<const void*>(&norm_grad_kernel<T, 2, 3>), \
      reinterpret_cast<const void*>(&norm_grad_kernel<T, 4, 0>), reinterpret_cast<const void*>(&norm_grad_any_kernel<T>)
#define HOC_NORM_V(T, V)                                                                                           \
  reinterpret_cast<const void*>(&norm_kernel<T, V, false, false>),                                                 \
      reinterpret_cast<const void*>(&norm_kernel<T, V, false, true>),                                              \
      reinterpret_cast<const void*>(&norm_kernel<T, V, true, false>), reinterpret_cast<const void*>(&norm_kernel<T, V, true, true>)
      HOC_NORM_OF(float), HOC_NORM_OF(__nv_bfloat16), HOC_NORM_V(float, 1), HOC_NORM_V(float, 4),
      HOC_NORM_V(__nv_bfloat16, 1), HOC_NORM_V(__nv_bfloat16, 4)};
#undef HOC_NORM_OF
#undef HOC_NORM_V
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
                   int64_t(ldh), int64_t(ldy), rows, width, *eps, weight_dtype == HOC_FLOAT32};
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
                       weight_dtype == HOC_FLOAT32};
  const bool vec = width * b % 16 == 0 && vector_rows(dy, lddy, b) && (!dy2 || vector_rows(dy2, lddy2, b)) &&
                   vector_rows(h, ldh, b) && (!dres || vector_rows(dres, lddres, b)) && vector_rows(dx, lddx, b) &&
                   aligned(weight, 16);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  int parts = 1;
  cudaError_t e = dtype == HOC_FLOAT32 ? start_grad<float>(A, vec, s, &parts) : start_grad<__nv_bfloat16>(A, vec, s, &parts);
  if (e == cudaSuccess && dw) {
    const dim3 grid((width + 31) / 32), cta(32, kSumRows);
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
  const int e = wide && width % 16 == 0 ? 16 : vec && width % 8 == 0 ? 8 : 1;
  while (A.log < 5 && (e << A.log) < width) ++A.log;
  const size_t want = ((most << A.log) + kWidenThreads) / kWidenThreads;  // one at least
  return launched(who, launch(e == 16 ? widen_kernel<16> : e == 8 ? widen_kernel<8> : widen_kernel<1>,
                              dim3(unsigned(want < size_t(kWidenCtas) ? want : size_t(kWidenCtas))), dim3(kWidenThreads), 0,
                              static_cast<cudaStream_t>(stream), A));
}
