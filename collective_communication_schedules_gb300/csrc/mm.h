// Matrix products on rows grouped by expert: what the host entry points
// (layer.cu) pass to the kernels (mm_any.cu, mm_few.cu, mm_tc.cu).
#pragma once

#include <cuda_bf16.h>

#include "hoc_internal.h"
#include "hoc_layer.h"

namespace hoc {

// The three products of a layer.  Each computes out[c][f] with f contiguous:
//   kForward  out[row][out feature] = sum over in  of W[f][k] x[row][k]
//   kDgrad    out[row][in feature]  = sum over out of W[k][f] dy[row][k]
//   kWgrad    out[out feature][in feature] = sum over an expert's rows of dy[row][c] x[row][f]
enum MmMode { kForward = 0, kDgrad = 1, kWgrad = 2 };

// Experts (over the rank buffers of one launch) whose tile counts a CTA keeps
// in shared memory; layer.cu splits calls with more into several launches.
constexpr int kMmMaxGroups = 1024;

struct MmParams {
  // read by every warp before its first tile: together, in as few constant-cache lines as can be
  const int64_t* seg;  // [nranks][sources * experts + 1] row offsets; null: one range, all rows
  int experts;         // experts of one rank (the seg layout)
  int sources;
  int part0, parts;    // rank buffers of this launch
  int group0, groups;  // experts of each of them in this launch
  int in, out;             // weight: [experts][out (x 2 when gated)][in]
  int act;                 // hocAct_t: forward, of the output; dgrad, of the layer below
  int out_f32, accumulate; // wgrad
  int32_t* status;
  int64_t ld_rows, ld_dy, ld_res, ld_y;
  int64_t ld_w;     // elements from one row of a weight to the next (in, but for a realigned copy)
  int64_t out_w;    // rows of an expert's weight, of its gates when gated (out, likewise)
  int64_t cap[kMaxRanks];  // rows of each rank buffer
  const __nv_bfloat16* rows[kMaxRanks];  // forward: x; dgrad: dy; wgrad: x
  const __nv_bfloat16* dy[kMaxRanks];    // wgrad
  const __nv_bfloat16* w[kMaxRanks];
  const __nv_bfloat16* bias[kMaxRanks];
  const __nv_bfloat16* res[kMaxRanks];
  const __nv_bfloat16* pre[kMaxRanks];  // dgrad: pre-activation of the layer below
  void* y[kMaxRanks];
  void* pre_out[kMaxRanks];  // forward: pre-activation to keep; wgrad: the bias gradient
};

// Device helpers ------------------------------------------------------------
// The rows [a, b) cut to a buffer of `cap` rows.
__device__ __forceinline__ void mm_cut(int64_t cap, int64_t a, int64_t b, int64_t& lo, int64_t& n) {
  lo = a < 0 ? 0 : (a < cap ? a : cap);
  const int64_t hi = b < lo ? lo : (b < cap ? b : cap);
  n = hi - lo;
}
// The row range of (rank buffer p, expert g, source s), cut to the buffer.
__device__ __forceinline__ void mm_range(const MmParams& P, int p, int g, int s, int64_t& lo, int64_t& n) {
  const int64_t cap = P.cap[p];
  if (P.seg == nullptr) {
    lo = 0;
    n = cap;
    return;
  }
  const int64_t* at = P.seg + int64_t(p) * (int64_t(P.sources) * P.experts + 1) + int64_t(s) * P.experts + g;
  mm_cut(cap, at[0], at[1], lo, n);
}

// Fills, for every (rank buffer, expert) pair i of the launch, vrows[i]: its
// rows, each source's count rounded up to `pad` (64: to 8, and the sum of every 32
// sources to 64), and tile0[i]: the tiles of the
// pairs before it, tiles(vrows) tiles each; tile0[n] is the total.  The whole
// CTA calls it (blockDim.x a multiple of 32).
template <class Tiles>
__device__ __forceinline__ void mm_count(const MmParams& P, int pad, int* vrows, unsigned* tile0, Tiles tiles) {
  const int n = P.parts * P.groups;
  const int ns = P.seg ? P.sources : 1;
  // The lanes of a warp take the sources of as many pairs as fit, then add up in
  // segments of `w` lanes.  32-bit sums: valid ranges of a buffer add up to less than
  // 2^31 rows, and whatever others wrap to is cut to the most there can be.
  int w = 1;
  while (w < ns && w < 32) w *= 2;
  const int sub = threadIdx.x & (w - 1), per = int(blockDim.x) / w;  // pairs at a time
  constexpr int kAhead = 2;  // loads of a thread in flight
  for (int at = 0; at < n; at += per * kAhead) {
    int sum[kAhead] = {};
    for (int base = 0; base < ns; base += 32) {
      int64_t lo, c[kAhead];
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        const int i = at + u * per + int(threadIdx.x) / w, part = i / P.groups;
        c[u] = 0;
        if (i < n && base + sub < ns) mm_range(P, P.part0 + part, P.group0 + i - part * P.groups, base + sub, lo, c[u]);
      }
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        const int to = pad < 8 ? pad : 8;
        int rows = int((c[u] + to - 1) / to * to);
        for (int off = w / 2; off; off >>= 1) rows += __shfl_xor_sync(0xFFFFFFFFu, rows, off);
        sum[u] += (rows + pad - 1) / pad * pad;
      }
    }
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int i = at + u * per + int(threadIdx.x) / w;
      if (i >= n || sub != 0) continue;
      const int64_t most = P.cap[P.part0 + i / P.groups] + int64_t(ns) * (pad - 1) + pad;  // more only if ranges overlap
      vrows[i] = int(sum[u] < 0 ? 0 : sum[u] < most ? sum[u] : most);
    }
  }
  __syncthreads();
  if (threadIdx.x < 32) {
    unsigned base = 0;
    for (int at = 0; at < n; at += 32) {
      const int i = at + int(threadIdx.x);
      const unsigned mine = i < n ? tiles(vrows[i]) : 0;
      unsigned incl = mine;
      for (int off = 1; off < 32; off <<= 1) {
        const unsigned v = __shfl_up_sync(0xFFFFFFFFu, incl, off);
        if (int(threadIdx.x) >= off) incl += v;
      }
      if (i < n) tile0[i] = base + incl - mine;
      base += __shfl_sync(0xFFFFFFFFu, incl, 31);
    }
    if (threadIdx.x == 0) tile0[n] = base;
  }
  __syncthreads();
}

// The pair that tile t belongs to: the last i with tile0[i] <= t (t below the total).
__device__ __forceinline__ int mm_find(const unsigned* tile0, int n, unsigned t) {
  int lo = 0, hi = n;  // tile0[lo] <= t < tile0[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (tile0[mid] <= t) lo = mid;
    else hi = mid;
  }
  return lo;
}

__device__ __forceinline__ float bf16_of(const __nv_bfloat16* p) { return __bfloat162float(*p); }

// 1 / (1 + exp(-z)) for every finite z: exp overflows to inf and the quotient to 0.
__device__ __forceinline__ float mm_sigmoid(float z) { return __fdividef(1.f, 1.f + __expf(-z)); }

// sqrt(2 / pi) and the cubic coefficient of the tanh form of GELU, of which
// 0.5 (1 + tanh v) = sigmoid(2 v).
constexpr float kGeluScale = 0.7978845608028654f;
constexpr float kGeluCubic = 0.044715f;

__device__ __forceinline__ float mm_act(int act, float z) {
  switch (act) {
    case HOC_ACT_RELU: return z > 0.f ? z : (z == z ? 0.f : z);
    case HOC_ACT_GELU: return z * mm_sigmoid(2.f * kGeluScale * (z + kGeluCubic * z * z * z));
    case HOC_ACT_SILU: return z * mm_sigmoid(z);
    default: return z;
  }
}

// d act(z) / dz (ReLU's is in mm_act_back); the products of a vanishing s (1 - s) with a
// huge z are cut where they are 0, at |z| = 30 and 120.
__device__ __forceinline__ float mm_act_slope(int act, float z) {
  switch (act) {
    case HOC_ACT_GELU: {
      const float s = mm_sigmoid(2.f * kGeluScale * (z + kGeluCubic * z * z * z));
      const float c = fminf(fmaxf(z, -30.f), 30.f);
      return s + c * s * (1.f - s) * 2.f * kGeluScale * (1.f + 3.f * kGeluCubic * c * c);
    }
    case HOC_ACT_SILU: {
      const float s = mm_sigmoid(z);
      const float c = fminf(fmaxf(z, -120.f), 120.f);
      return s * (1.f + c * (1.f - s));
    }
    default: return 1.f;
  }
}

// The gradient for z where d is that for act(z).  A closed ReLU is a choice and not a product: infinities
// and NaN do not come through it.
__device__ __forceinline__ float mm_act_back(int act, float z, float d) {
  return act == HOC_ACT_RELU ? (z > 0.f ? d : 0.f) : d * mm_act_slope(act, z);
}

// Host side -----------------------------------------------------------------
cudaError_t launch_mm_any(const MmParams& P, int mode, int sms, cudaStream_t s);
cudaError_t mm_any_preload();
// Whether the tensor-core kernel takes these operands (alignment and widths of
// what tensor copies fetch; the epilogue's rows may lie anywhere).
bool mm_tc_takes(const MmParams& P, int mode);
// Whether a row that the epilogue of this launch (rank buffers part0 .. part0 + parts)
// reads or writes is not whole 16-byte vectors.
bool mm_tc_loose(const MmParams& P, int mode);
// summed (weight gradient): whether the launch sums the columns of dy too, to P.pre_out[0].
cudaError_t launch_mm_tc(const MmParams& P, int mode, cudaStream_t s, bool* summed);
cudaError_t mm_tc_preload();
// Whether the kernel for a few rows takes this product (one range, at most 32 rows).
bool mm_few_takes(const MmParams& P, int mode);
cudaError_t launch_mm_few(const MmParams& P, cudaStream_t s);
cudaError_t mm_few_preload();

}  // namespace hoc
