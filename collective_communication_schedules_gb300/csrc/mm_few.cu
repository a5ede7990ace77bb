// Forward product for a few rows (a decoding step): y = act(x W^T + b) + r with at
// most 32 rows of x.
//
// Bound by reading the weights once: 2 in * out bytes against 2 rows in * out
// operations.  A tile kernel leaves most SMs without work here (4096 features are
// 16 tiles), so the contraction is split over the warps instead: a CTA owns 16
// features and its 8 warps take 64 or 128 elements of the contraction in turn, each
// lane with 16-byte loads straight into the fragments of mma.m16n8k16 -- the order of
// the contraction's elements within a fragment is free as long as both operands
// share it, so lane t of a row takes 8 consecutive elements.  The warps' binary32
// sums are added in warp order in shared memory.
//
// 4096 x 4096 weights from a flushed cache take 12.3 us at 1 row (2.7 TB/s; 8.8 us in a
// graph of calls, 3.8 TB/s), 14.3 at 16, 16.4 at 32; 2048 x 1408 at 1 row 8.2 us.  What
// bounds it at such sizes is latency: a warp makes four rounds of loads.
#include "mm.h"

namespace hoc {
namespace {

constexpr int kFewWarps = 8;
constexpr int kFewFeatures = 16;

__device__ __forceinline__ uint4 load_once(const void* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}
__device__ __forceinline__ uint4 load_x(const void* p) {  // volatile: issued where it stands
  uint4 v;
  asm volatile("ld.global.nc.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}
__device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Epilogue of one value: z holds the sums of feature f (gate and value where G is 2).
template <int G>
__device__ __forceinline__ void finish(const MmParams& P, int row, int f, float (&z)[G]) {
#pragma unroll
  for (int g = 0; g < G; ++g) {
    if (P.bias[0]) z[g] += bf16_of(P.bias[0] + int64_t(g) * P.out + f);
    if (P.pre_out[0])
      static_cast<__nv_bfloat16*>(P.pre_out[0])[(int64_t(row) * G + g) * P.out + f] = __float2bfloat16_rn(z[g]);
  }
  float y = G == 2 ? mm_act(HOC_ACT_SILU, z[0]) * z[G - 1] : mm_act(P.act, z[0]);
  if (P.res[0]) y += bf16_of(P.res[0] + row * P.ld_res + f);
  static_cast<__nv_bfloat16*>(P.y[0])[row * P.ld_y + f] = __float2bfloat16_rn(y);
}

// NB: blocks of 8 rows; G: 1, or 2 where a feature has a gate and a value.
template <int NB, int G>
__global__ void __launch_bounds__(32 * kFewWarps) mm_few_kernel(const __grid_constant__ MmParams P) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  __shared__ float part[kFewWarps][G][8 * NB][kFewFeatures + 1];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int r = lane >> 2, t = lane & 3;
  const int rows = int(P.cap[0]);
  const int f0 = int(blockIdx.x) * kFewFeatures;
  const __nv_bfloat16* w[G][2];  // this lane's two features; past the last one, the last (its sums are not stored)
#pragma unroll
  for (int g = 0; g < G; ++g)
#pragma unroll
    for (int h = 0; h < 2; ++h) w[g][h] = P.w[0] + (int64_t(g) * P.out_w + min(f0 + r + 8 * h, P.out - 1)) * P.ld_w + t * 8;
  const __nv_bfloat16* x = P.rows[0] + t * 8;
  float acc[G][NB][4] = {};
  // 32 elements deep: the operands of one step; two sets of kSteps steps, one loading while the other is used
  constexpr int kSteps = G == 1 && NB == 1 ? 4 : 2, kDepth = 32 * kSteps;
  struct Set {
    uint4 a[kSteps][G][2], b[kSteps][NB];
  };
  auto load = [&](Set& s, int k0) {
    const uint4 zero = make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int u = 0; u < kSteps; ++u) {
      const int k = k0 + u * 32;
      const bool in = k + t * 8 < P.in;  // in is a multiple of 8, or zeros make it one
#pragma unroll
      for (int g = 0; g < G; ++g)
#pragma unroll
        for (int h = 0; h < 2; ++h) s.a[u][g][h] = in ? load_once(w[g][h] + k) : zero;
#pragma unroll
      for (int n = 0; n < NB; ++n)
        s.b[u][n] = in && n * 8 + r < rows ? load_x(x + (n * 8 + r) * P.ld_rows + k) : zero;
    }
  };
  auto use = [&](const Set& s) {
#pragma unroll
    for (int u = 0; u < kSteps; ++u)
#pragma unroll
      for (int g = 0; g < G; ++g)
#pragma unroll
        for (int n = 0; n < NB; ++n) {
          mma(acc[g][n], s.a[u][g][0].x, s.a[u][g][1].x, s.a[u][g][0].y, s.a[u][g][1].y, s.b[u][n].x, s.b[u][n].y);
          mma(acc[g][n], s.a[u][g][0].z, s.a[u][g][1].z, s.a[u][g][0].w, s.a[u][g][1].w, s.b[u][n].z, s.b[u][n].w);
        }
  };
  Set one, two;
  load(one, warp * kDepth);
  for (int k0 = warp * kDepth; k0 < P.in; k0 += 2 * kFewWarps * kDepth) {
    load(two, k0 + kFewWarps * kDepth);
    use(one);
    load(one, k0 + 2 * kFewWarps * kDepth);
    use(two);
  }
#pragma unroll
  for (int g = 0; g < G; ++g)
#pragma unroll
    for (int n = 0; n < NB; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) part[warp][g][n * 8 + 2 * t + (e & 1)][r + 8 * (e >> 1)] = acc[g][n][e];
  __syncthreads();
  for (int i = threadIdx.x; i < rows * kFewFeatures; i += 32 * kFewWarps) {
    const int row = i / kFewFeatures, j = i % kFewFeatures, f = f0 + j;
    if (f >= P.out) continue;
    float z[G];
#pragma unroll
    for (int g = 0; g < G; ++g) {
      z[g] = 0.f;
#pragma unroll
      for (int v = 0; v < kFewWarps; ++v) z[g] += part[v][g][row][j];
    }
    finish<G>(P, row, f, z);
  }
}

using FewFn = void (*)(MmParams);
// By rows (at most 8, 16, 32) and whether features have gates.
const FewFn kFew[3][2] = {{mm_few_kernel<1, 1>, mm_few_kernel<1, 2>},
                          {mm_few_kernel<2, 1>, mm_few_kernel<2, 2>},
                          {mm_few_kernel<4, 1>, mm_few_kernel<4, 2>}};

}  // namespace

// Up to 32 rows.  Above 16 every load of weights meets four blocks of rows, and for
// large weights the tcgen05 kernel is faster (24 rows, us here and there): 4096 x 4096
// 16.4 and 18.5, with gates 30.7 and 24.6; 7168 x 7168 36.9 and 32.8, with gates 67.6
// and 53.2; 7168 x 512 with gates 24.6 and 18.4; 2048 x 1408 with gates 12.3 and 14.3.
bool mm_few_takes(const MmParams& P, int mode) {
  const bool large = P.cap[0] > 16 && int64_t(P.in) * P.out * (P.act == HOC_ACT_SWIGLU ? 5 : 1) > 1 << 24;
  return mode == kForward && P.seg == nullptr && P.cap[0] <= 32 && P.ld_rows % 8 == 0 && P.ld_w % 8 == 0 &&
         (P.in % 8 == 0 || P.ld_w != P.in) &&
         ((reinterpret_cast<uintptr_t>(P.rows[0]) | reinterpret_cast<uintptr_t>(P.w[0])) & 15u) == 0 &&
         !(large && mm_tc_takes(P, mode));
}

cudaError_t launch_mm_few(const MmParams& P, cudaStream_t s) {
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((P.out + kFewFeatures - 1) / kFewFeatures);
  cfg.blockDim = dim3(32 * kFewWarps);
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kFew[P.cap[0] <= 8 ? 0 : P.cap[0] <= 16 ? 1 : 2][P.act == HOC_ACT_SWIGLU], P);
}

cudaError_t mm_few_preload() {
  for (const auto& row : kFew)
    for (FewFn f : row) {
      cudaFuncAttributes a;
      const cudaError_t e = cudaFuncGetAttributes(&a, reinterpret_cast<const void*>(f));
      if (e != cudaSuccess) return e;
    }
  return cudaSuccess;
}

}  // namespace hoc
