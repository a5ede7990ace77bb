// Matrix products for operands of any alignment and width (mm.h): the general
// kernel behind the layer's entry points, for rows that are not a multiple of
// 16 bytes, which tensor copies cannot address, in products that are too small to
// gain by realigned copies (or without memory for those).
//
// A CTA of 4 warps computes a 64 x 64 tile of out[c][f] in steps of 32 along
// the contraction: both operands are gathered element by element into shared
// memory (the next step's elements are loaded into registers meanwhile) and
// multiplied with mma.m16n8k16 (bf16 in, binary32 sums).  Rows of a tile are
// named by a list, so the ranges that several sources sent to one expert share
// a tile.  With the gated activation the 64 columns are 32 gates and their 32
// values, placed so that one thread holds both of a feature.  Bound by issuing the
// element loads: 66 TFLOP/s at 4096 x 2047 x 2047.
#include "mm.h"

namespace hoc {
namespace {

constexpr int kAnyThreads = 128;
constexpr int kAnyTile = 64;
constexpr int kAnyStep = 32;
constexpr int kAnyPitch = kAnyStep + 8;  // 80-byte rows: the 8 rows of an ldmatrix fall in different banks

__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], const void* p) {
  const uint32_t a = uint32_t(__cvta_generic_to_shared(p));
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(a)
               : "memory");
}
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Global row of virtual row v of (buffer p, expert g): the sources' ranges one
// after another; -1 past the end.
__device__ __forceinline__ int64_t any_row(const MmParams& P, int p, int g, int64_t v) {
  const int ns = P.seg ? P.sources : 1;
  for (int s = 0; s < ns; ++s) {
    int64_t lo, n;
    mm_range(P, p, g, s, lo, n);
    if (v < n) return lo + v;
    v -= n;
  }
  return -1;
}

template <int MODE>
__global__ void __launch_bounds__(kAnyThreads) mm_any_kernel(const __grid_constant__ MmParams P) {
  __shared__ __align__(16) __nv_bfloat16 sm[kAnyTile][kAnyPitch];  // [c][k]
  __shared__ __align__(16) __nv_bfloat16 sn[kAnyTile][kAnyPitch];  // [f][k]
  __shared__ int64_t rowid[2][kAnyTile];
  extern __shared__ int counts[];  // vrows[n], tile0[n + 1]
  const int n = P.parts * P.groups;
  int* vrows = counts;
  unsigned* tile0 = reinterpret_cast<unsigned*>(counts + n);
  const bool gated = MODE == kForward && P.act == HOC_ACT_SWIGLU;
  const int fcount = MODE == kForward ? P.out : P.in;       // columns f of the result
  const int ftile = gated ? kAnyTile / 2 : kAnyTile;
  const unsigned ftiles = (fcount + ftile - 1) / ftile;
  const unsigned ctiles = MODE == kWgrad ? (P.out + kAnyTile - 1) / kAnyTile : 0;
  mm_count(P, 1, vrows, tile0, [&](int rows) {
    return (MODE == kWgrad ? ctiles : unsigned((rows + kAnyTile - 1) / kAnyTile)) * ftiles;
  });
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int wm = warp >> 1, wn = warp & 1;  // 32 x 32 part of the tile
  const int wrows = gated ? 2 * P.out : P.out;
  for (unsigned t = blockIdx.x; t < tile0[n]; t += gridDim.x) {
    const int i = mm_find(tile0, n, t);
    const int p = P.part0 + i / P.groups, g = P.group0 + i % P.groups;
    const unsigned lt = t - tile0[i];
    const int f0 = int(lt % ftiles) * ftile;
    const int c0 = int(lt / ftiles) * kAnyTile;  // wgrad: out feature; else virtual row
    const int len = MODE == kForward ? P.in : MODE == kDgrad ? P.out : vrows[i];
    const __nv_bfloat16* w = MODE == kWgrad ? nullptr : P.w[p] + int64_t(g) * wrows * P.in;
    __syncthreads();  // the tile before this one is done with rowid and the operands
    if (MODE != kWgrad && tid < kAnyTile) rowid[0][tid] = any_row(P, p, g, c0 + tid);

    // f-slot j of the tile: its feature, and its row of a gated weight
    auto feature = [&](int j) { return gated ? f0 + (j >> 5) * 16 + (j & 15) : f0 + j; };
    auto load = [&](int k0, uint16_t (&a)[16], uint16_t (&b)[16]) {
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        const int idx = e * kAnyThreads + tid;
        uint16_t va = 0, vb = 0;
        if (MODE == kWgrad) {
          const int m = idx & 63, k = idx >> 6;  // both operands have their rows' elements contiguous
          const int64_t row = k0 + k < len ? rowid[(k0 >> 5) & 1][k] : -1;
          if (row >= 0 && c0 + m < P.out) va = reinterpret_cast<const uint16_t*>(P.dy[p])[row * P.ld_dy + c0 + m];
          if (row >= 0 && f0 + m < P.in) vb = reinterpret_cast<const uint16_t*>(P.rows[p])[row * P.ld_rows + f0 + m];
        } else {
          const int k = idx & 31, m = idx >> 5;
          const int64_t row = rowid[0][m];
          if (row >= 0 && k0 + k < len) va = reinterpret_cast<const uint16_t*>(P.rows[p])[row * P.ld_rows + k0 + k];
          if (MODE == kForward) {
            const int f = feature(m);
            if (f < P.out && k0 + k < len)
              vb = reinterpret_cast<const uint16_t*>(w)[int64_t(f + (gated && (m & 16) ? P.out : 0)) * P.in + k0 + k];
          } else {
            const int f = f0 + (idx & 63), kk = k0 + (idx >> 6);
            if (f < P.in && kk < len) vb = reinterpret_cast<const uint16_t*>(w)[int64_t(kk) * P.in + f];
          }
        }
        a[e] = va;
        b[e] = vb;
      }
    };
    auto list = [&](int k0) {  // wgrad: the rows of one step
      if (MODE == kWgrad && tid < kAnyStep) rowid[(k0 >> 5) & 1][tid] = k0 + tid < len ? any_row(P, p, g, k0 + tid) : -1;
    };
    float acc[2][4][4] = {};
    uint16_t a[16], b[16];
    list(0);
    __syncthreads();
    if (len > 0) load(0, a, b);
    for (int k0 = 0; k0 < len; k0 += kAnyStep) {
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        const int idx = e * kAnyThreads + tid;
        uint16_t* da = MODE == kWgrad ? reinterpret_cast<uint16_t*>(&sm[idx & 63][idx >> 6])
                                      : reinterpret_cast<uint16_t*>(&sm[idx >> 5][idx & 31]);
        uint16_t* db = MODE == kForward ? reinterpret_cast<uint16_t*>(&sn[idx >> 5][idx & 31])
                                        : reinterpret_cast<uint16_t*>(&sn[idx & 63][idx >> 6]);
        *da = a[e];
        *db = b[e];
      }
      list(k0 + kAnyStep);
      __syncthreads();
      if (k0 + kAnyStep < len) load(k0 + kAnyStep, a, b);
#pragma unroll
      for (int kk = 0; kk < kAnyStep; kk += 16) {
        uint32_t ra[2][4], rb[2][4];
#pragma unroll
        for (int m = 0; m < 2; ++m) ldmatrix4(ra[m], &sm[wm * 32 + m * 16 + (lane & 15)][kk + (lane >> 4) * 8]);
#pragma unroll
        for (int q = 0; q < 2; ++q)  // two n8 columns each: rows f, halves of k
          ldmatrix4(rb[q], &sn[wn * 32 + q * 16 + (lane & 7) + (lane >> 4) * 8][kk + ((lane >> 3) & 1) * 8]);
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
          for (int j = 0; j < 4; ++j) mma16816(acc[m][j], ra[m], rb[j >> 1][(j & 1) * 2], rb[j >> 1][(j & 1) * 2 + 1]);
      }
      __syncthreads();
    }
    // thread: rows lane/4 (+8) of each 16-row block, columns 2 (lane % 4) (+1) of each 8-column block
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int c = wm * 32 + m * 16 + h * 8 + (lane >> 2);
        if (MODE == kWgrad) {
          if (c0 + c >= P.out) continue;
#pragma unroll
          for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int f = f0 + wn * 32 + j * 8 + (lane & 3) * 2 + e;
              if (f >= P.in) continue;
              const int64_t at = (int64_t(g) * P.out + c0 + c) * P.in + f;
              float v = acc[m][j][h * 2 + e];
              if (P.out_f32) {
                float* o = static_cast<float*>(P.y[p]) + at;
                *o = P.accumulate ? *o + v : v;
              } else {
                __nv_bfloat16* o = static_cast<__nv_bfloat16*>(P.y[p]) + at;
                *o = __float2bfloat16_rn(P.accumulate ? bf16_of(o) + v : v);
              }
            }
          continue;
        }
        const int64_t row = rowid[0][c];
        if (row < 0) continue;
        __nv_bfloat16* y = static_cast<__nv_bfloat16*>(P.y[p]) + row * P.ld_y;
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int slot = wn * 32 + j * 8 + (lane & 3) * 2 + e;
            float v = acc[m][j][h * 2 + e];
            if (MODE == kForward) {
              const int f = feature(slot);
              if (f >= P.out) continue;
              const __nv_bfloat16* bias = P.bias[p] ? P.bias[p] + int64_t(g) * wrows + f : nullptr;
              __nv_bfloat16* pre = P.pre_out[p] ? static_cast<__nv_bfloat16*>(P.pre_out[p]) + row * wrows + f : nullptr;
              if (gated) {
                if (j >= 2) continue;  // the value columns are read by their gates' turn
                float u = acc[m][j + 2][h * 2 + e];
                if (bias) {
                  v += bf16_of(bias);
                  u += bf16_of(bias + P.out);
                }
                if (pre) {
                  pre[0] = __float2bfloat16_rn(v);
                  pre[P.out] = __float2bfloat16_rn(u);
                }
                v = mm_act(HOC_ACT_SILU, v) * u;
              } else {
                if (bias) v += bf16_of(bias);
                if (pre) *pre = __float2bfloat16_rn(v);
                v = mm_act(P.act, v);
              }
              if (P.res[p]) v += bf16_of(P.res[p] + row * P.ld_res + f);
              y[f] = __float2bfloat16_rn(v);
            } else {
              const int f = f0 + slot;
              if (f >= P.in) continue;
              if (P.act == HOC_ACT_SWIGLU) {
                const __nv_bfloat16* pre = P.pre[p] + row * 2 * P.in + f;
                const float zg = bf16_of(pre), zu = bf16_of(pre + P.in);
                y[f] = __float2bfloat16_rn(v * zu * mm_act_slope(HOC_ACT_SILU, zg));
                y[P.in + f] = __float2bfloat16_rn(v * mm_act(HOC_ACT_SILU, zg));
              } else {
                if (P.act != HOC_ACT_NONE) v = mm_act_back(P.act, bf16_of(P.pre[p] + row * P.in + f), v);
                y[f] = __float2bfloat16_rn(v);
              }
            }
          }
      }
  }
}

using AnyFn = void (*)(MmParams);
const AnyFn kAny[3] = {mm_any_kernel<kForward>, mm_any_kernel<kDgrad>, mm_any_kernel<kWgrad>};

}  // namespace

cudaError_t launch_mm_any(const MmParams& P, int mode, int sms, cudaStream_t s) {
  const int n = P.parts * P.groups;
  // Tiles the launch can have at most: every range may leave one tile part full.
  const int64_t f = mode == kForward ? (P.act == HOC_ACT_SWIGLU ? 2 * int64_t(P.out) : P.out) : P.in;
  int64_t c = 0;
  if (mode == kWgrad)
    c = int64_t(n) * ((P.out + kAnyTile - 1) / kAnyTile);
  else
    for (int p = P.part0; p < P.part0 + P.parts; ++p) c += P.cap[p] / kAnyTile + P.groups;
  const int64_t tiles = c * ((f + kAnyTile - 1) / kAnyTile), cap = int64_t(sms) * 4;
  const int grid = int(tiles < 1 ? 1 : tiles < cap ? tiles : cap);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(kAnyThreads);
  cfg.dynamicSmemBytes = sizeof(int) * (2 * size_t(n) + 1);
  cfg.stream = s;
  return cudaLaunchKernelEx(&cfg, kAny[mode], P);
}

cudaError_t mm_any_preload() {
  for (AnyFn f : kAny) {
    cudaFuncAttributes a;
    const cudaError_t e = cudaFuncGetAttributes(&a, reinterpret_cast<const void*>(f));
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace hoc
