// Entry points of hoc_layer.h: argument checks, the choice of a product
// kernel, and the small kernels around the products (row ranges of a dispatch,
// activation gradient, bias gradient).
#include <atomic>
#include <cstdio>
#include <mutex>

#include "mm.h"

namespace hoc {
namespace {

// ------------------------------------------------------------ row ranges
struct SegIds {
  const int32_t* ids[kMaxRanks];
};

constexpr int kSegThreads = 256;
constexpr int kSegItems = 2048;     // pairs of one CTA
constexpr int kSegShared = 8192;    // experts whose counters fit in shared memory

// seg[d][1 + s * per + g] += pairs of source s (blockIdx.y) for expert g of
// rank d.  Integer atomics: the sums do not depend on their order.
__global__ void seg_count_kernel(const __grid_constant__ SegIds P, int n, int experts, int per, int nranks,
                                 unsigned long long* seg) {
  extern __shared__ int hist[];
  const int s = blockIdx.y;
  const bool shared = experts <= kSegShared;
  const size_t stride = size_t(nranks) * per + 1;
  for (int e = threadIdx.x; shared && e < experts; e += blockDim.x) hist[e] = 0;
  __syncthreads();
  const int64_t lo = int64_t(blockIdx.x) * kSegItems;
  for (int64_t i = lo + threadIdx.x; i < lo + kSegItems && i < n; i += blockDim.x) {
    const int e = P.ids[s][i];
    if (e < 0 || e >= experts) continue;
    if (shared) atomicAdd(&hist[e], 1);
    else atomicAdd(seg + (e / per) * stride + 1 + size_t(s) * per + e % per, 1ull);
  }
  __syncthreads();
  for (int e = threadIdx.x; shared && e < experts; e += blockDim.x)
    if (hist[e]) atomicAdd(seg + (e / per) * stride + 1 + size_t(s) * per + e % per, (unsigned long long)hist[e]);
}

// Counts to offsets: an inclusive scan of seg[d][1 ..] in place, one CTA per rank.
// Both and the zeroing before them are bound by their launches: 15 us for 8 x 4096
// tokens, top-6 of 64 experts.
__global__ void seg_scan_kernel(int m, int64_t* seg) {
  int64_t* v = seg + size_t(blockIdx.x) * (size_t(m) + 1) + 1;
  __shared__ int64_t part[kSegThreads / 32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int64_t base = 0;
  for (int at = 0; at < m; at += kSegThreads) {
    const int i = at + int(threadIdx.x);
    int64_t x = i < m ? v[i] : 0;
    for (int off = 1; off < 32; off <<= 1) {
      const int64_t y = __shfl_up_sync(0xFFFFFFFFu, x, off);
      if (lane >= off) x += y;
    }
    if (lane == 31) part[warp] = x;
    __syncthreads();
    int64_t before = base, all = 0;
    for (int w = 0; w < kSegThreads / 32; ++w) {
      if (w < warp) before += part[w];
      all += part[w];
    }
    if (i < m) v[i] = before + x;
    base += all;
    __syncthreads();
  }
}

// ------------------------------------------------------------ activation gradient
// dz = dy * act'(pre), in vectors of 8 values where rows are whole 16-byte vectors,
// else of one.  Bound by its bytes: dy and pre read, dz written.  A thread loads
// all its vectors before its arithmetic.  65,536 rows of 1280: GELU 93 us with two
// vectors (5.4 TB/s; 98 with one, 104 with four), the gated form, which loads three
// rows, 142 us with one (5.9 TB/s; 152 with two, 187 with four).
constexpr int kActThreads = 256;
constexpr int kGatedVecs = 1, kPlainVecs = 2;
template <int V, int ACT>
__global__ void __launch_bounds__(kActThreads)
    act_grad_kernel(const __nv_bfloat16* dy, const __nv_bfloat16* pre, __nv_bfloat16* dz, int64_t rows, int width) {
  struct alignas(2 * V) Vec {
    __nv_bfloat16 v[V];
  };
  const unsigned per = unsigned(width / V);
  const int64_t n = rows * per;
  constexpr bool gated = ACT == HOC_ACT_SWIGLU;
  constexpr int kVecs = gated ? kGatedVecs : kPlainVecs;
  for (int64_t base = int64_t(blockIdx.x) * kActThreads * kVecs; base < n; base += int64_t(gridDim.x) * kActThreads * kVecs) {
    Vec d[kVecs], z[kVecs], u[kVecs];
    int64_t at[kVecs];  // of pre and dz; -1 past the end
#pragma unroll
    for (int j = 0; j < kVecs; ++j) {
      const int64_t i = base + j * kActThreads + int(threadIdx.x);
      at[j] = -1;
      if (i >= n) continue;
      // a gated row is twice as wide
      const int64_t row = !gated ? 0 : i < (int64_t(1) << 32) ? int64_t(unsigned(i) / per) : i / per;
      at[j] = i * V + row * width;
      d[j] = *reinterpret_cast<const Vec*>(dy + i * V);
      z[j] = *reinterpret_cast<const Vec*>(pre + at[j]);
      if (gated) u[j] = *reinterpret_cast<const Vec*>(pre + at[j] + width);
    }
#pragma unroll
    for (int j = 0; j < kVecs; ++j) {
      if (at[j] < 0) continue;
      Vec o, o2;
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const float g = __bfloat162float(z[j].v[e]), dd = __bfloat162float(d[j].v[e]);
        if (gated) {
          o.v[e] = __float2bfloat16_rn(dd * __bfloat162float(u[j].v[e]) * mm_act_slope(HOC_ACT_SILU, g));
          o2.v[e] = __float2bfloat16_rn(dd * mm_act(HOC_ACT_SILU, g));
        } else {
          o.v[e] = __float2bfloat16_rn(mm_act_back(ACT, g, dd));
        }
      }
      *reinterpret_cast<Vec*>(dz + at[j]) = o;
      if (gated) *reinterpret_cast<Vec*>(dz + at[j] + width) = o2;
    }
  }
}

using ActFn = void (*)(const __nv_bfloat16*, const __nv_bfloat16*, __nv_bfloat16*, int64_t, int);
// By whether rows are whole 16-byte vectors, and the activation.
const ActFn kActGrad[2][4] = {{act_grad_kernel<1, HOC_ACT_RELU>, act_grad_kernel<1, HOC_ACT_GELU>,
                               act_grad_kernel<1, HOC_ACT_SILU>, act_grad_kernel<1, HOC_ACT_SWIGLU>},
                              {act_grad_kernel<8, HOC_ACT_RELU>, act_grad_kernel<8, HOC_ACT_GELU>,
                               act_grad_kernel<8, HOC_ACT_SILU>, act_grad_kernel<8, HOC_ACT_SWIGLU>}};
static_assert(HOC_ACT_RELU == 1 && HOC_ACT_GELU == 2 && HOC_ACT_SILU == 3 && HOC_ACT_SWIGLU == 4, "the order above");

// ------------------------------------------------------------ bias gradient
// db[e][n] (+)= sum over the expert's rows of dy[r][n]: bound by reading dy once
// more (after the weight gradient has read it, from L2 where it fits).  A cluster
// of 8 CTAs sums 64 columns of one expert, each warp taking 4 rows at a time of 8
// lanes x 8 columns (or, where rows are not whole 16-byte vectors, one row of 32
// lanes x 2 columns).  Binary32 sums; lanes, warps and CTAs are added in a fixed
// order.  With one CTA for the 64 columns the 4096 x 4096 gradient took 31 us; with
// eight it adds 8 us to the 78 us of 4096 rows of 4096 x 4096.
// For one range of rows the product's spare warps mostly do the same (mm_tc.cu).
// Launched right behind the product (programmatic dependent launch), it runs beside
// it where SMs have room: it needs nothing of it, and what both need was complete when the product's
// CTAs, which let it start, had passed their own wait.  Every kernel that is
// launched before it therefore waits before it lets dependents start.
constexpr int kBiasWarps = 8;
constexpr int kBiasCtas = 8;
template <bool VEC>
__global__ void __cluster_dims__(1, 1, kBiasCtas) __launch_bounds__(32 * kBiasWarps)
    bias_grad_kernel(const __grid_constant__ MmParams P) {
  __shared__ float sums[kBiasWarps][64];
  __shared__ float mine[64];
  const int i = blockIdx.y, p = P.part0 + i / P.groups, g = P.group0 + i % P.groups;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int part = int(blockIdx.z) * kBiasWarps + warp;
  const int c0 = int(blockIdx.x) * 64;
  const __nv_bfloat16* dy = P.dy[p];
  constexpr int N = VEC ? 8 : 2;
  constexpr int kRows = VEC ? 4 : 1;  // rows of a warp at a time
  const int c = c0 + (VEC ? (lane & 7) * 8 : lane * 2), sub = VEC ? lane >> 3 : 0;
  float acc[N] = {};
  const int ns = P.seg ? P.sources : 1;
  for (int s = 0; s < ns && c < P.out; ++s) {
    int64_t lo, n;
    mm_range(P, p, g, s, lo, n);
#pragma unroll 4
    for (int64_t r = int64_t(part) * kRows + sub; r < n; r += kBiasWarps * kBiasCtas * kRows) {
      const __nv_bfloat16* q = dy + (lo + r) * P.ld_dy + c;
      if constexpr (VEC) {
        const uint4 v = __ldg(reinterpret_cast<const uint4*>(q));
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          acc[2 * e] += __uint_as_float(w[e] << 16);
          acc[2 * e + 1] += __uint_as_float(w[e] & 0xFFFF0000u);
        }
      } else {
        acc[0] += bf16_of(q);
        if (c + 1 < P.out) acc[1] += bf16_of(q + 1);
      }
    }
  }
#pragma unroll
  for (int e = 0; e < N; ++e) {
    if (VEC) {
      acc[e] += __shfl_xor_sync(0xFFFFFFFFu, acc[e], 8);
      acc[e] += __shfl_xor_sync(0xFFFFFFFFu, acc[e], 16);
    }
    if (!VEC || lane < 8) sums[warp][lane * N + e] = acc[e];
  }
  __syncthreads();
  if (threadIdx.x < 64) {
    float v = 0.f;
    for (int w = 0; w < kBiasWarps; ++w) v += sums[w][threadIdx.x];
    mine[threadIdx.x] = v;
  }
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
  const int col = c0 + int(threadIdx.x);
  if (blockIdx.z == 0 && threadIdx.x < 64 && col < P.out) {
    float v = 0.f;
    const uint32_t here = uint32_t(__cvta_generic_to_shared(&mine[threadIdx.x]));
    for (int w = 0; w < kBiasCtas; ++w) {
      uint32_t there;
      float x;
      asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(there) : "r"(here), "r"(w));
      asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(x) : "r"(there) : "memory");
      v += x;
    }
    const int64_t at = int64_t(g) * P.out + col;
    if (P.out_f32) {
      float* o = static_cast<float*>(P.pre_out[p]) + at;
      *o = P.accumulate ? *o + v : v;
    } else {
      __nv_bfloat16* o = static_cast<__nv_bfloat16*>(P.pre_out[p]) + at;
      *o = __float2bfloat16_rn(P.accumulate ? bf16_of(o) + v : v);
    }
  }
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
  // Whatever follows on the stream waits for this grid; so this grid waits for the product's.
  asm volatile("griddepcontrol.wait;" ::: "memory");
}

// ------------------------------------------------------------ realigned copies
// Rows of `width` values from anywhere to rows of `to_ld` values on 16-byte
// boundaries, the rest of each row zero: a thread makes one 16-byte vector, from
// aligned words (and, where the source starts between two words, its first and last
// value).  Bound by its bytes; the widths where it pays are at kRealignLeast.
struct Realign {
  const uint16_t* from[kMaxRanks];
  uint4* to[kMaxRanks];
  int64_t rows[kMaxRanks];
  int64_t from_ld, to_ld;
  int64_t block, to_block;  // rows of a block, and of the place that it is copied to (an expert's gates, padded)
  int width;
};
__global__ void __launch_bounds__(256) realign_kernel(const __grid_constant__ Realign R) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int p = blockIdx.y, vecs = int(R.to_ld / 8);
  const int64_t n = R.rows[p] * vecs;
  for (int64_t i = int64_t(blockIdx.x) * blockDim.x + threadIdx.x; i < n; i += int64_t(gridDim.x) * blockDim.x) {
    const int64_t row = i / vecs;
    const int v = int(i - row * vecs), left = R.width - v * 8;
    const uint16_t* at = R.from[p] + row * R.from_ld + v * 8;
    uint32_t o[4] = {0, 0, 0, 0};
    if (left >= 8) {
      const bool odd = (reinterpret_cast<uintptr_t>(at) & 2u) != 0;
      const uint32_t* w = reinterpret_cast<const uint32_t*>(at + odd);
      if (odd) {
        const uint32_t a = __ldg(at), b = __ldg(w), c = __ldg(w + 1), d = __ldg(w + 2), e = __ldg(at + 7);
        o[0] = a | b << 16;
        o[1] = __funnelshift_r(b, c, 16);
        o[2] = __funnelshift_r(c, d, 16);
        o[3] = d >> 16 | e << 16;
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) o[j] = __ldg(w + j);
      }
    } else {
      for (int j = 0; j < left; ++j) o[j >> 1] |= uint32_t(__ldg(at + j)) << (16 * (j & 1));
    }
    const int64_t to = row / R.block * R.to_block + row % R.block;
    R.to[p][to * vecs + v] = make_uint4(o[0], o[1], o[2], o[3]);
  }
}

// ------------------------------------------------------------ host
constexpr int kMaxWidth = 1 << 20;
constexpr size_t kMaxRows = size_t(1) << 30;
// When realigned copies pay: where the contraction is long, which the general kernel's few
// CTAs walk alone (us here, with copies and without, from a flushed cache: forward 1 x 129 x
// 127 13 and 13, 1 x 257 x 255 13 and 17; data gradient 15 and 15, 15 and 21; weight gradient
// over 64 rows of 257 x 255 18 and 13, over 192 rows 19 and 21, over 2000 rows of 65 x 67 19
// and 142, over 16,000 of 33 x 31 36 and 1070); and in large products whatever its length
// (multiplications; forward 4 x 501 x 499 14 and 25, 4096 x 2047 x 2047 70 and 520; weight
// gradient of the latter 65 and 950).  Small ones gain nothing (1 x 65 x 63 13 and 11).
constexpr int64_t kRealignLong = 160;
constexpr double kRealignLeast[3] = {1 << 16, 1 << 16, 1 << 24};

hocResult_t refuse(const char* who, const char* what) {
  char msg[160];
  snprintf(msg, sizeof msg, "%s: %s", who, what);
  set_error_detail(msg);
  return HOC_ERR_INVALID_ARG;
}

// What a launch returned, and nothing else: the runtime's last error may be an earlier call's, which
// is the caller's to read.  Only a failed launch's own error is cleared.
hocResult_t launched(const char* who, cudaError_t e) {
  if (e == cudaSuccess) return HOC_SUCCESS;
  cudaGetLastError();
  char msg[160];
  snprintf(msg, sizeof msg, "%s: launch failed: %s", who, cudaGetErrorString(e));
  set_error_detail(msg);
  return HOC_ERR_CUDA;
}

// early: the kernel may start before the one before it on the stream has ended, and waits for that itself.
template <class... KArgs, class... Args>
cudaError_t launch(void (*kernel)(KArgs...), dim3 grid, int block, size_t smem, bool early, cudaStream_t s, Args... args) {
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(block);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = early;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

int sm_count() {
  static std::atomic<int> known[64];
  int dev = 0, sms = 1;
  if (cudaGetDevice(&dev) != cudaSuccess) return 1;
  if (dev < 64 && known[dev].load() > 0) return known[dev].load();
  cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (dev < 64) known[dev].store(sms);
  return sms;
}

bool widths_ok(int in, int out) { return in >= 1 && out >= 1 && in <= kMaxWidth && out <= kMaxWidth; }

bool act_ok(int act) { return act >= HOC_ACT_NONE && act <= HOC_ACT_SWIGLU; }

// Checks the groups and fills the layout part of P.
hocResult_t take_groups(const char* who, const hocRowGroups_t* G, MmParams& P) {
  if (!G || !G->seg || !G->capacity) return refuse(who, "groups, its seg and its capacity must be given");
  if (G->nranks < 1 || G->nranks > kMaxRanks || G->experts < 1 || G->experts > kMaxWidth || G->sources < 1 ||
      G->sources > 4096)
    return refuse(who, "rank, expert or source count out of range");
  for (int p = 0; p < G->nranks; ++p) {
    if (G->capacity[p] > kMaxRows) return refuse(who, "a buffer of more than 2^30 rows");
    P.cap[p] = int64_t(G->capacity[p]);
  }
  P.seg = G->seg;
  P.experts = G->experts;
  P.sources = G->sources;
  P.parts = G->nranks;
  P.groups = G->experts;
  return HOC_SUCCESS;
}

template <class T>
hocResult_t take(const char* who, const char* name, const void* const* from, const MmParams& P, bool rows, T** to) {
  char msg[96];
  snprintf(msg, sizeof msg, "%s holds a NULL pointer", name);
  if (!from) return refuse(who, msg);
  for (int p = 0; p < P.parts; ++p) {
    if (!from[p] && !(rows && P.cap[p] == 0)) return refuse(who, msg);
    to[p] = static_cast<T*>(const_cast<void*>(from[p]));
    if (reinterpret_cast<uintptr_t>(from[p]) & 1u) return refuse(who, "a pointer that is not aligned to its elements");
  }
  return HOC_SUCCESS;
}

int64_t up_to(int64_t v, int64_t step) { return (v + step - 1) / step * step; }

// Scratch for realigned operands: stream-ordered allocations from a pool of this
// library's own on the current device, which keeps what it has been given until
// hoc_layer_trim takes it back.  (Given back whenever a stream is waited for, as a pool does
// by default, it would have to be mapped again: 262,144 rows of 1023 -> 255 with a wait
// after every call 1890 us instead of 610, 1,048,576 rows 6880 instead of 2390.)
std::mutex pool_lock;
cudaMemPool_t pools[64] = {};
cudaError_t scratch(void** at, size_t bytes, cudaStream_t s) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 64) return cudaErrorNotSupported;
  cudaMemPool_t pool;
  {
    std::lock_guard<std::mutex> hold(pool_lock);
    if (!pools[dev]) {
      cudaMemPoolProps props = {};
      props.allocType = cudaMemAllocationTypePinned;
      props.location.type = cudaMemLocationTypeDevice;
      props.location.id = dev;
      uint64_t keep = UINT64_MAX;
      e = cudaMemPoolCreate(&pools[dev], &props);
      if (e == cudaSuccess) e = cudaMemPoolSetAttribute(pools[dev], cudaMemPoolAttrReleaseThreshold, &keep);
      if (e != cudaSuccess) return e;
    }
    pool = pools[dev];
  }
  return cudaMallocFromPoolAsync(at, bytes, pool, s);
}

// Copies the operands that tensor copies could not address into scratch and points
// P at them; the caller frees *used on the stream.  *used stays null where the
// product is too small to gain by it or no scratch is to be had: P is as it was,
// and the general kernel takes it.
void realign(MmParams& P, int mode, cudaStream_t s, void** used) {
  const bool gated = mode == kForward && P.act == HOC_ACT_SWIGLU;
  int64_t rows = 0, length = mode == kForward ? P.in : mode == kDgrad ? P.out : 0;
  for (int p = 0; p < P.parts; ++p) {
    rows += P.cap[p];
    // rows of an expert, on average: the ranges are not known here
    if (mode == kWgrad && P.cap[p] / P.experts > length) length = P.cap[p] / P.experts;
  }
  if (rows == 0 || (length < kRealignLong && double(rows) * P.in * P.out * (gated ? 2 : 1) < kRealignLeast[mode])) return;
  struct Operand {  // the rows, then dy (wgrad) or the weights
    const __nv_bfloat16* from[kMaxRanks];
    int64_t rows[kMaxRanks];
    int64_t from_ld, block, to_block;
    int width;
    bool copy;
    int64_t to_ld() const { return up_to(width, 8); }
    size_t bytes(int p) const { return size_t(up_to(rows[p], block) / block * to_block) * to_ld() * 2; }
  } op[2] = {};
  op[0].width = mode == kDgrad ? P.out : P.in;
  op[0].from_ld = P.ld_rows;
  op[1].width = mode == kWgrad ? P.out : P.in;
  op[1].from_ld = mode == kWgrad ? P.ld_dy : P.ld_w;
  size_t bytes = 0;
  for (int i = 0; i < 2; ++i) {
    Operand& o = op[i];
    const bool weights = i == 1 && mode != kWgrad;
    o.block = weights ? P.out : 1;
    o.to_block = weights && gated ? up_to(P.out, 8) : o.block;
    // (a width that is not whole vectors: the kernel for a few rows relies on the zeros behind both operands' rows)
    o.copy = o.from_ld % 8 != 0 || o.width % 8 != 0 || o.to_block != o.block;
    for (int p = 0; p < P.parts; ++p) {
      o.from[p] = i == 0 ? P.rows[p] : weights ? P.w[p] : P.dy[p];
      o.rows[p] = weights ? int64_t(P.experts) * P.out * (gated ? 2 : 1) : P.cap[p];
      o.copy = o.copy || (reinterpret_cast<uintptr_t>(o.from[p]) & 15u) != 0;
    }
    for (int p = 0; o.copy && p < P.parts; ++p) bytes += o.bytes(p);
  }
  void* at = nullptr;
  if (bytes == 0) return;
  if (scratch(&at, bytes, s) != cudaSuccess) {
    cudaGetLastError();
    return;
  }
  MmParams Q = P;
  char* next = static_cast<char*>(at);
  cudaError_t e = cudaSuccess;
  for (int i = 0; i < 2 && e == cudaSuccess; ++i) {
    const Operand& o = op[i];
    if (!o.copy) continue;
    Realign R{};
    R.from_ld = o.from_ld;
    R.to_ld = o.to_ld();
    R.block = o.block;
    R.to_block = o.to_block;
    R.width = o.width;
    int64_t most = 1;
    for (int p = 0; p < P.parts; ++p) {
      R.from[p] = reinterpret_cast<const uint16_t*>(o.from[p]);
      R.to[p] = reinterpret_cast<uint4*>(next);
      R.rows[p] = o.rows[p];
      if (o.rows[p] > most) most = o.rows[p];
      const __nv_bfloat16* to = reinterpret_cast<const __nv_bfloat16*>(next);
      if (i == 0) Q.rows[p] = to;
      else if (mode == kWgrad) Q.dy[p] = to;
      else Q.w[p] = to;
      next += o.bytes(p);
    }
    if (i == 0) Q.ld_rows = R.to_ld;
    else if (mode == kWgrad) Q.ld_dy = R.to_ld;
    else {
      Q.ld_w = R.to_ld;
      Q.out_w = o.to_block;
    }
    const int64_t want = (most * (R.to_ld / 8) + 255) / 256, cap = int64_t(sm_count()) * 16;
    e = launch(realign_kernel, dim3(unsigned(want < cap ? want : cap), P.parts), 256, 0, true, s, R);
  }
  if (e == cudaSuccess) {
    P = Q;
    *used = at;
  } else {
    cudaGetLastError();
    cudaFreeAsync(at, s);
  }
}

// Launches one product, in as many launches as kMmMaxGroups asks for.
hocResult_t launch_product(const char* who, MmParams P, int mode, cudaStream_t s, bool* summed) {
  const int sms = sm_count();
  const int nranks = P.parts, experts = P.groups;
  const bool few = mm_few_takes(P, mode), tc = !few && mm_tc_takes(P, mode);
  const int by_group = experts < kMmMaxGroups ? experts : kMmMaxGroups;
  const int by_part = kMmMaxGroups / by_group < nranks ? kMmMaxGroups / by_group : nranks;
  for (int p = 0; p < nranks; p += by_part)
    for (int g = 0; g < experts; g += by_group) {
      P.part0 = p;
      P.parts = nranks - p < by_part ? nranks - p : by_part;
      P.group0 = g;
      P.groups = experts - g < by_group ? experts - g : by_group;
      int64_t rows = 0;
      for (int q = p; q < p + P.parts; ++q) rows += P.cap[q];
      if (rows == 0 && mode != kWgrad) continue;
      const cudaError_t e = few  ? launch_mm_few(P, s)
                            : tc ? launch_mm_tc(P, mode, s, summed)
                                 : launch_mm_any(P, mode, sms, s);
      if (e != cudaSuccess) return launched(who, e);
    }
  return HOC_SUCCESS;
}

hocResult_t run_product(const char* who, const MmParams& given, int mode, cudaStream_t s, bool* summed = nullptr) {
  MmParams P = given;
  P.ld_w = P.in;
  P.out_w = P.out;
  void* held = nullptr;
  if (!mm_few_takes(P, mode) && !mm_tc_takes(P, mode)) realign(P, mode, s, &held);
  const hocResult_t r = launch_product(who, P, mode, s, summed);
  if (held && cudaFreeAsync(held, s) != cudaSuccess && r == HOC_SUCCESS) {
    set_error_detail("freeing scratch failed");
    return HOC_ERR_CUDA;
  }
  return r;
}

// 64-wide tiles bound every kernel's tile count; it has to fit the tile index.
bool tiles_ok(const MmParams& P, int mode, int width) {
  int64_t c = 0;
  for (int p = 0; p < P.parts; ++p)
    c += mode == kWgrad ? int64_t(P.groups) * ((P.out + 63) / 64)
                        : P.cap[p] / 64 + int64_t(P.groups) * (1 + P.sources / 8);
  return c * ((int64_t(width) + 63) / 64) < (int64_t(1) << 31);
}

hocResult_t run_wgrad(const char* who, MmParams& P, void* const* db, cudaStream_t s) {
  if (!tiles_ok(P, kWgrad, P.in)) return refuse(who, "more than 2^31 tiles");
  for (int p = 0; p < P.parts; ++p) P.pre_out[p] = db ? db[p] : nullptr;
  bool summed = false;
  hocResult_t r = run_product(who, P, kWgrad, s, &summed);
  if (r != HOC_SUCCESS || !db || summed) return r;
  const int pairs = P.parts * P.groups;
  bool vec = P.out % 8 == 0 && P.ld_dy % 8 == 0;
  for (int p = 0; p < P.parts; ++p) vec = vec && (reinterpret_cast<uintptr_t>(P.dy[p]) & 15u) == 0;
  MmParams Q = P;
  for (int at = 0; at < pairs;) {  // the grid's y extent ends at 65535
    const int p = at / P.groups, g = at % P.groups;
    Q.part0 = p;
    Q.group0 = g;
    Q.parts = 1;
    Q.groups = P.groups - g < 65535 ? P.groups - g : 65535;
    if (g == 0 && P.groups * int64_t(P.parts - p) <= 65535) {
      Q.parts = P.parts - p;
      Q.groups = P.groups;
    }
    const cudaError_t e = launch(vec ? bias_grad_kernel<true> : bias_grad_kernel<false>,
                                 dim3((P.out + 63) / 64, Q.parts * Q.groups, kBiasCtas), 32 * kBiasWarps, 0, true, s, Q);
    if (e != cudaSuccess) return launched(who, e);
    at += Q.parts * Q.groups;
  }
  return HOC_SUCCESS;
}

template <class V>
hocResult_t take_one(const char* who, const char* name, const void* v, V** to) {
  char msg[96];
  snprintf(msg, sizeof msg, "%s must be given", name);
  if (!v) return refuse(who, msg);
  if (reinterpret_cast<uintptr_t>(v) & 1u) return refuse(who, "a pointer that is not aligned to its elements");
  to[0] = static_cast<V*>(const_cast<void*>(v));
  return HOC_SUCCESS;
}

hocResult_t dense(const char* who, int rows, int in, int out, int32_t* status, MmParams& P) {
  if (rows < 0 || size_t(rows) > kMaxRows || !widths_ok(in, out)) return refuse(who, "row count or width out of range");
  if (!status) return refuse(who, "status must be given");
  P.parts = P.groups = P.experts = P.sources = 1;
  P.cap[0] = rows;
  P.in = in;
  P.out = out;
  P.status = status;
  return HOC_SUCCESS;
}

#define HOC_TRY(x)                                 \
  do {                                             \
    const hocResult_t try_r = (x);                 \
    if (try_r != HOC_SUCCESS) return try_r;        \
  } while (0)

}  // namespace

cudaError_t mm_preload() {
  const void* fns[] = {reinterpret_cast<const void*>(&seg_count_kernel), reinterpret_cast<const void*>(&seg_scan_kernel),
                       reinterpret_cast<const void*>(&realign_kernel),
                       reinterpret_cast<const void*>(&bias_grad_kernel<true>),
                       reinterpret_cast<const void*>(&bias_grad_kernel<false>)};
  for (const void* f : fns) {
    cudaFuncAttributes a;
    const cudaError_t e = cudaFuncGetAttributes(&a, f);
    if (e != cudaSuccess) return e;
  }
  for (const auto& row : kActGrad)
    for (ActFn f : row) {
      cudaFuncAttributes a;
      const cudaError_t e = cudaFuncGetAttributes(&a, reinterpret_cast<const void*>(f));
      if (e != cudaSuccess) return e;
    }
  cudaError_t e = mm_any_preload();
  if (e == cudaSuccess) e = mm_few_preload();
  return e == cudaSuccess ? mm_tc_preload() : e;
}

}  // namespace hoc

using namespace hoc;

extern "C" hocResult_t hoc_ep_segments(int nranks, const int32_t* const* expert_ids, int tokens, int topk, int experts,
                                       int64_t* seg, void* stream) {
  const char* who = "hoc_ep_segments";
  if (nranks < 1 || nranks > kMaxRanks || tokens < 0 || topk < 1 || experts < 1 || experts > kMaxWidth ||
      experts % nranks != 0)
    return refuse(who, "bad rank count, shape or expert count");
  if (!seg || size_t(tokens) * topk > size_t(INT32_MAX)) return refuse(who, "seg must be given, tokens * topk fit 31 bits");
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  SegIds P{};
  for (int r = 0; tokens > 0 && r < nranks; ++r) {
    if (!expert_ids || !expert_ids[r]) return refuse(who, "expert_ids holds a NULL pointer");
    P.ids[r] = expert_ids[r];
  }
  const size_t per_rank = size_t(experts) + 1;  // nranks * (experts / nranks) + 1
  cudaError_t e = cudaMemsetAsync(seg, 0, sizeof(int64_t) * per_rank * nranks, s);
  if (e == cudaSuccess && tokens > 0) {
    const int n = tokens * topk;
    e = launch(seg_count_kernel, dim3(unsigned((int64_t(n) + kSegItems - 1) / kSegItems), nranks), kSegThreads,
               experts <= kSegShared ? sizeof(int) * size_t(experts) : 0, false, s, P, n, experts, experts / nranks, nranks,
               reinterpret_cast<unsigned long long*>(seg));
    if (e == cudaSuccess) e = launch(seg_scan_kernel, dim3(nranks), kSegThreads, 0, false, s, experts, seg);
  }
  return launched(who, e);
}

extern "C" hocResult_t hoc_expert_mm(const hocRowGroups_t* groups, const void* const* x, const void* const* weight,
                                     const void* const* bias, int in, int out, int act, void* const* y,
                                     void* const* pre, int32_t* status, void* stream) {
  const char* who = "hoc_expert_mm";
  MmParams P{};
  HOC_TRY(take_groups(who, groups, P));
  if (!widths_ok(in, out) || !act_ok(act) || !status) return refuse(who, "bad width or activation, or no status");
  P.in = P.ld_rows = in;
  P.out = P.ld_y = out;
  P.act = act;
  P.status = status;
  HOC_TRY(take(who, "x", x, P, true, P.rows));
  HOC_TRY(take(who, "weight", weight, P, false, P.w));
  if (bias) HOC_TRY(take(who, "bias", bias, P, false, P.bias));
  HOC_TRY(take(who, "y", y, P, true, P.y));
  if (pre) HOC_TRY(take(who, "pre", pre, P, true, P.pre_out));
  if (!tiles_ok(P, kForward, 2 * out)) return refuse(who, "more than 2^31 tiles");
  return run_product(who, P, kForward, static_cast<cudaStream_t>(stream));
}

extern "C" hocResult_t hoc_expert_mm_dgrad(const hocRowGroups_t* groups, const void* const* dy,
                                           const void* const* weight, int in, int out, int act,
                                           const void* const* pre, void* const* dx, int32_t* status, void* stream) {
  const char* who = "hoc_expert_mm_dgrad";
  MmParams P{};
  HOC_TRY(take_groups(who, groups, P));
  if (!widths_ok(in, out) || !act_ok(act) || !status) return refuse(who, "bad width or activation, or no status");
  P.in = in;
  P.out = P.ld_rows = out;
  P.ld_y = act == HOC_ACT_SWIGLU ? 2 * int64_t(in) : in;
  P.act = act;
  P.status = status;
  HOC_TRY(take(who, "dy", dy, P, true, P.rows));
  HOC_TRY(take(who, "weight", weight, P, false, P.w));
  if (act != HOC_ACT_NONE) HOC_TRY(take(who, "pre", pre, P, true, P.pre));
  HOC_TRY(take(who, "dx", dx, P, true, P.y));
  if (!tiles_ok(P, kDgrad, in)) return refuse(who, "more than 2^31 tiles");
  return run_product(who, P, kDgrad, static_cast<cudaStream_t>(stream));
}

extern "C" hocResult_t hoc_expert_mm_wgrad(const hocRowGroups_t* groups, const void* const* dy, const void* const* x,
                                           int in, int out, hocDataType_t dtype, int accumulate, void* const* dw,
                                           void* const* db, int32_t* status, void* stream) {
  const char* who = "hoc_expert_mm_wgrad";
  MmParams P{};
  HOC_TRY(take_groups(who, groups, P));
  if (!widths_ok(in, out) || !status) return refuse(who, "bad width, or no status");
  if (dtype != HOC_BFLOAT16 && dtype != HOC_FLOAT32) return refuse(who, "dtype must be HOC_BFLOAT16 or HOC_FLOAT32");
  P.in = P.ld_rows = in;
  P.out = P.ld_dy = out;
  P.out_f32 = dtype == HOC_FLOAT32;
  P.accumulate = accumulate != 0;
  P.ld_y = in;
  P.status = status;
  HOC_TRY(take(who, "dy", dy, P, true, P.dy));
  HOC_TRY(take(who, "x", x, P, true, P.rows));
  HOC_TRY(take(who, "dw", dw, P, false, P.y));
  if (db) HOC_TRY(take(who, "db", db, P, false, P.pre_out));
  for (int p = 0; P.out_f32 && p < P.parts; ++p)
    if ((reinterpret_cast<uintptr_t>(P.y[p]) | reinterpret_cast<uintptr_t>(P.pre_out[p])) & 3u)
      return refuse(who, "a pointer that is not aligned to its elements");
  return run_wgrad(who, P, db, static_cast<cudaStream_t>(stream));
}

extern "C" hocResult_t hoc_linear(int rows, const void* x, size_t ldx, const void* weight, const void* bias,
                                  const void* residual, size_t ldr, int in, int out, int act, void* y, size_t ldy,
                                  void* pre, int32_t* status, void* stream) {
  const char* who = "hoc_linear";
  MmParams P{};
  HOC_TRY(dense(who, rows, in, out, status, P));
  if (!act_ok(act)) return refuse(who, "bad activation");
  if (rows == 0) return HOC_SUCCESS;
  if (ldx < size_t(in) || ldy < size_t(out) || (residual && ldr < size_t(out)) || ldx > (size_t(1) << 32) ||
      ldy > (size_t(1) << 32) || ldr > (size_t(1) << 32))
    return refuse(who, "a row stride shorter than its row, or past 2^32");
  P.act = act;
  P.ld_rows = int64_t(ldx);
  P.ld_y = int64_t(ldy);
  P.ld_res = int64_t(ldr);
  HOC_TRY(take_one(who, "x", x, P.rows));
  HOC_TRY(take_one(who, "weight", weight, P.w));
  HOC_TRY(take_one(who, "y", y, P.y));
  if (bias) HOC_TRY(take_one(who, "bias", bias, P.bias));
  if (residual) HOC_TRY(take_one(who, "residual", residual, P.res));
  if (pre) HOC_TRY(take_one(who, "pre", pre, P.pre_out));
  if (!tiles_ok(P, kForward, 2 * out)) return refuse(who, "more than 2^31 tiles");
  return run_product(who, P, kForward, static_cast<cudaStream_t>(stream));
}

extern "C" hocResult_t hoc_linear_dgrad(int rows, const void* dy, size_t lddy, const void* weight, int in, int out,
                                        int act, const void* pre, void* dx, int32_t* status, void* stream) {
  const char* who = "hoc_linear_dgrad";
  MmParams P{};
  HOC_TRY(dense(who, rows, in, out, status, P));
  if (!act_ok(act)) return refuse(who, "bad activation");
  if (rows == 0) return HOC_SUCCESS;
  if (lddy < size_t(out) || lddy > (size_t(1) << 32)) return refuse(who, "a row stride shorter than its row, or past 2^32");
  P.act = act;
  P.ld_rows = int64_t(lddy);
  P.ld_y = act == HOC_ACT_SWIGLU ? 2 * int64_t(in) : in;
  HOC_TRY(take_one(who, "dy", dy, P.rows));
  HOC_TRY(take_one(who, "weight", weight, P.w));
  HOC_TRY(take_one(who, "dx", dx, P.y));
  if (act != HOC_ACT_NONE) HOC_TRY(take_one(who, "pre", pre, P.pre));
  if (!tiles_ok(P, kDgrad, in)) return refuse(who, "more than 2^31 tiles");
  return run_product(who, P, kDgrad, static_cast<cudaStream_t>(stream));
}

extern "C" hocResult_t hoc_linear_wgrad(int rows, const void* dy, size_t lddy, const void* x, size_t ldx, int in,
                                        int out, hocDataType_t dtype, int accumulate, void* dw, void* db,
                                        int32_t* status, void* stream) {
  const char* who = "hoc_linear_wgrad";
  MmParams P{};
  HOC_TRY(dense(who, rows, in, out, status, P));
  if (dtype != HOC_BFLOAT16 && dtype != HOC_FLOAT32) return refuse(who, "dtype must be HOC_BFLOAT16 or HOC_FLOAT32");
  if (lddy < size_t(out) || ldx < size_t(in) || lddy > (size_t(1) << 32) || ldx > (size_t(1) << 32))
    return refuse(who, "a row stride shorter than its row, or past 2^32");
  P.out_f32 = dtype == HOC_FLOAT32;
  P.accumulate = accumulate != 0;
  P.ld_rows = int64_t(ldx);
  P.ld_dy = int64_t(lddy);
  P.ld_y = in;
  if (rows > 0) {
    HOC_TRY(take_one(who, "dy", dy, P.dy));
    HOC_TRY(take_one(who, "x", x, P.rows));
  }
  HOC_TRY(take_one(who, "dw", dw, P.y));
  if (db) HOC_TRY(take_one(who, "db", db, P.pre_out));
  if (P.out_f32 && ((reinterpret_cast<uintptr_t>(dw) | reinterpret_cast<uintptr_t>(db)) & 3u))
    return refuse(who, "a pointer that is not aligned to its elements");
  return run_wgrad(who, P, db ? P.pre_out : nullptr, static_cast<cudaStream_t>(stream));
}

extern "C" hocResult_t hoc_layer_trim(size_t keep) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) {
    cudaGetLastError();
    return HOC_ERR_NO_DEVICE;
  }
  if (dev >= 64) return HOC_SUCCESS;  // (no pool there)
  {
    std::lock_guard<std::mutex> hold(pool_lock);
    if (pools[dev]) e = cudaMemPoolTrimTo(pools[dev], keep);
  }
  if (e == cudaSuccess) return HOC_SUCCESS;
  cudaGetLastError();
  set_error_detail("hoc_layer_trim: the pool could not be trimmed");
  return HOC_ERR_CUDA;
}

extern "C" hocResult_t hoc_act_grad(int rows, int width, int act, const void* dy, const void* pre, void* dz,
                                    void* stream) {
  const char* who = "hoc_act_grad";
  if (rows < 0 || size_t(rows) > kMaxRows || !widths_ok(width, width) || act <= HOC_ACT_NONE || !act_ok(act))
    return refuse(who, "row count, width or activation out of range");
  if (rows == 0) return HOC_SUCCESS;
  const __nv_bfloat16 *d[1], *z[1];
  __nv_bfloat16* o[1];
  HOC_TRY(take_one(who, "dy", dy, d));
  HOC_TRY(take_one(who, "pre", pre, z));
  HOC_TRY(take_one(who, "dz", dz, o));
  const bool vec = width % 8 == 0 && ((reinterpret_cast<uintptr_t>(dy) | reinterpret_cast<uintptr_t>(pre) |
                                       reinterpret_cast<uintptr_t>(dz)) & 15u) == 0;
  const int64_t n = int64_t(rows) * (vec ? width / 8 : width);
  const int64_t each = kActThreads * (act == HOC_ACT_SWIGLU ? kGatedVecs : kPlainVecs), want = (n + each - 1) / each;
  const int grid = int(want < 1 << 20 ? want : 1 << 20);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return launched(who, launch(kActGrad[vec][act - HOC_ACT_RELU], dim3(grid), kActThreads, 0, false, s, d[0], z[0], o[0],
                              int64_t(rows), width));
}
