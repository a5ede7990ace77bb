// Global gradient norm and clipping over a list of tensors (hoc_grad.h).
//
// norm = sqrt(sum g^2), then dst = min(1, max_norm / (norm + 1e-6)) * src.  Both
// passes are bound by their bytes: the first reads every element, the second
// reads it again and writes it (the coefficient needs every element, so the
// second read can only be saved where L2 still holds the data; the second pass
// therefore walks the tiles backwards, starting with those read last).  The first
// pass leaves one binary64 partial sum per CTA.  Few tiles: every CTA of the second
// pass adds the partial sums up itself, in the same order, which saves a launch.
// Many tiles: one CTA adds them up in a launch between the passes, and the second
// pass has one CTA per tile, handed out as SMs become free (32 tensors of 13.1 M
// bf16: 378 us, 6.7 TB/s of the three passes' bytes, against 405 us with a fixed share
// of the tiles per CTA).  48 tensors, 1.5 M binary32: 10.6 us for the two launches in a row of
// calls, 17 for one call from a flushed cache, bound by their latencies; the partial
// sums added by four warps or by one take the same.
#include <cstdio>
#include <new>
#include <vector>

#include <cuda_bf16.h>

#include "hoc_grad.h"
#include "hoc_internal.h"

// A tile of one tensor: the unit of work of a CTA.
struct hocTensorList {
  struct Tile {
    char* ptr;
    uint64_t n;  // elements
  };
  Tile* tiles;  // device
  size_t ntiles;
  std::vector<size_t> count;
  hocDataType_t dtype;
  int device;
};

namespace hoc {
namespace {

using Tile = hocTensorList::Tile;

constexpr int kGradThreads = 256;
constexpr int kGradUnroll = 4;          // 16-byte loads a thread has in flight
constexpr size_t kTileMost = 8192;      // elements: one set of a thread's bf16 loads
constexpr size_t kTileLeast = 2048;
constexpr int kGradCtas = 152 * 8;      // at most: partial sums in the workspace

template <class T>
__device__ __forceinline__ float widen(T v);
template <>
__device__ __forceinline__ float widen(float v) { return v; }
template <>
__device__ __forceinline__ float widen(__nv_bfloat16 v) { return __bfloat162float(v); }
template <class T>
__device__ __forceinline__ T narrow(float v);
template <>
__device__ __forceinline__ float narrow(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 narrow(float v) { return __float2bfloat16_rn(v); }

template <class T>
union Vec {
  uint4 q;
  T v[16 / sizeof(T)];
};

// Elements of a tile before its first 16-byte boundary.
template <class T>
__device__ __forceinline__ uint64_t head_of(const char* p, uint64_t n) {
  const uint64_t h = ((16u - (reinterpret_cast<uintptr_t>(p) & 15u)) & 15u) / sizeof(T);
  return h < n ? h : n;
}

template <class T>
__global__ void __launch_bounds__(kGradThreads) grad_square_kernel(const Tile* __restrict__ tiles, uint64_t ntiles,
                                                                   double* __restrict__ partial) {
  Tile next = blockIdx.x < ntiles ? tiles[blockIdx.x] : Tile{};  // (a list does not change: before the wait)
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  constexpr int V = 16 / sizeof(T);
  __shared__ double sh[kGradThreads / 32];
  double mine = 0;  // lane 0: the warp's sum.  This GPU adds few binary64 values a cycle, so that is once a tile.
  for (uint64_t t = blockIdx.x; t < ntiles; t += gridDim.x) {
    const Tile tile = next;
    if (t + gridDim.x < ntiles) next = tiles[t + gridDim.x];
    const T* p = reinterpret_cast<const T*>(tile.ptr);
    const uint64_t head = head_of<T>(tile.ptr, tile.n), nvec = (tile.n - head) / V;
    const uint64_t tail0 = head + nvec * V;
    const uint4* v = reinterpret_cast<const uint4*>(p + head);
    float s[kGradUnroll] = {};
    if (threadIdx.x < head) s[0] = widen(p[threadIdx.x]) * widen(p[threadIdx.x]);
    if (threadIdx.x < tile.n - tail0) {
      const float x = widen(p[tail0 + threadIdx.x]);
      s[1] = x * x;
    }
    for (uint64_t i = threadIdx.x; i < nvec; i += kGradThreads * kGradUnroll) {
      Vec<T> x[kGradUnroll];
#pragma unroll
      for (int u = 0; u < kGradUnroll; ++u)
        x[u].q = i + u * kGradThreads < nvec ? __ldg(v + i + u * kGradThreads) : make_uint4(0, 0, 0, 0);
#pragma unroll
      for (int u = 0; u < kGradUnroll; ++u)
#pragma unroll
        for (int e = 0; e < V; ++e) {
          const float f = widen(x[u].v[e]);
          s[u] = fmaf(f, f, s[u]);
        }
    }
    float sum = (s[0] + s[1]) + (s[2] + s[3]);
    for (int off = 16; off; off >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, off);
    if ((threadIdx.x & 31) == 0) mine += double(sum);
  }
  if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = mine;
  __syncthreads();
  if (threadIdx.x == 0) {
    double all = 0;
    for (int w = 0; w < kGradThreads / 32; ++w) all += sh[w];
    partial[blockIdx.x] = all;
  }
}

// sqrt of the partial sums' total, added up by one warp in a fixed order.
__device__ __forceinline__ float norm_of(const double* partial, int n, float* sh) {
  if (threadIdx.x < 32) {
    double v = 0;
    for (int i = threadIdx.x; i < n; i += 32) v += partial[i];
    for (int off = 16; off; off >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, off);
    if (threadIdx.x == 0) *sh = float(sqrt(v));
  }
  __syncthreads();
  return *sh;
}

__global__ void __launch_bounds__(kGradThreads) grad_norm_kernel(const double* __restrict__ partial, int n,
                                                                 float* norm) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  __shared__ float sh;
  const float v = norm_of(partial, n, &sh);
  if (threadIdx.x == 0) *norm = v;
}

// partial: the first pass's n partial sums, of which this kernel makes the norm; or
// null where norm holds it already.
template <class T>
__global__ void __launch_bounds__(kGradThreads) grad_scale_kernel(const Tile* src, const Tile* dst, uint64_t ntiles,
                                                                  const double* __restrict__ partial, int n,
                                                                  float max_norm, float* norm, int in_place) {
  Tile next{}, next_dst{};
  if (blockIdx.x < ntiles) {  // (a list does not change: before the wait)
    next = src[ntiles - 1 - blockIdx.x];
    next_dst = dst[ntiles - 1 - blockIdx.x];
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  constexpr int V = 16 / sizeof(T);
  __shared__ float sh;
  const float nv = partial ? norm_of(partial, n, &sh) : *norm;
  if (partial && blockIdx.x == 0 && threadIdx.x == 0) *norm = nv;
  float c = max_norm / (nv + 1e-6f);
  if (c > 1.f) c = 1.f;  // NaN stays
  if ((in_place && c == 1.f) || blockIdx.x >= ntiles) return;
  for (uint64_t k = blockIdx.x; k < ntiles; k += gridDim.x) {
    const Tile a = next, b = next_dst;
    if (k + gridDim.x < ntiles) {
      next = src[ntiles - 1 - (k + gridDim.x)];
      next_dst = dst[ntiles - 1 - (k + gridDim.x)];
    }
    const T* p = reinterpret_cast<const T*>(a.ptr);
    T* q = reinterpret_cast<T*>(b.ptr);
    if (((reinterpret_cast<uintptr_t>(p) ^ reinterpret_cast<uintptr_t>(q)) & 15u) != 0) {
      for (uint64_t i = threadIdx.x; i < a.n; i += kGradThreads) q[i] = narrow<T>(c * widen(p[i]));
      continue;
    }
    const uint64_t head = head_of<T>(a.ptr, a.n), nvec = (a.n - head) / V, tail0 = head + nvec * V;
    if (threadIdx.x < head) q[threadIdx.x] = narrow<T>(c * widen(p[threadIdx.x]));
    if (threadIdx.x < a.n - tail0) q[tail0 + threadIdx.x] = narrow<T>(c * widen(p[tail0 + threadIdx.x]));
    const uint4* v = reinterpret_cast<const uint4*>(p + head);
    uint4* o = reinterpret_cast<uint4*>(q + head);
    for (uint64_t i = threadIdx.x; i < nvec; i += kGradThreads * kGradUnroll) {
      Vec<T> x[kGradUnroll];
#pragma unroll
      for (int u = 0; u < kGradUnroll; ++u)
        if (i + u * kGradThreads < nvec) x[u].q = __ldcs(v + i + u * kGradThreads);
#pragma unroll
      for (int u = 0; u < kGradUnroll; ++u)
        if (i + u * kGradThreads < nvec) {
#pragma unroll
          for (int e = 0; e < V; ++e) x[u].v[e] = narrow<T>(c * widen(x[u].v[e]));
          __stcs(o + i + u * kGradThreads, x[u].q);
        }
    }
  }
}

hocResult_t refuse(const char* who, const char* what) {
  char msg[160];
  snprintf(msg, sizeof msg, "%s: %s", who, what);
  set_error_detail(msg);
  return HOC_ERR_INVALID_ARG;
}

template <class... KArgs, class... Args>
cudaError_t launch(void (*kernel)(KArgs...), int grid, cudaStream_t s, Args... args) {
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(kGradThreads);
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// What a launch returned; a failed launch's error is not left for the next call to read.
hocResult_t launched(const char* who, cudaError_t e) {
  if (e == cudaSuccess) return HOC_SUCCESS;
  cudaGetLastError();
  char msg[160];
  snprintf(msg, sizeof msg, "%s: launch failed: %s", who, cudaGetErrorString(e));
  set_error_detail(msg);
  return HOC_ERR_CUDA;
}

int grid_of(const hocTensorList* l) {
  return int(l->ntiles < 1 ? 1 : l->ntiles < size_t(kGradCtas) ? l->ntiles : size_t(kGradCtas));
}

// Whether the list was made on the current device: its table is there, and a launch would run here.
bool is_here(const hocTensorList* l) {
  int device = -1;
  return cudaGetDevice(&device) == cudaSuccess && device == l->device;
}

// Sum of squares of every tile into the workspace's partial sums.
hocResult_t squares(const char* who, const hocTensorList_t* src, const float* norm, int32_t* workspace,
                    size_t workspace_ints, cudaStream_t s) {
  if (!src || !norm || !workspace) return refuse(who, "list, norm and workspace must be given");
  if (!is_here(src)) return refuse(who, "the list belongs to another device than the current one");
  size_t need = 0;
  hoc_grad_workspace(src, &need);
  if (workspace_ints < need) return refuse(who, "workspace smaller than hoc_grad_workspace() asks for");
  if (reinterpret_cast<uintptr_t>(workspace) & 7u) return refuse(who, "workspace must be aligned to 8 bytes");
  double* partial = reinterpret_cast<double*>(workspace);
  const Tile* tiles = src->tiles;
  const uint64_t n = src->ntiles;
  const auto kernel = src->dtype == HOC_FLOAT32 ? grad_square_kernel<float> : grad_square_kernel<__nv_bfloat16>;
  return launched(who, launch(kernel, grid_of(src), s, tiles, n, partial));
}

}  // namespace

cudaError_t grad_preload() {
  const void* fns[] = {reinterpret_cast<const void*>(&grad_square_kernel<float>),
                       reinterpret_cast<const void*>(&grad_square_kernel<__nv_bfloat16>),
                       reinterpret_cast<const void*>(&grad_norm_kernel),
                       reinterpret_cast<const void*>(&grad_scale_kernel<float>),
                       reinterpret_cast<const void*>(&grad_scale_kernel<__nv_bfloat16>)};
  for (const void* f : fns) {
    cudaFuncAttributes a;
    const cudaError_t e = cudaFuncGetAttributes(&a, f);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace hoc

using namespace hoc;

extern "C" hocResult_t hoc_tensor_list_create(hocTensorList_t** list, int n, const void* const* ptr,
                                              const size_t* count, hocDataType_t dtype) {
  const char* who = "hoc_tensor_list_create";
  if (!list || n < 0 || (n > 0 && (!ptr || !count))) return refuse(who, "bad list, count or array");
  *list = nullptr;
  if (dtype != HOC_FLOAT32 && dtype != HOC_BFLOAT16) return refuse(who, "dtype must be HOC_FLOAT32 or HOC_BFLOAT16");
  const size_t b = dtype == HOC_FLOAT32 ? 4 : 2;
  size_t total = 0;
  for (int i = 0; i < n; ++i) {
    if (count[i] > (size_t(1) << 40) / b) return refuse(who, "a tensor of more than 2^40 bytes");
    if (count[i] && (!ptr[i] || reinterpret_cast<uintptr_t>(ptr[i]) % b))
      return refuse(who, "a NULL pointer, or one that is not aligned to its elements");
    total += count[i];
  }
  // Tiles of kTileMost elements, smaller in a list that has too few of them to
  // give every SM several; a rule on the counts alone, so that two lists of
  // the same counts have the same tiles.
  size_t tile = kTileMost;
  while (tile > kTileLeast && total / tile < size_t(kGradCtas)) tile /= 2;
  try {
    hocTensorList* l = new hocTensorList{};
    std::vector<Tile> tiles;
    try {
      l->count.assign(count, count + n);
      for (int i = 0; i < n; ++i)
        for (size_t at = 0; at < count[i]; at += tile)
          tiles.push_back({static_cast<char*>(const_cast<void*>(ptr[i])) + at * b,
                           count[i] - at < tile ? count[i] - at : tile});
    } catch (...) {
      delete l;
      throw;
    }
    l->dtype = dtype;
    l->ntiles = tiles.size();
    int devices = 0;
    if (cudaGetDeviceCount(&devices) != cudaSuccess || devices == 0) {
      cudaGetLastError();
      delete l;
      return HOC_ERR_NO_DEVICE;
    }
    cudaError_t e = cudaGetDevice(&l->device);
    const size_t bytes = sizeof(Tile) * (tiles.empty() ? 1 : tiles.size());
    if (e == cudaSuccess) e = cudaMalloc(&l->tiles, bytes);
    if (e == cudaSuccess && !tiles.empty())
      e = cudaMemcpy(l->tiles, tiles.data(), sizeof(Tile) * tiles.size(), cudaMemcpyHostToDevice);
    // A copy from pageable memory may return before the data is on the device, ordered with nothing
    // but the default stream; the kernels read the table on any stream, ahead of what they wait for.
    if (e == cudaSuccess) e = cudaStreamSynchronize(cudaStreamLegacy);
    if (e != cudaSuccess) {
      set_error_detail("hoc_tensor_list_create: allocating or filling the table failed");
      if (l->tiles) cudaFree(l->tiles);
      cudaGetLastError();
      delete l;
      return e == cudaErrorMemoryAllocation ? HOC_ERR_OOM : HOC_ERR_CUDA;
    }
    *list = l;
    return HOC_SUCCESS;
  } catch (const std::bad_alloc&) {
    return HOC_ERR_OOM;
  }
}

extern "C" hocResult_t hoc_tensor_list_destroy(hocTensorList_t* list) {
  if (!list) return refuse("hoc_tensor_list_destroy", "NULL list");
  const cudaError_t e = cudaFree(list->tiles);  // waits for work that still reads the table
  delete list;
  return e == cudaSuccess ? HOC_SUCCESS : HOC_ERR_CUDA;
}

extern "C" hocResult_t hoc_grad_workspace(const hocTensorList_t* list, size_t* ints) {
  if (!list || !ints) return refuse("hoc_grad_workspace", "list and ints must be given");
  *ints = size_t(grid_of(list)) * 2;
  return HOC_SUCCESS;
}

extern "C" hocResult_t hoc_grad_norm(const hocTensorList_t* src, float* norm, int32_t* workspace, size_t workspace_ints,
                                     void* stream) {
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const hocResult_t r = squares("hoc_grad_norm", src, norm, workspace, workspace_ints, s);
  if (r != HOC_SUCCESS) return r;
  return launched("hoc_grad_norm",
                  launch(grad_norm_kernel, 1, s, reinterpret_cast<const double*>(workspace), grid_of(src), norm));
}

extern "C" hocResult_t hoc_grad_clip(const hocTensorList_t* src, const hocTensorList_t* dst, const float* max_norm,
                                     float* norm, int32_t* workspace, size_t workspace_ints, void* stream) {
  const char* who = "hoc_grad_clip";
  if (!src || !dst) return refuse(who, "both lists must be given");
  if (!max_norm || !(*max_norm >= 0.f)) return refuse(who, "max_norm must be at least 0");
  if (src->dtype != dst->dtype || src->count != dst->count) return refuse(who, "the lists differ in counts or dtype");
  if (src->device != dst->device) return refuse(who, "the lists belong to different devices");
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const hocResult_t r = squares(who, src, norm, workspace, workspace_ints, s);
  if (r != HOC_SUCCESS) return r;
  const Tile *a = src->tiles, *b = dst->tiles;
  const uint64_t n = src->ntiles;
  const double* partial = reinterpret_cast<const double*>(workspace);
  const int sums = grid_of(src), same = src == dst;
  const bool few = n <= uint64_t(kGradCtas);
  cudaError_t e = few ? cudaSuccess : launch(grad_norm_kernel, 1, s, partial, sums, norm);
  if (!few) partial = nullptr;
  const int g = few ? sums : int(n < (1u << 30) ? n : (1u << 30));
  const auto kernel = src->dtype == HOC_FLOAT32 ? grad_scale_kernel<float> : grad_scale_kernel<__nv_bfloat16>;
  if (e == cudaSuccess) e = launch(kernel, g, s, a, b, n, partial, sums, *max_norm, norm, same);
  return launched(who, e);
}
