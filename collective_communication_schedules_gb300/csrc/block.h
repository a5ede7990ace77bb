// Shared by the operators around the dispatch (hoc_block.h): refusals, launches,
// and rows in vectors of 16 bytes or element by element.
#pragma once

#include <cstdint>
#include <cstdio>

#include <cuda_bf16.h>

#include "hoc_block.h"
#include "hoc_internal.h"

namespace hoc {
namespace block {

constexpr int kSms = 152;
constexpr unsigned kAll = 0xFFFFFFFFu;

// The kernel before this one in the stream is done, and the one after may start
// its launch.
__device__ __forceinline__ void after_the_last() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

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

// N values of T that are moved in one access.
template <class T, int N>
struct alignas(sizeof(T) * N) Vec {
  T v[N];
};

inline hocResult_t refuse(const char* who, const char* what) {
  char msg[192];
  snprintf(msg, sizeof msg, "%s: %s", who, what);
  set_error_detail(msg);
  return HOC_ERR_INVALID_ARG;
}

// What a launch returned; a failed launch's error is not left for the next call to read.
inline hocResult_t launched(const char* who, cudaError_t e) {
  if (e == cudaSuccess) return HOC_SUCCESS;
  cudaGetLastError();
  char msg[192];
  snprintf(msg, sizeof msg, "%s: launch failed: %s", who, cudaGetErrorString(e));
  set_error_detail(msg);
  return HOC_ERR_CUDA;
}

template <class... KArgs, class... Args>
cudaError_t launch(void (*kernel)(KArgs...), dim3 grid, dim3 cta, size_t smem, cudaStream_t s, Args... args) {
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = cta;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

inline bool row_dtype(int dtype) { return dtype == HOC_BFLOAT16 || dtype == HOC_FLOAT32; }
inline size_t bytes_of(int dtype) { return dtype == HOC_FLOAT32 ? 4 : 2; }
inline bool aligned(const void* p, size_t bytes) { return reinterpret_cast<uintptr_t>(p) % bytes == 0; }

// Whether rows that start at p, ld elements apart, start on 16-byte boundaries.
inline bool vector_rows(const void* p, size_t ld, size_t elem) { return aligned(p, 16) && ld * elem % 16 == 0; }

// A row operand: NULL only where it may be; its pointer on an element, its stride not
// below the width, its extent below 2^60 bytes.
inline const char* bad_rows(const void* p, size_t ld, int64_t rows, int width, size_t elem, bool optional) {
  if (!p) return optional ? nullptr : "a NULL pointer";
  if (!aligned(p, elem)) return "a pointer that is not aligned to its elements";
  if (ld < size_t(width)) return "a row stride below the width";
  if (rows > 0 && ld > (size_t(1) << 60) / elem / size_t(rows)) return "rows that lie too far apart";
  return nullptr;
}

}  // namespace block
}  // namespace hoc
