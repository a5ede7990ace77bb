// A CUDA runtime of two devices without a GPU, for host code that is linked against it instead of the real one: it
// keeps what the runtime's documentation leaves open open.  A copy from pageable host memory reaches the "device" (the
// heap) only when its stream is waited for; the launches are counted, and may be made to fail; an error stays the last
// one until it is read.
#include "fake_cudart.h"

#include <cstdlib>
#include <cstring>
#include <vector>

#include <cuda.h>
#include <cuda_runtime_api.h>

namespace fake {
int device = 0, launches = 0, last = 0;
unsigned widest = 0;
bool refuse = false;
static cudaError_t now(cudaError_t e) { return e == cudaSuccess ? e : cudaError_t(last = e); }
static cudaError_t launch() { return refuse ? now(cudaErrorInvalidConfiguration) : (++launches, cudaSuccess); }
struct Copy {
  void* to;
  std::vector<char> bytes;
};
static std::vector<Copy> under_way;
int copies_under_way() { return int(under_way.size()); }
static cudaError_t arrive() {
  for (auto& c : under_way) memcpy(c.to, c.bytes.data(), c.bytes.size());
  under_way.clear();
  return cudaSuccess;
}
}  // namespace fake

extern "C" {
cudaError_t cudaGetDeviceCount(int* n) { return *n = 2, cudaSuccess; }
cudaError_t cudaGetDevice(int* d) { return *d = fake::device, cudaSuccess; }
cudaError_t cudaGetLastError() {
  const cudaError_t e = cudaError_t(fake::last);
  fake::last = cudaSuccess;
  return e;
}
cudaError_t cudaMalloc(void** p, size_t n) { return (*p = calloc(1, n)) ? cudaSuccess : cudaErrorMemoryAllocation; }
cudaError_t cudaFree(void* p) {
  fake::arrive();
  free(p);
  return cudaSuccess;
}
cudaError_t cudaMemcpy(void* to, const void* from, size_t n, cudaMemcpyKind) {
  const char* c = static_cast<const char*>(from);
  fake::under_way.push_back({to, std::vector<char>(c, c + n)});
  return cudaSuccess;
}
cudaError_t cudaStreamSynchronize(cudaStream_t) { return fake::arrive(); }
cudaError_t cudaLaunchKernelExC(const cudaLaunchConfig_t* cfg, const void*, void**) {
  if (cfg->gridDim.x > fake::widest) fake::widest = cfg->gridDim.x;
  return fake::launch();
}
cudaError_t cudaFuncGetAttributes(cudaFuncAttributes*, const void*) { return cudaSuccess; }
cudaError_t cudaFuncSetAttribute(const void*, cudaFuncAttribute, int) { return cudaSuccess; }
cudaError_t cudaOccupancyMaxActiveClusters(int* n, const void*, const cudaLaunchConfig_t*) { return *n = 8, cudaSuccess; }
cudaError_t cudaDeviceGetAttribute(int* v, cudaDeviceAttr, int) { return *v = 16, cudaSuccess; }
const char* cudaGetErrorString(cudaError_t) { return "an error"; }
cudaError_t cudaMemsetAsync(void* p, int v, size_t n, cudaStream_t) { return memset(p, v, n), cudaSuccess; }
cudaError_t cudaMemPoolCreate(cudaMemPool_t* pool, const cudaMemPoolProps*) {
  static int one;
  return *pool = reinterpret_cast<cudaMemPool_t>(&one), cudaSuccess;
}
cudaError_t cudaMemPoolSetAttribute(cudaMemPool_t, cudaMemPoolAttr, void*) { return cudaSuccess; }
cudaError_t cudaMemPoolTrimTo(cudaMemPool_t, size_t) { return cudaSuccess; }
cudaError_t cudaMallocFromPoolAsync(void** p, size_t n, cudaMemPool_t, cudaStream_t) { return cudaMalloc(p, n); }
cudaError_t cudaFreeAsync(void* p, cudaStream_t) { return free(p), cudaSuccess; }
static CUresult encode(...) { return CUDA_SUCCESS; }
cudaError_t cudaGetDriverEntryPointByVersion(const char*, void** fn, unsigned, unsigned long long,
                                             cudaDriverEntryPointQueryResult* r) {
  *fn = reinterpret_cast<void*>(&encode);
  return *r = cudaDriverEntryPointSuccess, cudaSuccess;
}

// What the compiler's host code for kernels refers to.
static void* nothing[8];
void** __cudaRegisterFatBinary(void*) { return nothing; }
void __cudaRegisterFatBinaryEnd(void**) {}
void __cudaUnregisterFatBinary(void**) {}
void __cudaRegisterFunction(void**, const char*, char*, const char*, int, uint3*, uint3*, dim3*, dim3*, int*) {}
cudaError_t __cudaGetKernel(cudaKernel_t*, const void*) { return cudaSuccess; }
cudaError_t __cudaLaunchKernel(cudaKernel_t, dim3, dim3, void**, size_t, cudaStream_t) { return fake::launch(); }
unsigned __cudaPushCallConfiguration(dim3, dim3, size_t, CUstream_st*) { return 0; }
cudaError_t __cudaPopCallConfiguration(dim3*, dim3*, size_t*, void*) { return cudaSuccess; }
}
