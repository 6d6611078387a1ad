// cache_common.cuh - device helpers of the cache operators' kernels.
#pragma once

#include <atomic>

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "cache_internal.h"

namespace cmdx {

// ---- launches ------------------------------------------------------------------
// As the executors' launches, these may begin while the previous kernel on
// their stream still runs (programmatic dependent launch): each CTA waits for
// it before its first access to memory, and lets the next launch start.
__device__ __forceinline__ void wait_for_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void let_next_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// (with cluster > 1: in clusters of that many CTAs)
template <class K, class... P>
inline cudaError_t launch_clusters(K kernel, int cluster, dim3 grid, int block, size_t smem, cudaStream_t stream,
                                   const P&... params) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3((unsigned)block);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)cluster;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, params...);
}
template <class K, class... P>
inline cudaError_t launch_grid(K kernel, dim3 grid, int block, size_t smem, cudaStream_t stream, const P&... params) {
  return launch_clusters(kernel, 1, grid, block, smem, stream, params...);
}
template <class K, class... P>
inline cudaError_t launch_chained(K kernel, int grid, int block, size_t smem, cudaStream_t stream, const P&... params) {
  return launch_grid(kernel, dim3((unsigned)grid), block, smem, stream, params...);
}

// Whether something was done once for a device (relaxed atomics: a race only
// repeats it). Static storage: no, before first use.
struct PerDevice {
  static constexpr int kDevices = 64;
  std::atomic<bool> done[kDevices];
};

// Lets a kernel use smem bytes of dynamic shared memory, once per device.
template <class K>
inline cudaError_t allow_smem(K kernel, int smem, PerDevice& ready) {
  int dev = 0;
  cudaGetDevice(&dev);
  const bool listed = dev >= 0 && dev < PerDevice::kDevices;
  if (listed && ready.done[dev].load(std::memory_order_relaxed)) return cudaSuccess;
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e == cudaSuccess && listed) ready.done[dev].store(true, std::memory_order_relaxed);
  return e;
}

// ---- numbers ---------------------------------------------------------------------

__device__ __forceinline__ uint32_t fast_div32(const FastDiv32& f, uint32_t n) {
  if (f.l == 0) return n;
  const uint32_t t = __umulhi(f.m, n);
  return (t + ((n - t) >> 1)) >> (f.l - 1);
}

__device__ __forceinline__ float to_float(float x) { return x; }
__device__ __forceinline__ float to_float(__half x) { return __half2float(x); }
__device__ __forceinline__ float to_float(__nv_bfloat16 x) { return __bfloat162float(x); }
template <class T>
__device__ __forceinline__ T from_float(float x);
template <>
__device__ __forceinline__ float from_float<float>(float x) { return x; }
template <>
__device__ __forceinline__ __half from_float<__half>(float x) { return __float2half_rn(x); }
template <>
__device__ __forceinline__ __nv_bfloat16 from_float<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }

__device__ __forceinline__ void report(int32_t* status, int32_t bit) {
  if (status) atomicOr(status, bit);
}

}  // namespace cmdx
