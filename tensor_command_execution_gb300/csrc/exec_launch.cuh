// exec_launch.cuh - how this library's kernels are launched: programmatic
// dependent launch, per-device caches of host-side values, and the grid size
// of persistent kernels.
#pragma once

#include <atomic>
#include <cstdint>

#include <cuda_runtime.h>

namespace cmdx {

// ---- programmatic dependent launch ------------------------------------------
// Every executor launch may begin while the previous kernel on its stream is
// still running: its CTAs are scheduled early, and each one first waits
// (griddepcontrol.wait) until that kernel has completed and its memory is
// visible, so no data access overlaps it and a Command that reads what the
// previous one wrote stays correct. Each CTA then lets the next launch start
// (griddepcontrol.launch_dependents). What overlaps is launch processing and
// CTA scheduling, which dominate small launches. Without the launch
// attribute both instructions are no-ops.
__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void pdl_trigger() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

template <class K, class... P>
inline cudaError_t launch_pdl(K kernel, int grid, int block, size_t smem, cudaStream_t stream, const P&... params) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3((unsigned)block);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, params...);
}

// A value computed once per device by host code (a grid size, a flag that a
// kernel attribute is set), read and written from any host thread: relaxed
// atomics suffice, since every thread that computes it computes the same
// value and a race only repeats the computation. Zero means "not yet"; a
// device index outside the table is never cached.
struct DeviceCache {
  static constexpr int kDevices = 64;
  std::atomic<int> v[kDevices];
  int get(int dev) const { return dev >= 0 && dev < kDevices ? v[dev].load(std::memory_order_relaxed) : 0; }
  void put(int dev, int x) {
    if (dev >= 0 && dev < kDevices) v[dev].store(x, std::memory_order_relaxed);
  }
};

// Lets a kernel use smem bytes of dynamic shared memory, once per device.
template <class K>
inline cudaError_t allow_smem(K kernel, int smem, DeviceCache& ready) {
  int dev = 0;
  cudaGetDevice(&dev);
  if (ready.get(dev)) return cudaSuccess;
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e == cudaSuccess) ready.put(dev, 1);
  return e;
}

// Grid size for a persistent grid-stride kernel: enough CTAs to fill the
// device at the kernel's occupancy, and no more than the work needs.
template <class K>
inline int persistent_grid(K kernel, int block, size_t smem, int64_t work_blocks) {
  int dev = 0, sms = 0, per_sm = 0;
  cudaGetDevice(&dev);
  cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kernel, block, smem);
  if (per_sm < 1) per_sm = 1;
  if (sms < 1) sms = 1;
  int64_t g = (int64_t)sms * per_sm;
  if (work_blocks < g) g = work_blocks;
  return g < 1 ? 1 : (int)g;
}

}  // namespace cmdx
