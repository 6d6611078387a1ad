// cache_tc.cuh - what the kernels on the CTA-wide tensor instructions share:
// their parameters with the maps of the pools for TMA, waits, pairs of numbers.
#pragma once

#include <cudaTypedefs.h>

#include <cstring>

#include "cache_drafts.cuh"
#include "exec_pipe.cuh"
#include "tcgen05.cuh"

namespace cmdx {

PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder();  // (exec_host.cpp)

constexpr int kTcTile = 128;                // tokens
constexpr uint64_t kPatience = 2000000000;  // ns: no wait takes longer

struct TcParams : DraftParams {
  CUtensorMap maps[2];  // keys, values: [page][kv head][slot][dim] (by TMA only)
  int32_t box;          // tokens of a copy: a power of two, 8 to 128
};

// The maps of a call's pools (drafts_tma_fits).
inline cudaError_t pool_maps(int dtype, const DraftParams& d, TcParams* out) {
  TcParams& p = *out;
  static_cast<DraftParams&>(p) = d;
  p.box = kTcTile;
  while (p.page.d % p.box) p.box /= 2;
  for (int i = 0; i < 2; ++i) {
    const int64_t* st = i == 0 ? p.k_st : p.v_st;  // page, slot, head
    // (a stride of a dim of one element may be anything)
    const auto bytes = [&](int64_t n, int64_t stride) { return (cuuint64_t)(n > 1 ? 2 * stride : 16); };
    const cuuint64_t sizes[4] = {(cuuint64_t)p.dim, p.page.d, (cuuint64_t)p.kv_heads, (cuuint64_t)p.n_pages};
    const cuuint64_t strides[3] = {bytes(p.page.d, st[1]), bytes(p.kv_heads, st[2]), bytes(p.n_pages, st[0])};
    const cuuint32_t box[4] = {64, (cuuint32_t)p.box, 1, 1}, step[4] = {1, 1, 1, 1};
    const CUresult r = tensor_map_encoder()(
        &p.maps[i], dtype == CMD_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4,
        const_cast<void*>(i == 0 ? p.k : p.v), sizes, strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
        CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) return cudaErrorInvalidValue;
  }
  return cudaSuccess;
}

// A wait that gives up (for the whole CTA, whose word it sets) after kPatience. (The clock is read
// now and then only: a read takes about as long as a wait should.)
__device__ __forceinline__ void wait(uint32_t& stop_word, uint32_t bar, uint32_t parity) {
  volatile uint32_t* stop = &stop_word;
  uint64_t t0 = 0;
  for (uint32_t n = 1; !mbar_try_wait(bar, parity); ++n) {
    if (n % 256) continue;
    if (*stop) return;
    const uint64_t now = global_ns();
    if (t0 == 0) t0 = now;
    if (now - t0 > kPatience) {
      *stop = 1;
      return;
    }
  }
}

// ---- pairs of binary32 numbers in one instruction --------------------------------
__device__ __forceinline__ uint64_t pair(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float2 unpair(uint64_t x) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(x));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
}  // namespace cmdx
