// cache_tc.cuh - what the kernels on the CTA-wide tensor instructions share:
// their parameters with the maps of the pools for TMA, waits, pairs of numbers.
#pragma once

#include <cudaTypedefs.h>

#include <cstring>

#include "cache_drafts.cuh"
#include "cache_wait.cuh"
#include "exec_pipe.cuh"
#include "tcgen05.cuh"

namespace cmdx {

PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder();  // (exec_host.cpp)

constexpr int kTcTile = 128;  // tokens

struct TcParams : DraftParams {
  CUtensorMap maps[2];  // keys, values: [page][kv head][slot][dim] (by TMA only)
  int32_t box;          // tokens of a copy: a power of two, 8 to 128
};

// The maps of a call's pools (drafts_tma_fits).
inline cudaError_t pool_maps(int dtype, const DraftParams& d, TcParams* out) {
  TcParams& p = *out;
  static_cast<DraftParams&>(p) = d;
  const auto encode = tensor_map_encoder();
  if (!encode) return cudaErrorNotSupported;
  p.box = kTcTile;
  while (p.page.d % p.box) p.box /= 2;
  for (int i = 0; i < 2; ++i) {
    const int64_t* st = i == 0 ? p.k_st : p.v_st;  // page, slot, head
    // (a stride of a dim of one element may be anything)
    const auto bytes = [&](int64_t n, int64_t stride) { return (cuuint64_t)(n > 1 ? 2 * stride : 16); };
    const cuuint64_t sizes[4] = {(cuuint64_t)p.dim, p.page.d, (cuuint64_t)p.kv_heads, (cuuint64_t)p.n_pages};
    const cuuint64_t strides[3] = {bytes(p.page.d, st[1]), bytes(p.kv_heads, st[2]), bytes(p.n_pages, st[0])};
    const cuuint32_t box[4] = {64, (cuuint32_t)p.box, 1, 1}, step[4] = {1, 1, 1, 1};
    // (bytes that L2 fetches at once: no more than lie together. Of rows of 128 bytes between other heads' 256 would be
    // half theirs.)
    const cuuint64_t run = (st[1] == p.dim ? p.page.d : 1) * (cuuint64_t)p.dim * 2;
    const CUtensorMapL2promotion fetch = run % 256 == 0   ? CU_TENSOR_MAP_L2_PROMOTION_L2_256B
                                         : run % 128 == 0 ? CU_TENSOR_MAP_L2_PROMOTION_L2_128B
                                                          : CU_TENSOR_MAP_L2_PROMOTION_NONE;
    const CUresult r = encode(
        &p.maps[i], dtype == CMD_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4,
        const_cast<void*>(i == 0 ? p.k : p.v), sizes, strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
        fetch, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) return cudaErrorInvalidValue;
  }
  return cudaSuccess;
}

// Waits of a thread (cache_wait.cuh). One that gives up sets the CTA's word before
// it does anything else. Whoever then goes on without what it waited for may tell
// others that something is there which is not, but they hear of it after the word
// was set: so a thread that finds the word clear after the last of its waits has
// had all that its results rest on. (Going on keeps warps in step at their
// barriers; who copies by TMA stops, since no barrier may be armed twice.)
__device__ __forceinline__ bool wait(uint32_t& stop, uint32_t bar, uint32_t parity) {
  return wait_until(&stop, [&] { return mbar_try_wait(bar, parity); }, [] { return global_ns(); });
}
__device__ __forceinline__ bool gave_up(const uint32_t& stop) { return *static_cast<const volatile uint32_t*>(&stop) != 0; }
// ... of a whole warp, which is told one thing.
__device__ __forceinline__ bool warp_wait(uint32_t& stop, uint32_t bar, uint32_t parity) { return __all_sync(~0u, wait(stop, bar, parity)); }
// ... for what this warp has on its way, whatever the word says.
__device__ __forceinline__ void wait_own(uint32_t& stop, uint32_t bar, uint32_t parity) {
  wait_anyway(&stop, [&] { return mbar_try_wait(bar, parity); }, [] { return global_ns(); });
  __syncwarp();
}

// What a warp needs to copy the tiles of a segment by TMA. Table entries are
// read for as many tiles at once as there are lanes (one to each box of tokens),
// and so many again ahead of the copies. (A copy takes 80 cycles to issue,
// whether by a lane each or by one lane in a loop.)
struct TmaTiles {
  const TcParams& p;
  const int lane, boxes, each, slabs;  // each: tiles to a batch of entries
  const uint32_t one;
  AttendSegment g;
  int page = 0, next = 0;              // of this lane's tile of the batch and box, and of the next batch
  uint32_t good = 0;                   // which lanes' boxes are there
  int batch = 0, sub = 0;
  // the tile at hand: its first token, which boxes are there, which of tokens
  // 32 * lane .. + 31 are (lanes 0 to 3)
  int t0 = 0;
  uint32_t taken = 0, here = 0;

  __device__ __forceinline__ TmaTiles(const TcParams& p_)
      : p(p_), lane(threadIdx.x % 32), boxes(kTcTile / p_.box), each(32 / boxes), slabs((p_.dim + 63) / 64), one(elected()) {}

  // this lane's entry of a batch; -1: it has none, and -2: it has one that is negative
  __device__ __forceinline__ int entry(int b) const {
    const int i = b * each + lane / boxes, t = (g.tile0 + i) * kTcTile + lane % boxes * p.box;
    if (i >= g.tiles || t >= g.n || t + p.box <= g.lo) return -1;
    const int e = p.tables[g.row * p.table_st[0] + fast_div32(p.page, (uint32_t)t) * p.table_st[1]];
    return e < 0 ? -2 : e;
  }
  __device__ __forceinline__ void begin(const AttendSegment& segment) {
    g = segment;
    batch = -1;
    next = entry(0);
  }
  // Tile i of the segment (in order). REPORT: entries that name no page.
  template <bool REPORT>
  __device__ __forceinline__ void look(int i) {
    sub = i & (each - 1);
    if (i - sub != batch * each) {
      page = next;
      next = entry(++batch + 1);
      if (REPORT && (page < -1 || page >= p.n_pages)) report(p.status, CMD_CACHE_BAD_PAGE);
      good = __ballot_sync(~0u, page >= 0 && page < p.n_pages);
    }
    t0 = (g.tile0 + i) * kTcTile;
    const uint32_t all = (1u << boxes) - 1u;  // (at most 16)
    taken = good >> (sub * boxes) & all;
    here = ~0u;
    if (taken != all || t0 < g.lo || t0 + kTcTile > g.n) {
      const int mine = t0 + 32 * lane, begin = max(g.lo - mine, 0), end = min(g.n - mine, 32);
      here = begin < end ? (~0u >> (32 - (end - begin))) << begin : 0u;
      for (int k = 0; k < 32; k += min(p.box, 32))
        if (lane < 4 && !(taken >> ((32 * lane + k) / p.box) & 1)) here &= ~((p.box < 32 ? (1u << p.box) - 1u : ~0u) << k);
    }
  }
  // Copies one kv head's tile into a slot, completing on the mbarrier `bar`: a
  // lane to each box and slab of 64 dims.
  __device__ __forceinline__ void copy(const CUtensorMap& map, int kv, uint32_t slot, uint32_t bar) const {
    if (one) mbar_arrive_expect_tx(bar, (uint32_t)(__popc(taken) * slabs * p.box * 128));
    __syncwarp();
    const int box = lane & (boxes - 1), t = t0 + box * p.box;
    const int from = __shfl_sync(~0u, page, sub * boxes + box), first = t - (int)(fast_div32(p.page, (uint32_t)t) * p.page.d);
    if (taken >> box & 1) {
#pragma unroll 1
      for (int slab = lane / boxes; slab < slabs; slab += 32 / boxes)  // (once, up to 128 dims)
        asm volatile("cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(
                         slot + slab * kTcTile * 128 + box * p.box * 128),
                     "l"(&map), "r"(64 * slab), "r"(first), "r"(kv), "r"(from), "r"(bar)
                     : "memory");
    }
    __syncwarp();
  }
};

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
