// cache_pages.cu - selecting the sequences that go on (fork, free, grow), and
// compaction, of a paged cache.
//
// Both are two launches. The first works out which page goes where, on one
// cluster of 8 CTAs: its tables are small (one count per page, one entry per
// row), its steps depend on one another, and a cluster's barrier is far
// cheaper than a launch between steps. Free pages are ranked by an exclusive
// sum over the pool's counts, each thread summing a run of consecutive pages,
// then warps, CTAs and (through distributed shared memory) the cluster. The
// second launch, over the whole device, rewrites the tables and moves the
// pages: bound by memory, 16 bytes a thread and access with four in flight.
//
// Only integer atomics are used where threads meet, so the results do not
// depend on their order (the list of pages to copy has no order of its own:
// no page is both source and destination).
#include <cooperative_groups.h>

#include "cache_common.cuh"

namespace cg = cooperative_groups;

namespace cmdx {

namespace {

constexpr int kMetaCtas = 8;
constexpr int kMetaThreads = 1024;
constexpr int kMetaAll = kMetaCtas * kMetaThreads;

// head[] of the workspace
enum { kCopies = 0, kFree = 1, kUsedBefore = 2 };

// Sum over the cluster of each thread's x: returns the sum over the threads
// before this one (CTA-major order), and the total in *all. Every thread of
// the cluster calls it.
__device__ __forceinline__ int cluster_before(cg::cluster_group& cluster, int x, int* all) {
  __shared__ int s_warp[kMetaThreads / 32];
  __shared__ int s_cta;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int incl = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(~0u, incl, o);
    if (lane >= o) incl += y;
  }
  if (lane == 31) s_warp[warp] = incl;
  __syncthreads();
  if (warp == 0) {
    int w = s_warp[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(~0u, w, o);
      if (lane >= o) w += y;
    }
    s_warp[lane] = w;
    if (lane == 31) s_cta = w;
  }
  cluster.sync();
  int before = incl - x + (warp ? s_warp[warp - 1] : 0), total = 0;
#pragma unroll
  for (int c = 0; c < kMetaCtas; ++c) {
    const int v = *cluster.map_shared_rank(&s_cta, c);
    if (c < (int)cluster.block_rank()) before += v;
    total += v;
  }
  cluster.sync();  // nobody's sums are overwritten, or gone, while another reads them
  *all = total;
  return before;
}

__device__ __forceinline__ int pages_of(int n, int page_size) { return (int)(((int64_t)n + page_size - 1) / page_size); }

// One old row's length, held to its table.
__device__ __forceinline__ int row_length(const SelectParams& p, int row) {
  const int64_t most = (int64_t)p.columns * p.page_size;
  int64_t n = p.lengths[row];
  if (n < 0 || n > most) {
    report(p.status, CMD_CACHE_BAD_INDEX);
    n = n < 0 ? 0 : most;
  }
  return (int)n;
}

// What becomes of new row i: its parent (-1: none), its length, the pages it
// shares and the pages it has in all. A row that its table is too short for
// has all = columns + 1. first[] is read unless the caller is filling it.
struct Plan {
  int parent, length, keep, all;
  bool split, fits;
};
__device__ __forceinline__ Plan plan_row(const SelectParams& p, int i, bool with_first = true) {
  Plan r;
  r.parent = p.parents[i];
  int grow = p.grow ? p.grow[i] : 0;
  if (r.parent < -1 || r.parent >= p.old_rows || grow < 0) {
    if (with_first) report(p.status, CMD_CACHE_BAD_INDEX);
    if (grow < 0) grow = 0;
    if (r.parent >= p.old_rows) r.parent = -1;
    if (r.parent < -1) r.parent = -1;
  }
  const int n = r.parent >= 0 ? row_length(p, r.parent) : 0;
  const int old = pages_of(n, p.page_size);
  const int64_t length = (int64_t)n + grow;
  const int64_t all = (length + p.page_size - 1) / p.page_size;
  r.fits = all <= p.columns;
  r.all = r.fits ? (int)all : p.columns + 1;
  r.length = r.fits ? (int)length : 0;
  r.split = with_first && r.parent >= 0 && n % p.page_size != 0 && p.first[r.parent] != i;
  r.keep = old - (r.split ? 1 : 0);
  return r;
}

__global__ void __cluster_dims__(kMetaCtas, 1, 1) __launch_bounds__(kMetaThreads)
    select_plan_kernel(const __grid_constant__ SelectParams p) {
  cg::cluster_group cluster = cg::this_cluster();
  const int me = blockIdx.x * kMetaThreads + threadIdx.x;
  pdl_wait();
  // counts start from refs, families empty
  for (int i = me; i < p.pages; i += kMetaAll) p.refs_out[i] = p.refs[i];
  for (int i = me; i < p.old_rows; i += kMetaAll) {
    p.first[i] = 0x7fffffff;
    p.children[i] = 0;
  }
  if (me == 0) p.head[kCopies] = 0;
  cluster.sync();
  for (int i = me; i < p.new_rows; i += kMetaAll) {
    const Plan r = plan_row(p, i, false);
    if (r.parent >= 0 && r.fits) atomicMin(&p.first[r.parent], i);
  }
  cluster.sync();
  // pages each new row needs, summed in row order; children that fit
  const int run = (p.new_rows + kMetaAll - 1) / kMetaAll;
  const int i0 = min(me * run, p.new_rows), i1 = min(i0 + run, p.new_rows);
  int need = 0, all_need;
  for (int i = i0; i < i1; ++i) {
    const Plan r = plan_row(p, i);
    p.keep[i] = r.keep;
    if (!r.fits) {
      report(p.status, CMD_CACHE_FULL_TABLE);
      continue;
    }
    need += r.all - r.keep;
    if (r.parent >= 0) atomicAdd(&p.children[r.parent], 1);
  }
  int base = cluster_before(cluster, need, &all_need);
  for (int i = i0; i < i1; ++i) {
    const Plan r = plan_row(p, i);
    p.base[i] = r.fits ? base : -1;
    if (r.fits) base += r.all - r.keep;
  }
  cluster.sync();  // (children complete, base of every row written)
  // counts: each page of an old row changes hands from one row to its
  // children; the page in progress to the first child alone. A warp per row.
  const int lane = threadIdx.x & 31;
  for (int r = me >> 5; r < p.old_rows; r += kMetaAll / 32) {
    const int n = row_length(p, r), old = pages_of(n, p.page_size), kids = p.children[r];
    const bool partial = n % p.page_size != 0;
    const int last = partial ? (kids ? 1 : 0) : kids;
    if (kids == 1 && last == 1) continue;
    for (int j = lane; j < old; j += 32) {
      const int page = p.tables[r * p.table_st + j];
      if (page < 0 || page >= p.pages) {
        report(p.status, CMD_CACHE_BAD_PAGE);
        continue;
      }
      const int change = (j == old - 1 ? last : kids) - 1;
      if (change) atomicAdd(&p.refs_out[page], change);
    }
  }
  cluster.sync();
  // the free pages in ascending order
  const int prun = (p.pages + kMetaAll - 1) / kMetaAll;
  const int p0 = min(me * prun, p.pages), p1 = min(p0 + prun, p.pages);
  int free = 0, all_free;
  for (int i = p0; i < p1; ++i) free += __ldcg(&p.refs_out[i]) == 0;
  int rank = cluster_before(cluster, free, &all_free);
  for (int i = p0; i < p1; ++i)
    if (__ldcg(&p.refs_out[i]) == 0) p.free_list[rank++] = i;
  cluster.sync();
  // which rows the pool has room for, and the pages to copy
  for (int i = me; i < p.new_rows; i += kMetaAll) {
    const Plan r = plan_row(p, i);
    int at = p.base[i];
    const int wants = r.all - r.keep;
    if (at >= 0 && wants > 0 && (int64_t)at + wants > all_free) {
      report(p.status, CMD_CACHE_NO_PAGES);
      at = p.base[i] = -2;  // dropped, although its shared pages were counted
    }
    p.lengths_out[i] = at >= 0 ? r.length : 0;
    if (at >= 0 && r.split) {
      const int src = p.tables[r.parent * p.table_st + r.keep];
      if (src >= 0 && src < p.pages) {
        const int c = atomicAdd(&p.head[kCopies], 1);
        p.copy_src[c] = src;
        p.copy_dst[c] = __ldcg(&p.free_list[at]);
      }
    }
  }
  pdl_trigger();
}

// Moves the pages: pair k goes from src[k] to dst[k] in every pool.
template <class U>
__device__ __forceinline__ void move_pages(const PoolList& pools, const int32_t* src, const int32_t* dst, int pairs) {
  constexpr int kEach = 4;
  const int64_t span = (int64_t)blockDim.x * kEach * sizeof(U);
  for (int k = 0; k < pools.n; ++k) {
    const int64_t bytes = pools.bytes[k], stride = pools.stride[k];
    const int pieces = (int)((bytes + span - 1) / span);
    const int64_t items = (int64_t)pairs * pieces;
    for (int64_t it = blockIdx.x; it < items; it += gridDim.x) {
      const int pair = (int)(it / pieces);
      const int64_t at = (it - (int64_t)pair * pieces) * span;
      const U* from = reinterpret_cast<const U*>(pools.ptr[k] + src[pair] * stride + at);
      U* to = reinterpret_cast<U*>(pools.ptr[k] + dst[pair] * stride + at);
      const int64_t n = (bytes - at) / (int64_t)sizeof(U);
      U x[kEach];
#pragma unroll
      for (int j = 0; j < kEach; ++j) {
        const int64_t e = j * (int64_t)blockDim.x + threadIdx.x;
        if (e < n) x[j] = from[e];
      }
#pragma unroll
      for (int j = 0; j < kEach; ++j) {
        const int64_t e = j * (int64_t)blockDim.x + threadIdx.x;
        if (e < n) to[e] = x[j];
      }
    }
  }
}

constexpr int kMoveThreads = 256;

template <class U>
__global__ void __launch_bounds__(kMoveThreads) select_apply_kernel(const __grid_constant__ SelectParams p,
                                                                    const __grid_constant__ PoolList pools) {
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31, warps = gridDim.x * (kMoveThreads / 32);
  for (int i = blockIdx.x * (kMoveThreads / 32) + (threadIdx.x >> 5); i < p.new_rows; i += warps) {
    const int base = p.base[i], keep = p.keep[i], parent = p.parents[i];
    const int all = base >= 0 ? pages_of(p.lengths_out[i], p.page_size) : 0;
    for (int j = lane; j < p.columns; j += 32) {
      int page = -1;
      if (j < all) {
        if (j < keep) {
          page = p.tables[parent * p.table_st + j];
        } else {
          page = p.free_list[base + j - keep];
          p.refs_out[page] = 1;
        }
      }
      p.tables_out[i * p.table_out_st + j] = page;
    }
    if (base == -2 && parent >= 0 && parent < p.old_rows)  // the pages it would have shared
      for (int j = lane; j < keep; j += 32) {
        const int page = p.tables[parent * p.table_st + j];
        if (page >= 0 && page < p.pages) atomicSub(&p.refs_out[page], 1);
      }
  }
  move_pages<U>(pools, p.copy_src, p.copy_dst, p.head[kCopies]);
}

__global__ void __cluster_dims__(kMetaCtas, 1, 1) __launch_bounds__(kMetaThreads)
    compact_plan_kernel(const __grid_constant__ CompactParams p) {
  cg::cluster_group cluster = cg::this_cluster();
  const int me = blockIdx.x * kMetaThreads + threadIdx.x;
  pdl_wait();
  const int run = (p.pages + kMetaAll - 1) / kMetaAll;
  const int i0 = min(me * run, p.pages), i1 = min(i0 + run, p.pages);
  int used = 0, n;
  for (int i = i0; i < i1; ++i) used += p.refs[i] > 0;
  const int before = cluster_before(cluster, used, &n);
  // used pages before index n: the thread whose run holds n says
  if (i0 <= n && n < i1) {
    int c = before;
    for (int i = i0; i < n; ++i) c += p.refs[i] > 0;
    p.head[kUsedBefore] = c;
    p.head[kCopies] = n - c;
  } else if (me == 0 && n == p.pages) {
    p.head[kUsedBefore] = n;
    p.head[kCopies] = 0;
  }
  cluster.sync();
  const int used_before = __ldcg(&p.head[kUsedBefore]);
  int rank = before;
  for (int i = i0; i < i1; ++i) {
    const bool u = p.refs[i] > 0;
    if (u && i >= n) p.movers[rank - used_before] = i;
    if (!u && i < n) p.holes[i - rank] = i;
    rank += u;
  }
  cluster.sync();
  rank = before;
  for (int i = i0; i < i1; ++i) {
    const int r = p.refs[i];
    const bool u = r > 0;
    p.map_out[i] = !u ? -1 : i < n ? i : __ldcg(&p.holes[rank - used_before]);
    p.refs_out[i] = i >= n ? 0 : u ? r : p.refs[__ldcg(&p.movers[i - rank])];
    rank += u;
  }
  pdl_trigger();
}

template <class U>
__global__ void __launch_bounds__(kMoveThreads) compact_apply_kernel(const __grid_constant__ CompactParams p,
                                                                     const __grid_constant__ PoolList pools) {
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31, warps = gridDim.x * (kMoveThreads / 32);
  for (int i = blockIdx.x * (kMoveThreads / 32) + (threadIdx.x >> 5); i < p.rows; i += warps) {
    int64_t n = p.lengths[i];
    const int64_t most = (int64_t)p.columns * p.page_size;
    if (n < 0 || n > most) {
      if (lane == 0) report(p.status, CMD_CACHE_BAD_INDEX);
      n = n < 0 ? 0 : most;
    }
    const int all = pages_of((int)n, p.page_size);
    for (int j = lane; j < p.columns; j += 32) {
      int page = -1;
      if (j < all) {
        const int old = p.tables[i * p.table_st + j];
        if (old >= 0 && old < p.pages) page = p.map_out[old];
        if (page < 0) report(p.status, CMD_CACHE_BAD_PAGE);
      }
      p.tables_out[i * p.table_out_st + j] = page;
    }
  }
  move_pages<U>(pools, p.movers, p.holes, p.head[kCopies]);
}

template <class P>
cudaError_t run(void (*plan)(P), void (*apply)(P, PoolList), const P& p, const PoolList& pools, cudaStream_t stream) {
  cudaError_t e = launch_pdl(plan, kMetaCtas, kMetaThreads, 0, stream, p);
  if (e != cudaSuccess) return e;
  return launch_pdl(apply, 152 * 8, kMoveThreads, 0, stream, p, pools);
}

// calls f with a value of the pools' access type
template <class F>
cudaError_t by_unit(int unit, F f) {
  switch (unit) {
    case 16: return f(uint4{});
    case 8: return f(uint2{});
    case 4: return f(uint32_t{});
    case 2: return f(uint16_t{});
  }
  return f(uint8_t{});
}

}  // namespace

cudaError_t select_launch(const SelectParams& p, const PoolList& pools, cudaStream_t stream) {
  return by_unit(pools.unit, [&](auto u) { return run(select_plan_kernel, select_apply_kernel<decltype(u)>, p, pools, stream); });
}

cudaError_t compact_launch(const CompactParams& p, const PoolList& pools, cudaStream_t stream) {
  return by_unit(pools.unit,
                 [&](auto u) { return run(compact_plan_kernel, compact_apply_kernel<decltype(u)>, p, pools, stream); });
}

}  // namespace cmdx
