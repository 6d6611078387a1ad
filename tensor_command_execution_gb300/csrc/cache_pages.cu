// cache_pages.cu - selecting the sequences that go on (fork, free, grow), and
// compaction, of a paged cache.
//
// Both are two launches. The first works out which page goes where; its
// tables are small (one count per page, one entry per row) and its steps
// depend on one another, so it is one CTA, whose barriers are far cheaper than
// launches between steps, or for large pools one cluster of 8 CTAs. Free pages
// are ranked by an exclusive sum over the pool's counts, each thread summing a
// run of consecutive pages, then warps, CTAs and (through distributed shared
// memory) the cluster. The second launch, over the whole device, rewrites the
// tables and moves the pages: bound by memory, 16 bytes a thread and access
// with four in flight.
//
// Only integer atomics are used where threads meet, so the results do not
// depend on their order (the list of pages to copy has no order of its own:
// no page is both source and destination).
#include <cooperative_groups.h>

#include "cache_common.cuh"

namespace cg = cooperative_groups;

namespace cmdx {

namespace {

constexpr int kTeamThreads = 1024;

// head[] of the workspace
enum { kCopies = 0, kUsedBefore = 1 };

// The threads of the first launch: one CTA, or a cluster of CTAS.
template <int CTAS>
struct Team {
  static constexpr int kThreads = CTAS * kTeamThreads;
  const int me = blockIdx.x * kTeamThreads + threadIdx.x;

  // (orders global memory among the team's threads)
  __device__ __forceinline__ void sync() const {
    if constexpr (CTAS == 1) __syncthreads();
    else cg::this_cluster().sync();
  }

  // The sum of x over the threads before this one, and over all in *all.
  // Every thread of the team calls it.
  __device__ __forceinline__ int before(int x, int* all) const {
    __shared__ int s_warp[kTeamThreads / 32];
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
    sync();
    int sum = incl - x + (warp ? s_warp[warp - 1] : 0);
    if constexpr (CTAS == 1) {
      *all = s_cta;
    } else {
      int total = 0;
#pragma unroll
      for (int c = 0; c < CTAS; ++c) {
        const int v = *cg::this_cluster().map_shared_rank(&s_cta, c);
        if (c < (int)blockIdx.x) sum += v;
        total += v;
      }
      *all = total;
    }
    sync();  // nobody's sums are overwritten, or gone, while another reads them
    return sum;
  }
};

// Pages of n tokens (n and a page's size are below 2^31).
__device__ __forceinline__ int pages_of(int n, const FastDiv32& page) {
  return (int)fast_div32(page, (uint32_t)n + page.d - 1);
}

// The items [0, n) that have a property, ranked: warps take runs of items, 32
// at a time, so that reads are whole lines and a ballot does the counting.
template <int CTAS>
struct Ranks {
  int from, to, start;  // this warp's run (from is a multiple of 32), and how many before it have the property

  // (every thread of the team calls it; *all: how many have it)
  template <class F>
  __device__ __forceinline__ Ranks(const Team<CTAS>& team, int n, F has, int* all) {
    const int lane = threadIdx.x & 31;
    const int run = (n + Team<CTAS>::kThreads - 1) / Team<CTAS>::kThreads * 32;
    from = (int)min((int64_t)(team.me >> 5) * run, (int64_t)n);
    to = (int)min((int64_t)from + run, (int64_t)n);
    int mine = 0;
#pragma unroll 8
    for (int i = from + lane; i < to; i += 32) mine += has(i);
    const int before = team.before(mine, all);
    start = __shfl_sync(~0u, before, 0);
  }
  // Calls f(item, has it, how many before it have it) on this warp's items.
  template <class F, class G>
  __device__ __forceinline__ void each(F has, G f) const {
    const int lane = threadIdx.x & 31;
    int rank = start;
#pragma unroll 4
    for (int i = from; i < to; i += 32) {
      const bool h = i + lane < to && has(i + lane);
      const uint32_t b = __ballot_sync(~0u, h);
      if (i + lane < to) f(i + lane, h, rank + __popc(b & ((1u << lane) - 1u)));
      rank += __popc(b);
    }
  }
};

// One old row's length, held to its table.
__device__ __forceinline__ int row_length(const SelectParams& p, int row) {
  const int64_t most = (int64_t)p.columns * p.page.d;
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
  const int old = pages_of(n, p.page);
  const int64_t length = (int64_t)n + grow;
  r.fits = length <= (int64_t)p.columns * p.page.d;
  r.length = r.fits ? (int)length : 0;
  r.all = r.fits ? pages_of(r.length, p.page) : p.columns + 1;
  r.split = with_first && r.parent >= 0 && n != old * (int)p.page.d && p.first[r.parent] != i;
  r.keep = old - (r.split ? 1 : 0);
  return r;
}

template <int CTAS>
__device__ __forceinline__ void select_plan(const SelectParams& p) {
  using All = Team<CTAS>;
  const All team;
  const int me = team.me;
  pdl_wait();
  pdl_trigger();
  // counts start from refs, families empty
  for (int i = me; i < p.pages; i += All::kThreads) p.refs_out[i] = p.refs[i];
  for (int i = me; i < p.old_rows; i += All::kThreads) {
    p.first[i] = 0x7fffffff;
    p.children[i] = 0;
  }
  if (me == 0) p.head[kCopies] = 0;
  team.sync();
  for (int i = me; i < p.new_rows; i += All::kThreads) {
    const Plan r = plan_row(p, i, false);
    if (r.parent >= 0 && r.fits) atomicMin(&p.first[r.parent], i);
  }
  team.sync();
  // pages each new row needs, summed in row order; children that fit
  const int run = (p.new_rows + All::kThreads - 1) / All::kThreads;
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
  int base = team.before(need, &all_need);
  for (int i = i0; i < i1; ++i) {
    const Plan r = plan_row(p, i);
    p.base[i] = r.fits ? base : -1;
    if (r.fits) base += r.all - r.keep;
  }
  team.sync();  // (children complete, base of every row written)
  // counts: each page of an old row changes hands from one row to its
  // children; the page in progress to the first child alone. A warp per row.
  const int lane = threadIdx.x & 31;
  for (int r = me >> 5; r < p.old_rows; r += All::kThreads / 32) {
    const int n = row_length(p, r), old = pages_of(n, p.page), kids = p.children[r];
    const bool partial = n != old * (int)p.page.d;
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
  team.sync();
  // the free pages in ascending order
  int all_free;
  const auto is_free = [&](int i) { return __ldcg(&p.refs_out[i]) == 0; };
  const Ranks<CTAS> ranks(team, p.pages, is_free, &all_free);
  ranks.each(is_free, [&](int i, bool f, int rank) {
    if (f) p.free_list[rank] = i;
  });
  team.sync();
  // which rows the pool has room for, and the pages to copy
  for (int i = me; i < p.new_rows; i += All::kThreads) {
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
}

// Moves the pages: pair k goes from src[k] to dst[k] in every pool.
template <class U, class L>
__device__ __forceinline__ void move_pages(const L& pools, const int32_t* src, const int32_t* dst, int pairs) {
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

template <class U, class L>
__global__ void __launch_bounds__(kMoveThreads) select_apply_kernel(const __grid_constant__ SelectParams p, const __grid_constant__ L pools) {
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31, warps = gridDim.x * (kMoveThreads / 32);
  for (int i = blockIdx.x * (kMoveThreads / 32) + (threadIdx.x >> 5); i < p.new_rows; i += warps) {
    const int base = p.base[i], keep = p.keep[i], parent = p.parents[i];
    const int all = base >= 0 ? pages_of(p.lengths_out[i], p.page) : 0;
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
  move_pages<U, L>(pools, p.copy_src, p.copy_dst, p.head[kCopies]);
}

template <int CTAS>
__device__ __forceinline__ void compact_plan(const CompactParams& p) {
  const Team<CTAS> team;
  const int me = team.me;
  pdl_wait();
  pdl_trigger();
  int n;
  const auto is_used = [&](int i) { return p.refs[i] > 0; };
  const Ranks<CTAS> ranks(team, p.pages, is_used, &n);
  // the free pages before index n take the used pages from n on, in turn: the
  // first of these has rank `kept`
  ranks.each(is_used, [&](int i, bool u, int rank) {
    if (i == n || (i == n - 1 && n == p.pages)) {
      const int kept = rank + (i == n - 1 && u);
      p.head[kUsedBefore] = kept;
      p.head[kCopies] = n - kept;
    }
    if (!u && i < n) p.holes[i - rank] = i;
  });
  if (me == 0 && n == 0) p.head[kCopies] = 0;
  team.sync();
  const int kept = n ? __ldcg(&p.head[kUsedBefore]) : 0;
  ranks.each(is_used, [&](int i, bool u, int rank) {
    int where = u ? i : -1;
    if (u && i >= n) {
      where = __ldcg(&p.holes[rank - kept]);
      p.movers[rank - kept] = i;
      p.refs_out[where] = p.refs[i];
    }
    p.map_out[i] = where;
    if (i >= n) p.refs_out[i] = 0;
    else if (u) p.refs_out[i] = p.refs[i];
  });
}

template <class U, class L>
__global__ void __launch_bounds__(kMoveThreads) compact_apply_kernel(const __grid_constant__ CompactParams p, const __grid_constant__ L pools) {
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31, warps = gridDim.x * (kMoveThreads / 32);
  for (int i = blockIdx.x * (kMoveThreads / 32) + (threadIdx.x >> 5); i < p.rows; i += warps) {
    int64_t n = p.lengths[i];
    const int64_t most = (int64_t)p.columns * p.page.d;
    if (n < 0 || n > most) {
      if (lane == 0) report(p.status, CMD_CACHE_BAD_INDEX);
      n = n < 0 ? 0 : most;
    }
    const int all = pages_of((int)n, p.page);
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
  move_pages<U, L>(pools, p.movers, p.holes, p.head[kCopies]);
}

__global__ void __launch_bounds__(kTeamThreads) select_plan_one(const __grid_constant__ SelectParams p) { select_plan<1>(p); }
__global__ void __cluster_dims__(8, 1, 1) __launch_bounds__(kTeamThreads)
    select_plan_cluster(const __grid_constant__ SelectParams p) {
  select_plan<8>(p);
}
__global__ void __launch_bounds__(kTeamThreads) compact_plan_one(const __grid_constant__ CompactParams p) { compact_plan<1>(p); }
__global__ void __cluster_dims__(8, 1, 1) __launch_bounds__(kTeamThreads)
    compact_plan_cluster(const __grid_constant__ CompactParams p) {
  compact_plan<8>(p);
}

// Pages or rows above which the first launch is a cluster.
constexpr int kLargePool = 2048, kManyRows = 256;

template <class P, class L>
cudaError_t run(void (*plan)(P), int ctas, void (*apply)(P, L), const P& p, const PoolList& pools, cudaStream_t stream) {
  cudaError_t e = launch_pdl(plan, ctas, kTeamThreads, 0, stream, p);
  if (e != cudaSuccess) return e;
  L l;
  constexpr int most = sizeof l.ptr / sizeof l.ptr[0];
  for (int i = 0; i < most; ++i) {
    l.ptr[i] = pools.ptr[i];
    l.stride[i] = pools.stride[i];
    l.bytes[i] = pools.bytes[i];
  }
  l.n = pools.n;
  l.unit = pools.unit;
  return launch_pdl(apply, 152 * 8, kMoveThreads, 0, stream, p, l);
}

// calls f with a value of the pools' access type, and an empty list that holds them
template <class F>
cudaError_t by_unit(const PoolList& pools, F f) {
  auto sized = [&](auto u) { return pools.n <= 8 ? f(u, PoolListOf<8>{}) : f(u, PoolList{}); };
  switch (pools.unit) {
    case 16: return sized(uint4{});
    case 8: return sized(uint2{});
    case 4: return sized(uint32_t{});
    case 2: return sized(uint16_t{});
  }
  return sized(uint8_t{});
}

}  // namespace

cudaError_t select_launch(const SelectParams& p, const PoolList& pools, cudaStream_t stream) {
  const bool large = p.pages > kLargePool || p.new_rows > kManyRows || p.old_rows > kManyRows;
  return by_unit(pools, [&](auto u, auto l) {
    return run(large ? select_plan_cluster : select_plan_one, large ? 8 : 1, select_apply_kernel<decltype(u), decltype(l)>, p,
               pools, stream);
  });
}

cudaError_t compact_launch(const CompactParams& p, const PoolList& pools, cudaStream_t stream) {
  const bool large = p.pages > kLargePool;
  return by_unit(pools, [&](auto u, auto l) {
    return run(large ? compact_plan_cluster : compact_plan_one, large ? 8 : 1, compact_apply_kernel<decltype(u), decltype(l)>,
               p, pools, stream);
  });
}

}  // namespace cmdx
