// cache_pages.cu - selecting the sequences that go on (fork, free, grow), and
// compaction, of a paged cache.
//
// Both are two launches. The first works out which page goes where; its
// tables are small (one count per page, one entry per row) and its steps
// depend on one another, so it is one CTA, whose barriers are far cheaper than
// launches between steps, or for large pools one cluster of 8 CTAs. Free pages
// are ranked by an exclusive sum over the pool's counts: ballots within a
// warp's run of pages, then warps, CTAs and (through distributed shared
// memory) the cluster. The second launch, over the whole device, rewrites the
// tables and moves the pages: bound by memory, 16 bytes a thread and access
// with four in flight.
//
// Measured: compaction moving 1703 pages of 4 x 64 KB among 7001, 143.2 us,
// 6.24 TB/s, 92% of the copy peak (the moves alone 6.75 TB/s), and 437 pages of
// 64 x 64 KB, 563 us, 96%; selection of 509 rows among 6300 pages, 200 of 4 x 128
// KB copied, 41.7 us, 75% (13 us of it the plan, bound by the latency of its
// steps); 64 beams 8.6 us, 601 pages' compaction 5.7 us, both fixed parts. Pools
// are gone over one after another: 64 beams on 64 pools of a few copies each take
// 72.7 us.
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
  const int me = (CTAS == 1 ? 0 : (int)blockIdx.x * kTeamThreads) + threadIdx.x;

  // (orders global memory among the team's threads)
  __device__ __forceinline__ void sync() const {
    if constexpr (CTAS == 1) __syncthreads();
    else cg::this_cluster().sync();
  }

  // The sum of x over the threads before this one, and over all in *all.
  // Every thread of the team calls it.
  template <class N>
  __device__ __forceinline__ N before(N x, N* all) const {
    __shared__ N s_warp[kTeamThreads / 32];
    __shared__ N s_cta;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    N incl = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const N y = __shfl_up_sync(~0u, incl, o);
      if (lane >= o) incl += y;
    }
    if (lane == 31) s_warp[warp] = incl;
    __syncthreads();
    if (warp == 0) {
      N w = s_warp[lane];
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const N y = __shfl_up_sync(~0u, w, o);
        if (lane >= o) w += y;
      }
      s_warp[lane] = w;
      if (lane == 31) s_cta = w;
    }
    sync();
    N sum = incl - x + (warp ? s_warp[warp - 1] : 0);
    if constexpr (CTAS == 1) {
      *all = s_cta;
    } else {
      N total = 0;
#pragma unroll
      for (int c = 0; c < CTAS; ++c) {
        const N v = *cg::this_cluster().map_shared_rank(&s_cta, c);
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

// What becomes of new row i: its parent (-1: none), its length and its pages
// (where its table has room), the parent's pages, and whether the last of
// those is in progress.
struct Plan {
  int parent, length, all, old;
  bool fits, partial;
  // pages it shares, when `first` is the first of its parent's children that fits
  __device__ __forceinline__ int keep(bool first) const { return old - (partial && !first); }
};
__device__ __forceinline__ Plan plan_row(const SelectParams& p, int i) {
  Plan r;
  r.parent = p.parents[i];
  int grow = p.grow ? p.grow[i] : 0;
  if (r.parent < -1 || r.parent >= p.old_rows || grow < 0) {
    report(p.status, CMD_CACHE_BAD_INDEX);
    grow = max(grow, 0);
    if (r.parent >= p.old_rows || r.parent < -1) r.parent = -1;
  }
  const int n = r.parent >= 0 ? row_length(p, r.parent) : 0;
  const int64_t length = (int64_t)n + grow;
  r.old = pages_of(n, p.page);
  r.partial = n != r.old * (int)p.page.d;
  r.fits = length <= (int64_t)p.columns * p.page.d;
  if (!r.fits) report(p.status, CMD_CACHE_FULL_TABLE);
  r.length = r.fits ? (int)length : 0;
  r.all = r.fits ? pages_of(r.length, p.page) : 0;
  return r;
}

constexpr int kNobody = 0x7fffffff;  // as a row's first child

// Counts of the pages of old row r, by a warp: each changes hands from the row
// to its children (those that fit), the page in progress to the first of them.
__device__ __forceinline__ void hand_over(const SelectParams& p, int r, int kids) {
  const int n = row_length(p, r), old = pages_of(n, p.page);
  const bool partial = n != old * (int)p.page.d;
  const int last = partial ? min(kids, 1) : kids;
  if (kids == 1) return;
  for (int j = threadIdx.x & 31; j < old; j += 32) {
    const int page = p.tables[r * p.table_st + j];
    if (page < 0 || page >= p.pages) {
      report(p.status, CMD_CACHE_BAD_PAGE);
      continue;
    }
    const int change = (j == old - 1 ? last : kids) - 1;
    if (change) atomicAdd(&p.refs_out[page], change);
  }
}

// New row i, whose new pages begin at the base-th free one: its length, and
// the page to copy. Returns the base, or what stands for none: -1 for a row
// whose table is too short, -2 where the pool had no room (and the pages it
// would have shared were counted).
__device__ __forceinline__ int settle(const SelectParams& p, int i, const Plan& r, bool first, int64_t base, int all_free) {
  const int keep = r.keep(first), wants = r.all - keep;
  const bool room = wants <= 0 || base + wants <= all_free;
  if (r.fits && !room) report(p.status, CMD_CACHE_NO_PAGES);
  const int at = !r.fits ? -1 : !room ? -2 : (int)min(base, (int64_t)all_free);
  p.lengths_out[i] = at >= 0 ? r.length : 0;
  if (at >= 0 && r.partial && !first) {
    const int src = p.tables[r.parent * p.table_st + keep];
    if (src >= 0 && src < p.pages) {
      const int c = atomicAdd(&p.head[kCopies], 1);
      p.copy_src[c] = src;
      p.copy_dst[c] = __ldcg(&p.free_list[at]);
    }
  }
  return at;
}

// The free pages in ascending order; returns their number.
template <int CTAS>
__device__ __forceinline__ int list_free(const SelectParams& p, const Team<CTAS>& team) {
  int all_free;
  const auto is_free = [&](int i) { return __ldcg(&p.refs_out[i]) == 0; };
  const Ranks<CTAS> ranks(team, p.pages, is_free, &all_free);
  ranks.each(is_free, [&](int i, bool f, int rank) {
    if (f) p.free_list[rank] = i;
  });
  return all_free;
}

// Rows enough for a thread each and families in shared memory: every CTA of
// the team works out all rows, and the team meets over the counts alone.
constexpr int kFewRows = kTeamThreads, kFewOldRows = 4096;

template <int CTAS>
__device__ __forceinline__ void select_plan_few(const SelectParams& p) {
  __shared__ int s_first[kFewOldRows], s_children[kFewOldRows];
  const Team<CTAS> team;
  const Team<1> cta;
  const int i = threadIdx.x;
  wait_for_previous();
  let_next_start();
  Plan r = {};
  if (i < p.new_rows) r = plan_row(p, i);
  for (int k = team.me; k < p.pages; k += Team<CTAS>::kThreads) p.refs_out[k] = p.refs[k];
  for (int k = i; k < p.old_rows; k += kTeamThreads) {
    s_first[k] = kNobody;
    s_children[k] = 0;
  }
  if (team.me == 0) p.head[kCopies] = 0;
  __syncthreads();
  const bool goes_on = i < p.new_rows && r.parent >= 0;
  if (goes_on && r.fits) {
    atomicMin(&s_first[r.parent], i);
    atomicAdd(&s_children[r.parent], 1);
  }
  team.sync();  // (and the counts are copied)
  const bool first = !goes_on || s_first[r.parent] == i;
  int64_t all_need;
  const int64_t base = cta.before<int64_t>(r.fits ? r.all - r.keep(first) : 0, &all_need);
  for (int k = team.me >> 5; k < p.old_rows; k += Team<CTAS>::kThreads / 32) hand_over(p, k, s_children[k]);
  team.sync();
  const int all_free = list_free(p, team);
  team.sync();
  if (i < p.new_rows && i % CTAS == (CTAS == 1 ? 0 : (int)blockIdx.x)) {
    p.base[i] = settle(p, i, r, first, base, all_free);
    p.keep[i] = r.keep(first);
  }
}

template <int CTAS>
__device__ __forceinline__ void select_plan_many(const SelectParams& p) {
  using All = Team<CTAS>;
  const All team;
  const int me = team.me;
  wait_for_previous();
  let_next_start();
  for (int i = me; i < p.pages; i += All::kThreads) p.refs_out[i] = p.refs[i];
  for (int i = me; i < p.old_rows; i += All::kThreads) {
    p.first[i] = kNobody;
    p.children[i] = 0;
  }
  if (me == 0) p.head[kCopies] = 0;
  team.sync();
  for (int i = me; i < p.new_rows; i += All::kThreads) {
    const Plan r = plan_row(p, i);
    if (r.parent < 0 || !r.fits) continue;
    atomicMin(&p.first[r.parent], i);
    atomicAdd(&p.children[r.parent], 1);
  }
  team.sync();
  // pages each new row needs, summed in row order
  const int run = (p.new_rows + All::kThreads - 1) / All::kThreads;
  const int i0 = min(me * run, p.new_rows), i1 = min(i0 + run, p.new_rows);
  const auto is_first = [&](int i, const Plan& r) { return r.parent < 0 || p.first[r.parent] == i; };
  int64_t need = 0, all_need;
  for (int i = i0; i < i1; ++i) {
    const Plan r = plan_row(p, i);
    if (r.fits) need += r.all - r.keep(is_first(i, r));
  }
  int64_t base = team.template before<int64_t>(need, &all_need);
  for (int k = me >> 5; k < p.old_rows; k += All::kThreads / 32) hand_over(p, k, p.children[k]);
  team.sync();
  const int all_free = list_free(p, team);
  team.sync();
  for (int i = i0; i < i1; ++i) {
    const Plan r = plan_row(p, i);
    const bool first = is_first(i, r);
    p.base[i] = settle(p, i, r, first, base, all_free);
    p.keep[i] = r.keep(first);
    if (r.fits) base += r.all - r.keep(first);
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
__global__ void __launch_bounds__(kMoveThreads)
    select_apply_kernel(const __grid_constant__ SelectParams p, const __grid_constant__ L pools) {
  wait_for_previous();
  let_next_start();
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
  wait_for_previous();
  let_next_start();
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
__global__ void __launch_bounds__(kMoveThreads)
    compact_apply_kernel(const __grid_constant__ CompactParams p, const __grid_constant__ L pools) {
  wait_for_previous();
  let_next_start();
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

__global__ void __launch_bounds__(kTeamThreads) select_plan_one(const __grid_constant__ SelectParams p) { select_plan_few<1>(p); }
__global__ void __cluster_dims__(8, 1, 1) __launch_bounds__(kTeamThreads)
    select_plan_cluster(const __grid_constant__ SelectParams p) {
  select_plan_few<8>(p);
}
__global__ void __cluster_dims__(8, 1, 1) __launch_bounds__(kTeamThreads)
    select_plan_many_rows(const __grid_constant__ SelectParams p) {
  select_plan_many<8>(p);
}
__global__ void __launch_bounds__(kTeamThreads) compact_plan_one(const __grid_constant__ CompactParams p) { compact_plan<1>(p); }
__global__ void __cluster_dims__(8, 1, 1) __launch_bounds__(kTeamThreads)
    compact_plan_cluster(const __grid_constant__ CompactParams p) {
  compact_plan<8>(p);
}

// Pages (and for a selection rows) above which the first launch is a cluster
// of 8 CTAs. Measured, whole calls, one CTA against the cluster: compaction of
// 601 pages 5.8 and 7.6 us, of 7001 147.6 and 143.6 (131.7 of them the moves);
// selection of 64 rows among 1400 pages 12.6 and 14.7, 3000 pages 13.4 and
// 14.8, 6000 pages 16.5 and 15.4; of 509 rows among 6300 pages 54.5 and 41.7.
constexpr int kLargePool = 4096, kManyRows = 256;

// Takes bits off the status word that were read from it, and no others: an
// operator on another stream may have set some since.
__global__ void status_clear_kernel(int32_t* status, int32_t bits) {
  wait_for_previous();
  let_next_start();
  atomicAnd(status, ~bits);
}

template <class P, class L>
cudaError_t run(void (*plan)(P), int ctas, void (*apply)(P, L), const P& p, const PoolList& pools, cudaStream_t stream) {
  cudaError_t e = launch_chained(plan, ctas, kTeamThreads, 0, stream, p);
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
  return launch_chained(apply, 152 * 8, kMoveThreads, 0, stream, p, l);
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
  const bool few = p.new_rows <= kFewRows && p.old_rows <= kFewOldRows;
  const bool large = p.pages > kLargePool || p.new_rows > kManyRows || p.old_rows > kManyRows;
  const auto plan = !few ? select_plan_many_rows : large ? select_plan_cluster : select_plan_one;
  return by_unit(pools, [&](auto u, auto l) {
    return run(plan, !few || large ? 8 : 1, select_apply_kernel<decltype(u), decltype(l)>, p, pools, stream);
  });
}

cudaError_t status_clear_launch(int32_t* status, int32_t bits, cudaStream_t stream) {
  return launch_chained(status_clear_kernel, 1, 1, 0, stream, status, bits);
}

cudaError_t compact_launch(const CompactParams& p, const PoolList& pools, cudaStream_t stream) {
  const bool large = p.pages > kLargePool;
  return by_unit(pools, [&](auto u, auto l) {
    return run(large ? compact_plan_cluster : compact_plan_one, large ? 8 : 1, compact_apply_kernel<decltype(u), decltype(l)>,
               p, pools, stream);
  });
}

}  // namespace cmdx
