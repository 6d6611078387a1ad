// cache_keep.cu - what a paged cache keeps: the accepted branch of a tree of
// drafts (cmd_draft_path finds it, cmd_cache_accept moves its slots together),
// and the tokens of the largest weights (cmd_cache_evict).
//
// Both move tokens towards the front of their row, in order: the j-th kept one
// from slot of[j] >= j to slot j. So whoever takes tokens in order may read as
// far ahead as it likes: what it writes lies before everything that it has yet
// to read. A plan (a warp to a row) says first which rows are cut, and copies
// the counts; pages past a row's new end are released by the move.
#include <math_constants.h>

#include "cache_common.cuh"

namespace cmdx {

namespace {

__device__ __forceinline__ int pages_of(const KeepParams& p, int n) { return (int)fast_div32(p.page, (uint32_t)n + p.page.d - 1); }

// ---- the accepted branch ---------------------------------------------------------
// A warp walks a row's tree: each lane holds every 32nd draft, and a step is a
// minimum over the drafts that go on from the present one with the token that
// the model chose there. Bound by the steps' latency.
constexpr int kPathRows = 4;

__global__ void __launch_bounds__(kPathRows * 32) path_kernel(const __grid_constant__ PathParams p) {
  constexpr int kEach = CMD_CACHE_MAX_DRAFTS / 32;
  __shared__ int32_t s_choice[kPathRows][CMD_CACHE_MAX_DRAFTS];
  __shared__ int32_t s_path[kPathRows][CMD_CACHE_MAX_DRAFTS];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int row = blockIdx.x * kPathRows + warp;
  wait_for_previous();
  let_next_start();
  if (row >= p.rows) return;
  int token[kEach], parent[kEach];
#pragma unroll
  for (int k = 0; k < kEach; ++k) {
    const int i = lane + 32 * k;
    token[k] = 0;
    parent[k] = -2;
    if (i < p.drafts) {
      token[k] = p.tokens[row * p.token_st[0] + i * p.token_st[1]];
      parent[k] = p.parents ? p.parents[row * p.parent_st[0] + i * p.parent_st[1]] : i - 1;
      s_choice[warp][i] = p.choices[row * p.choice_st[0] + i * p.choice_st[1]];
      s_path[warp][i] = -1;
      if (parent[k] >= i) {
        report(p.status, CMD_CACHE_BAD_INDEX);
        parent[k] = -2;
      }
    }
  }
  __syncwarp();
  int at = __shfl_sync(~0u, parent[0], 0) == -1 ? 0 : -1, steps = 0, last = -1;
  while (at >= 0) {  // (`at` grows: at most as many steps as there are drafts)
    if (lane == 0) s_path[warp][steps] = at;
    ++steps;
    last = s_choice[warp][at];
    uint32_t next = ~0u;
#pragma unroll
    for (int k = kEach - 1; k >= 0; --k)
      if (parent[k] == at && token[k] == last) next = lane + 32 * k;
    next = __reduce_min_sync(~0u, next);
    at = next == ~0u ? -1 : (int)next;
  }
  __syncwarp();
  for (int i = lane; i < p.drafts; i += 32) p.path[row * p.path_st[0] + i * p.path_st[1]] = s_path[warp][i];
  if (lane == 0) {
    p.counts[row * p.counts_st] = steps;
    p.last[row * p.last_st] = last;
  }
}

// ---- the plan ----------------------------------------------------------------------
constexpr int kPlanThreads = 256;

// Whether the row's pages [from, to) exist and only it holds them (`shared`
// asks for the latter); every lane of a warp calls it.
__device__ __forceinline__ bool pages_usable(const KeepParams& p, int row, int from, int to, bool shared) {
  const int lane = threadIdx.x & 31;
  bool ok = true;
  for (int c = from + lane; c < to; c += 32) {
    const int page = p.tables[row * p.table_st + c];
    if (page < 0 || page >= p.pages) {
      report(p.status, CMD_CACHE_BAD_PAGE);
      ok = false;
    } else if (shared && p.refs[page] != 1) {
      report(p.status, CMD_CACHE_SHARED_PAGE);
      ok = false;
    }
  }
  return __all_sync(~0u, ok);
}

// Row r's length, held to its table.
__device__ __forceinline__ int keep_length(const KeepParams& p, int row) {
  const int n = p.lengths[row], most = p.columns * (int)p.page.d;
  if (n >= 0 && n <= most) return n;
  report(p.status, CMD_CACHE_BAD_INDEX);
  return n < 0 ? 0 : most;
}

// A row's new length when its accepted drafts are kept.
__device__ __forceinline__ int accepted_length(const KeepParams& p, int row) {
  const int lane = threadIdx.x & 31;
  const int n = keep_length(p, row), base = n - p.drafts;
  if (base < 0) {
    if (n > 0) report(p.status, CMD_CACHE_BAD_INDEX);
    return n;
  }
  const int32_t* path = p.path + row * p.path_st;
  int count = p.counts[row];
  bool ok = count >= 0 && count <= p.drafts;
  if (!ok) count = 0;
  bool moves = false;
  int furthest = 0;
  for (int j = lane; j < count; j += 32) {
    const int of = path[j];
    ok = ok && of >= j && of < p.drafts && (j == 0 || path[j - 1] < of);
    moves = moves || of != j;
    furthest = max(furthest, of);
  }
  ok = __all_sync(~0u, ok);
  if (!ok) {
    report(p.status, CMD_CACHE_BAD_INDEX);
    return base;
  }
  if (!__any_sync(~0u, moves)) return base + count;
  furthest = __reduce_max_sync(~0u, furthest);
  const int from = (int)fast_div32(p.page, (uint32_t)base), to = pages_of(p, base + count);
  ok = pages_usable(p, row, from, to, true);
  ok = pages_usable(p, row, to, pages_of(p, base + furthest + 1), false) && ok;
  return ok ? base + count : base;
}

// ... and when it is held to the budget.
__device__ __forceinline__ int evicted_length(const KeepParams& p, int row) {
  const int n = keep_length(p, row);
  if (n <= p.budget) return n;
  const int to = pages_of(p, p.budget);
  bool ok = pages_usable(p, row, 0, to, true);
  ok = pages_usable(p, row, to, pages_of(p, n), false) && ok;
  return ok ? p.budget : n;
}

template <bool ACCEPT>
__global__ void __launch_bounds__(kPlanThreads) keep_plan_kernel(const __grid_constant__ KeepParams p) {
  wait_for_previous();
  let_next_start();
  const int64_t me = (int64_t)blockIdx.x * kPlanThreads + threadIdx.x, all = (int64_t)gridDim.x * kPlanThreads;
  for (int64_t i = me; i < p.pages; i += all) p.refs_out[i] = p.refs[i];
  for (int64_t row = me >> 5; row < p.rows; row += all >> 5) {
    const int n = ACCEPT ? accepted_length(p, (int)row) : evicted_length(p, (int)row);
    if ((threadIdx.x & 31) == 0) p.lengths_out[row] = n;
  }
}

// The pages past a row's new length are released (each thread of the CTA calls it).
__device__ __forceinline__ void release_pages(const KeepParams& p, int row, int now, int before) {
  for (int c = pages_of(p, now) + (int)threadIdx.x; c < pages_of(p, before); c += blockDim.x) {
    const int page = p.tables[row * p.table_st + c];
    if (page >= 0 && page < p.pages) atomicSub(&p.refs_out[page], 1);
    else report(p.status, CMD_CACHE_BAD_PAGE);
  }
}

// ---- the accepted branch's tokens ----------------------------------------------------
// A thread takes one piece of a token (16 bytes where all rows allow it) in
// one pool, and moves it for all tokens of a row, in order.
constexpr int kAcceptThreads = 128;

template <class U>
__global__ void __launch_bounds__(kAcceptThreads) accept_kernel(const __grid_constant__ KeepParams p, const __grid_constant__ KeepPools pools) {
  constexpr int kAtOnce = 4;
  wait_for_previous();
  let_next_start();
  const uint32_t at = blockIdx.x * kAcceptThreads + threadIdx.x;
  const uint32_t head = fast_div32(p.per_head, at);
  const KeepPool& pool = pools.pool[blockIdx.y];
  uint8_t* base_ptr = pool.ptr + head * pool.st[2] + (int64_t)(at - head * p.per_head.d) * sizeof(U);
  for (int row = blockIdx.z; row < p.rows; row += gridDim.z) {
    const int before = keep_length(p, row), base = before - p.drafts, now = p.lengths_out[row];
    if (base < 0) continue;
    if (blockIdx.x == 0 && blockIdx.y == 0) release_pages(p, row, now, before);
    if (at >= (uint32_t)(p.heads * p.pieces)) continue;
    const int32_t* path = p.path + row * p.path_st;
    const int32_t* table = p.tables + row * p.table_st;
    const auto slot = [&](int t) {
      const uint32_t column = fast_div32(p.page, (uint32_t)t);
      return reinterpret_cast<U*>(base_ptr + table[column] * pool.st[0] + (int64_t)(t - column * p.page.d) * pool.st[1]);
    };
    for (int j = 0; j < now - base; j += kAtOnce) {
      U x[kAtOnce];
      bool moves[kAtOnce];
#pragma unroll
      for (int k = 0; k < kAtOnce; ++k) {
        const int of = j + k < now - base ? path[j + k] : j + k;
        moves[k] = of != j + k;
        if (moves[k]) x[k] = *slot(base + of);
      }
#pragma unroll
      for (int k = 0; k < kAtOnce; ++k)
        if (moves[k]) *slot(base + j + k) = x[k];
    }
  }
}

// ---- eviction --------------------------------------------------------------------------
// Which tokens one kv head of one layer and row keeps: those whose key (the
// weight's bits, in the order of the numbers) is above the threshold, and of
// those at it the first. The threshold is found digit by digit from a
// histogram. Weights are read once where they fit in shared memory.
constexpr int kSelectThreads = 512, kSelectWarps = kSelectThreads / 32;
constexpr int kBins = 2048;
constexpr int kCached = 48 * 1024;  // keys

__device__ __forceinline__ uint32_t order_of(float x) {
  if (x != x) return 0;  // below all numbers
  const uint32_t b = __float_as_uint(x == 0.0f ? 0.0f : x);
  return b >> 31 ? ~b : b | 0x80000000u;
}

__global__ void __launch_bounds__(kSelectThreads) evict_select_kernel(const __grid_constant__ KeepParams p,
                                                                       const __grid_constant__ KeepLayers layers, int cached) {
  extern __shared__ uint32_t s_keys[];
  __shared__ uint32_t s_bins[kBins];
  __shared__ uint32_t s_warp[kSelectWarps], s_more[kSelectWarps];
  __shared__ uint32_t s_digit, s_above;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  wait_for_previous();
  let_next_start();
  const int head = blockIdx.x % p.heads, task = blockIdx.x / p.heads, layer = task % p.layers, row = task / p.layers;
  const int n = keep_length(p, row);
  if (n <= p.budget || p.lengths_out[row] != p.budget) return;
  const float* weights = layers.weights[layer] + row * layers.w_st[layer][0] + head * layers.w_st[layer][1];
  int32_t* kept = p.kept + (int64_t)blockIdx.x * p.budget;
  const int count = n - p.recent, want = p.budget - p.recent;
  const bool in_shared = count <= cached;
  if (in_shared)
    for (int t = threadIdx.x; t < count; t += kSelectThreads) s_keys[t] = order_of(weights[t]);
  __syncthreads();
  const auto key_of = [&](int t) { return in_shared ? s_keys[t] : order_of(weights[t]); };
  uint32_t top = 0, left = want;  // the threshold's digits so far; how many are still to be taken among its equals
  if (want > 0) {
#pragma unroll 1
    for (int pass = 0; pass < 3; ++pass) {
      const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, width = pass == 2 ? 10 : 11;
      for (int i = threadIdx.x; i < kBins; i += kSelectThreads) s_bins[i] = 0;
      __syncthreads();
      for (int t0 = warp * 32; t0 < count; t0 += kSelectThreads) {
        const int t = t0 + lane;
        const uint32_t key = t < count ? key_of(t) : 0u;
        const bool mine = t < count && (pass == 0 || key >> (shift + width) == top);
        const uint32_t digit = key >> shift & ((1u << width) - 1);
        const uint32_t who = __ballot_sync(~0u, mine);
        if (!mine) continue;
        int same;
        __match_all_sync(who, digit, &same);  // (equal weights would meet in one counter)
        if (!same) atomicAdd(&s_bins[digit], 1u);
        else if (lane == __ffs(who) - 1) atomicAdd(&s_bins[digit], (uint32_t)__popc(who));
      }
      __syncthreads();
      // this thread's 4 bins, the largest first
      constexpr int kEach = kBins / kSelectThreads;
      const int first = kBins - 1 - (int)threadIdx.x * kEach;
      uint32_t sum = 0;
#pragma unroll
      for (int k = 0; k < kEach; ++k) sum += s_bins[first - k];
      uint32_t incl = sum;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t y = __shfl_up_sync(~0u, incl, o);
        if (lane >= o) incl += y;
      }
      if (lane == 31) s_warp[warp] = incl;
      __syncthreads();
      uint32_t above = incl - sum;
      for (int w = 0; w < warp; ++w) above += s_warp[w];
      if (above < left && above + sum >= left) {  // (one thread)
#pragma unroll
        for (int k = 0; k < kEach; ++k) {
          const uint32_t here = s_bins[first - k];
          if (above < left && above + here >= left) {
            s_digit = first - k;
            s_above = above;
            break;
          }
          above += here;
        }
      }
      __syncthreads();
      top = top << width | s_digit;
      left -= s_above;
      __syncthreads();  // (the next pass clears the bins)
    }
  }
  // the kept ones in order: warps take runs, and count before they write
  const int run = (count + kSelectThreads - 1) / kSelectThreads * 32;
  const int from = min(warp * run, count), to = min(from + run, count);
  uint32_t more = 0, equal = 0;
  if (want > 0)
    for (int t = from + lane; t < to; t += 32) {
      const uint32_t key = key_of(t);
      more += key > top;
      equal += key == top;
    }
  more = __reduce_add_sync(~0u, more);
  equal = __reduce_add_sync(~0u, equal);
  if (lane == 0) {
    s_more[warp] = more;
    s_warp[warp] = equal;
  }
  __syncthreads();
  more = equal = 0;
  for (int w = 0; w < warp; ++w) {
    more += s_more[w];
    equal += s_warp[w];
  }
  if (want > 0)
    for (int t0 = from; t0 < to; t0 += 32) {
      const int t = t0 + lane;
      const uint32_t key = t < to ? key_of(t) : 0u, below = (1u << lane) - 1u;
      const uint32_t is_more = __ballot_sync(~0u, t < to && key > top), is_equal = __ballot_sync(~0u, t < to && key == top);
      const uint32_t m = more + __popc(is_more & below), e = equal + __popc(is_equal & below);
      if (is_more >> lane & 1) kept[m + min(e, left)] = t;
      else if ((is_equal >> lane & 1) && e < left) kept[m + e] = t;
      more += __popc(is_more);
      equal += __popc(is_equal);
    }
  for (int i = threadIdx.x; i < p.recent; i += kSelectThreads) kept[want + i] = count + i;
}

// A CTA moves the kept keys, values or weights of one kv head of one layer and
// row, chunks of tokens in order: the next chunk is read before this one is
// written, and the barrier between stands for its reads by all threads.
constexpr int kMoveThreads = 256, kMoveAtOnce = 8;

template <class U, class A>
__device__ __forceinline__ void move_kept(const int32_t* kept, int n, int pieces, const A& address) {
  const int over = kMoveThreads / pieces;  // tokens side by side
  const int mine = threadIdx.x / pieces, piece = threadIdx.x - mine * pieces;
  const int chunk = over * kMoveAtOnce;
  const bool busy = mine < over;
  U x[kMoveAtOnce];
  const auto read = [&](int j0) {
#pragma unroll
    for (int k = 0; k < kMoveAtOnce; ++k) {
      const int j = j0 + k * over + mine;
      if (busy && j < n) x[k] = *address(kept[j], piece);
    }
  };
  read(0);
  for (int j0 = 0; j0 < n; j0 += chunk) {
    U y[kMoveAtOnce];
#pragma unroll
    for (int k = 0; k < kMoveAtOnce; ++k) y[k] = x[k];
    read(j0 + chunk);
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kMoveAtOnce; ++k) {
      const int j = j0 + k * over + mine;
      if (busy && j < n) *address(j, piece) = y[k];
    }
  }
}

template <class U>
__global__ void __launch_bounds__(kMoveThreads) evict_move_kernel(const __grid_constant__ KeepParams p, const __grid_constant__ KeepLayers layers) {
  wait_for_previous();
  let_next_start();
  const int what = blockIdx.x % 3, list = blockIdx.x / 3;
  const int head = list % p.heads, task = list / p.heads, layer = task % p.layers, row = task / p.layers;
  const int n = keep_length(p, row), now = p.lengths_out[row];
  if (n <= p.budget || now != p.budget) return;
  const int32_t* kept = p.kept + (int64_t)list * p.budget;
  if (what == 2) {
    float* weights = layers.weights[layer] + row * layers.w_st[layer][0] + head * layers.w_st[layer][1];
    move_kept<float>(kept, now, 1, [&](int t, int) { return weights + t; });
    __syncthreads();
    for (int t = now + threadIdx.x; t < n; t += kMoveThreads) weights[t] = 0.0f;
    if (layer == 0 && head == 0) release_pages(p, row, now, n);
    return;
  }
  const KeepPool& pool = layers.pool[layer][what];
  uint8_t* base = pool.ptr + head * pool.st[2];
  const int32_t* table = p.tables + row * p.table_st;
  move_kept<U>(kept, now, p.pieces, [&](int t, int piece) {
    const uint32_t column = fast_div32(p.page, (uint32_t)t);
    return reinterpret_cast<U*>(base + table[column] * pool.st[0] + (int64_t)(t - column * p.page.d) * pool.st[1]) + piece;
  });
}

// calls f with a value of the access type
template <class F>
cudaError_t by_unit(int unit, F f) {
  switch (unit) {
    case 16: return f(uint4{});
    case 8: return f(uint2{});
    case 4: return f(uint32_t{});
  }
  return f(uint16_t{});
}

template <bool ACCEPT>
cudaError_t plan_launch(const KeepParams& p, cudaStream_t stream) {
  const int64_t work = (int64_t)p.rows * 32 > p.pages ? (int64_t)p.rows * 32 : p.pages;
  const int64_t ctas = (work + kPlanThreads - 1) / kPlanThreads;
  return launch_chained(keep_plan_kernel<ACCEPT>, (int)(ctas < 152 * 8 ? ctas : 152 * 8), kPlanThreads, 0, stream, p);
}

}  // namespace

cudaError_t path_launch(const PathParams& p, cudaStream_t stream) {
  return launch_chained(path_kernel, (p.rows + kPathRows - 1) / kPathRows, kPathRows * 32, 0, stream, p);
}

cudaError_t accept_launch(const KeepParams& p, const KeepPools& pools, cudaStream_t stream) {
  const cudaError_t e = plan_launch<true>(p, stream);
  if (e != cudaSuccess || p.rows == 0) return e;
  return by_unit(p.unit, [&](auto u) {
    const dim3 grid((unsigned)((p.heads * p.pieces + kAcceptThreads - 1) / kAcceptThreads), (unsigned)pools.n,
                    (unsigned)(p.rows < 32768 ? p.rows : 32768));
    return launch_grid(accept_kernel<decltype(u)>, grid, kAcceptThreads, 0, stream, p, pools);
  });
}

cudaError_t evict_launch(const KeepParams& p, const KeepLayers& layers, cudaStream_t stream) {
  cudaError_t e = plan_launch<false>(p, stream);
  if (e != cudaSuccess || p.rows == 0) return e;
  const int lists = p.rows * p.layers * p.heads;
  if (p.budget > 0) {
    const int64_t most = (int64_t)p.columns * p.page.d;
    const int cached = (int)(most < kCached ? most : kCached);
    static PerDevice ready;  // (static storage: zero before first use)
    e = allow_smem(evict_select_kernel, kCached * 4, ready);
    if (e == cudaSuccess) e = launch_chained(evict_select_kernel, lists, kSelectThreads, (size_t)cached * 4, stream, p, layers, cached);
  }
  if (e != cudaSuccess) return e;
  return by_unit(p.unit, [&](auto u) { return launch_chained(evict_move_kernel<decltype(u)>, 3 * lists, kMoveThreads, 0, stream, p, layers); });
}

}  // namespace cmdx
