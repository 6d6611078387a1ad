// cache_keep.cu - what a paged cache keeps: the accepted branch of a tree of
// drafts (cmd_draft_path finds it, cmd_cache_accept moves its slots together),
// and the tokens of the largest weights (cmd_cache_evict).
//
// Both move tokens towards the front of their row, in order: the j-th kept one
// from slot of[j] >= j to slot j. So whoever takes tokens in order may read as
// far ahead as it likes: what it writes lies before everything that it has yet
// to read. A plan (a warp to a row) says first which rows are cut, and copies
// the counts; pages past a row's new end are released by the move.
#include <cooperative_groups.h>
#include <math_constants.h>

#include "cache_common.cuh"

namespace cmdx {

namespace {

namespace cg = cooperative_groups;

__device__ __forceinline__ int pages_of(const KeepParams& p, int n) { return (int)fast_div32(p.page, (uint32_t)n + p.page.d - 1); }

// ---- the accepted branch ---------------------------------------------------------
// A warp walks a row's tree: each lane holds every 32nd draft, and a step is a
// minimum over the drafts that go on from the present one with the token that
// the model chose there. Bound by the steps' latency, one after another (16 rows
// of 24 drafts 2.1 us, 512 of 256 3.8).
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

// Whether the page in column c of a row exists and only it holds it (`shared`
// asks for the latter); what is wrong is reported.
__device__ __forceinline__ bool page_usable(const KeepParams& p, int row, int c, bool shared) {
  const int page = p.tables[row * p.table_st + c];
  if (page < 0 || page >= p.pages) {
    report(p.status, CMD_CACHE_BAD_PAGE);
    return false;
  }
  if (shared && p.refs[page] > 1) {
    report(p.status, CMD_CACHE_SHARED_PAGE);
    return false;
  }
  return true;
}
// ... all of columns [from, to); every lane of a warp calls it.
__device__ __forceinline__ bool pages_usable(const KeepParams& p, int row, int from, int to, bool shared) {
  bool ok = true;
  for (int c = from + (int)(threadIdx.x & 31); c < to; c += 32) ok = page_usable(p, row, c, shared) && ok;
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
  for (int j = lane; j < count; j += 32) {
    const int of = path[j];
    ok = ok && of >= j && of < p.drafts && (j == 0 || path[j - 1] < of);
  }
  ok = __all_sync(~0u, ok);
  if (!ok) {
    report(p.status, CMD_CACHE_BAD_INDEX);
    return base;
  }
  // the pages that the moves meet, and no others
  for (int j = lane; j < count; j += 32) {
    const int of = path[j];
    if (of == j) continue;
    ok = page_usable(p, row, (int)fast_div32(p.page, (uint32_t)(base + j)), true) && ok;
    ok = page_usable(p, row, (int)fast_div32(p.page, (uint32_t)(base + of)), false) && ok;
  }
  return __all_sync(~0u, ok) ? base + count : base;
}

// ... and when it is held to the budget.
__device__ __forceinline__ int evicted_length(const KeepParams& p, int row) {
  const int n = keep_length(p, row);
  // (a length beyond the table names no tokens that are known to be the last ones: nothing is dropped by it)
  if (n <= p.budget || p.lengths[row] != n) return n;
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
// A CTA takes some pieces of a token (16 bytes each where all rows allow it) of
// one row in one pool, a thread one piece of every accepted token, in order.
// Where the tokens lie is worked out once for the CTA, all at the same time.
// 61 rows of 64 drafts in 32 pools of 8 heads of 128 dims: 14 us with the plan
// (18.8 MB read and as many written: 5.6), the chain of plan, path, tables and
// data; from Python 52, of which 24 are the caller's 32 views of its pools.
constexpr int kAcceptThreads = 128;

template <class U>
__global__ void __launch_bounds__(kAcceptThreads) accept_kernel(const __grid_constant__ KeepParams p, const __grid_constant__ KeepPools pools) {
  constexpr int kAtOnce = 8;
  __shared__ int64_t s_from[CMD_CACHE_MAX_DRAFTS], s_to[CMD_CACHE_MAX_DRAFTS];  // (from -1: it stays)
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
    const int count = now - base;
    const int32_t* path = p.path + row * p.path_st;
    const int32_t* table = p.tables + row * p.table_st;
    const auto slot = [&](int t) {
      const uint32_t column = fast_div32(p.page, (uint32_t)t);
      return table[column] * pool.st[0] + (int64_t)(t - column * p.page.d) * pool.st[1];
    };
    for (int j = threadIdx.x; j < count; j += kAcceptThreads) {
      const int of = path[j];
      s_from[j] = of == j ? -1 : slot(base + of);
      s_to[j] = of == j ? 0 : slot(base + j);
    }
    __syncthreads();
    if (at < (uint32_t)(p.heads * p.pieces)) {
      for (int j = 0; j < count; j += kAtOnce) {
        U x[kAtOnce];
#pragma unroll
        for (int k = 0; k < kAtOnce; ++k)
          if (j + k < count && s_from[j + k] >= 0) x[k] = *reinterpret_cast<const U*>(base_ptr + s_from[j + k]);
#pragma unroll
        for (int k = 0; k < kAtOnce; ++k)
          if (j + k < count && s_from[j + k] >= 0) *reinterpret_cast<U*>(base_ptr + s_to[j + k]) = x[k];
      }
    }
    __syncthreads();
  }
}

// ---- eviction --------------------------------------------------------------------------
// Which tokens one kv head of one layer and row keeps: those whose key (the
// weight's bits, in the order of the numbers) is above the threshold, and of
// those at it the first. The threshold's first 11 bits come from a histogram of
// all keys; the few with the same first bits are then gathered, and its others
// come from histograms of them. Keys are read once where they fit in shared
// memory; in the last pass each warp writes the kept ones of its run of tokens
// behind those of the runs before. Bound by instructions (issue slots 65%) and by
// lists to a CTA: 256 lists of 20011 to 32768 weights 49 us, their 27 MB 4.
constexpr int kSelectThreads = 1024, kSelectWarps = kSelectThreads / 32;
constexpr int kBins = 2048;
constexpr int kCached = 44 * 1024;  // keys
constexpr int kGathered = 1024;     // of equal first bits, at most: more are gone over where they lie

__device__ __forceinline__ uint32_t order_of(float x) {
  if (x != x) return 0;  // below all numbers
  const uint32_t b = __float_as_uint(x == 0.0f ? 0.0f : x);
  return b >> 31 ? ~b : b | 0x80000000u;
}

struct SelectState {
  uint32_t bins[kBins];
  uint32_t warp[kSelectWarps], more[kSelectWarps], equal[kSelectWarps];
  uint32_t digit, above, gathered;
  uint32_t key[kGathered];
  int32_t token[kGathered];
};

// Counts a warp's keys' digits (those with `mine`).
__device__ __forceinline__ void count_digit(SelectState& s, uint32_t digit, bool mine) {
  const uint32_t who = __ballot_sync(~0u, mine);
  const int first = __ffs(who) - 1;
  // (equal weights would meet in one counter)
  const uint32_t lead = __shfl_sync(~0u, digit, first & 31);
  const bool same = __all_sync(~0u, !mine || digit == lead);
  if (mine && (!same || (int)(threadIdx.x & 31) == first)) atomicAdd(&s.bins[digit], same ? (uint32_t)__popc(who) : 1u);
}
// The digit at which the counts from the largest down reach `left`; *left then
// counts on among the keys of that digit. Every thread calls it.
__device__ __forceinline__ uint32_t find_digit(SelectState& s, uint32_t* left) {
  constexpr int kEach = kBins / kSelectThreads;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  __syncthreads();
  const int first = kBins - 1 - (int)threadIdx.x * kEach;
  uint32_t sum = 0;
#pragma unroll
  for (int k = 0; k < kEach; ++k) sum += s.bins[first - k];
  uint32_t incl = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t y = __shfl_up_sync(~0u, incl, o);
    if (lane >= o) incl += y;
  }
  if (lane == 31) s.warp[warp] = incl;
  __syncthreads();
  uint32_t w = lane < warp ? s.warp[lane] : 0u;
  uint32_t above = __reduce_add_sync(~0u, w) + incl - sum;
  if (above < *left && above + sum >= *left) {  // (one thread)
#pragma unroll
    for (int k = 0; k < kEach; ++k) {
      const uint32_t here = s.bins[first - k];
      if (above < *left && above + here >= *left) {
        s.digit = first - k;
        s.above = above;
        break;
      }
      above += here;
    }
  }
  __syncthreads();
  *left -= s.above;
  const uint32_t digit = s.digit;
  for (int i = threadIdx.x; i < kBins; i += kSelectThreads) s.bins[i] = 0;
  __syncthreads();
  return digit;
}

__global__ void __launch_bounds__(kSelectThreads) evict_select_kernel(const __grid_constant__ KeepParams p,
                                                                       const __grid_constant__ KeepLayers layers, int cached) {
  extern __shared__ uint32_t s_keys[];
  __shared__ SelectState s;
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
  for (int i = threadIdx.x; i < kBins; i += kSelectThreads) s.bins[i] = 0;
  if (threadIdx.x < kSelectWarps) s.more[threadIdx.x] = s.equal[threadIdx.x] = 0;
  if (threadIdx.x == 0) s.gathered = 0;
  __syncthreads();
  const auto key_of = [&](int t) { return in_shared ? s_keys[t] : order_of(weights[t]); };
  // runs of tokens for the warps of the last pass, whole 32s each
  const int run = (count + kSelectThreads - 1) / kSelectThreads * 32;
  uint32_t top = 0, left = want;  // the threshold; how many are still to be taken among its equals
  if (want > 0) {
    constexpr int kAtOnce = 8;
    for (int t0 = 0; t0 < count; t0 += kSelectThreads * kAtOnce) {
      float x[kAtOnce];
#pragma unroll
      for (int k = 0; k < kAtOnce; ++k) {
        const int t = t0 + k * kSelectThreads + (int)threadIdx.x;
        if (t < count) x[k] = weights[t];
      }
#pragma unroll
      for (int k = 0; k < kAtOnce; ++k) {
        const int t = t0 + k * kSelectThreads + (int)threadIdx.x;
        const uint32_t key = t < count ? order_of(x[k]) : 0u;
        if (in_shared && t < count) s_keys[t] = key;
        count_digit(s, key >> 21, t < count);
      }
    }
    top = find_digit(s, &left);
    // those with its first bits, gathered; those above counted, for each run
    for (int t0 = 0; t0 < count; t0 += kSelectThreads * kAtOnce) {
      uint32_t key[kAtOnce];
#pragma unroll
      for (int k = 0; k < kAtOnce; ++k) {
        const int t = t0 + k * kSelectThreads + (int)threadIdx.x;
        key[k] = t < count ? key_of(t) : 0u;
      }
#pragma unroll
      for (int k = 0; k < kAtOnce; ++k) {
        const int t = t0 + k * kSelectThreads + (int)threadIdx.x;
        const bool more = t < count && key[k] >> 21 > top, same = t < count && key[k] >> 21 == top;
        const uint32_t is_more = __ballot_sync(~0u, more);
        if (lane == 0 && is_more) atomicAdd(&s.more[t / run], (uint32_t)__popc(is_more));  // (a run is whole 32s)
        if (same) {
          const uint32_t at = atomicAdd(&s.gathered, 1u);
          if (at < kGathered) {
            s.key[at] = key[k];
            s.token[at] = t;
          }
        }
      }
    }
    __syncthreads();
    const uint32_t gathered = s.gathered;
    const bool few = gathered <= kGathered;
    const int items = few ? (int)gathered : count;
    const auto item_key = [&](int i) { return few ? s.key[i] : key_of(i); };
#pragma unroll 1
    for (int pass = 0; pass < 2; ++pass) {
      const int shift = pass == 0 ? 10 : 0, width = pass == 0 ? 11 : 10;
      for (int i0 = 0; i0 < items; i0 += kSelectThreads) {
        const int i = i0 + (int)threadIdx.x;
        const uint32_t key = i < items ? item_key(i) : 0u;
        count_digit(s, key >> shift & ((1u << width) - 1), i < items && key >> (shift + width) == top);
      }
      top = top << width | find_digit(s, &left);
    }
    for (int i = threadIdx.x; i < items; i += kSelectThreads) {
      const uint32_t key = item_key(i);
      if (key >> 21 != top >> 21) continue;
      const int t = few ? s.token[i] : i;
      if (key > top) atomicAdd(&s.more[t / run], 1u);
      if (key == top) atomicAdd(&s.equal[t / run], 1u);
    }
    __syncthreads();
    uint32_t more = __reduce_add_sync(~0u, lane < warp ? s.more[lane] : 0u);
    uint32_t equal = __reduce_add_sync(~0u, lane < warp ? s.equal[lane] : 0u);
    const int from = min(warp * run, count), to = min(from + run, count);
    const uint32_t below = (1u << lane) - 1u;
    for (int t0 = from; t0 < to; t0 += 32 * kAtOnce) {
      uint32_t key[kAtOnce];
#pragma unroll
      for (int k = 0; k < kAtOnce; ++k) {
        const int t = t0 + 32 * k + lane;
        key[k] = t < to ? key_of(t) : 0u;
      }
#pragma unroll
      for (int k = 0; k < kAtOnce; ++k) {
        const int t = t0 + 32 * k + lane;
        const uint32_t is_more = __ballot_sync(~0u, t < to && key[k] > top), is_equal = __ballot_sync(~0u, t < to && key[k] == top);
        const uint32_t m = more + __popc(is_more & below), e = equal + __popc(is_equal & below);
        if (is_more >> lane & 1) kept[m + min(e, left)] = t;
        else if ((is_equal >> lane & 1) && e < left) kept[m + e] = t;
        more += __popc(is_more);
        equal += __popc(is_equal);
      }
    }
  }
  for (int i = threadIdx.x; i < p.recent; i += kSelectThreads) kept[want + i] = count + i;
}

// A team (a cluster of CTAs) moves the kept keys or values of one kv head of one
// layer and row (some of each token's pieces), or its weights: chunks of tokens
// in order, one to each CTA at a time. No token moves up, so that what a chunk is
// written over lies in its own place or before it, and all that is left to see to
// is that the team has read its chunks before any of them is written: a barrier
// of the team. While a chunk's data is on its way, the next one's places are
// looked up. (A lone CTA takes 2 us for 256 tokens; CTAs without a row to cut cost
// as much as they are many, so that teams stand where the lists are few.) 4 rows'
// 4096 of up to 32768 tokens in 8 layers of 8 heads of 128 dims: 192 us, 1.08 GB
// read and written, 84% of the copy peak.
constexpr int kMoveThreads = kEvictMoveThreads, kMoveAtOnce = kEvictMoveAtOnce;

// tokens: of a chunk (threads / pieces * kMoveAtOnce); from, to: their places,
// two chunks of each
template <class U, class F>
__device__ __forceinline__ void move_kept(int n, int team, int pieces, int64_t* from, int64_t* to, uint8_t* base, const F& place) {
  const int over = kMoveThreads / pieces;  // tokens side by side
  const int mine = threadIdx.x / pieces, piece = threadIdx.x - mine * pieces;
  const int chunk = over * kMoveAtOnce, first = blockIdx.x % team * chunk;
  const bool busy = mine < over;
  base += (int64_t)piece * sizeof(U);
  U x[kMoveAtOnce];
  const auto look = [&](int j0) {
    for (int i = threadIdx.x; i < chunk && j0 + i < n; i += kMoveThreads) place(j0 + i, &from[i], &to[i]);
  };
  look(first);
  __syncthreads();
  for (int all0 = 0; all0 < n; all0 += team * chunk) {
    const int j0 = all0 + first;
    int64_t d[kMoveAtOnce];
#pragma unroll
    for (int k = 0; k < kMoveAtOnce; ++k) {
      const int i = k * over + mine;
      if (busy && j0 + i < n) {
        x[k] = *reinterpret_cast<const U*>(base + from[i]);
        d[k] = to[i];
      }
    }
    __syncthreads();  // (the places have been read; so has, after the next barrier, the data)
    look(j0 + team * chunk);
    if (team > 1) cg::this_cluster().sync();
    else __syncthreads();
#pragma unroll
    for (int k = 0; k < kMoveAtOnce; ++k)
      if (busy && j0 + k * over + mine < n) *reinterpret_cast<U*>(base + d[k]) = x[k];
  }
}

template <class U>
__global__ void __launch_bounds__(kMoveThreads) evict_move_kernel(const __grid_constant__ KeepParams p, const __grid_constant__ KeepLayers layers) {
  __shared__ int64_t s_from[kMoveThreads * kMoveAtOnce], s_to[kMoveThreads * kMoveAtOnce];
  wait_for_previous();
  let_next_start();
  // the slices of a list: keys, values, and at the end the weights
  const int slices = 2 * p.slices + 1, what = blockIdx.x / p.team % slices, list = blockIdx.x / p.team / slices;
  const int head = list % p.heads, task = list / p.heads, layer = task % p.layers, row = task / p.layers;
  const int n = keep_length(p, row), now = p.lengths_out[row];
  if (n <= p.budget || now != p.budget) return;
  const int32_t* kept = p.kept + (int64_t)list * p.budget;
  if (what == slices - 1) {
    float* weights = layers.weights[layer] + row * layers.w_st[layer][0] + head * layers.w_st[layer][1];
    move_kept<float>(now, p.team, 1, s_from, s_to, reinterpret_cast<uint8_t*>(weights), [&](int j, int64_t* from, int64_t* to) {
      *from = 4 * (int64_t)kept[j];
      *to = 4 * (int64_t)j;
    });
    // (the team has read all that it will, now that its last chunks are written)
    const int rank = blockIdx.x % p.team;
    for (int t = now + rank * kMoveThreads + (int)threadIdx.x; t < n; t += p.team * kMoveThreads) weights[t] = 0.0f;
    if (layer == 0 && head == 0 && rank == 0) release_pages(p, row, now, n);
    return;
  }
  const int each = (p.pieces + p.slices - 1) / p.slices, piece0 = what / 2 * each, pieces = min(each, p.pieces - piece0);
  if (pieces <= 0) return;
  const KeepPool& pool = layers.pool[layer][what & 1];
  const int32_t* table = p.tables + row * p.table_st;
  const auto slot = [&](int t) {
    const uint32_t column = fast_div32(p.page, (uint32_t)t);
    return table[column] * pool.st[0] + (int64_t)(t - column * p.page.d) * pool.st[1];
  };
  move_kept<U>(now, p.team, pieces, s_from, s_to, pool.ptr + head * pool.st[2] + (int64_t)piece0 * sizeof(U), [&](int j, int64_t* from, int64_t* to) {
    *from = slot(kept[j]);
    *to = slot(j);
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
  return by_unit(p.unit, [&](auto u) {
    return launch_clusters(evict_move_kernel<decltype(u)>, p.team, (unsigned)((2 * p.slices + 1) * lists * p.team), kMoveThreads, 0, stream, p, layers);
  });
}

}  // namespace cmdx
