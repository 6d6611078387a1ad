// cache_drafts.cuh - what the attention of drafted tokens adds to that of one
// (cache_attend.cuh), shared by its kernels.
//
// Row r's last `drafts` tokens in the cache are guesses, a tree: draft i goes
// on from draft parents[i] (or from the tokens before the drafts: -1), and sees
// those tokens, its ancestors and itself. The queries of all drafts and of all
// query heads of a kv head are the rows of one product with that head's keys:
// "query head" q of cache_attend.cuh is draft q / per, head q % per of the kv
// head's. So each key and value crosses from memory once for up to a block of
// them, and the split over CTAs and its join are the same.
//
// A tile all of whose tokens every draft sees needs no mask. In the others (the
// last ones of a row, and the first of a window) a draft's ancestors are bits
// of a word list in shared memory, and its first token a number.
#pragma once

#include "cache_attend.cuh"

namespace cmdx {

constexpr int kDraftWords = CMD_CACHE_MAX_DRAFTS / 32;
constexpr int kNever = 0x7fffffff;

// Row r's length, held to its table; none where the drafts do not fit in it.
__device__ __forceinline__ int attend_length(const DraftParams& p, int r) {
  const int n = attend_length(static_cast<const AttendParams&>(p), r);
  if (n >= p.drafts) return n;
  if (n > 0) report(p.status, CMD_CACHE_BAD_INDEX);
  return 0;
}
__device__ __forceinline__ AttendPlace attend_place(const DraftParams& p, int row, int h) {
  const int kv = h / p.group, q = h - kv * p.group;
  const int draft = (int)fast_div32(p.per, (uint32_t)q), head = kv * (int)p.per.d + q - draft * (int)p.per.d;
  return {row * p.out_st[0] + draft * p.out_draft + head * p.out_st[1],
          row * p.lse_st[0] + draft * p.lse_draft + head * p.lse_st[1]};
}
// The maximum that a part of padding is given (with a sum of zero): the parts
// of tokens that every draft sees are worked out without the tree, as if it
// were none.
constexpr float kPadding = 3e38f;
__device__ __forceinline__ bool attend_void(const DraftParams&, float m) { return m == kPadding; }

// The drafts of a row: which each sees (a bit each; itself among them), its
// first token (kNever: the draft is padding and sees nothing).
struct DraftTree {
  uint32_t seen[CMD_CACHE_MAX_DRAFTS][kDraftWords];
  int32_t from[CMD_CACHE_MAX_DRAFTS];
  int32_t depth[CMD_CACHE_MAX_DRAFTS];

  // Whether draft i sees token t, the drafts beginning at `base`.
  __device__ __forceinline__ bool sees(const DraftParams& p, int i, int t, int base) const {
    if (t < base) return t >= from[i];
    const uint32_t j = (uint32_t)(t - base);
    return j < (uint32_t)p.drafts && (seen[i][j >> 5] >> (j & 31) & 1);
  }
  // Which of the tokens t .. t + 31 draft i sees, a bit each.
  __device__ __forceinline__ uint32_t sees_of_32(const DraftParams& p, int i, int t, int base) const {
    const int first = max(from[i] - t, 0), last = min(base - t, 32);  // (context tokens: bits [first, last))
    uint32_t bits = first < last ? (~0u >> (32 - (last - first))) << first : 0u;
    const int j = t - base;  // bit k stands for draft j + k
    if (j > -32 && from[i] != kNever) {
      const int word = j >> 5;  // (rounded down: j may be negative)
      const uint32_t lo = word >= 0 && word < kDraftWords && word * 32 < p.drafts ? seen[i][word] : 0u;
      const uint32_t hi = word + 1 < kDraftWords && (word + 1) * 32 < p.drafts ? seen[i][word + 1] : 0u;
      bits |= __funnelshift_r(lo, hi, j & 31);
    }
    return bits;
  }
};

// ... where a row is that of many drafts: every warp of the launch takes some of
// their heads. (One CTA took 50 us to clear 24 drafts of 32 heads of 128.)
template <class T>
__device__ __forceinline__ void attend_empty_rows(const DraftParams& p, const AttendRows& s) {
  const int heads = p.kv_heads * p.group, groups = p.kv_heads * p.blocks, lane = threadIdx.x & 31;
  const int warps = blockDim.x >> 5, me = blockIdx.x * warps + (threadIdx.x >> 5);
  for (int r0 = 0; r0 < p.rows; r0 += 32) {
    uint32_t empty = __ballot_sync(~0u, r0 + lane < p.rows && s.at[min(r0 + lane, p.rows - 1) + 1] == s.at[min(r0 + lane, p.rows - 1)]);
    for (; empty; empty &= empty - 1) {
      const int r = r0 + __ffs(empty) - 1;
      for (int h = me; h < heads; h += gridDim.x * warps) {
        const AttendPlace at = attend_place(p, r, h);
        T* out = static_cast<T*>(p.out) + at.out;
        for (int d = lane; d < p.dim; d += 32) out[d] = from_float<T>(0.0f);
        if (p.lse && lane == 0) p.lse[at.lse] = -CUDART_INF_F;
      }
      if (p.split_by_row)
        for (int i = me * 32 + lane; i < groups; i += gridDim.x * warps * 32) p.splits[r * groups + i].parts = 0;
    }
  }
}

// A barrier of all threads of the CTA, and one of THREADS of them (whole warps).
struct WholeCta {
  static __device__ __forceinline__ void sync() { __syncthreads(); }
  static __device__ __forceinline__ bool any(bool x) { return __syncthreads_or(x); }
};
template <int THREADS, int ID>
struct SomeThreads {
  static __device__ __forceinline__ void sync() { asm volatile("bar.sync %0, %1;" ::"n"(ID), "n"(THREADS) : "memory"); }
  static __device__ __forceinline__ bool any(bool x) {
    uint32_t r;
    asm volatile("{\n .reg .pred p, q;\n setp.ne.u32 p, %1, 0;\n bar.red.or.pred q, %2, %3, p;\n selp.u32 %0, 1, 0, q;\n}\n"
                 : "=r"(r) : "r"((uint32_t)x), "n"(ID), "n"(THREADS) : "memory");
    return r != 0;
  }
};

// Fills s for a row whose drafts begin at `base`; THREADS threads, the
// CTA's first, call it. Ancestors are found by doubling: a draft's list takes in
// that of the draft it points to, which then points where that one did.
template <int THREADS, class B = WholeCta>
__device__ __forceinline__ void draft_tree(const DraftParams& p, DraftTree& s, int row, int base) {
  constexpr int kEach = (CMD_CACHE_MAX_DRAFTS + THREADS - 1) / THREADS;
  const int words = (p.drafts + 31) >> 5;
  B::sync();  // the tree before it is no longer read
  bool going = false;
#pragma unroll
  for (int e = 0; e < kEach; ++e) {
    const int i = threadIdx.x + e * THREADS;
    if (i >= p.drafts) break;
    int parent = -1;
    if (p.parents) {
      parent = p.parents[row * p.parent_st[0] + i * p.parent_st[1]];
      if (parent >= i) {
        report(p.status, CMD_CACHE_BAD_INDEX);
        parent = -2;
      }
      parent = max(parent, -2);
      for (int w = 0; w < words; ++w) s.seen[i][w] = w == i >> 5 ? 1u << (i & 31) : 0u;
    } else {
      for (int w = 0; w < words; ++w) s.seen[i][w] = w < i >> 5 ? ~0u : w == i >> 5 ? ~0u >> (31 - (i & 31)) : 0u;
    }
    s.from[i] = parent;
    going = going || parent >= 0;
  }
  while (B::any(going)) {
    uint32_t add[kEach][kDraftWords];
    int next[kEach];
#pragma unroll
    for (int e = 0; e < kEach; ++e) {
      const int i = threadIdx.x + e * THREADS;
      next[e] = -1;
      if (i >= p.drafts) break;
      const int at = s.from[i];
      next[e] = at;
#pragma unroll
      for (int w = 0; w < kDraftWords; ++w) add[e][w] = at >= 0 && w < words ? s.seen[at][w] : 0u;
      if (at >= 0) next[e] = s.from[at];
    }
    B::sync();
    going = false;
#pragma unroll
    for (int e = 0; e < kEach; ++e) {
      const int i = threadIdx.x + e * THREADS;
      if (i >= p.drafts) break;
#pragma unroll
      for (int w = 0; w < kDraftWords; ++w)
        if (w < words) s.seen[i][w] |= add[e][w];
      s.from[i] = next[e];
      going = going || next[e] >= 0;
    }
  }
#pragma unroll
  for (int e = 0; e < kEach; ++e) {
    const int i = threadIdx.x + e * THREADS;
    if (i >= p.drafts) break;
    int depth = -1;
    for (int w = 0; w < words; ++w) depth += __popc(s.seen[i][w]);
    s.depth[i] = depth;
    s.from[i] = s.from[i] == -2 ? kNever : p.near ? max(0, base + depth + 1 - p.near) : 0;
  }
  B::sync();
  if (p.near && p.near < p.drafts) {  // (a chain of ancestors may be longer than the window)
    for (int e = 0; e < kEach; ++e) {
      const int i = threadIdx.x + e * THREADS;
      if (i >= p.drafts) break;
      for (int w = 0; w < words; ++w) {
        uint32_t mine = s.seen[i][w];
        for (uint32_t rest = mine; rest; rest &= rest - 1) {
          const int j = __ffs(rest) - 1;
          if (s.depth[i] - s.depth[32 * w + j] >= p.near) mine &= ~(1u << j);
        }
        s.seen[i][w] = mine;
      }
    }
    B::sync();
  }
}

// Whether every draft sees every token of [t, end) of a row.
__device__ __forceinline__ bool draft_all_seen(const DraftParams& p, int t, int end, int base) {
  return end <= base && (p.near == 0 || t >= base + p.drafts - p.near);
}

// Where a tile's tokens lie: offsets (in elements, for one kv head) of their
// keys and values, -1 for none. The thread of each token looks it up a tile
// before the copies that need it.
template <int TOKENS>
struct DraftTile {
  int64_t k[TOKENS], v[TOKENS];
  uint32_t here[(TOKENS + 31) / 32];
};
struct DraftLook {
  int page, slot;
  bool inside;
};
__device__ __forceinline__ DraftLook draft_look(const DraftParams& p, const AttendSegment& g, int tile, int tokens, bool valid) {
  DraftLook x = {0, 0, false};
  const int t = tile * tokens + (int)threadIdx.x;
  if (valid && (int)threadIdx.x < tokens && t >= g.lo && t < g.n) {
    const uint32_t column = fast_div32(p.page, (uint32_t)t);
    x.inside = true;
    x.slot = t - (int)(column * p.page.d);
    x.page = p.tables[g.row * p.table_st[0] + column * p.table_st[1]];
  }
  return x;
}
template <int TOKENS>
__device__ __forceinline__ void draft_place(const DraftParams& p, DraftTile<TOKENS>& s, const DraftLook& x, int kv) {
  if ((int)threadIdx.x >= (TOKENS + 31) / 32 * 32) return;  // (whole warps)
  bool in = x.inside;
  if (in && (x.page < 0 || x.page >= p.n_pages)) {
    report(p.status, CMD_CACHE_BAD_PAGE);
    in = false;
  }
  if ((int)threadIdx.x < TOKENS) {
    s.k[threadIdx.x] = in ? x.page * p.k_st[0] + x.slot * p.k_st[1] + kv * p.k_st[2] : -1;
    s.v[threadIdx.x] = in ? x.page * p.v_st[0] + x.slot * p.v_st[1] + kv * p.v_st[2] : -1;
  }
  const uint32_t here = __ballot_sync(~0u, in);
  if (threadIdx.x % 32 == 0) s.here[threadIdx.x / 32] = here;
}

// Query row q (of the kv head's) of a row of the batch.
template <class T>
__device__ __forceinline__ const T* draft_query(const DraftParams& p, int row, int kv, int q) {
  const int draft = (int)fast_div32(p.per, (uint32_t)q), head = kv * (int)p.per.d + q - draft * (int)p.per.d;
  return static_cast<const T*>(p.q) + row * p.q_st[0] + draft * p.q_draft + head * p.q_st[1];
}

}  // namespace cmdx
