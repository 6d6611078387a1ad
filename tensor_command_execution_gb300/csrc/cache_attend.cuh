// cache_attend.cuh - how the one-token attention's work is split and joined,
// shared by its kernels.
//
// A unit of work is a tile of tokens of one row, for one kv head and a block
// of the query heads that share it; a CTA's warps share its tokens. The units
// of a launch, ordered by row, then head, then token, are cut into equal runs,
// one for each CTA, whatever the rows' lengths: no CTA waits for a long row.
// The beginning of a row counts as start_units more units (before its first
// tile; a CTA whose run ends with them does nothing for the row), since
// fetching queries and writing a result take as long as some tiles. A CTA
// whose run holds all of a row's tiles writes the result; one that holds some
// writes a part (maximum, sum and weighted values) to the workspace, and a
// second, small launch joins the parts of each split row in their order, so
// that the result does not depend on timing. At most two of a CTA's segments
// are parts (its first and its last), so the workspace does not grow with the
// rows, and at most one row that is split begins in a CTA, so neither does the
// list of them.
//
// Where the CTAs can be divided among the groups (`sides` of them), each group's
// CTAs share its units alone, so that the groups' CTAs walk the same tokens at
// the same time: where heads lie side by side in a page, a row of one head
// that is no whole number of 128-byte lines shares lines with the next head's.
//
// A few short rows are not worth that: there a cluster of CTAs (a team) takes
// each row and group and joins its parts through distributed shared memory,
// in the same launch and without the workspace.
#pragma once

#include <cooperative_groups.h>
#include <math_constants.h>

#include <type_traits>

#include "cache_common.cuh"

namespace cmdx {

// The rows of a launch, in shared memory: where each row's units begin (in
// units of one kv head and block of query heads), and the row's length.
struct AttendRows {
  int32_t at[kAttendRows + 4];  // (one more than the rows, and a multiple of 16 bytes)
  int32_t n[kAttendRows];
  __device__ __forceinline__ int lo(const AttendParams& p, int r) const {
    return p.window > 0 && n[r] > p.window ? n[r] - p.window : 0;
  }
};

// Row r's length, held to its table; none where its one draft is padding.
__device__ __forceinline__ int attend_length(const AttendParams& p, int r) {
  int n = p.lengths[r * p.len_st];
  const int most = p.columns * (int)p.page.d;
  if (n < 0 || n > most) {
    report(p.status, CMD_CACHE_BAD_INDEX);
    n = n < 0 ? 0 : most;
  }
  if (p.roots && n > 0) {
    const int parent = p.roots[r * p.root_st];
    if (parent >= 0) report(p.status, CMD_CACHE_BAD_INDEX);
    if (parent != -1) n = 0;
  }
  return n;
}

// Fills s for tiles of `tile` tokens (aligned to the row's start); all
// threads of the CTA call it. (The host sees to it that the units of a launch,
// of all heads, are below 2^31.)
template <class P>
__device__ __forceinline__ void attend_rows(const P& p, AttendRows& s, int tile) {
  __shared__ int32_t s_warp[32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int run = (p.rows + blockDim.x - 1) / blockDim.x;
  const int r0 = min(tid * run, p.rows), r1 = min(r0 + run, p.rows);
  int sum = 0;
  for (int r = r0; r < r1; ++r) {
    const int n = s.n[r] = attend_length(p, r);
    s.at[r + 1] = n > 0 ? (n + tile - 1) / tile - s.lo(p, r) / tile + p.start_units : 0;
    sum += s.at[r + 1];
  }
  int incl = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(~0u, incl, o);
    if (lane >= o) incl += y;
  }
  if (lane == 31) s_warp[warp] = incl;
  __syncthreads();
  int at = incl - sum;
  for (int w = 0; w < warp; ++w) at += s_warp[w];
  if (tid == 0) s.at[0] = 0;
  for (int r = r0; r < r1; ++r) {
    at += s.at[r + 1];
    s.at[r + 1] = at;
  }
  __syncthreads();
}

// A CTA's share of a launch: units [begin, end) of the `units` that it and
// ctas - 1 others share; it is the index-th of them.
struct AttendShare {
  int units, ctas, begin, end, index;
  int groups;  // groups (a kv head and a block of query heads) that these units are of,
  int group0;  // and the first of them
  // the first unit of CTA c: c * units / ctas (each < 2^31; the product of c and the remainder is small)
  __device__ __forceinline__ int begin_of(int c) const {
    const int each = units / ctas;
    return c * each + c * (units - each * ctas) / ctas;
  }
  // the CTA that works on unit u
  __device__ __forceinline__ int owner(int u) const { return (int)((((int64_t)u + 1) * ctas - 1) / units); }
};
__device__ __forceinline__ AttendShare attend_share(const AttendParams& p, const AttendRows& s) {
  AttendShare w;
  w.index = blockIdx.x / p.sides;
  w.group0 = blockIdx.x - w.index * p.sides;
  w.groups = p.kv_heads * p.blocks / p.sides;
  w.units = s.at[p.rows] * w.groups;
  w.ctas = min(w.units, (int)gridDim.x / p.sides);
  w.begin = w.end = 0;
  if (w.index < w.ctas) {
    w.begin = w.begin_of(w.index);
    w.end = w.begin_of(w.index + 1);
  }
  return w;
}

// A stretch of one row's tiles for one kv head and block of query heads.
struct AttendSegment {
  int row, group;           // group = kv head * blocks + block
  int lo, n;                // the row's tokens
  int tile0, tiles;         // this stretch, in tiles from the row's start; no tiles: the share has ended
  int first;                // the unit of the row's and group's first tile
  int row_tiles;            // and their number
  __device__ __forceinline__ bool whole() const { return tiles == row_tiles; }
};
// The stretch of row `row` and the share's group `group`, whose first unit is u, that lies in the share.
__device__ __forceinline__ AttendSegment attend_stretch(const AttendParams& p, const AttendRows& s, const AttendShare& w,
                                                        int u, int row, int group, int tile) {
  AttendSegment g;
  g.row = row;
  g.group = w.group0 + group;
  g.n = s.n[row];
  g.lo = s.lo(p, row);
  g.row_tiles = s.at[row + 1] - s.at[row] - p.start_units;
  g.first = u + p.start_units;
  const int from = max(w.begin, g.first), to = min(w.end, g.first + g.row_tiles);
  g.tile0 = g.lo / tile + from - g.first;
  g.tiles = max(to - from, 0);
  return g;
}
__device__ __forceinline__ AttendSegment attend_first(const AttendParams& p, const AttendRows& s, const AttendShare& w,
                                                      int tile) {
  const int x = w.begin / w.groups;
  int a = 0, b = p.rows;  // the last row that begins at or before x
  while (b - a > 1) {
    const int m = (a + b) >> 1;
    if (s.at[m] <= x) a = m; else b = m;
  }
  const int row_units = s.at[a + 1] - s.at[a], row0 = s.at[a] * w.groups;
  const int group = (w.begin - row0) / row_units;
  return attend_stretch(p, s, w, row0 + group * row_units, a, group, tile);
}
// The one after g (no tiles: there is none).
__device__ __forceinline__ AttendSegment attend_next(const AttendParams& p, const AttendRows& s, const AttendShare& w,
                                                     const AttendSegment& g, int tile) {
  const int u = g.first + g.row_tiles;
  int row = g.row, group = g.group - w.group0 + 1;
  if (u >= w.end) {
    AttendSegment none = g;
    none.tiles = 0;
    return none;
  }
  if (group == w.groups) {
    group = 0;
    do ++row;
    while (s.at[row + 1] == s.at[row]);
  }
  return attend_stretch(p, s, w, u, row, group, tile);
}

// The state of a query head over some of its tokens: the maximum m of the
// scores (in powers of two), the sum l of exp2(score - m) and the values
// weighted by the same, o[dim]. -infinity, zero and zeros for no token. In
// memory: o, then m and l at attend_pitch - 4 and - 3, all aligned to 16
// bytes.
__host__ __device__ constexpr int attend_pitch(int dim) { return (dim + 3) / 4 * 4 + 4; }

// What a state with maximum m weighs in one with maximum top.
__device__ __forceinline__ float attend_weight(float m, float top) {
  return m == -CUDART_INF_F ? 0.0f : exp2f(m - top);
}

__device__ __forceinline__ void add_scaled(float4& o, const float4& x, float c) {
  o.x = fmaf(x.x, c, o.x);
  o.y = fmaf(x.y, c, o.y);
  o.z = fmaf(x.z, c, o.z);
  o.w = fmaf(x.w, c, o.w);
}
__device__ __forceinline__ void scale_by(float4& o, float c) {
  o.x *= c;
  o.y *= c;
  o.z *= c;
  o.w *= c;
}

// Where query head h of a row is written (elements from out and lse), and what
// is kept of its maximum and sum.
struct AttendPlace {
  int64_t out, lse;
};
__device__ __forceinline__ AttendPlace attend_place(const AttendParams& p, int row, int h) {
  return {row * p.out_st[0] + h * p.out_st[1], row * p.lse_st[0] + h * p.lse_st[1]};
}
__device__ __forceinline__ void attend_note(const AttendParams& p, int row, int h, float top, float l) {
  if (p.stats) p.stats[(int64_t)row * p.kv_heads * p.group + h] = make_float2(top, l);
}
// Whether a part with this maximum says that its row is empty, whatever the others hold.
__device__ __forceinline__ bool attend_void(const AttendParams&, float) { return false; }

// Writes elements d .. d + 3 (those below dim) of a finished head. NOTE: its
// maximum and sum may be asked for.
template <class T, bool NOTE = true, class P>
__device__ __forceinline__ void attend_write(const P& p, int row, int h, int d, float top, float l, float4 o) {
  const AttendPlace at = attend_place(p, row, h);
  T* out = static_cast<T*>(p.out) + at.out + d;
  const float r = l == 0.0f ? 0.0f : 1.0f / l;
  if (l == 0.0f) o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  const float x[4] = {o.x, o.y, o.z, o.w};
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (d + i < p.dim) out[i] = from_float<T>(x[i] * r);
  if (d == 0 && p.lse) p.lse[at.lse] = l == 0.0f ? -CUDART_INF_F : (top + log2f(l)) * CUDART_LN2_F;
  if (NOTE && d == 0) attend_note(p, row, h, top, l);
}

// A segment's kv head and its query heads [head0, head0 + heads).
struct AttendHeads {
  int kv, head0, heads;
};
__device__ __forceinline__ AttendHeads attend_heads(const AttendParams& p, int group) {
  AttendHeads h;
  h.kv = group / p.blocks;
  h.head0 = h.kv * p.group + (group - h.kv * p.blocks) * p.block_heads;
  h.heads = min(p.block_heads, (h.kv + 1) * p.group - h.head0);
  return h;
}

// Elements d .. d + 3 of a head over the warps' states of it, WARPS of them
// warp_pitch apart; the maximum and sum in *top and *l.
template <int WARPS>
__device__ __forceinline__ float4 attend_merged(const float* s, int warp_pitch, int pitch, int d, float* top, float* l) {
  float m[WARPS];
  *top = -CUDART_INF_F;
  *l = 0.0f;
#pragma unroll
  for (int t = 0; t < WARPS; ++t) *top = fmaxf(*top, m[t] = s[t * warp_pitch + pitch - 4]);
  float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
  for (int t = 0; t < WARPS; ++t) {
    const float* x = s + t * warp_pitch;
    const float c = attend_weight(m[t], *top);
    *l = fmaf(x[pitch - 3], c, *l);
    add_scaled(o, *reinterpret_cast<const float4*>(x + d), c);
  }
  return o;
}

// Where a segment's part goes (NULL: the segment is all of its row and group);
// one thread says in the list of splits where the parts of a row that begins
// here are.
__device__ __forceinline__ float* attend_part(const AttendParams& p, const AttendShare& w, const AttendSegment& g, bool one) {
  const int slot = 2 * blockIdx.x + (g.first <= w.begin ? 0 : 1);
  float* part = g.whole() ? nullptr : p.parts + (int64_t)slot * p.block_heads * attend_pitch(p.dim);
  if (one && g.first >= w.begin) {
    AttendSplit split = {g.row, g.group, slot, 0};
    if (part) split.parts = w.owner(g.first + g.row_tiles - 1) - w.index + 1;
    if (p.split_by_row) p.splits[g.row * p.kv_heads * p.blocks + g.group] = split;
    else if (part) p.splits[blockIdx.x] = split;
  }
  return part;
}

// Ends a segment. The warps' states lie in shared memory, query head q of
// warp w (of WARPS that hold states of the same heads) at state + w *
// warp_pitch + q * pitch (pitch = attend_pitch of something at least dim). All
// threads call it, once their states are written.
template <class T, int WARPS, int THREADS = WARPS * 32, class P>
__device__ __forceinline__ void attend_finish(const P& p, const AttendShare& w, const AttendSegment& g,
                                              const AttendHeads& h, const float* state, int warp_pitch, int pitch) {
  const int part_pitch = attend_pitch(p.dim), quads = part_pitch / 4 - 1;
  float* part = attend_part(p, w, g, threadIdx.x == 0);
  __syncthreads();  // the warps' states are complete
  for (int i = threadIdx.x; i < h.heads * quads; i += THREADS) {
    const int q = i / quads, d = 4 * (i - q * quads);
    float top, l;
    const float4 o = attend_merged<WARPS>(state + q * pitch, warp_pitch, pitch, d, &top, &l);
    if (part) {
      float* x = part + q * part_pitch;
      if (d == 0) {
        x[part_pitch - 4] = top;
        x[part_pitch - 3] = l;
      }
      *reinterpret_cast<float4*>(x + d) = o;
    } else {
      attend_write<T>(p, g.row, h.head0 + q, d, top, l, o);
    }
  }
  __syncthreads();  // the states may be overwritten
}

// Zeros, and a log-sum of -infinity, for the rows without a token: a row to a CTA.
template <class T>
__device__ __forceinline__ void attend_empty_rows(const AttendParams& p, const AttendRows& s) {
  const int heads = p.kv_heads * p.group, groups = p.kv_heads * p.blocks;
  for (int r = blockIdx.x; r < p.rows; r += gridDim.x) {
    if (s.at[r + 1] != s.at[r]) continue;
    for (int i = threadIdx.x; i < heads * p.dim; i += blockDim.x) {
      const int h = i / p.dim;
      static_cast<T*>(p.out)[r * p.out_st[0] + h * p.out_st[1] + (i - h * p.dim)] = from_float<T>(0.0f);
    }
    if (p.lse)
      for (int h = threadIdx.x; h < heads; h += blockDim.x) p.lse[r * p.lse_st[0] + h * p.lse_st[1]] = -CUDART_INF_F;
    if (p.split_by_row)
      for (int i = threadIdx.x; i < groups; i += blockDim.x) p.splits[r * groups + i].parts = 0;
  }
}

// What a CTA does before its first segment: the rows, those of them that are
// empty (zeros, and a log-sum of -infinity), and its share. False: no work.
template <class T, class P>
__device__ __forceinline__ bool attend_begin(const P& p, AttendRows& s, int tile, AttendShare* w) {
  attend_rows(p, s, tile);
  attend_empty_rows<T>(p, s);
  *w = attend_share(p, s);
  if (!p.split_by_row && threadIdx.x == 0) p.splits[blockIdx.x].parts = 0;  // (unless a row is split here, below)
  return w->begin != w->end;
}

// A team's CTA: its stretch of the team's row and group (no tiles where the row
// is short), and a share that ends with it.
template <class P>
__device__ __forceinline__ AttendSegment attend_team(const P& p, int tile, AttendShare* w) {
  const int team = blockIdx.x / p.team, rank = blockIdx.x - team * p.team;
  w->groups = p.kv_heads * p.blocks;
  w->units = w->ctas = w->begin = w->end = w->index = w->group0 = 0;
  AttendSegment g;
  g.row = team / w->groups;
  g.group = team - g.row * w->groups;
  g.n = attend_length(p, g.row);
  g.lo = p.window > 0 && g.n > p.window ? g.n - p.window : 0;
  const int all = g.n > 0 ? (g.n + tile - 1) / tile - g.lo / tile : 0;
  const int each = all / p.team, more = all - each * p.team;  // the first `more` CTAs take one more
  g.tile0 = g.lo / tile + rank * each + min(rank, more);
  g.tiles = each + (rank < more);
  g.first = 0;
  g.row_tiles = 0;
  return g;
}

// Joins a team's row: every CTA's `part` holds its states of the heads, and the
// CTAs of the team write the result, a run of elements each. Every thread of
// the team calls it.
template <class T, int THREADS, class P>
__device__ __forceinline__ void attend_join_team(const P& p, const AttendSegment& g, const AttendHeads& h, float* part) {
  namespace cg = cooperative_groups;
  const cg::cluster_group team = cg::this_cluster();
  const int part_pitch = attend_pitch(p.dim), quads = part_pitch / 4 - 1;
  team.sync();
  constexpr int kMost = 8;
  const int rank = blockIdx.x % p.team;
  for (int i = rank * THREADS + threadIdx.x; i < h.heads * quads; i += p.team * THREADS) {
    const int q = i / quads, d = 4 * (i - q * quads);
    float m[kMost], pl[kMost], top = -CUDART_INF_F, l = 0.0f;
    float4 po[kMost], o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    bool empty = false;
#pragma unroll
    for (int k = 0; k < kMost; ++k) {
      m[k] = -CUDART_INF_F;
      if (k < p.team) {
        const float* x = team.map_shared_rank(part, k) + q * part_pitch;
        m[k] = x[part_pitch - 4];
        pl[k] = x[part_pitch - 3];
        po[k] = *reinterpret_cast<const float4*>(x + d);
      }
      top = fmaxf(top, m[k]);
      empty = empty || attend_void(p, m[k]);
    }
#pragma unroll
    for (int k = 0; k < kMost; ++k)
      if (k < p.team) {
        const float c = attend_weight(m[k], top);
        l = fmaf(pl[k], c, l);
        add_scaled(o, po[k], c);
      }
    if (empty) l = 0.0f;
    attend_write<T>(p, g.row, h.head0 + q, d, top, l, o);
  }
  team.sync();  // nobody leaves while its part is read
}

// Ends a team's row: the warps' states (as in attend_finish) go to `part` of
// each CTA, and are joined. Every thread of the team calls it.
template <class T, int WARPS, int THREADS = WARPS * 32, class P>
__device__ __forceinline__ void attend_finish_team(const P& p, const AttendSegment& g, const AttendHeads& h, const float* state,
                                                   int warp_pitch, int pitch, float* part) {
  const int part_pitch = attend_pitch(p.dim), quads = part_pitch / 4 - 1;
  __syncthreads();  // the warps' states are complete
  for (int i = threadIdx.x; i < h.heads * quads; i += THREADS) {
    const int q = i / quads, d = 4 * (i - q * quads);
    float top, l;
    const float4 o = attend_merged<WARPS>(state + q * pitch, warp_pitch, pitch, d, &top, &l);
    float* x = part + q * part_pitch;
    if (d == 0) {
      x[part_pitch - 4] = top;
      x[part_pitch - 3] = l;
    }
    *reinterpret_cast<float4*>(x + d) = o;
  }
  attend_join_team<T, THREADS>(p, g, h, part);
}

// Joins the parts of query head q of a split row: WARPS warps take every
// WARPS-th run of 8 parts, a lane 4 elements of the head (and 128 further).
template <class T, int WARPS, bool NOTE, class P>
__device__ __forceinline__ void attend_join(const P& p, int task, float (*s_state)[CMD_CACHE_MAX_DIM + 4]) {
  constexpr int kAtOnce = 8;
  constexpr bool kVoid = !std::is_same<P, AttendParams>::value;  // (attend_void may be true)
  const int lane = threadIdx.x & 31, warp = WARPS == 1 ? 0 : threadIdx.x >> 5;
  const AttendSplit split = p.splits[task / p.block_heads];
  const int q = task % p.block_heads;
  if (split.parts == 0) return;
  const AttendHeads h = attend_heads(p, split.group);
  if (q >= h.heads) return;
  const int pitch = attend_pitch(p.dim);
  const int64_t size = (int64_t)p.block_heads * pitch;
  const float* base = p.parts + (int64_t)q * pitch;
  for (int d = 4 * lane; d < pitch - 4 || WARPS > 1; d += 128) {
    if (WARPS > 1 && d - 4 * lane >= pitch - 4) break;  // (the same for all of the CTA)
    const bool mine = d < pitch - 4;
    float top = -CUDART_INF_F, l = 0.0f;
    bool empty = false;
    float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    for (int c = warp * kAtOnce; c < split.parts; c += WARPS * kAtOnce) {
      float m[kAtOnce], pl[kAtOnce];
      float4 po[kAtOnce];
#pragma unroll
      for (int k = 0; k < kAtOnce; ++k) {
        const float* x = base + (c + k == 0 ? split.first : (split.first & ~1) + 2 * (int64_t)(c + k) * p.sides) * size;
        m[k] = -CUDART_INF_F;
        if (c + k < split.parts && mine) {
          m[k] = x[pitch - 4];
          pl[k] = x[pitch - 3];
          po[k] = *reinterpret_cast<const float4*>(x + d);
        }
      }
      float up = top;
#pragma unroll
      for (int k = 0; k < kAtOnce; ++k) {
        up = fmaxf(up, m[k]);
        empty = empty || attend_void(p, m[k]);
      }
      const float a = attend_weight(top, up);
      l *= a;
      scale_by(o, a);
      top = up;
#pragma unroll
      for (int k = 0; k < kAtOnce; ++k)
        if (c + k < split.parts && mine) {
          const float b = attend_weight(m[k], up);
          l = fmaf(pl[k], b, l);
          add_scaled(o, po[k], b);
        }
    }
    if (kVoid && empty) top = CUDART_NAN_F;  // (a maximum is never that)
    if constexpr (WARPS > 1) {
      if (mine) {
        *reinterpret_cast<float4*>(&s_state[warp][d]) = o;
        if (d == 0) {
          s_state[warp][CMD_CACHE_MAX_DIM] = top;
          s_state[warp][CMD_CACHE_MAX_DIM + 1] = l;
        }
      }
      __syncthreads();
      if (warp == 0 && mine) {
        top = -CUDART_INF_F;
#pragma unroll
        for (int t = 0; t < WARPS; ++t) {
          const float x = s_state[t][CMD_CACHE_MAX_DIM];
          top = fmaxf(top, x);
          if (kVoid) empty = empty || x != x;
        }
        l = 0.0f;
        o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
        for (int t = 0; t < WARPS; ++t) {
          const float c = attend_weight(s_state[t][CMD_CACHE_MAX_DIM], top);
          l = fmaf(s_state[t][CMD_CACHE_MAX_DIM + 1], c, l);
          add_scaled(o, *reinterpret_cast<const float4*>(&s_state[t][d]), c);
        }
      }
      // (a second run of dims reads the m and l that the first wrote, unchanged)
    }
    if (empty) l = 0.0f;
    if (warp == 0 && mine) attend_write<T, NOTE>(p, split.row, h.head0 + q, d, top, l, o);
  }
}

template <class T, int WARPS, bool NOTE, class P>
__global__ void __launch_bounds__(WARPS == 1 ? 256 : WARPS * 32) attend_join_kernel(const __grid_constant__ P p) {
  __shared__ __align__(16) float s_state[WARPS == 1 ? 1 : WARPS][CMD_CACHE_MAX_DIM + 4];
  wait_for_previous();
  let_next_start();
  const int task = WARPS == 1 ? blockIdx.x * 8 + (threadIdx.x >> 5) : blockIdx.x;
  if (task < p.tasks) attend_join<T, WARPS, NOTE>(p, task, s_state);
}

// CTAs of the teams of a launch of tiles of `tile` tokens, 0 for none: up to 8
// for each row and group, where a CTA has four tiles at most and the teams
// leave a third of the device's places (`ctas`) free. Measured against units
// dealt out evenly, bf16, 8 kv heads of 128, 64 tokens to a tile: one row of 64
// tokens 4.3 and 5.1 us, 700 6.6 and 8.3, 2000 (4 tiles) 8.4 and 9.3, 4000 (8
// tiles) 12.3 and 10.8; 4 rows of 1000 (256 CTAs of 456) 8.8 and 11.9, 14 of
// 250 (448) 10.8 and 10.5, 7 of 2000 (448) 22.1 and 18.1; dim 256, 2 rows of
// 900 (128 of 152) 16.5 and 14.4.
constexpr int kTeamTiles = 4;

inline int attend_team_size(const AttendParams& p, int ctas, int tile) {
  int64_t most = (int64_t)p.columns * p.page.d;
  if (p.window > 0) most = most < p.window ? most : p.window;
  const int64_t tiles = (most + tile - 1) / tile + (p.window > 0);  // (a window may begin inside a tile)
  int team = 1;
  while (team < 8 && team < tiles) team *= 2;
  return tiles <= team * kTeamTiles && (int64_t)p.rows * p.kv_heads * p.blocks * team * 3 <= ctas * 2 ? team : 0;
}

// The CTAs of a launch of at most `ctas`, and how many groups work side by side:
// all groups, where that leaves at most a twentieth of the places
// empty. Measured on 64 rows of 4096 tokens, 8 kv heads (bf16, heads side by
// side in a page), against units of all groups in one order: dim 72 (144-byte
// rows) 119 and 159 us, 96 138 and 165, 128 176.5 and 179.5, f32 of 72 189 and
// 233; heads outermost, dim 128, 180 and 182.5; 64 ragged rows 48.5 and 48.5.
inline int attend_sides(int groups, int ctas, int32_t* sides) {
  *sides = ctas / groups * groups * 20 >= ctas * 19 ? groups : 1;
  return *sides > 1 ? ctas / groups * groups : ctas;
}

// Launches a kernel of `ctas` CTAs of `threads` threads that splits its work
// as above in tiles of `tile` tokens (teams: it can also work in teams), and
// the join. The joining warps: 16 to a
// head where few rows can have many parts each, one where each has few.
// Measured, one against 16, whole calls: one row of 393217 tokens and one kv
// head (456 parts) 116 and 47.7 us; one of 32768 and 8 kv heads 39.3 and 30.2;
// four of those 93.5 and 94.5; 64 rows of 4096 tokens 179 and 227.
template <class T, class K, class P>
cudaError_t attend_launch(K kernel, P p, int start_units, int ctas, int threads, int smem, int tile,
                          cudaStream_t stream, bool teams = true) {
  p.start_units = start_units;
  p.team = teams ? attend_team_size(p, ctas, tile) : 0;
  if (p.team)
    return launch_clusters(kernel, p.team, p.rows * p.kv_heads * p.blocks * p.team, threads, (size_t)smem, stream, p);
  const int groups = p.kv_heads * p.blocks;
  const int64_t rows = (int64_t)p.rows * groups;
  ctas = attend_sides(groups, ctas, &p.sides);
  p.split_by_row = rows <= ctas;
  const int lists = p.split_by_row ? (int)rows : ctas;
  p.tasks = lists * p.block_heads;
  cudaError_t e = launch_chained(kernel, ctas, threads, (size_t)smem, stream, p);
  if (e != cudaSuccess || (int64_t)p.columns * p.page.d <= tile) return e;  // (a row of one tile is never split)
  const auto join = [&](auto note) {
    if (lists * 16 <= ctas) return launch_chained(attend_join_kernel<T, 16, note, P>, p.tasks, 512, 0, stream, p);
    return launch_chained(attend_join_kernel<T, 1, note, P>, (p.tasks + 7) / 8, 256, 0, stream, p);
  };
  // (of one token's attention the maxima and sums are seldom wanted, and the join that may note them spills registers)
  if (std::is_same<P, AttendParams>::value && !p.stats) return join(std::integral_constant<bool, !std::is_same<P, AttendParams>::value>());
  return join(std::true_type());
}

// A score in powers of two from a dot product.
__device__ __forceinline__ float attend_score(const AttendParams& p, float dot) {
  return p.cap_out != 0.0f ? p.cap_out * tanhf(dot * p.cap_in) : dot * p.scale_log2;
}

}  // namespace cmdx
