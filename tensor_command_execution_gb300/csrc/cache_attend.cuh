// cache_attend.cuh - how the one-token attention's work is split and joined,
// shared by its kernels.
//
// A unit of work is a tile of tokens of one row and one group of heads. The
// units of a launch, ordered by row, then head group, then token, are cut
// into equal runs, one for each CTA, whatever the rows' lengths: no CTA waits
// for a long row. A CTA whose run holds all of a row's tiles writes the
// result; one that holds some writes a partial result (running maximum, sum
// and weighted values) to the workspace, and the CTA that arrives last at a
// row's counter joins the row's parts, in their order, so that the result does
// not depend on which CTA that was. At most two of a CTA's segments are
// partial (its first and its last), so the workspace does not grow with the
// rows.
#pragma once

#include <math_constants.h>

#include "cache_common.cuh"

namespace cmdx {

// Where each row's units begin (in units of one head group), in shared memory.
struct AttendSpan {
  int64_t at[kAttendRows + 1];
};

// Row r's tokens [lo, n) that are attended to.
__device__ __forceinline__ void attend_range(const AttendParams& p, int r, int* lo, int* n) {
  int64_t len = p.lengths[r * p.len_st];
  const int64_t most = (int64_t)p.columns * p.page.d;
  if (len < 0 || len > most) {
    if (blockIdx.x == 0) report(p.status, CMD_CACHE_BAD_INDEX);
    len = len < 0 ? 0 : most;
  }
  *n = (int)len;
  *lo = p.window > 0 && len > p.window ? (int)(len - p.window) : 0;
}

// The rows' first units for tiles of `tile` tokens (aligned to the row's
// start), by all threads of the CTA (256 of them or fewer).
__device__ __forceinline__ void attend_spans(const AttendParams& p, AttendSpan& s, int tile) {
  __shared__ int64_t s_warp[32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int run = (p.rows + blockDim.x - 1) / blockDim.x;
  const int r0 = min(tid * run, p.rows), r1 = min(r0 + run, p.rows);
  int64_t sum = 0;
  for (int r = r0; r < r1; ++r) {
    int lo, n;
    attend_range(p, r, &lo, &n);
    s.at[r + 1] = n > lo ? (n + tile - 1) / tile - lo / tile : 0;
    sum += s.at[r + 1];
  }
  int64_t incl = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t y = __shfl_up_sync(~0u, incl, o);
    if (lane >= o) incl += y;
  }
  if (lane == 31) s_warp[warp] = incl;
  __syncthreads();
  int64_t at = incl - sum;
  for (int w = 0; w < warp; ++w) at += s_warp[w];
  if (tid == 0) s.at[0] = 0;
  for (int r = r0; r < r1; ++r) {
    at += s.at[r + 1];
    s.at[r + 1] = at;
  }
  __syncthreads();
}

// A CTA's share of a launch.
struct AttendShare {
  int64_t units, ctas, begin, end;
};
__device__ __forceinline__ AttendShare attend_share(const AttendParams& p, const AttendSpan& s) {
  AttendShare w;
  w.units = s.at[p.rows] * ((p.kv_heads / p.heads_per_cta) * p.blocks);
  w.ctas = w.units < gridDim.x ? w.units : gridDim.x;
  w.begin = w.ctas ? blockIdx.x * w.units / w.ctas : 0;
  w.end = blockIdx.x < w.ctas ? (blockIdx.x + 1) * w.units / w.ctas : w.begin;
  return w;
}
// The CTA that works on unit u.
__device__ __forceinline__ int attend_owner(const AttendShare& w, int64_t u) {
  return (int)(((u + 1) * w.ctas - 1) / w.units);
}

// A stretch of one row's tiles for one head group.
struct AttendSegment {
  int row, head0, qblock;   // first kv head, block of query heads
  int lo, n;                // the row's tokens
  int tile0, tiles;         // this stretch, in tiles from the row's start
  int64_t first, last;      // the first and last unit of the row and head group
  int64_t unit;             // the stretch's first unit
  bool whole;
};
__device__ __forceinline__ AttendSegment attend_segment(const AttendParams& p, const AttendSpan& s, const AttendShare& w,
                                                        int64_t u, int tile) {
  const int groups = (p.kv_heads / p.heads_per_cta) * p.blocks;
  const int64_t x = u / groups;
  int a = 0, b = p.rows;  // the last row that begins at or before x
  while (b - a > 1) {
    const int m = (a + b) >> 1;
    if (s.at[m] <= x) a = m; else b = m;
  }
  AttendSegment g;
  g.row = a;
  const int64_t row_tiles = s.at[a + 1] - s.at[a];
  const int64_t in_row = u - s.at[a] * groups;
  const int group = (int)(in_row / row_tiles);
  const int64_t t = in_row - group * row_tiles;
  g.head0 = group / p.blocks * p.heads_per_cta;
  g.qblock = group % p.blocks;
  attend_range(p, a, &g.lo, &g.n);
  g.tile0 = (int)(g.lo / tile + t);
  const int64_t left = w.end - u;
  g.tiles = (int)(row_tiles - t < left ? row_tiles - t : left);
  g.unit = u;
  g.first = u - t;
  g.last = g.first + row_tiles - 1;
  g.whole = g.tiles == row_tiles;
  return g;
}

// Rows with no tokens: zeros, and a log-sum of -infinity.
template <class T>
__device__ __forceinline__ void attend_empty_rows(const AttendParams& p, const AttendSpan& s) {
  const int heads = p.kv_heads * p.group;
  for (int r = blockIdx.x; r < p.rows; r += gridDim.x) {
    if (s.at[r + 1] != s.at[r]) continue;
    for (int i = threadIdx.x; i < heads * p.dim; i += blockDim.x) {
      const int h = i / p.dim;
      static_cast<T*>(p.out)[r * p.out_st[0] + h * p.out_st[1] + (i - h * p.dim)] = from_float<T>(0.0f);
    }
    if (p.lse)
      for (int h = threadIdx.x; h < heads; h += blockDim.x) p.lse[r * p.lse_st[0] + h * p.lse_st[1]] = -CUDART_INF_F;
  }
}

// The merged state of one query head over the warps that shared its tokens.
// o[] of a warp: unnormalised, relative to its maximum m (in powers of two;
// -infinity where it saw no token, with l and o zero).
__device__ __forceinline__ float attend_weight(float m, float top) {
  return m == -CUDART_INF_F ? 0.0f : exp2f(m - top);
}

// Writes the result of (row, kv head, query head g of its block), element d.
template <class T>
__device__ __forceinline__ void attend_write(const AttendParams& p, int row, int kv_head, int qblock, int g, int d,
                                             float top, float l, float o) {
  const int h = kv_head * p.group + qblock * p.block_heads + g;
  static_cast<T*>(p.out)[row * p.out_st[0] + h * p.out_st[1] + d] = from_float<T>(l == 0.0f ? 0.0f : o / l);
  if (d == 0 && p.lse)
    p.lse[row * p.lse_st[0] + h * p.lse_st[1]] = l == 0.0f ? -CUDART_INF_F : (top + log2f(l)) * CUDART_LN2_F;
}

// Ends a segment. The warps' states lie in shared memory: query head g of warp
// w has its m, its l and its o[dim] at state + w * warp_pitch + g * pitch. Warp
// w worked on kv head head0 + w % heads_per_cta and every (warps /
// heads_per_cta)-th tile. All threads call it.
template <class T>
__device__ __forceinline__ void attend_finish(const AttendParams& p, const AttendShare& w, const AttendSegment& g,
                                              const float* state, int warp_pitch, int pitch, int* s_last) {
  const int hw = p.heads_per_cta, phases = (int)(blockDim.x >> 5) / hw;
  const int gh = min(p.block_heads, p.group - g.qblock * p.block_heads);
  const int heads = hw * gh, dim = p.dim;
  const int part_pitch = dim + 2;
  const int64_t part_size = (int64_t)hw * p.block_heads * part_pitch;
  __syncthreads();  // the warps' states are complete
  float* part = nullptr;
  if (!g.whole) part = p.parts + (2 * (int64_t)blockIdx.x + (g.unit == w.begin ? 0 : 1)) * part_size;
  for (int i = threadIdx.x; i < heads * dim; i += blockDim.x) {
    const int hg = i / dim, d = i - hg * dim, hh = hg / gh, q = hg - hh * gh;
    const float* s = state + hh * warp_pitch + q * pitch;
    float top = -CUDART_INF_F;
    for (int t = 0; t < phases; ++t) top = fmaxf(top, s[t * hw * warp_pitch]);
    float l = 0.0f, o = 0.0f;
    for (int t = 0; t < phases; ++t) {
      const float* x = s + t * hw * warp_pitch;
      const float c = attend_weight(x[0], top);
      l = fmaf(x[1], c, l);
      o = fmaf(x[2 + d], c, o);
    }
    if (part) {
      float* x = part + (hh * p.block_heads + q) * part_pitch;
      if (d == 0) {
        x[0] = top;
        x[1] = l;
      }
      x[2 + d] = o;
    } else {
      attend_write<T>(p, g.row, g.head0 + hh, g.qblock, q, d, top, l, o);
    }
  }
  if (part) {
    const int c0 = attend_owner(w, g.first), c1 = attend_owner(w, g.last);
    const int groups = (p.kv_heads / hw) * p.blocks;
    int32_t* arrived = p.arrived + (int64_t)g.row * groups + g.head0 / hw * p.blocks + g.qblock;
    __threadfence();
    __syncthreads();
    if (threadIdx.x == 0) {
      const int seen = atomicAdd(arrived, 1);
      *s_last = seen == c1 - c0;
      if (seen == c1 - c0) *arrived = 0;  // for the next launch
    }
    __syncthreads();
    if (*s_last) {
      __threadfence();
      // the first part is the second of its CTA unless that CTA's run begins with this row
      const int64_t begin0 = c0 * w.units / w.ctas;
      const float* first = p.parts + (2 * (int64_t)c0 + (begin0 == g.first ? 0 : 1)) * part_size;
      for (int i = threadIdx.x; i < heads * dim; i += blockDim.x) {
        const int hg = i / dim, d = i - hg * dim, hh = hg / gh, q = hg - hh * gh;
        const int64_t off = (hh * p.block_heads + q) * part_pitch;
        float top = __ldcg(first + off);
        float l = __ldcg(first + off + 1), o = __ldcg(first + off + 2 + d);
        for (int c = c0 + 1; c <= c1; ++c) {
          const float* x = p.parts + 2 * (int64_t)c * part_size + off;
          const float m = __ldcg(x), pl = __ldcg(x + 1), po = __ldcg(x + 2 + d);
          const float up = fmaxf(top, m);
          const float a = attend_weight(top, up), b = attend_weight(m, up);
          l = fmaf(l, a, pl * b);
          o = fmaf(o, a, po * b);
          top = up;
        }
        attend_write<T>(p, g.row, g.head0 + hh, g.qblock, q, d, top, l, o);
      }
    }
  }
  __syncthreads();  // the states may be overwritten
}

// A score in powers of two from a dot product.
__device__ __forceinline__ float attend_score(const AttendParams& p, float dot) {
  return p.cap_out != 0.0f ? p.cap_out * tanhf(dot * p.cap_in) : dot * p.scale_log2;
}

}  // namespace cmdx
