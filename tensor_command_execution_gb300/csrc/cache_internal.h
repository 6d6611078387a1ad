// cache_internal.h - launch parameters of the cache operators' kernels, shared
// by their host side (cache_api.cpp) and the CUDA sources (cache_*.cu). Not
// public.
#pragma once

#include <cstdint>

#include <cuda_runtime.h>

#include "../../include/cmd_cache.h"

namespace cmdx {

// Unsigned 32-bit division by an invariant divisor with a multiply-high
// (Granlund and Montgomery, PLDI 1994, section 4, as FastDiv in
// cmd_internal.h): l = 0 marks a divisor of 1.
struct FastDiv32 {
  uint32_t m, l, d;
};
inline FastDiv32 fast_div_by(uint32_t d) {
  FastDiv32 f = {0, 0, d};
  if (d < 2) return f;
  while ((uint64_t(1) << f.l) < d) ++f.l;
  f.m = (uint32_t)(((uint64_t(1) << 32) * ((uint64_t(1) << f.l) - d)) / d + 1);
  return f;
}

// ---- rotation and append (cache_rope.cu) --------------------------------------
// What a tensor of the launch is: rotated or copied, into a tensor or into a
// cache's pages.
struct RopeStream {
  const void* in;
  void* out;           // a tensor's first element, or the pool's
  int64_t in_st[3];    // batch, token, head strides (elements)
  int64_t out_st[3];   // the same of a tensor; page, slot, head of a pool
  int32_t heads;
  uint8_t rotate, cache;
};

struct RopeParams {
  RopeStream s[3];
  int32_t n_streams;
  int32_t heads;       // of all streams together
  const int32_t* positions;
  int64_t pos_st[2];   // batch, token
  const uint64_t* turns;
  int32_t n_pairs;
  int32_t dim;
  float scale, sine_scale;  // of the cosine; of the sine (negative: backward)
  int64_t tokens;      // per batch
  FastDiv32 per_batch; // by that number
  int32_t batch;
  // the cache (append)
  const int32_t* tables;
  const int32_t* rows;
  int64_t table_st[2], rows_st;
  int32_t n_rows, columns, n_pages;  // (columns -1: no cache)
  FastDiv32 page;
  int32_t* status;
};

// bytes: 16, 8 or 4 where every row of every stream may be accessed so many at
// a time and every stride is below 2^31, else 0
cudaError_t rope_launch(int dtype, int layout, int bytes, const RopeParams& p, cudaStream_t stream);

// ---- attention of one token (cache_attend*.cu) --------------------------------
constexpr int kAttendMaxCtas = 152 * 4;  // bounds the workspace
constexpr int kAttendRows = 512;         // rows of one launch, at most (the host splits larger calls)
constexpr int kAttendLeastTile = 32;     // tokens of a CTA's tile, at least, and
constexpr int kAttendMostStart = 4;      // units of a row's beginning, at most: they bound a launch's units

// A row (for one kv head and block of query heads) whose tiles went to several
// CTAs: part k lies at index `first` for k = 0, (first & ~1) + 2 k sides after.
struct AttendSplit {
  int32_t row, group, first;
  int32_t parts;  // 0: none
};

struct AttendParams {
  const void* q;
  void* out;
  float* lse;
  const void* k;
  const void* v;
  const int32_t* tables;
  const int32_t* lengths;
  int64_t q_st[2], out_st[2], lse_st[2];  // row, head
  int64_t k_st[3], v_st[3];               // page, slot, head
  int64_t table_st[2], len_st;
  int32_t rows, kv_heads, group, dim;
  int32_t n_pages, columns;
  FastDiv32 page;
  float scale_log2;    // scale * log2 e: scores are kept in powers of two
  float cap_in, cap_out;  // scale / softcap, softcap * log2 e (cap_out 0: none)
  int32_t window;
  int32_t blocks;      // blocks of query heads of one kv head
  int32_t block_heads; // query heads of a block (the last may have fewer)
  float* parts;        // partial results, [2 CTAs][block_heads][attend_pitch(dim)]
  AttendSplit* splits; // one for each CTA, or for each row and group
  int32_t tasks;       // of the join
  int32_t start_units; // what the beginning of a row counts, in tiles
  int32_t sides;       // groups whose CTAs work side by side: all of them, or 1: units of all groups are shared
  int32_t team;        // CTAs of a cluster that takes one row and group; 0: units are dealt out evenly
  uint8_t split_by_row;
  int32_t* status;
  uint8_t q_pairs;     // q rows may be read two 16-bit elements at a time
};

// 16-bit types whose cache rows are not whole 4-byte words; at most 8 query
// heads of a block
cudaError_t attend_simt_launch(int dtype, const AttendParams& p, cudaStream_t stream);
// the others, with rows of whole 16-byte or 4-byte pieces: 32-bit, at most 8
// query heads of a block; 16-bit, at most 16
#define CMDX_COPY_NAME_(f, n) f##n
#define CMDX_COPY_NAME__(f, n) CMDX_COPY_NAME_(f, n)
#define CMDX_COPY_NAME(f) CMDX_COPY_NAME__(f, CMDX_COPY)
cudaError_t attend_f32_launch16(const AttendParams& p, cudaStream_t stream);
cudaError_t attend_f32_launch4(const AttendParams& p, cudaStream_t stream);
cudaError_t attend_mma_launch16(int dtype, const AttendParams& p, cudaStream_t stream);
cudaError_t attend_mma_launch4(int dtype, const AttendParams& p, cudaStream_t stream);
constexpr int kAttendHeads = 8, kAttendMmaHeads = 16;

// ---- pages (cache_pages.cu) -----------------------------------------------------
// The pools of a call; MAX of them at most (a launch's parameters are copied
// to the device with it, so few pools go in a short list).
template <int MAX>
struct PoolListOf {
  uint8_t* ptr[MAX];
  int64_t stride[MAX];
  int64_t bytes[MAX];
  int32_t n;
  int32_t unit;        // bytes of one access: every address and size is a multiple of it
};
using PoolList = PoolListOf<CMD_CACHE_MAX_POOLS>;

struct SelectParams {
  const int32_t *tables, *lengths, *refs, *parents, *grow;
  int32_t *tables_out, *lengths_out, *refs_out;
  int64_t table_st, table_out_st;  // rows; a row's entries are dense
  int32_t old_rows, new_rows, columns, pages;
  FastDiv32 page;
  int32_t *first, *children, *keep, *base, *free_list, *copy_src, *copy_dst, *head;  // workspace
  int32_t* status;
};

struct CompactParams {
  const int32_t *tables, *lengths, *refs;
  int32_t *tables_out, *refs_out, *map_out;
  int64_t table_st, table_out_st;
  int32_t rows, columns, pages;
  FastDiv32 page;
  int32_t *holes, *movers, *head;  // workspace
  int32_t* status;
};

cudaError_t select_launch(const SelectParams& p, const PoolList& pools, cudaStream_t stream);
cudaError_t status_clear_launch(int32_t* status, int32_t bits, cudaStream_t stream);
cudaError_t compact_launch(const CompactParams& p, const PoolList& pools, cudaStream_t stream);

}  // namespace cmdx
