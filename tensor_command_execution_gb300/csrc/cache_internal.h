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
  float2* stats;       // optional: a row's maximum and sum for each head, [rows][kv_heads * group]
  float* scores;       // optional (16-bit types, copies of 16 bytes): every token's, [rows][kv_heads][scores_tokens][group]
  int64_t scores_tokens;
  const int32_t* roots;  // optional: a row where this is not -1 is as one without a token
  int64_t root_st;
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

// ---- attention of drafted tokens (cache_drafts*.cu) ----------------------------
// The attention above with drafts * (query heads to a kv head) rows in the
// place of a kv head's query heads: `group` counts them, draft outermost.
// lengths include the drafts; `window` reaches from the last token back to the
// first that any draft sees. One draft is one token's attention, of the rows
// where its parent is -1 (roots).
struct DraftParams : AttendParams {
  int32_t drafts;
  FastDiv32 per;              // by query heads to a kv head
  int64_t q_draft, out_draft, lse_draft;  // strides of the drafts
  const int32_t* parents;     // NULL: each draft goes on from the one before
  int64_t parent_st[2];
  int32_t near;               // the caller's window, 0: none
  float* weights;             // optional: [rows, kv heads, tokens], added to
  int64_t w_st[2];
  uint8_t q_vectors, out_vectors;  // their rows may be accessed 16 bytes at a time
};
// CTAs of a launch and rows of a block, at most: they bound the workspace
constexpr int kDraftCtas = 152 * 2, kDraftRows = 64;
constexpr int kDraftTcCtas = 152, kDraftTcRows = 256;
// copy: bytes of a copy that suits every row of the cache, 16 or 4, or 0
cudaError_t drafts_mma_launch16(int dtype, const DraftParams& p, cudaStream_t stream);
cudaError_t drafts_mma_launch4(int dtype, const DraftParams& p, cudaStream_t stream);
cudaError_t drafts_mma_launch0(int dtype, const DraftParams& p, cudaStream_t stream);
// 16-byte copies, dims up to 128; by TMA, where pages of `sizes` and these
// strides (page, slot, head, dim; elements) in device memory suit it
cudaError_t drafts_tc_launch(int dtype, const DraftParams& p, cudaStream_t stream);
cudaError_t drafts_tma_launch(int dtype, const DraftParams& p, cudaStream_t stream);
bool drafts_tma_fits(int64_t page_size, const int64_t (&sizes)[4], const int64_t (&k_st)[4], const int64_t (&v_st)[4]);
cudaError_t drafts_f32_launch16(const DraftParams& p, cudaStream_t stream);
cudaError_t drafts_f32_launch4(const DraftParams& p, cudaStream_t stream);
// The weights, from the maxima and sums that the attention has left in p.stats.
cudaError_t weigh_mma_launch16(int dtype, const DraftParams& p, cudaStream_t stream);
cudaError_t weigh_mma_launch4(int dtype, const DraftParams& p, cudaStream_t stream);
cudaError_t weigh_mma_launch0(int dtype, const DraftParams& p, cudaStream_t stream);
cudaError_t weigh_scores_launch(const DraftParams& p, cudaStream_t stream);  // (from p.scores)
cudaError_t weigh_tma_launch(int dtype, const DraftParams& p, cudaStream_t stream);  // (where drafts_tma_launch may be)
cudaError_t weigh_f32_launch16(const DraftParams& p, cudaStream_t stream);
cudaError_t weigh_f32_launch4(const DraftParams& p, cudaStream_t stream);

// ---- what is kept (cache_keep.cu) -----------------------------------------------
struct PathParams {
  const int32_t *tokens, *choices, *parents;  // (parents NULL: a chain)
  int64_t token_st[2], choice_st[2], parent_st[2];
  int32_t *path, *counts, *last;
  int64_t path_st[2], counts_st, last_st;
  int32_t rows, drafts;
  int32_t* status;
};
cudaError_t path_launch(const PathParams& p, cudaStream_t stream);

// What the accepted tokens' move and the eviction share: rows that are cut.
constexpr int kEvictMoveThreads = 256, kEvictMoveAtOnce = 8;  // of a CTA that moves what an eviction keeps
struct KeepParams {
  const int32_t *tables, *lengths, *refs;
  int32_t *lengths_out, *refs_out;
  int64_t table_st;
  int32_t rows, columns, pages;
  FastDiv32 page;
  int32_t heads, pieces;      // a token's access units: heads times the pieces of one
  int32_t unit;               // bytes of one
  FastDiv32 per_head;         // by pieces
  int32_t* status;
  // accept
  const int32_t *path, *counts;
  int64_t path_st;            // rows; a row's entries are dense
  int32_t drafts;
  // evict
  int32_t budget, recent, layers;
  int32_t slices, team;       // a token's pieces go to so many clusters of so many CTAs
  int32_t* kept;              // [rows][layers][heads][budget]
};
struct KeepPool {
  uint8_t* ptr;
  int64_t st[3];              // page, slot, head (bytes)
};
struct KeepPools {
  KeepPool pool[CMD_CACHE_MAX_POOLS];
  int32_t n;
};
struct KeepLayers {
  KeepPool pool[CMD_CACHE_MAX_LAYERS][2];
  float* weights[CMD_CACHE_MAX_LAYERS];
  int64_t w_st[CMD_CACHE_MAX_LAYERS][2];
};
cudaError_t accept_launch(const KeepParams& p, const KeepPools& pools, cudaStream_t stream);
cudaError_t evict_launch(const KeepParams& p, const KeepLayers& layers, cudaStream_t stream);

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
